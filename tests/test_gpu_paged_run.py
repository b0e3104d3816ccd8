"""The paged cache, its attention and the next token as they are used: whole steps of
a model's attention layer from prompts through single tokens and drafts to the end,
batches padded to a captured size, HIP graphs, several streams, caches past 32 bits,
random shapes."""
import random

import numpy as np
import pytest
import torch

import paged_ref as R
from test_gpu_kv import Cache, f64, filled, layout, up, values

pytestmark = pytest.mark.gpu
F32, BF, I32, F8 = torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(int)


class Model:
    """One layer of attention and an output projection over random weights; the
    host keeps every request's keys and values as they were given."""

    def __init__(self, K, rows, blocks, bs, H, Hq, D, vocab, io, seed):
        self.K, self.bs, self.dims, self.io = K, bs, (H, Hq, D), io
        g = torch.Generator().manual_seed(seed)
        self.cache = Cache(blocks, H, bs, D)
        self.lens, self.held, self.count = (torch.zeros(n, dtype=I32, device="cuda") for n in (rows, rows, 1))
        self.table = torch.full((rows, 32), -1, dtype=I32, device="cuda")
        self.free = torch.randperm(blocks, generator=g).to(I32).cuda()
        self.count.fill_(blocks)
        self.emb = torch.randn(vocab, (Hq + 2 * H) * D, generator=g).to(io).cuda()
        self.out = (torch.randn(Hq * D, vocab, generator=g) / 4).cuda()
        self.kept = {}                     # row -> tokens that stand, in order

    def tables(self):
        return self.lens, self.held, self.table, self.free, self.count

    def step(self, idx, tokens, pad=0):
        """Logits of every token; tokens: a list a request."""
        H, Hq, D = self.dims
        lens = [len(t) for t in tokens]
        cu = up(np.concatenate([offsets(lens), [sum(lens)] * pad]))
        rows = up(list(idx) + [-1] * pad)
        flat = torch.tensor([t for s in tokens for t in s] + [0] * pad, dtype=torch.long, device="cuda")
        qkv = self.emb[flat].view(len(flat), Hq + 2 * H, D)
        slots, totals = self.K.kv_reserve(cu, len(flat), rows, *self.tables(), block_size=self.bs)
        self.K.kv_store(qkv[:, Hq:Hq + H], qkv[:, Hq + H:], slots, *self.cache.all())
        o = self.K.kv_attention(qkv[:, :Hq], cu, totals, rows, self.table, *self.cache.all())
        self.cu, self.rows = cu, rows
        return o[:sum(lens)], o[:sum(lens)].float().reshape(sum(lens), -1) @ self.out

    def check(self, idx, tokens, o, name):
        """o against attention over keys and values rounded to the cache's values."""
        H, Hq, D = self.dims
        table, lens = self.table.cpu().numpy(), offsets([len(t) for t in tokens])
        q = f64(self.emb)[[t for s in tokens for t in s]].reshape(-1, Hq + 2 * H, D)
        totals = [len(self.kept[r]) + len(t) for r, t in zip(idx, tokens)]
        ref, tol = R.attention(q[:, :Hq], lens, totals, idx, table, values(self.cache.kc), values(self.cache.vc), f64(self.cache.ks),
                               f64(self.cache.vs), D ** -0.5, self.io)
        R.check(name, o, ref, tol, self.io)
        # what the cache holds is what was given, to half a step of e4m3 under the scale that fits the block, twice where it grew
        for r, t in zip(idx, tokens):
            whole = f64(self.emb)[self.kept[r] + list(t)].reshape(-1, Hq + 2 * H, D)
            n = len(whole)
            for part, c, s, last in ((whole[:, Hq:Hq + H], self.cache.kc, self.cache.ks, False), (whole[:, Hq + H:], self.cache.vc, self.cache.vs, True)):
                pages = torch.from_numpy(table[r][:-(-n // self.bs)]).long().cuda()
                got = c[pages].float() * s[pages][:, :, None, None]
                got = (got.permute(0, 3, 1, 2) if last else got.permute(0, 2, 1, 3)).reshape(-1, H, D)[:n]
                least = f64(s[pages]).repeat(self.bs, 0)[:n, :, None] * 2.0 ** -6      # e4m3's least normal number
                assert (np.abs(f64(got) - part) <= 2.0 ** -4 * np.maximum(np.abs(part), least)).all(), name


@pytest.mark.parametrize("io,bs,D", [(BF, 16, 64), (BF, 64, 128), (F32, 32, 64)])
def test_serving(K, io, bs, D):
    """Prompts, single tokens, runs of drafts of which some stand, requests that end
    and others in their place: the attention of every step, the cache, the tokens drawn
    and verified, and at the end a full list."""
    r = random.Random(bs + D)
    vocab, rows, blocks = 211, 7, 90
    m = Model(K, rows, blocks, bs, 2, 4, D, vocab, io, bs)
    live = {}
    for step in range(9):
        ended = [x for x in list(live) if r.random() < 0.15]
        if ended:
            m.K.kv_release(up(ended), *m.tables(), block_size=bs)
            for x in ended:
                del live[x], m.kept[x]
        fresh = [x for x in range(rows) if x not in live][:r.randint(0, 3)]
        for x in fresh:
            m.kept[x] = []
        idx = fresh + list(live)
        r.shuffle(idx)
        if not idx:
            continue
        tokens = [[live[x]] + [r.randrange(vocab) for _ in range(r.choice([0, 0, 2, 3]))] if x in live else
                  [r.randrange(vocab) for _ in range(r.choice([1, bs, 70, 33]))] for x in idx]
        o, logits = m.step(idx, tokens, pad=r.choice([0, 2]))
        m.check(idx, tokens, o, "step %d" % step)
        lens = [len(t) for t in tokens]
        T, cu = sum(lens), offsets(lens)
        flat = torch.tensor([t for s in tokens for t in s], dtype=I32, device="cuda")
        u, un = (torch.rand(n, generator=torch.Generator().manual_seed(step + n)).cuda() for n in (T, len(idx)))
        limit = dict(temperature=torch.full((T,), 0.8, device="cuda"), top_p=torch.full((T,), 0.9, device="cuda"),
                     top_k=torch.full((T,), 40, dtype=I32, device="cuda"))
        p = K.token_probs(logits, **limit)
        accepted, nxt, _ = K.verify_drafts(flat, p, up(cu), u, un)
        # a prompt's tokens all stand: its next one is drawn after the last
        last = torch.tensor([cu[i + 1] - 1 for i in range(len(idx))], device="cuda")
        drawn = K.sample_tokens(logits[last], un, **{k: v[:len(idx)] for k, v in limit.items()})
        steps = [lens[i] - 1 if x not in live else int(accepted[i]) for i, x in enumerate(idx)]
        want, _ = R.sample(f64(logits[last]), f64(un), [float(torch.tensor(0.8))] * len(idx), [40] * len(idx), [float(torch.tensor(0.9))] * len(idx))
        assert drawn.tolist() == want
        pad = len(m.rows) - len(idx)
        K.kv_commit(m.cu, m.rows, m.lens, m.held, block_size=bs, steps=up(steps + [-1] * pad))
        for i, x in enumerate(idx):
            m.kept[x] = m.kept[x] + tokens[i][:steps[i] + 1]
            live[x] = int(drawn[i]) if steps[i] == lens[i] - 1 else int(nxt[i])
        assert [int(m.lens[x]) for x in idx] == [len(m.kept[x]) for x in idx]
    K.kv_release(up(list(range(rows))), *m.tables(), block_size=bs)
    assert int(m.count) == blocks and sorted(m.free.tolist()) == list(range(blocks)) and not bool(m.held.any())


def test_store_by_parts_is_store_at_once(K):
    """A prompt in one call, in chunks and token by token: attention over the three
    caches agrees to what the rounding of grown blocks leaves (none: equal scales)."""
    bs, H, D, n = 32, 2, 64, 100
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(n, H, D, generator=g).clamp(-3, 3).cuda() for _ in range(2))
    k[::bs, :, 0], v[::bs, :, 0] = 3.0, 3.0            # a block's first token has its largest value
    slots = list(range(bs, bs + n))
    got = []
    for parts in ([n], [1] * n, [37, 1, 2, 60]):
        c, t = Cache(6, H, bs, D), 0
        for m in parts:
            K.kv_store(k[t:t + m], v[t:t + m], up(slots[t:t + m]), *c.all())
            t += m
        got.append([x.view(torch.uint8) if x.dtype == F8 else x for x in c.all()])
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a.nan_to_num(-1.0) if a.is_floating_point() else a, b.nan_to_num(-1.0) if b.is_floating_point() else b)


def test_padded_batch(K):
    """Arrays for more tokens and requests than there are: nothing of the rest is
    read, its slots are nowhere, its rows of o are not written."""
    bs, H, Hq, D = 16, 2, 4, 64
    g = torch.Generator().manual_seed(2)
    lens, old = [3, 1], [40, 9]
    table, at, cu = layout(lens, old, bs, 12, 7)
    cache = filled(K, table, at, lens, old, 12, H, bs, D, g)
    totals = [43, 10]
    q = torch.randn(9, Hq, D, generator=g).to(BF).cuda()
    want = K.kv_attention(q[:4], up(cu), up(totals), up(at), up(table), *cache.all())
    q[4:] = float("nan")
    more = K.kv_attention(q, up(list(cu) + [4, 4]), up(totals + [7, 99]), up(list(at) + [-1, 100]), up(table), *cache.all())
    assert torch.equal(more[:4], want)
    more = K.kv_attention(q, up(cu), up(totals + [7]), up(list(at) + [1]), up(table), *cache.all())
    assert torch.equal(more[:4], want)
    k = torch.randn(9, H, D, generator=g).cuda()
    k[4:] = float("nan")
    before = [x.clone() for x in cache.all()]
    K.kv_store(k, k, up([-1] * 9), *cache.all())
    for a, b in zip(before, cache.all()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_long_cache(K):
    """A cache of more than 2^32 bytes: blocks at its far end give the bits of a small
    one."""
    bs, H, Hq, D, blocks = 128, 8, 16, 128, 34000
    assert blocks * bs * H * D > 1 << 32
    lens, old = [1, 5, 70], [1000, 300, 200]
    g = torch.Generator().manual_seed(3)
    table, at, cu = layout(lens, old, bs, 20, 8)
    small = filled(K, table, at, lens, old, 20, H, bs, D, g, io=BF)
    big = [torch.empty(blocks, *x.shape[1:], dtype=x.dtype, device="cuda") for x in small.all()]
    far = np.where(table < 20, blocks - 1 - table * 7, table)
    slots = [int(far[at[i], p // bs]) * bs + p % bs for i in range(3) for p in range(lens[i] + old[i])]
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(len(slots), H, D, generator=g).to(BF).cuda() for _ in range(2))
    K.kv_store(k, v, up(slots), *big)
    q = torch.randn(int(cu[-1]), Hq, D, generator=g).to(BF).cuda()
    totals = [a + b for a, b in zip(lens, old)]
    a = K.kv_attention(q, up(cu), up(totals), up(at), up(table), *small.all())
    b = K.kv_attention(q, up(cu), up(totals), up(at), up(far), *big)
    assert torch.equal(a, b)


def test_shared_prefix_and_equal_rows(K):
    """Requests whose rows name the same blocks, and requests on one row, read them
    alike."""
    bs, H, Hq, D = 16, 1, 2, 64
    g = torch.Generator().manual_seed(9)
    table, at, cu = layout([1], [79], bs, 8, 9)
    cache = filled(K, table, at, [1], [79], 8, H, bs, D, g)
    q = torch.randn(1, Hq, D, generator=g).to(BF).cuda().repeat(3, 1, 1)
    both = np.stack([table[at[0]], table[at[0]]])
    o = K.kv_attention(q, up([0, 1, 2, 3]), up([80, 80, 80]), up([0, 1, 0]), up(both), *cache.all())
    assert torch.equal(o[0], o[1]) and torch.equal(o[0], o[2])


def _work(K, seed, n, old, bs=64, H=2, Hq=8, D=128):
    g = torch.Generator().manual_seed(seed)
    lens = [1] * n
    blocks = sum(-(-(a + b) // bs) for a, b in zip(lens, old)) + 3
    table, at, cu = layout(lens, old, bs, blocks, seed)
    cache = filled(K, table, at, lens, old, blocks, H, bs, D, g, io=BF)
    q = torch.randn(n, Hq, D, generator=g).to(BF).cuda()
    x, u = (torch.randn(n, 5000, generator=g) * 3).cuda(), torch.rand(n, generator=g).cuda()
    p = torch.full((n,), 0.9, device="cuda")
    args = (up(cu), up([a + b for a, b in zip(lens, old)]), up(at), up(table), *cache.all())
    return lambda: (K.kv_attention(q, *args), *K.sample_tokens(x, u, top_p=p, return_probs=True))


def test_streams(K):
    """Two streams at once, each with its own work: what the lone calls gave."""
    works = [_work(K, 1, 5, [3000, 10, 700, 64, 1]), _work(K, 2, 40, [random.Random(5).randint(1, 900) for _ in range(40)])]
    want = [w() for w in works]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in works]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(works[i]())
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            for a, b in zip(out, want[i]):
                assert torch.equal(a, b)


def test_graph(K):
    """Two steps of decoding captured into two graphs (blocks reserved, keys stored,
    attended to, a token drawn, the token counted), replayed in turn with eager work
    between: every replay equals the eager steps."""
    bs, H, Hq, D, n, vocab = 16, 2, 4, 64, 3, 300

    def fresh():
        m = Model(K, 5, 40, bs, H, Hq, D, vocab, BF, 11)
        idx, prompts = [4, 0, 2], [[5, 6, 7] * 7, [1] * 15, [9]]
        m.step(idx, prompts)
        K.kv_commit(m.cu, m.rows, m.lens, m.held, block_size=bs)
        return m

    def one(m, token, u):
        qkv = m.emb[token.long()].view(n, Hq + 2 * H, D)
        slots, totals = K.kv_reserve(m.dcu, n, m.drows, *m.tables(), block_size=bs)
        K.kv_store(qkv[:, Hq:Hq + H], qkv[:, Hq + H:], slots, *m.cache.all())
        o = K.kv_attention(qkv[:, :Hq], m.dcu, totals, m.drows, m.table, *m.cache.all())
        logits = o.float().reshape(n, -1) @ m.out
        token.copy_(K.sample_tokens(logits, u, top_p=m.p, top_k=m.k))
        K.kv_commit(m.dcu, m.drows, m.lens, m.held, block_size=bs)
        return o

    def setup():
        m = fresh()
        m.dcu, m.drows = up([0, 1, 2, 3]), up([4, 0, 2])
        m.p, m.k = torch.full((n,), 0.95, device="cuda"), torch.full((n,), 30, dtype=I32, device="cuda")
        return m, up([3, 4, 5]), torch.tensor([0.3, 0.6, 0.9], device="cuda")

    m, token, u = setup()
    want = []
    for i in range(24):
        o = one(m, token, u)
        want.append((o.clone(), token.clone()))
        u.copy_((u + 0.37) % 1.0)
    final = [x.clone() for x in m.tables()]
    m, token, u = setup()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    keep = [x.clone() for x in (*m.tables(), token)]
    with torch.cuda.stream(side):
        one(m, token, u)                      # the libraries' own first calls
    torch.cuda.synchronize()
    m, token, u = setup()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(one(m, token, u))
        graphs.append(graph)
    for a, b in zip((*m.tables(), token), keep):      # capturing ran nothing
        assert torch.equal(a, b)
    for i in range(24):
        graphs[i % 2].replay()
        assert torch.equal(outs[i % 2], want[i][0]) and torch.equal(token, want[i][1]), i
        u.copy_((u + 0.37) % 1.0)
        torch.empty(1 << 20, device="cuda").fill_(float(i))
    for a, b in zip(m.tables(), final):
        assert torch.equal(a, b)


@pytest.mark.parametrize("seed", range(16))
def test_random_shapes(K, seed):
    """Mixed batches of prompts, single tokens and drafts, any heads, dims, block
    sizes and types, against 64 bits."""
    r = random.Random(seed)
    H, D, bs, io = r.choice([1, 2, 3, 5]), r.choice([64, 128]), r.choice([16, 32, 64, 128]), r.choice([BF, BF, F32])
    Hq = H * r.choice([1, 2, 3, 4, 8, 17])
    n = r.randint(1, 9)
    lens = [r.choice([0, 1, 1, 1, 2, 5, 17, r.randint(1, 150)]) for _ in range(n)]
    old = [r.choice([0, 1, 63, 64, 65, r.randint(0, 1200)]) for _ in range(n)]
    g = torch.Generator().manual_seed(seed)
    blocks = sum(-(-(a + b) // bs) for a, b in zip(lens, old)) + 2
    table, at, cu = layout(lens, old, bs, blocks, seed)
    cache = filled(K, table, at, lens, old, blocks, H, bs, D, g, size=r.choice([0.1, 1.0, 5.0]))
    q = (torch.randn(int(cu[-1]), Hq + 2, D, generator=g) * r.choice([0.5, 2.0])).to(io).cuda()[:, 1:Hq + 1]
    totals = [a + b for a, b in zip(lens, old)]
    o = K.kv_attention(q, up(cu), up(totals), up(at), up(table), *cache.all())
    ref, tol = R.attention(f64(q), cu, totals, at, table, values(cache.kc), values(cache.vc), f64(cache.ks), f64(cache.vs), D ** -0.5, io)
    R.check("o", o, ref, tol, io)


def test_many_requests(K):
    """More requests than a workgroup's threads, some far longer than the others."""
    r = random.Random(3)
    n, bs, H, Hq, D = 700, 16, 1, 2, 64
    old = [r.randint(0, 30) for _ in range(n)]
    old[13], old[600] = 5000, 2500
    lens = [1] * n
    lens[50], lens[51] = 0, 40
    g = torch.Generator().manual_seed(4)
    blocks = sum(-(-(a + b) // bs) for a, b in zip(lens, old)) + 2
    table, at, cu = layout(lens, old, bs, blocks, 4)
    cache = filled(K, table, at, lens, old, blocks, H, bs, D, g)
    q = torch.randn(int(cu[-1]), Hq, D, generator=g).to(BF).cuda()
    totals = [a + b for a, b in zip(lens, old)]
    o = K.kv_attention(q, up(cu), up(totals), up(at), up(table), *cache.all())
    ref, tol = R.attention(f64(q), cu, totals, at, table, values(cache.kc), values(cache.vc), f64(cache.ks), f64(cache.vs), D ** -0.5, BF)
    R.check("o", o, ref, tol, BF)


def test_many_prompts(K):
    """More requests than a workgroup's threads with prompts, some empty, one long."""
    r = random.Random(8)
    n, bs, H, Hq, D = 290, 32, 1, 2, 64
    lens = [r.choice([0, 17, 40, 55]) for _ in range(n)]
    old = [r.randint(0, 20) for _ in range(n)]
    lens[100], old[100], old[200] = 600, 300, 900
    g = torch.Generator().manual_seed(8)
    blocks = sum(-(-(a + b) // bs) for a, b in zip(lens, old)) + 2
    table, at, cu = layout(lens, old, bs, blocks, 8)
    cache = filled(K, table, at, lens, old, blocks, H, bs, D, g)
    q = torch.randn(int(cu[-1]), Hq, D, generator=g).to(BF).cuda()
    totals = [a + b for a, b in zip(lens, old)]
    o = K.kv_attention(q, up(cu), up(totals), up(at), up(table), *cache.all())
    ref, tol = R.attention(f64(q), cu, totals, at, table, values(cache.kc), values(cache.vc), f64(cache.ks), f64(cache.vs), D ** -0.5, BF)
    R.check("o", o, ref, tol, BF)
