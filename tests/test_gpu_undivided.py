"""Attention of prompts whose units fill the chip undivided, the longest first: any
number of requests up to, at and beyond what a wave and a workgroup look through,
empty and padded ones, totals below the length, totals up to the largest.  And the
opposite: columns cut into more chunks than a wave has lanes."""
import ctypes
import random

import numpy as np
import pytest
import torch

import paged_ref as R
from test_gpu_kv import Cache, f64, up, values

pytestmark = pytest.mark.gpu
F32, BF, I32 = torch.float32, torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


def workspace(K, n, T, Hq, H, D, bs, io):
    d = K.KvDesc(num_seqs=n, total_tokens=T, q_heads=Hq, kv_heads=H, head_dim=D, block_size=bs, num_blocks=1, rows=1, max_blocks=1,
                 io_dtype=int(io == BF), scale=1.0, q_stride=Hq * D, k_stride=H * D, v_stride=H * D)
    return K.lib().kda_kv_attention_workspace_size(ctypes.byref(d))


def undivided(K, n, T, Hq, H, D, bs, io):
    """Such a call needs room for no sums: nothing, or where many requests' places begin."""
    return workspace(K, n, T, Hq, H, D, bs, io) <= (0 if n <= 256 else 4 * n + 512)


def definition(q, cu, totals, at, table, cache, scale, io):
    """o and its bound (paged_ref.attention's) in 64 bits, whole requests at once."""
    kc, vc, ks, vs = (x.float().double() for x in cache.all())
    B, H, bs, D = kc.shape
    T, Hq, _ = q.shape
    g, q = Hq // H, q.double()
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    for n in range(len(cu) - 1):
        lo, hi, L = int(cu[n]), int(cu[n + 1]), int(cu[n + 1] - cu[n])
        if L == 0 or not 0 <= at[n] < len(table):
            continue
        total = min(max(int(totals[n]), 0), table.shape[1] * bs)
        if total == 0:
            continue
        page = torch.as_tensor(np.asarray(table[at[n]][:-(-total // bs)], np.int64)).cuda()
        assert int(page.min()) >= 0 and int(page.max()) < B
        last = total - L + torch.arange(L, device="cuda")
        see = torch.arange(total, device="cuda")[None, :] <= last[:, None]
        for h in range(H):
            k = (kc[page, h] * ks[page, h][:, None, None]).reshape(-1, D)[:total]
            v = (vc[page, h].transpose(1, 2) * vs[page, h][:, None, None]).reshape(-1, D)[:total]
            # a value that nobody stored is no number, and no column may see it
            k, v = k.nan_to_num(0.0), v.nan_to_num(0.0)
            kt, kta = k.t().contiguous(), k.abs().t().contiguous()
            for i in range(h * g, h * g + g):
                x = q[lo:hi, i].contiguous()
                z = (scale * (x @ kt)).masked_fill(~see, -float("inf"))
                A = (scale * (x.abs() @ kta)).masked_fill(~see, 0).amax(1)
                top = z.amax(1)
                p = torch.exp(z - torch.where(top.isinf(), torch.zeros_like(top), top)[:, None])
                s = p.sum(1)[:, None].clamp_min(1e-300)
                out, spread = p @ v / s, p @ v.abs() / s
                ep = R.E32 * ((D + 10) * A + 8)
                near = 2 * ep + (2.0 ** -8 if io == BF else 4 * R.E32) + 2 * (see.sum(1) + 64) * R.E32
                o[lo:hi, i] = out
                tol[lo:hi, i] = near[:, None] * spread + (2.0 ** -8 * out.abs() if io == BF else 0)
    return f64(o), f64(tol)


class Batch:
    """Requests on scattered rows and blocks, their tokens stored; `short`: totals as
    far below what the request has."""

    def __init__(self, K, lens, old, H, Hq, D, bs, io, seed, short=None, pad=()):
        self.K, self.io = K, io
        g = torch.Generator().manual_seed(seed)
        r = np.random.RandomState(seed)
        n, have = len(lens), [-(-(a + b) // bs) for a, b in zip(lens, old)]
        blocks, wide = sum(have) + 3, max(have) + 2
        self.table = np.full((n + 2, wide), -1, np.int32)
        self.at, order, used = r.permutation(n + 2)[:n], r.permutation(blocks), 0
        for i in range(n):
            self.table[self.at[i], :have[i]] = order[used:used + have[i]]
            used += have[i]
        self.cache = Cache(blocks, H, bs, D)
        slots = np.concatenate([np.repeat(self.table[self.at[i], :have[i]] * bs, bs)[:a + b] + np.arange(a + b) % bs
                                for i, (a, b) in enumerate(zip(lens, old))])
        k, v = (torch.randn(len(slots), H, D, generator=g).cuda() for _ in range(2))
        K.kv_store(k, v, up(slots), *self.cache.all())
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(int)
        self.totals = [a + b - (short[i] if short else 0) for i, (a, b) in enumerate(zip(lens, old))]
        for i in pad:
            self.at[i] = -1 if i % 2 else n + 5
        self.q = (torch.randn(int(self.cu[-1]), Hq, D, generator=g) * 2).to(io).cuda()
        self.shape = (n, int(self.cu[-1]), Hq, H, D, bs, io)

    def run(self, table=None):
        table = up(self.table) if table is None else table
        # where o is allocated lie NaN of the call before: a row that is not written shows
        torch.full_like(self.q, float("nan"))
        return self.K.kv_attention(self.q, up(self.cu), up(self.totals), up(self.at), table, *self.cache.all())

    def check(self, name, o):
        ref, tol = definition(self.q, self.cu, self.totals, self.at, self.table, self.cache, self.q.shape[-1] ** -0.5, self.io)
        R.check(name, o, ref, tol, self.io)


def spread(n, most, seed, empty=True):
    r = random.Random(seed)
    return [r.choice([0, most, r.randint(1, most), r.randint(1, most)] if empty else [r.randint(most // 2, most)]) for _ in range(n)]


CASES = [   # requests, longest, H, Hq, D, block size, io
    (1, 4103, 8, 32, 64, 64, BF),
    (1, 2049, 16, 32, 128, 128, F32),
    (5, 2300, 8, 32, 128, 64, BF),
    (3, 1500, 16, 32, 64, 16, F32),
    (64, 150, 8, 24, 64, 32, BF),
    (65, 150, 8, 16, 128, 64, BF),
    (64, 90, 8, 16, 64, 64, F32),
    (65, 70, 9, 27, 64, 16, F32),
    (256, 90, 2, 6, 64, 32, BF),
    (256, 60, 2, 6, 128, 64, F32),
    (257, 100, 2, 4, 128, 16, BF),
    (300, 60, 2, 6, 64, 128, F32),
]


@pytest.mark.parametrize("n,most,H,Hq,D,bs,io", CASES, ids=["%d-%s" % (c[0], "bf16" if c[-1] == BF else "f32") + "-%d" % i for i, c in enumerate(CASES)])
def test_prompts(K, n, most, H, Hq, D, bs, io):
    """Unequal lengths, empty ones among them, behind tokens held or none."""
    lens = spread(n, most, n + D) if n > 5 else [most] * n
    if n > 5:
        lens[0], lens[n // 2] = most, 0
    r = random.Random(n)
    old = [r.choice([0, 0, 1, 70, r.randint(0, 200)]) for _ in range(n)]
    b = Batch(K, lens, old, H, Hq, D, bs, io, n + most)
    assert undivided(K, *b.shape), workspace(K, *b.shape)
    o = b.run()
    b.check("o", o)
    assert torch.equal(o, b.run())


@pytest.mark.parametrize("n", [6, 64, 70, 260])
@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
def test_equal_prompts(K, n, io):
    """Ties everywhere: all requests of one length, none held, and one of them twice."""
    L, H, Hq, D = {6: 700, 64: 45, 70: 45, 260: 45}[n], 8, 32, 64
    b = Batch(K, [L] * n, [0] * n, H, Hq, D, 64, io, n)
    assert undivided(K, *b.shape)
    b.q[L:2 * L] = b.q[:L]
    b.table[b.at[1]] = b.table[b.at[0]]
    o = b.run()
    b.check("o", o)
    assert torch.equal(o[L:2 * L], o[:L])


@pytest.mark.parametrize("n,L", [(7, 700), (80, 70), (270, 40)])
@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
def test_padding_and_short_totals(K, n, L, io):
    """Rows that do not exist see nothing; a total below the length leaves the first
    tokens without a position, one of 0 all of them: zeros, rows of o behind the last
    request are not written."""
    H, Hq, D = 8, 32, 64
    r = random.Random(n)
    lens = [r.choice([L, L + 3, 0]) for _ in range(n)]
    lens[:4] = [L, L, L, L + 1]
    short = [r.choice([0, 0, 5, 3 * L]) for _ in range(n)]
    short[:4] = [0, 10, 5 * L, 1]
    b = Batch(K, lens, [r.choice([0, 33]) for _ in range(n)], H, Hq, D, 32, io, n, short, pad=(3, n - 2))
    assert undivided(K, *b.shape)
    o = b.run()
    b.check("o", o)
    assert not bool(o[int(b.cu[2]):int(b.cu[4])].any())
    # the same in arrays for more tokens, which hold anything
    more = torch.full((b.q.shape[0] + 9, Hq, D), float("nan"), dtype=io, device="cuda")
    more[:-9] = b.q
    again = K.kv_attention(more, up(b.cu), up(b.totals), up(b.at), up(b.table), *b.cache.all())
    assert torch.equal(again[:-9], o)


@pytest.mark.parametrize("total", [(1 << 30) - 300, 1 << 30, (1 << 31) - 1])
def test_largest_total(K, total):
    """A request without new tokens, but with as many held as a row can have, beside
    prompts: they are what they are without it."""
    lens, H, Hq, D, bs = [4000, 0, 150], 8, 32, 64, 128
    b = Batch(K, lens, [0, 100, 40], H, Hq, D, bs, BF, 9)
    assert undivided(K, *b.shape)
    want = b.run()
    b.check("o", want)
    table = torch.full((len(b.table), (1 << 30) // bs), -1, dtype=I32, device="cuda")
    table[:, :b.table.shape[1]] = up(b.table)
    b.totals[1] = total
    assert torch.equal(b.run(table), want)


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 290])
def test_many_chunks(K, n, io):
    """One token behind 60,000 others, and a prompt behind 40,000 in another call:
    each column has more chunks than a wave has lanes."""
    D, bs = 64, 128
    lens, old = [1] * n, [5] * n
    old[1] = 60000
    lens[2] = 0
    b = Batch(K, lens, old, 1, 2, D, bs, io, n)
    b.check("token", b.run())
    if n == 3:
        b = Batch(K, [45, 1], [40000, 3], 2, 2, 128, 64, io, n)
        b.check("prompt", b.run())


def test_captured_and_on_streams(K):
    """Undivided prompts, cut prompts and many requests in one graph, replayed with other
    queries and eager work between, and on two streams at once: each equals its lone
    call."""
    works = [Batch(K, [1700, 0, 400], [0, 9, 50], 8, 64, 64, 64, BF, 1), Batch(K, [200, 90], [300, 2000], 2, 8, 128, 32, BF, 2),
             Batch(K, [40] * 259, [3] * 259, 2, 6, 64, 16, F32, 3), Batch(K, [4] * 30, [700] * 30, 2, 8, 128, 16, BF, 4)]
    assert undivided(K, *works[0].shape) and not undivided(K, *works[1].shape) and undivided(K, *works[2].shape)
    fixed = [(up(b.cu), up(b.totals), up(b.at), up(b.table), *b.cache.all()) for b in works]
    want = [[], []]
    queries = [[b.q.clone(), b.q.roll(1, 0).contiguous()] for b in works]
    for i in (0, 1):
        want[i] = [K.kv_attention(q[i], *f) for q, f in zip(queries, fixed)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for b, f in zip(works, fixed):
            K.kv_attention(b.q, *f)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [K.kv_attention(b.q, *f) for b, f in zip(works, fixed)]
    for n in range(6):
        for b, q in zip(works, queries):
            b.q.copy_(q[n % 2])
        graph.replay()
        for o, w in zip(outs, want[n % 2]):
            assert torch.equal(o, w), n
        torch.empty(1 << 22, device="cuda").fill_(float("nan"))
    streams, got = [torch.cuda.Stream() for _ in works], []
    torch.cuda.synchronize()
    for _ in range(3):
        for q, f, w, s in zip(queries, fixed, want[0], streams):
            with torch.cuda.stream(s):
                got.append((K.kv_attention(q[0], *f), w))
    torch.cuda.synchronize()
    for o, w in got:
        assert torch.equal(o, w)
