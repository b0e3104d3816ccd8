"""The 8-bit cache and the attention over it against 64 bits: block sizes, head
counts and dims, single tokens, runs of drafts, prompts, long contexts, odd lengths,
pages that do not exist, NaN and infinities in masked places."""
import numpy as np
import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu
F32, BF, I32, F8 = torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn
IO = {"bf16": BF, "f32": F32}


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


def f64(t):
    return t.detach().cpu().double().numpy()


def up(a):
    return torch.as_tensor(np.asarray(a), dtype=I32).cuda()


def values(cache):
    return cache.float().cpu().double().numpy()


class Cache:
    """A cache whose every byte is NaN and every scale NaN until it is stored."""

    def __init__(self, blocks, H, bs, D):
        self.kc = torch.full((blocks, H, bs, D), 0x7f, dtype=torch.uint8, device="cuda").view(F8)
        self.vc = torch.full((blocks, H, D, bs), 0xff, dtype=torch.uint8, device="cuda").view(F8)
        self.ks = torch.full((blocks, H), float("nan"), device="cuda")
        self.vs = torch.full((blocks, H), float("nan"), device="cuda")

    def all(self):
        return self.kc, self.vc, self.ks, self.vs

    def host(self):
        return values(self.kc), values(self.vc).transpose(0, 1, 3, 2).copy(), f64(self.ks), f64(self.vs)


def same(a, b):
    return np.array_equal(a, b, equal_nan=True)


def store_both(K, cache, k, v, slots):
    kc, vc, ks, vs = cache.host()
    R.store(f64(k), slots, kc, ks)
    R.store(f64(v), slots, vc, vs)
    K.kv_store(k, v, up(slots), *cache.all())
    for a, b, name in zip(cache.host(), (kc, vc, ks, vs), ("keys", "values", "key scales", "value scales")):
        assert same(a, b), name


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("D,H", [(64, 3), (128, 2)])
def test_store(K, io, bs, D, H):
    """Runs that start and end anywhere in a block, in any order of blocks, rows cut
    out of wider ones, slots that are nowhere; then more tokens behind them that
    need larger and smaller scales."""
    g = torch.Generator().manual_seed(bs + D)
    cache = Cache(9, H, bs, D)
    first = list(range(3 * bs, 4 * bs)) + list(range(bs, bs + 5)) + [-1, -1, 9 * bs, 1 << 30] + list(range(7 * bs, 7 * bs + 1)) \
        + list(range(5 * bs, 7 * bs - 3)) + list(range(0, bs - 1))
    then = [bs + 5, bs + 6] + [7 * bs - 3, 7 * bs - 2, 7 * bs - 1] + list(range(7 * bs + 1, 8 * bs)) + [bs - 1, -1] + list(range(2 * bs, 2 * bs + 7))
    for slots, size in ((first, 1.0), (then, 30.0), ([bs + 7, 2 * bs + 7], 1e-3), ([bs + 8], 1e5)):
        row = (torch.randn(len(slots), 4 * H + 1, D, generator=g) * size).to(IO[io]).cuda()
        store_both(K, cache, row[:, H:2 * H], row[:, 2 * H:3 * H], slots)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_store_borders(K, io):
    """Largest values at and beside a scale's border, zeros, the smallest and largest
    numbers, infinities and NaN (stored as NaN, without a part in the scale)."""
    H, D, bs = 2, 64, 16
    tops = [448.0, 449.0, 452.0, 447.0, 7.0, 7.0625, 0.875, 1e-30, 0.0, 3e38, 1e-38]
    cache = Cache(len(tops) + 2, H, bs, D)
    x = torch.rand(len(tops) + 1, H, D, generator=torch.Generator().manual_seed(1)) * 2 - 1
    for i, t in enumerate(tops):
        x[i] *= t
        x[i, :, 5] = -t
    x[-1, 0, 3], x[-1, 0, 4], x[-1, 1] = float("inf"), float("nan"), float("-inf")
    x = x.to(IO[io]).cuda()
    store_both(K, cache, x, -x, [bs * i for i in range(len(tops) + 1)])
    assert bool(cache.kc.float()[len(tops), 1, 0].isnan().all())


def test_store_every_value(K):
    """Every e4m3 value and every midpoint of two, under a scale of one."""
    vals = torch.arange(127, dtype=torch.uint8).view(F8).float()
    mids = (vals[1:] + vals[:-1]) / 2
    x = torch.cat([vals, mids, torch.full((3,), 448.0)])
    x = torch.cat([x, -x]).view(-1, 1, 64)[:8].contiguous().cuda()
    assert float(x.abs().amax(2).min()) >= 0
    x[:, :, 0] = 448.0
    cache = Cache(8, 1, 16, 64)
    store_both(K, cache, x, x, [16 * i for i in range(8)])
    assert bool((cache.ks == 1).all())


def test_grown_twice(K):
    """A block's tokens are stored again under every larger scale, subnormal values
    rounded each time."""
    H, D, bs = 2, 128, 32
    cache = Cache(2, H, bs, D)
    g = torch.Generator().manual_seed(4)
    for t in range(20):
        x = (torch.randn(1, H, D, generator=g) * 4.0 ** (t // 4)).cuda()
        store_both(K, cache, x, x * 3, [bs + t])


def layout(lens, old, bs, blocks, seed, rows=None, spare=3):
    """Tables of requests at scattered rows with scattered blocks, entries behind
    what they hold not of the cache."""
    r = np.random.RandomState(seed)
    n = len(lens)
    rows = rows or n + 2
    wide = max([-(-(a + b) // bs) for a, b in zip(lens, old)] + [1]) + spare
    table = np.full((rows, wide), 1 << 28, np.int32)
    order = r.permutation(blocks)
    at = r.permutation(rows)[:n]
    used = 0
    for i in range(n):
        have = -(-(lens[i] + old[i]) // bs)
        table[at[i], :have] = order[used:used + have]
        used += have
    assert used <= blocks
    return table, at, np.concatenate([[0], np.cumsum(lens)]).astype(int)


def filled(K, table, at, lens, old, blocks, H, bs, D, g, size=1.0, io=F32):
    """Every request's tokens stored in one call."""
    cache = Cache(blocks, H, bs, D)
    slots = [int(table[at[i], p // bs]) * bs + p % bs for i in range(len(lens)) for p in range(lens[i] + old[i])]
    if slots:
        k, v = ((torch.randn(len(slots), H, D, generator=g) * size).to(io).cuda() for _ in range(2))
        K.kv_store(k, v, up(slots), *cache.all())
    return cache


CASES = [   # new lengths, held lengths, query heads, heads, D, block size, io
    ([1], [0], 1, 1, 64, 16, "bf16"),
    ([1], [62], 4, 1, 128, 64, "bf16"),
    ([1, 1, 1], [63, 64, 65], 8, 2, 128, 32, "bf16"),
    ([1, 0, 1, 1], [0, 0, 500, 1], 6, 3, 64, 16, "bf16"),
    ([1, 1], [1000, 130], 16, 1, 128, 128, "bf16"),
    ([1, 1], [700, 10], 40, 2, 64, 64, "bf16"),
    ([4, 4, 4], [100, 3, 259], 4, 4, 64, 16, "bf16"),
    ([3, 0, 5, 1], [64, 10, 250, 300], 8, 2, 128, 64, "bf16"),
    ([7], [2000], 4, 2, 128, 16, "bf16"),
    ([130], [0], 4, 2, 128, 64, "bf16"),
    ([65, 1, 0, 200], [0, 300, 5, 77], 8, 2, 128, 64, "bf16"),
    ([257], [33], 5, 1, 64, 32, "bf16"),
    ([100, 63], [0, 500], 12, 4, 64, 16, "bf16"),
    ([1], [0], 1, 1, 64, 16, "f32"),
    ([1, 1], [300, 64], 8, 2, 128, 64, "f32"),
    ([4, 2], [100, 31], 6, 2, 64, 32, "f32"),
    ([5, 1], [200, 31], 8, 2, 128, 16, "f32"),
    ([90, 0, 35], [10, 0, 140], 6, 3, 64, 128, "f32"),
    ([131], [20], 4, 1, 128, 64, "f32"),
]


@pytest.mark.parametrize("lens,old,Hq,H,D,bs,io", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention(K, lens, old, Hq, H, D, bs, io):
    g = torch.Generator().manual_seed(sum(lens) + sum(old))
    blocks = sum(-(-(a + b) // bs) for a, b in zip(lens, old)) + 5
    table, at, cu = layout(lens, old, bs, blocks, 3)
    cache = filled(K, table, at, lens, old, blocks, H, bs, D, g)
    T = int(cu[-1])
    q = (torch.randn(T, 2 * Hq + 1, D, generator=g) * 2).to(IO[io]).cuda()[:, 1:Hq + 1]
    totals = [a + b for a, b in zip(lens, old)]
    o = K.kv_attention(q, up(cu), up(totals), up(at), up(table), *cache.all())
    ref, tol = R.attention(f64(q), cu, totals, at, table, values(cache.kc), values(cache.vc), f64(cache.ks), f64(cache.vs), D ** -0.5, IO[io])
    R.check("o", o, ref, tol, IO[io])
    again = K.kv_attention(q.contiguous(), up(cu), up(totals), up(at), up(table), *cache.all(), scale=D ** -0.5)
    assert torch.equal(o, again)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("scale,size", [(1.0, 4.0), (1e-6, 1.0), (30.0, 1.0)], ids=["peaked", "flat", "one key"])
def test_scores(K, io, scale, size):
    """Scores of hundreds (one key takes all, the reference is raised again and
    again), and scores near nothing."""
    lens, old, bs, H, D = [40, 1], [300, 500], 32, 2, 64
    g = torch.Generator().manual_seed(5)
    blocks = 40
    table, at, cu = layout(lens, old, bs, blocks, 4)
    cache = filled(K, table, at, lens, old, blocks, H, bs, D, g, size)
    q = (torch.randn(41, 4, D, generator=g) * size).to(IO[io]).cuda()
    totals = [340, 501]
    o = K.kv_attention(q, up(cu), up(totals), up(at), up(table), *cache.all(), scale=scale)
    ref, tol = R.attention(f64(q), cu, totals, at, table, values(cache.kc), values(cache.vc), f64(cache.ks), f64(cache.vs), scale, IO[io])
    R.check("o", o, ref, tol, IO[io])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[5, 1, 1, 3], [70, 1, 33, 90]], ids=["tokens", "prompts"])
def test_nothing_to_see(K, io, lens):
    """Tokens before the first position, requests without anything, padding, rows that
    do not exist, totals beyond the table, missing pages: zeros, or what is left."""
    bs, H, D, Hq = 16, 2, 64, 4
    g = torch.Generator().manual_seed(6)
    old = [40, 20, 30, 50]
    blocks = 60
    table, at, cu = layout(lens, old, bs, blocks, 5, rows=5, spare=0)
    cache = filled(K, table, at, lens, old, blocks, H, bs, D, g)
    table[at[3], 1] = -1          # the tokens 16 .. 31 of the last are nowhere
    table[at[3], 2] = blocks
    at = np.array([at[0], -1, 9, at[3]])
    totals = [lens[0] - 2, 21, 31, 1 << 30]
    reach = table.shape[1] * bs
    table[at[3], -(-(lens[3] + old[3]) // bs):] = -5
    q = torch.randn(int(cu[-1]), Hq, D, generator=g).to(IO[io]).cuda()
    o = K.kv_attention(q, up(cu), up(totals), up(at), up(table), *cache.all())
    # positions past what was stored hold NaN: see only what is there
    host = [values(cache.kc), values(cache.vc), f64(cache.ks), f64(cache.vs)]
    ref, tol = R.attention(f64(q), cu, [lens[0] - 2, 0, 0, reach], at, table, *host, D ** -0.5, IO[io])
    R.check("o", o, ref, tol, IO[io])
    assert not bool(o[:2].any()) and not bool(o[cu[1]:cu[3]].any())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,old", [([6], [130]), ([200], [0]), ([80, 1], [64, 90])], ids=["drafts", "prompt", "mixed"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_tokens_stay_where_they_are(K, io, lens, old, bad):
    """A NaN or infinity in a later token's key or value reaches no earlier token, in
    a value no other channel, in a query no other token."""
    bs, H, D, Hq = 64, 2, 128, 4
    g = torch.Generator().manual_seed(7)
    blocks = 12
    table, at, cu = layout(lens, old, bs, blocks, 6)
    total = lens[0] + old[0]
    cache = filled(K, table, at, lens, old, blocks, H, bs, D, g)
    q = torch.randn(int(cu[-1]), Hq, D, generator=g).to(IO[io]).cuda()
    totals = [a + b for a, b in zip(lens, old)]
    args = (up(cu), up(totals), up(at), up(table))
    want = K.kv_attention(q, *args, *cache.all())
    p = total - 2                                   # seen by the last two tokens of the first request
    j = lens[0] - 2
    slot = int(table[at[0], p // bs]) * bs + p % bs
    code = 0x7f
    kc = cache.kc.clone()
    kc.view(torch.uint8)[slot // bs, 1, slot % bs, 3] = code
    o = K.kv_attention(q, *args, kc, *cache.all()[1:])
    assert bool(o[j:j + 2, 2:].isnan().all())
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[j:j + 2, 2:] = False
    assert torch.equal(o[keep], want[keep])
    vc = cache.vc.clone()
    vc.view(torch.uint8)[slot // bs, 1, 9, slot % bs] = code
    o = K.kv_attention(q, *args, cache.kc, vc, cache.ks, cache.vs)
    assert bool(o[j:j + 2, 2:, 9].isnan().all())
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[j:j + 2, 2:, 9] = False
    assert torch.equal(o[keep], want[keep])
    q2 = q.clone()
    q2[1, 0, 5] = bad
    o = K.kv_attention(q2, *args, *cache.all())
    assert bool(o[1, 0].isnan().all())
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[1, 0] = False
    assert torch.equal(o[keep], want[keep])


def test_empty_calls(K):
    cache = Cache(3, 2, 16, 64)
    none = torch.zeros(0, 4, 64, dtype=BF, device="cuda")
    assert K.kv_attention(none, up([0]), up([]), up([]), up([[0]]), *cache.all()).shape == (0, 4, 64)
    assert K.kv_attention(none, up([0, 0]), up([0]), up([0]), up([[0]]), *cache.all()).shape == (0, 4, 64)
    K.kv_store(none[:, :2], none[:, 2:], up([]), *cache.all())
    assert bool(cache.ks.isnan().all())
