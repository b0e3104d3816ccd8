"""The short causal convolution against a 64-bit token-by-token reference:
prompts (dense and pool mode, strided rows, empty and one-token sequences, tile
borders), one token a request, and the commit of accepted inputs."""
import pytest
import torch

import serve_ref as R

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


def make(seed, T, D, W, dtype, bias=True, wide=0):
    g = torch.Generator().manual_seed(seed)
    row = torch.randn(T, D + wide, generator=g).to(dtype)
    w = (torch.rand(D, W, generator=g) * 2 - 1).to(dtype)
    b = torch.randn(D, generator=g).to(dtype) if bias else None
    return row, w, b, g


def offsets(lens):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
    return cu


RAGGED = [3, 0, 1, 70, 32, 2, 31, 33, 0, 64, 5, 1, 1, 97]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D,wide", [(64, 0), (1, 0), (37, 0), (2056, 24), (264, 3)])
def test_prompts(K, dtype, W, D, wide):
    lens = RAGGED
    T, N = sum(lens), len(lens)
    row, w, b, g = make(W * 100 + D, T, D, W, dtype, bias=W != 3, wide=wide)
    x = row.cuda()[:, :D]
    cu = offsets(lens).cuda()
    bc = None if b is None else b.cuda()
    first = torch.randn(N, W - 1, D, generator=g).to(dtype)
    # dense, from given states
    y, last = K.conv_prefill(x, w.cuda(), bc, cu, initial_state=first.cuda())
    ref, tol, end = R.conv(x, w, b, lens, first)
    R.check("dense", y, ref, tol, dtype)
    assert (R.f64(last) == end).all()
    # dense, from nothing, no final state asked for
    y0, none = K.conv_prefill(x, w.cuda(), bc, cu, output_final_state=False, activation=None)
    ref0, tol0, _ = R.conv(x, w, b, lens, torch.zeros_like(first), activation=False)
    R.check("zeros, no SiLU", y0, ref0, tol0, dtype)
    assert none is None
    # pool: the same values in rows of a pool, others as they were
    slots = N + 6
    pool0 = torch.randn(slots, W - 1, D, generator=g).to(dtype)
    idx = torch.randperm(slots - 1, generator=g)[:N].to(torch.int32)
    idx[4] = -1
    at = torch.from_numpy(R.slots_of(idx, slots)).long()
    pool0[at] = first
    pool = pool0.cuda()
    yr, same = K.conv_prefill(x, w.cuda(), bc, cu, initial_state=pool, state_indices=idx.cuda(), update_pool=False)
    assert same is pool and torch.equal(pool.cpu(), pool0) and torch.equal(yr, y)
    yp, _ = K.conv_prefill(x, w.cuda(), bc, cu, initial_state=pool, state_indices=idx.cuda())
    want = pool0.clone()
    want[at] = last.cpu()
    assert torch.equal(yp, y) and torch.equal(pool.cpu(), want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,D,wide,W", [(1, 8, 0, 4), (5, 4099, 0, 3), (130, 512, 16, 2), (33, 2048, 5, 4)])
def test_tokens(K, dtype, B, D, wide, W):
    row, w, b, g = make(B + D, B, D, W, dtype, wide=wide)
    x = row.cuda()[:, :D]
    slots = B + 3
    pool0 = torch.randn(slots, W - 1, D, generator=g).to(dtype)
    idx = torch.randperm(slots - 1, generator=g)[:B].to(torch.int32)
    idx[-1] = -1
    at = torch.from_numpy(R.slots_of(idx, slots)).long()
    pool = pool0.cuda()
    y = K.conv_decode(x, w.cuda(), b.cuda(), pool, idx.cuda())
    ref, tol, end = R.conv(x, w, b, [1] * B, pool0[at])
    R.check("tokens", y, ref, tol, dtype)
    want = pool0.clone()
    want[at] = torch.from_numpy(end).to(dtype)
    assert torch.equal(pool.cpu(), want)
    # the prompt form over the same tokens gives the same bits
    pool2 = pool0.cuda()
    y2, _ = K.conv_prefill(x, w.cuda(), b.cuda(), offsets([1] * B).cuda(), initial_state=pool2, state_indices=idx.cuda())
    assert torch.equal(y2, y) and torch.equal(pool2, pool)


def test_large_values(K):
    """Sums whose exponential overflows: SiLU's ends are s and -0."""
    x = torch.tensor([[200.0, -200.0, 1e30, -1e30]]).cuda()
    w = torch.zeros(4, 2).cuda()
    w[:, 1] = 1
    y, _ = K.conv_prefill(x, w, None, offsets([1]).cuda())
    assert torch.equal(y, torch.tensor([[200.0, 0.0, 1e30, 0.0]]).cuda())


@pytest.mark.parametrize("dtype,D", [(BF, 520), (F32, 33)])
def test_commit(K, dtype, D):
    W, lens = 4, [4, 1, 0, 6, 2, 3, 5]
    steps = [3, 0, -1, 2, 1, 3, -5]          # the sixth is beyond its request: left as it is
    row, _, _, g = make(3, sum(lens), D, W, dtype, wide=8)
    x = row.cuda()[:, :D]
    slots = 12
    pool0 = torch.randn(slots, W - 1, D, generator=g).to(dtype)
    idx = torch.tensor([5, 2, 9, 0, -1, 3, 7], dtype=torch.int32)
    pool = pool0.cuda()
    K.conv_commit(x, offsets(lens).cuda(), torch.tensor(steps, dtype=torch.int32).cuda(), pool, idx.cuda())
    want, t = pool0.clone(), 0
    for n, (L, s) in enumerate(zip(lens, steps)):
        a = int(R.slots_of(idx, slots)[n])
        if 0 <= s < L:
            want[a] = torch.cat([pool0[a], row[t:t + s + 1, :D]])[-(W - 1):]
        t += L
    assert torch.equal(pool.cpu(), want)


def test_empty_calls(K):
    w = torch.zeros(16, 4, device="cuda")
    x = torch.zeros(0, 16, device="cuda")
    y, last = K.conv_prefill(x, w, None, offsets([]).cuda())
    assert y.shape == (0, 16) and last.shape == (0, 3, 16)
    first = torch.randn(2, 3, 16, device="cuda")
    y, last = K.conv_prefill(x, w, None, offsets([0, 0]).cuda(), initial_state=first)
    assert torch.equal(last, first)
    assert K.conv_decode(x, w, None, first, torch.zeros(0, dtype=torch.int32, device="cuda")).shape == (0, 16)
