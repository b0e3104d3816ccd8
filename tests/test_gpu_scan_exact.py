"""The scan where fp32 arithmetic is exact: inputs whose products and sums are
whole numbers (times one power of 2) that fit 24 bits, while the state, or the
factors between two tokens, need 20.  A kernel that holds those in fp32, or
splits them without loss, gives the 64-bit result rounded once; one that keeps
17 bits of them is off by far more than that, as the large parts cancel in y.
So the tolerance is zero."""
import pytest
import torch

import gated_delta_rule_51_amd as kda

pytestmark = pytest.mark.gpu
F32, BF, I32 = torch.float32, torch.bfloat16, torch.int32
HIGH, MIDDLE = 173 << 12, 107 << 4   # whole numbers of 8 bits, so bf16 values; with an odd number added they make 20 bits
SHAPES = [(32, 32), (32, 64), (32, 128), (64, 32), (64, 64), (64, 128), (128, 32), (128, 64), (128, 128)]
LENS = [1, 64, 0, 65, 700, 3]


def offsets(lens):
    cu = torch.zeros(len(lens) + 1, dtype=I32)
    cu[1:] = torch.tensor(lens, dtype=I32).cumsum(0)
    return cu.cuda()


def odd(g, *shape):
    return torch.randint(-64, 64, shape, generator=g).double() * 2 + 1


def calls(args, kw, lens, first):
    """y and the last states of the prompt form and of runs of tokens, and of
    one token a request where every length is 1."""
    cu, n = offsets(lens), len(lens)
    yield "prompt", *kda.ssm_prefill(*args, cu, initial_state=first.cuda(), **kw)
    idx = torch.arange(n, dtype=I32, device="cuda")
    pool = torch.cat([first, first[:1]]).cuda()
    yield "run", kda.ssm_decode_multi(*args, cu, pool, idx, **kw), pool[:n]
    if all(x == 1 for x in lens):
        pool = torch.cat([first, first[:1]]).cuda()
        yield "token", kda.ssm_decode(*args, pool, idx, **kw), pool[:n]


def same(name, got, want, dtype):
    """got equals the 64-bit values rounded to dtype."""
    want = want.to(dtype).double()
    off = (got.cpu().double() - want).abs()
    print("%s: %d of %d off, most %.3g" % (name, int((off != 0).sum()), off.numel(), float(off.max()) if off.numel() else 0.0), flush=True)
    assert torch.equal(got.cpu().double(), want), name


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("P,S", SHAPES)
@pytest.mark.parametrize("lens", [LENS, [1] * 5], ids=["lengths", "ones"])
def test_state_against_c(io, P, S, lens):
    """Steps of zero keep the state as it is; C takes the difference of two
    pairs of its columns, whose common part of 20 to 22 bits cancels."""
    g = torch.Generator().manual_seed(P + S)
    H, G, T, N = 6, 2, sum(lens), len(lens)
    first = ((HIGH + MIDDLE) * torch.randint(1, 4, (N, H, P, 1), generator=g) + odd(g, N, H, P, S)).to(F32)
    C = torch.zeros(T, G, S)
    for k, v in enumerate((1.0, 1.0, -1.0, -1.0)):
        C.scatter_add_(2, torch.randint(0, S // 4, (T, G, 1), generator=g) + k * (S // 4), torch.full((T, G, 1), v))
    x, B = torch.randint(-9, 9, (T, H, P), generator=g), torch.randint(-9, 9, (T, G, S), generator=g)
    D = torch.randint(-3, 4, (H,), generator=g).float()
    args = (x.to(io).cuda(), torch.full((T, H), -300.0, dtype=io).cuda(), torch.zeros(H).cuda(), B.to(io).cuda(), C.to(io).cuda())
    seq = torch.repeat_interleave(torch.arange(N), torch.tensor(lens))
    want = D.double()[:, None] * x
    for t in range(T):
        want[t] += (first[seq[t]].double() * C[t].double().repeat_interleave(H // G, 0)[:, None]).sum(-1)
    for name, y, last in calls(args, dict(D=D.cuda()), lens, first):
        same(name, y, want, io)
        same(name + " states", last, first.double(), F32)


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("P,S", SHAPES)
def test_tokens_against_tokens(io, P, S):
    """Steps of 64 without any decay: C_t . B_s has 20 bits, and x changes its
    sign from token to token, so that the large parts cancel."""
    g = torch.Generator().manual_seed(P * S)
    H, G, T, N = 6, 2, sum(LENS), len(LENS)
    at = torch.stack([torch.randperm(S, generator=g)[:3] for _ in range(G)])      # three columns of each group
    B, C = torch.zeros(T, G, S), torch.zeros(T, G, S)
    for k in range(G):
        B[:, k, at[k, 0]], B[:, k, at[k, 1]], B[:, k, at[k, 2]] = HIGH, MIDDLE, odd(g, T).float()
        C[:, k, at[k]] = 1
    sign = (1 - 2 * (torch.arange(T) % 2)).double()
    x = sign[:, None, None] * (1 - 2 * torch.randint(0, 2, (1, H, P), generator=g)).double()
    D = torch.randint(-3, 4, (H,), generator=g) * 64.0
    args = (x.to(io).cuda(), torch.full((T, H), 64.0, dtype=io).cuda(), torch.full((H,), -200.0).cuda(), B.to(io).cuda(), C.to(io).cuda())
    first = torch.zeros(N, H, P, S)
    Bh, Ch = B.double().repeat_interleave(H // G, 1), C.double().repeat_interleave(H // G, 1)
    want, ends = torch.zeros(T, H, P, dtype=torch.float64), torch.zeros(N, H, P, S, dtype=torch.float64)
    t = 0
    for n, length in enumerate(LENS):
        for _ in range(length):
            ends[n] += 64 * x[t][:, :, None] * Bh[t][:, None]
            want[t] = (ends[n] * Ch[t][:, None]).sum(-1) + D.double()[:, None] * x[t]
            t += 1
    for name, y, last in calls(args, dict(D=D.cuda()), LENS, first):
        same(name, y, want, io)
        same(name + " states", last, ends, F32)


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("P,S", [(32, 64), (64, 64), (128, 128)])
def test_largest_values(io, P, S):
    """States, factors between tokens and weighted inputs between bf16's largest
    value and fp32's: finite results stay finite."""
    top, small = 3.4e38, 2.0 ** -100
    H, T, N = 4, 70, 1
    x, B, C = torch.zeros(T, H, P), torch.zeros(T, 1, S), torch.zeros(T, 1, S)
    first = torch.zeros(N, H, P, S)
    first[:, :, :, 1] = top
    C[:, :, 1] = small                # y takes the large state, made small
    x[5], B[5, :, 2] = 2.0 ** 127, small  # a weighted x of 2^127 step, made small in the state
    step = 1.9985                     # (as bf16: 2; so of a bias that is fp32)
    args = (x.to(io).cuda(), torch.zeros(T, H, dtype=io).cuda(), torch.full((H,), -200.0).cuda(), B.to(io).cuda(), C.to(io).cuda())
    bias = torch.full((H,), step).double().expm1().log().float()
    real = bias.double().exp().log1p()
    assert float(real[0]) * 2.0 ** 127 > float(torch.finfo(BF).max)
    want = torch.full((T, H, P), float(torch.tensor(top)) * small, dtype=torch.float64)
    ends = first.double()
    ends[:, :, :, 2] += (real[:, None] * 2.0 ** 127 * small)
    for name, y, last in calls(args, dict(dt_bias=bias.cuda()), [T], first):
        off = (y.cpu().double() / want - 1).abs().max()
        end = ((last.cpu().double() - ends).abs() / ends.abs().clamp_min(1.0)).max()
        print("%s: y off by %.3g, states by %.3g" % (name, float(off), float(end)), flush=True)
        # y: one product and its rounding; the states: softplus to 4 units of fp32 and three roundings
        assert float(off) <= 2.0 ** -22 + torch.finfo(io).eps / 2 and float(end) <= 2.0 ** -20
