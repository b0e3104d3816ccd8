"""Calls of the convolution, scan, verification and commit that the documentation
allows and that the other tests do not make."""
import ctypes

import pytest
import torch

import gated_delta_rule_51_amd as kda
from test_gpu_ssm import Layer, offsets, states

pytestmark = pytest.mark.gpu
F32, BF, I32 = torch.float32, torch.bfloat16, torch.int32


@pytest.mark.parametrize("P,S", [(32, 32), (64, 128), (128, 64)])
@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("given", [True, False])
def test_no_tokens_and_no_arrays(io, P, S, given):
    """Sequences without any token: the states are copied (or zeros), and
    neither the tokens' arrays nor A_log are read."""
    N, H = 3, 2
    first = torch.randn(N, H, P, S, device="cuda") if given else None
    last = torch.full((N, H, P, S), 7.0, device="cuda")
    cu = torch.zeros(N + 1, dtype=I32, device="cuda")
    d = kda.SsmDesc(N, 0, H, 1, P, S, io, 0, 0, 0, 0, 0, H * P, H, S, S, H * P)
    status = kda.lib().kda_ssm_prefill(ctypes.byref(d), *[None] * 8, cu.data_ptr(), first.data_ptr() if given else None, None,
                                       last.data_ptr(), None, None, 0, torch.cuda.current_stream().cuda_stream)
    assert status == 0
    assert torch.equal(last, first if given else torch.zeros_like(last))


@pytest.mark.parametrize("P,S", [(32, 128), (64, 64), (128, 32)])
@pytest.mark.parametrize("io,wide", [(BF, 10), (BF, 2), (F32, 5), (F32, 10)])
def test_z_from_a_projection(io, wide, P, S):
    """z is read in place from rows [z | dt] of a projection with any number of
    heads, whose rows start on words, not on 16 bytes: the bits of a copy."""
    H, lens = 10, [200, 0, 1, 700, 66]
    T, N = sum(lens), len(lens)
    m = Layer(P + wide, T, H, P, S, 2, io)
    proj = torch.randn(T, H * P + wide, generator=m.g).to(io).cuda()
    z = proj[:, :H * P].unflatten(1, (H, P))
    first, cu = states(m, N + 1, F32), offsets(lens)
    idx = torch.arange(N, dtype=I32, device="cuda")

    def run(z):
        kw = dict(m.kw, z=z)
        y, last = kda.ssm_prefill(*m.args, cu, initial_state=first[:N].cuda(), **kw)
        pool, one = first.cuda(), first.cuda()
        x, dt, A, B, C = m.args
        return (y, last, kda.ssm_decode_multi(*m.args, cu, pool, idx, **kw), pool,
                kda.ssm_decode(x[:N], dt[:N], A, B[:N], C[:N], one, idx, **dict(kw, z=z[:N])), one)

    for a, b in zip(run(z), run(z.contiguous())):
        assert torch.equal(a, b)


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
def test_rate_beyond_fp32(io):
    """A rate of e^89, above fp32's largest, and steps that are zero in fp32: the
    decay is 1 (the exponent is below 1e-45), and after a step of 1 it is 0."""
    H, P, S = 8, 32, 32      # a row of dt is 16 bytes or more, so that every one starts on 16
    x, B = torch.ones(3, H, P, dtype=io, device="cuda"), torch.ones(3, 1, S, dtype=io, device="cuda")
    dt = torch.tensor([-200.0, -200.0, 40.0], device="cuda").to(io)[:, None].expand(3, H).contiguous()
    A = torch.full((H,), 89.0, device="cuda")
    first = torch.randn(1, H, P, S, device="cuda")
    idx = torch.zeros(1, dtype=I32, device="cuda")
    for lens in ([2], [3]):
        n = lens[0]
        cut = (x[:n], dt[:n], A, B[:n], B[:n])
        want = first if n == 2 else torch.full_like(first, 40.0)
        _, last = kda.ssm_prefill(*cut, offsets(lens), initial_state=first)
        pool, one = first.clone(), first.clone()
        kda.ssm_decode_multi(*cut, offsets(lens), pool, idx)
        for t in range(n):
            kda.ssm_decode(x[t:t + 1], dt[t:t + 1], A, B[t:t + 1], B[t:t + 1], one, idx)
        assert torch.equal(last, want) and torch.equal(pool, want) and torch.equal(one, want)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_one_bad_input(bad):
    """An infinity or NaN in x at one token spoils its column from that token's
    32 on, not the tokens before, nor other columns or sequences."""
    H, P, S, lens, at = 2, 64, 64, [200, 50], 101
    m = Layer(9, sum(lens), H, P, S, 1, BF)
    want, ends = kda.ssm_prefill(*m.args, offsets(lens), **m.kw)
    x = m.args[0].clone()
    x[at, 1, 5] = bad
    y, last = kda.ssm_prefill(x, *m.args[1:], offsets(lens), **m.kw)
    assert not bool(y[at:200, 1, 5].isfinite().any())
    some = torch.ones_like(y, dtype=torch.bool)
    some[at // 32 * 32:200, 1, 5] = False
    assert torch.equal(y[some], want[some])
    ok = torch.ones_like(last, dtype=torch.bool)
    ok[0, 1, 5] = False
    assert torch.equal(last[ok], ends[ok])
