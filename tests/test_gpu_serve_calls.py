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
