"""Calls of the convolution, scan, verification and commit that the documentation
allows and that the other tests do not make."""
import ctypes

import pytest
import torch

import gated_delta_rule_51_amd as kda

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
