"""Further refusals of the convolution, scan, verification and commit that need
no GPU: through the C ABI with fake, never dereferenced addresses, and through
the binding with host tensors."""
import ctypes

import pytest
import torch

import gated_delta_rule_51_amd as kda
from test_serve_abi import ALIAS, L, fake, ssm, ssm_desc  # noqa: F401  (L: fixture)


@pytest.mark.parametrize("name", ["x", "dt", "A", "B", "C", "D", "z", "bias", "cu", "state", "final", "y"])
def test_scan_workspace_overlaps_nothing(L, name):  # noqa: F811
    """A prompt cut into segments writes its workspace before it has read its
    inputs again."""
    long = ssm_desc(num_seqs=1, total_tokens=100000)
    need = L.kda_ssm_prefill_workspace_size(ctypes.byref(long))
    assert need > 1 << 20
    for at in (0, need - 16):
        assert ssm(L, long, ws=fake(20), n=need, **{name: fake(20, at)}) == ALIAS, name
    pool = dict(idx=fake(13), state=fake(14), final=None)
    assert ssm(L, long, ws=fake(20), n=need, **dict(pool, idx=fake(20, 64))) == ALIAS
    assert ssm(L, long, ws=fake(20), n=need, **dict(pool, state=fake(20, 4096))) == ALIAS
