"""Further refusals of the convolution, scan, verification and commit that need
no GPU: through the C ABI with fake, never dereferenced addresses, and through
the binding with host tensors."""
import ctypes

import pytest
import torch

import gated_delta_rule_51_amd as kda
from test_serve_abi import ALIAS, ALIGN, L, fake, ssm, ssm_desc  # noqa: F401  (L: fixture)


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


def no_heads(device):
    """A pool and a step cache of states without heads, whose pitch in steps
    would be a division by zero."""
    pool, cache = torch.zeros(4, 0, 64, 64, device=device), torch.zeros(2, 2, 0, 64, 64, device=device)
    return pool, cache.as_strided((2, 2, 0, 64, 64), (0, 0, 64 * 64, 64, 1)), torch.zeros(2, dtype=torch.int32, device=device)


def test_commit_of_no_heads():
    pool, cache, idx = no_heads("cpu")
    with pytest.raises(ValueError, match="heads and rows"):
        kda.commit_states(pool, idx, cache, idx)


@pytest.mark.gpu
def test_commit_of_no_heads_natively():
    pool, cache, idx = no_heads("cuda")
    assert kda._native().commit_states(0, pool, idx, cache, idx) is None
    with pytest.raises(ValueError, match="heads and rows"):
        kda.commit_states(pool, idx, cache, idx)


def test_scan_z_rows_of_whole_words(L):  # noqa: F811
    """Rows of z need not start on 16 bytes, as beside [T, H] steps of any H in
    one projection: such a call passes that check and gets to the next one."""
    for io, stride, want in ((1, 258, ALIAS), (1, 266, ALIAS), (1, 259, ALIGN), (0, 257, ALIAS)):
        assert ssm(L, ssm_desc(io_dtype=io, z_stride=stride), y=fake(7, 512)) == want, (io, stride)


def test_empty_sizes_are_named():
    """What the native call declines for its sizes is named, not called a tensor
    of a strange kind."""
    i32, z = torch.int32, torch.zeros
    cu, idx = torch.tensor([0, 4], dtype=i32), z(4, dtype=i32)
    x, X = z(4, 8), z(4, 2, 32)
    for call, msg in (
            (lambda: kda.conv_prefill(x, z(8, 0), None, cu), "2 to 4 taps"),
            (lambda: kda.conv_decode(x, z(8, 5), None, z(2, 4, 8), idx), "2 to 4 taps"),
            (lambda: kda.ssm_prefill(z(4, 0, 32), z(4, 0), z(0), z(4, 1, 32), z(4, 1, 32), cu), "must have heads"),
            (lambda: kda.ssm_decode(X, z(4, 2), z(2), z(4, 1, 0), z(4, 1, 0), z(5, 2, 32, 0), idx), "must have heads"),
            (lambda: kda.ssm_prefill(X, z(4, 2), z(2), z(4, 0, 32), z(4, 0, 32), cu), "must have heads"),
            (lambda: kda.verify_drafts(idx, z(4, 0), cu, z(4), z(1)), "vocabulary")):
        with pytest.raises(ValueError, match=msg):
            call()
