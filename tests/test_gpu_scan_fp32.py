"""fp32 io stays fp32 in every form of the scan: the whole output against 64
bits, by its norm, on inputs of ordinary size.

Bound of the relative 2-norm.  A value is a sum of at most n = S + 64 + 2
products (prompts; S + 1 for tokens), the matrix cores may truncate, so one
addition is off by up to d = 2^-23 of the partial sum.  With terms of random
sign the partial sums grow with the root of their number: the errors add up to
d sqrt(n / 6) of the sum's size where they are independent and to
(d / 2) sqrt(n / 3) where they all go one way: for n = 194 5.7 d and 4.0 d, of
which rounding to nearest takes half.  The softplus, the exponential and its
argument add up to 4 d to each term, independently: 2.3 d.  Together below
sqrt(5.7^2 + 4^2 + 2.3^2) d = 7.4 d = 8.8e-7.  Operands of 17 bits are off by
2^-17 / sqrt(3) = 4.4e-6 each, those of 16 and fewer by more."""
import numpy as np
import pytest
import torch

import gated_delta_rule_51_amd as kda
import serve_ref as R
from test_gpu_ssm import Layer, offsets, states

pytestmark = pytest.mark.gpu
F32, I32 = torch.float32, torch.int32
MOST = 7.4 * 2.0 ** -23


def off(name, got, want):
    got = R.f64(got)
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    print("%s: rel-L2 %.3e" % (name, rel), flush=True)
    assert rel <= MOST, name


@pytest.mark.parametrize("P,S", [(32, 32), (32, 128), (64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens", [[300, 64, 0, 1, 77], [1] * 40], ids=["lengths", "ones"])
def test_fp32(P, S, lens):
    H, G, T, N = 6, 3, sum(lens), len(lens)
    m = Layer(P * 3 + S, T, H, P, S, G, F32)
    first = states(m, N, F32)
    ref = m.ref(lens, first)
    some = [n for n, length in enumerate(lens) if length]
    y, last = kda.ssm_prefill(*m.args, offsets(lens), initial_state=first.cuda(), **m.kw)
    off("prompt", y, ref["y"])
    off("prompt states", last[some], ref["last"][some])
    idx, pool = torch.arange(N, dtype=I32, device="cuda"), torch.cat([first, first[:1]]).cuda()
    cache = torch.zeros(N, 80, H, P, S, device="cuda") if T < 1000 and P * S < 8192 else None
    y = kda.ssm_decode_multi(*m.args, offsets(lens), pool, idx, intermediate_states=cache, **m.kw)
    off("run", y, ref["y"])
    off("run states", pool[some], ref["last"][some])
    if cache is not None:
        off("run steps", torch.cat([cache[n, :lens[n]] for n in some]), np.concatenate([np.stack(ref["steps"][n][:80]) for n in some]))
    if max(lens) == 1:
        pool = torch.cat([first, first[:1]]).cuda()
        off("token", kda.ssm_decode(*m.args, pool, idx, **m.kw), ref["y"])
        off("token states", pool[:N], ref["last"])
