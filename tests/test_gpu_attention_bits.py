"""Single tokens and runs of drafts in bf16 keep 16 bits of softmax's numerators: only
the output is rounded to bf16.

The bound is paged_ref.attention's with the numerators' rounding replaced: as the sum
of two bf16 terms each is off by at most 2^-16, and their sum is formed in fp32 from
what is not rounded, so sum p |v| / sum p is the only factor."""
import numpy as np
import pytest
import torch

import paged_ref as R
from test_gpu_kv import f64, filled, layout, up, values

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


def bound(q, cu, totals, at, table, host, scale):
    """fp32's part of paged_ref.attention's bound, and the two terms'."""
    ref, tol = R.attention(q, cu, totals, at, table, *host, scale, F32)
    # of fp32 io the bound has 4 e sum p |v| / sum p for three terms: here 2^-16
    flat = [np.abs(host[1])] + list(host[2:])
    spread, _ = R.attention(q, cu, totals, at, table, host[0], *flat, scale, F32)
    return ref, tol + 2.0 ** -16 * spread


CASES = [   # new lengths, held lengths, query heads, heads, D, block size
    ([1, 1, 1], [7, 15, 3], 8, 2, 128, 16),
    ([1, 1], [40, 900], 16, 1, 64, 64),
    ([1], [3000], 4, 1, 128, 128),
    ([4, 4, 3], [0, 9, 100], 8, 2, 128, 32),          # two column tiles for some
    ([5, 6], [10, 70], 16, 4, 64, 16),
    ([7, 8], [2, 30], 4, 1, 128, 64),
    ([8, 8], [2, 600], 12, 3, 64, 64),
]


@pytest.mark.parametrize("lens,old,Hq,H,D,bs", CASES, ids=[str(i) for i in range(len(CASES))])
def test_numerators(K, lens, old, Hq, H, D, bs):
    g = torch.Generator().manual_seed(sum(old))
    blocks = sum(-(-(a + b) // bs) for a, b in zip(lens, old)) + 2
    table, at, cu = layout(lens, old, bs, blocks, 11)
    cache = filled(K, table, at, lens, old, blocks, H, bs, D, g)
    q = (torch.randn(int(cu[-1]), Hq, D, generator=g) * 0.3).to(BF).cuda()
    totals = [a + b for a, b in zip(lens, old)]
    o = K.kv_attention(q, up(cu), up(totals), up(at), up(table), *cache.all())
    host = [np.nan_to_num(values(cache.kc)), np.nan_to_num(values(cache.vc)), np.nan_to_num(f64(cache.ks)), np.nan_to_num(f64(cache.vs))]
    ref, tol = bound(f64(q), cu, totals, at, table, host, D ** -0.5)
    R.check("o", o, ref, tol, BF)
