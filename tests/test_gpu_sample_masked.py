"""Rows masked with minus infinity, as guided decoding makes them, and rows so flat that
a cut's bin holds thousands of logits: the ways through a whole row."""
import pytest
import torch

from test_gpu_sample import IO, both

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


TOPS = [1e-30, 0.02, 0.3, 0.7, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 8.0, 100.0, 1e10, -0.0, -0.5, -1.5, -3.0, -6.0, -1e30]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("mask", ["infinite", "lowest"])
@pytest.mark.parametrize("v", [400, 3000, 6000])
def test_largest_logit_of_any_size(K, v, mask, io):
    """Masks at the end of the numbers and a largest logit in any octave: what is left
    of the numbers between them is cut into pieces again and again."""
    g = torch.Generator().manual_seed(v)
    n = len(TOPS)
    low = -INF if mask == "infinite" else torch.finfo(IO[io]).min
    x = torch.full((n, v), low)
    for i, top in enumerate(TOPS):
        at = torch.randperm(v, generator=g)[:12]
        x[i, at] = top - torch.rand(12, generator=g) * abs(top)
        x[i, at[5]] = top
    x, u = x.to(IO[io]).cuda(), torch.rand(n, generator=g).cuda()
    both(K, x, u, k=[300] * n)
    both(K, x, u, k=[v - 50] * n, p=[0.9] * n)
    both(K, x, u, p=[0.999] * n, t=[1e30] * n)
