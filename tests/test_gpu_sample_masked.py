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


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("v,allowed", [(9000, 20), (40000, 1), (40000, 300), (131072, 20)])
def test_masked(K, io, v, allowed):
    """Fewer tokens allowed than top_k takes: the k-th lies among the masked ones, which
    weigh nothing."""
    g = torch.Generator().manual_seed(v + allowed)
    n = 3
    x = torch.full((n, v), -INF)
    for i in range(n):
        at = torch.randperm(v, generator=g)[:allowed]
        x[i, at] = torch.randn(allowed, generator=g) * 3
    x, u = x.to(IO[io]).cuda(), torch.tensor([0.0, 0.37, 1 - 2.0 ** -24], device="cuda")
    both(K, x, u)
    both(K, x, u, k=[50, 1000, 2000])
    both(K, x, u, k=[50] * n, p=[0.9, 0.5, 1.0], t=[0.7, 1.0, 3.0])
    both(K, x, u, k=[4000, 1, 30], m=[0.1, 0.0, 1e-6])
    both(K, x, u, p=[0.95] * n, t=[0.3, 1.5, 1.0])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_flat(K, io):
    """High temperatures and small logits: nearly equal weights, cuts far down."""
    g = torch.Generator().manual_seed(9)
    n, v = 3, 50000
    x, u = (torch.randn(n, v, generator=g)).to(IO[io]).cuda(), torch.rand(n, generator=g).cuda()
    t = [5.0, 20.0, 100.0]
    both(K, x, u, t=t, p=[0.9, 0.5, 0.99])
    both(K, x, u, t=t, k=[20000, 1000, 49999], p=[0.9, 0.5, 0.7])
    both(K, x, u, t=t, m=[0.5, 0.9, 0.97], k=[1000, 30000, 700])
