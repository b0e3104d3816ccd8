"""top_k as large as the number of logits in the leading bins: the cut lies between two
bins, and what follows is not kept."""
import pytest
import torch

from test_gpu_sample import IO, both

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("k", [3, 255, 256, 257, 300, 1000, 1024, 1025, 3000])
def test_gap_behind_the_last_kept(K, k, io):
    """k logits near the top, the others a step below, in numbers of either sign."""
    v, n = 4500, 4
    g = torch.Generator().manual_seed(k)
    x = torch.zeros(n, v)
    for i, (high, low) in enumerate([(5.0, 3.0), (0.5, -0.5), (-1.0, -4.0), (300.0, 299.0)]):
        x[i] = low - torch.rand(v, generator=g) * 0.01
        x[i, torch.randperm(v, generator=g)[:k]] = high
    x, u = x.to(IO[io]).cuda(), torch.tensor([0.0, 0.3, 0.9, 1 - 2.0 ** -24], device="cuda")
    for kk in (k - 1, k, k + 1):
        both(K, x, u, k=[kk] * n)
        both(K, x, u, k=[kk] * n, t=[0.5, 1.0, 2.0, 0.1])
        both(K, x, u, k=[kk] * n, m=[1e-9, 0.5, 1e-3, 0.0])
        both(K, x, u, k=[kk] * n, p=[0.99, 1.0, 0.5, 0.999])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("v", [257, 300, 1014, 2052, 4096])
def test_all_but_a_few(K, v, io):
    """top_k from a few below the vocabulary on."""
    n = 8
    g = torch.Generator().manual_seed(v)
    x, u = (torch.randn(n, v, generator=g) * 3).to(IO[io]).cuda(), torch.rand(n, generator=g).cuda()
    both(K, x, u, k=[v - 1 - i for i in range(n)])
    both(K, x, u, k=[v // 2 + 7 * i for i in range(n)], m=[1e-4] * n)
    x = (x * 2).round() / 2
    both(K, x, u, k=[v - 1 - i for i in range(n)])
