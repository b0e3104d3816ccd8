"""The next token against the definition in 64 bits: every limit alone and
together, types, odd and large vocabularies, ties, infinities and NaN, rows cut
out of wider ones."""
import numpy as np
import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu
F32, BF, I32 = torch.float32, torch.bfloat16, torch.int32
IO = {"bf16": BF, "f32": F32}


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


def cuda(a, dtype=F32):
    return None if a is None else torch.tensor(a, dtype=dtype, device="cuda")


def both(K, x, u, t=None, k=None, p=None, m=None):
    """Tokens are equal; a probability is rounded once, its 64-bit sum holds to
    2^-28 (2^-46 a weight), and it is 0 exactly where the definition's is (or where
    that is below the least weight, 2^-40 of the largest)."""
    one = lambda a: None if a is None else [float(torch.tensor(y, dtype=F32)) for y in a]  # noqa: E731
    want, probs = R.sample(x.detach().cpu().double().numpy(), u.cpu().double().numpy(), one(t), k, one(p), one(m))
    kw = dict(temperature=cuda(t), top_k=cuda(k, I32), top_p=cuda(p), min_p=cuda(m))
    tokens, got = K.sample_tokens(x, u, return_probs=True, **kw)
    assert tokens.tolist() == want
    assert torch.equal(K.sample_tokens(x, u, **kw), tokens) and torch.equal(K.token_probs(x, **kw), got)
    got = got.cpu().double().numpy()
    off = np.abs(got - probs) - probs * (2.0 ** -24 + 2.0 ** -27)
    assert off.max() <= 2.0 ** -40 * probs.max(), off.max()
    assert not ((got > 0) & (probs == 0)).any()


def logits(n, v, io, seed, size=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, v, generator=g) * size).to(IO[io]).cuda(), torch.rand(n, generator=g).cuda()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("v", [1, 2, 17, 63, 64, 65, 257, 1000, 5000, 32001, 70000])
def test_limits(K, io, v):
    n = 6
    x, u = logits(n, v, io, v)
    t = [0.0, 0.5, 0.7, 1.0, 1.3, 5.0]
    k = [0, 1, 5, 50, 200, v]
    p = [0.1, 0.9, 0.95, 1.0, 0.0, 0.999]
    m = [0.0, 0.1, 0.5, 1.0, 0.01, 2.0]
    both(K, x, u)
    both(K, x, u, t=t)
    both(K, x, u, k=k)
    both(K, x, u, p=p)
    both(K, x, u, m=m)
    both(K, x, u, t=t, k=k[::-1], p=p, m=m)
    both(K, x, u, t=t[::-1], k=k, p=p[::-1])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_ties(K, io):
    """Equal logits are taken by rising index: all of a row, a few values over and
    over, both zeros, in numbers above and below what one list of a bin holds."""
    n, v = 5, 9000
    g = torch.Generator().manual_seed(1)
    x = torch.zeros(n, v)
    x[1] = torch.randint(-3, 3, (v,), generator=g).float()
    x[2, ::2] = -0.0
    x[3] = torch.randint(0, 2, (v,), generator=g).float() * 1e-3 + 5
    x[4, 4000:] = 1.0
    x, u = x.to(IO[io]).cuda(), torch.rand(n, generator=g).cuda()
    for k in (1, 7, 4096, 4097, 8999):
        both(K, x, u, k=[k] * n)
    for p in (1e-4, 0.3, 0.5, 0.99):
        both(K, x, u, p=[p] * n)
        both(K, x, u, k=[5000] * n, p=[p] * n)
        both(K, x, u, p=[p] * n, m=[0.2] * n)
    both(K, x, u, m=[0.5] * n)
    both(K, x, u, k=[3000] * n, m=[0.9] * n)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_odd_logits(K, io):
    """Infinities, NaN, rows without any logit, numbers of every size."""
    inf, nan, v = float("inf"), float("nan"), 700
    x, u = logits(9, v, io, 2)
    x[0] = -inf
    x[1] = nan
    x[2, 5:] = -inf
    x[3, 100], x[3, 300] = inf, inf
    x[4, ::3] = nan
    x[5] *= 1e30
    x[6] *= 1e-30
    x[7, 1:] = nan
    x[8, :350] = -inf
    both(K, x, u)
    both(K, x, u, t=[0.0] * 9)
    both(K, x, u, k=[400] * 9, p=[0.8] * 9)
    both(K, x, u, m=[0.05] * 9)
    both(K, x, u, k=[30] * 9, m=[0.3] * 9)
    both(K, x, u, p=[0.9] * 9, m=[1e-9] * 9)
    both(K, x, u, t=[1e-20, 1e-20, 1e30, 1.0, 1e-3, 1e25, 1e-38, 1e-20, 3e38], p=[0.9] * 9)


def test_random_numbers_at_the_ends(K):
    """u of 0 gives the first token with weight, the largest below 1 the last."""
    x, _ = logits(4, 5000, "f32", 3)
    x[:, :10], x[:, -7:] = -float("inf"), -float("inf")
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 0.5, 0.25], device="cuda")
    both(K, x, u)
    both(K, x, u, k=[3] * 4)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_of_a_wider_tensor(K, io):
    """Rows apart, and rows that start anywhere."""
    x, u = logits(4, 3001, io, 4)
    both(K, x[:, 1:2900], u, k=[30] * 4, p=[0.9] * 4)
    both(K, x[1:, 7:40], u[1:], p=[0.9] * 3)


@pytest.mark.parametrize("io,v", [("f32", 131072), ("bf16", 151111), ("bf16", 1 << 20)])
def test_large(K, io, v):
    x, u = logits(2, v, io, 5)
    both(K, x, u, t=[0.8, 1.2], p=[0.9, 0.99])
    both(K, x, u, k=[50, 5000], p=[0.9, 0.99])
    both(K, x, u, k=[2000, 1025], m=[0.01, 1e-3])
    both(K, x, u, k=[1024, 700], p=[0.999, 1.0], m=[1e-4, 0.0])


def test_many_rows_alike(K):
    """Rows do not disturb each other, and a call gives what the call before gave."""
    x, u = logits(600, 2000, "bf16", 6)
    x, u = x[:200].repeat(3, 1), u[:200].repeat(3)
    p = torch.full((600,), 0.9, device="cuda")
    tokens, probs = K.sample_tokens(x, u, top_p=p, return_probs=True)
    assert torch.equal(tokens[:200], tokens[200:400]) and torch.equal(probs[:200], probs[400:])
    for _ in range(3):
        assert torch.equal(K.sample_tokens(x, u, top_p=p), tokens)


def test_empty(K):
    none = torch.zeros(0, 50, device="cuda")
    assert K.sample_tokens(none, none[:, 0].contiguous()).shape == (0,)
    assert K.token_probs(none).shape == (0, 50)
