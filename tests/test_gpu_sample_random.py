"""Random rows of every kind under random limits against the definition in 64 bits:
stretches of masked, missing and lowest logits over whole parts of a row, values over
and over, steps, infinities, any temperature."""
import random

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


def row(r, g, v, io):
    x = torch.randn(v, generator=g) * r.choice([0.01, 1.0, 3.0, 20.0]) + r.choice([0.0, 5.0, -40.0, 300.0])
    for _ in range(r.randint(0, 4)):
        lo = r.randrange(v)
        hi = min(v, lo + r.choice([1, 5, v // 20 + 1, v // 3 + 1, v]))
        if lo == 0 and hi == v:
            lo = 1
        kind = r.choice(["mask", "mask", "nan", "lowest", "equal", "steps", "sparse"])
        if kind == "steps":
            x[lo:hi] = (x[lo:hi] * 4).round() / 4
        elif kind == "sparse":
            away = torch.rand(hi - lo, generator=g) < 0.99
            x[lo:hi] = torch.where(away, torch.full((), -INF), x[lo:hi])
        else:
            x[lo:hi] = {"mask": -INF, "nan": float("nan"), "lowest": torch.finfo(io).min, "equal": float(x[lo])}[kind]
    if r.random() < 0.05:
        x[r.randrange(v)] = INF
    return x.to(io)


@pytest.mark.parametrize("seed", range(20))
def test_random_rows(K, seed):
    r, g = random.Random(seed), torch.Generator().manual_seed(seed)
    io = IO[r.choice(["bf16", "f32"])]
    v = r.choice([r.randint(2, 300), r.randint(300, 5000), r.randint(5000, 40000)])
    n = 6
    x = torch.stack([row(r, g, v, io) for _ in range(n)]).cuda()
    u = torch.rand(n, generator=g).cuda()
    for _ in range(4):
        kw = {}
        if r.random() < 0.6:
            kw["k"] = [r.choice([0, 1, 50, 300, 1024, 1025, v // 2, v - 1, v]) for _ in range(n)]
        if r.random() < 0.6:
            kw["p"] = [r.choice([0.1, 0.5, 0.9, 0.99, 0.9999, 1.0]) for _ in range(n)]
        if r.random() < 0.4:
            kw["m"] = [r.choice([0.0, 1e-12, 1e-3, 0.1, 0.7]) for _ in range(n)]
        if r.random() < 0.6:
            kw["t"] = [r.choice([0.0, 0.01, 0.7, 1.0, 4.0, 1e4]) for _ in range(n)]
        print(v, io, kw, flush=True)
        both(K, x, u, **kw)
