"""Next tokens of rows in which whole stretches of logits weigh nothing beside the
largest (below half of the unit that weights are summed in): no token without a
weight is drawn, whatever the random number."""
import numpy as np
import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu
F32, BF, I32 = torch.float32, torch.bfloat16, torch.int32
INF = float("inf")
LAST = 1 - 2.0 ** -24          # the largest fp32 below one


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


def bits(v):
    """Weights are whole multiples of 2^-46 up to 65,536 logits, of twice that for
    every doubling."""
    return 46 if v <= 65536 else 62 - (v - 1).bit_length()


def drawn(x, u, probs):
    """Tokens by the whole weights of the logits that the limits keep: first with
    a running sum above u times all of it."""
    out = []
    for row, r, p in zip(x, u, probs):
        w = np.where(p > 0, np.rint(2.0 ** bits(len(row)) * np.exp(row - row.max())), 0)
        cum = np.cumsum(w.astype(np.int64))
        out.append(int(np.searchsorted(cum, int(r * float(cum[-1])), side="right")))
    return out


def rows(kind, v, dtype):
    """One row: its heavy logits at `heavy`, all else too light to count."""
    x = torch.full((v,), -INF)
    if kind == "light first":            # 0.6 of 2^-50 and less, thousands of them, before the only heavy one
        x[1:] = 0.0
        x[v // 2 + min(100, v // 4)] = 35.0
    elif kind == "light last":
        x[:-3] = 0.0
        x[v // 3] = 35.0
    elif kind == "few":                  # three below half a unit in the first part
        x[5:8] = -32.9
        x[2 * v // 3], x[2 * v // 3 + 9] = 0.0, -1.0
    elif kind == "nan":
        x[:] = float("nan")
        x[3:40] = 1.0
        x[v - 200], x[v - 100] = 40.0, 38.0
    elif kind == "both sides":
        x[:] = 2.0
        x[0], x[-1] = -INF, -INF
        x[v // 2] = 37.5
    return x.to(dtype)


KINDS = ["light first", "light last", "few", "nan", "both sides"]
LIMITS = {"none": {}, "top_p": dict(top_p=0.9999), "min_p": dict(min_p=1e-30), "top_k": dict(top_k=2000), "few": dict(top_k=40),
          "all": dict(top_k=3000, top_p=0.999, min_p=1e-25)}


@pytest.mark.parametrize("limits", list(LIMITS))
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("v", [50, 5000, 16384, 70001])
def test_light_stretches(K, v, dtype, limits):
    u = [0.0, 2.0 ** -60, 2.0 ** -37, 0.5, LAST]
    kinds = [k for k in KINDS if v > 500 or k != "nan"]
    one = torch.stack([rows(k, v, dtype) for k in kinds])
    x, n = one.repeat_interleave(len(u), 0), len(u) * len(kinds)
    random = torch.tensor(u * len(kinds), device="cuda")
    kw = LIMITS[limits]
    on = {k: torch.full((n,), y, dtype=I32 if k == "top_k" else F32, device="cuda") for k, y in kw.items()}
    host = {k: [float(torch.tensor(y, dtype=F32))] * len(kinds) for k, y in kw.items()}
    _, probs = R.sample(one.double().numpy(), **host)
    full = np.nan_to_num(x.double().numpy(), nan=-INF, neginf=-INF)
    want = drawn(full, random.cpu().double().numpy(), np.repeat(probs, len(u), 0))
    tokens, got = K.sample_tokens(x.cuda(), random, return_probs=True, **on)
    tokens, got = tokens.tolist(), got.cpu().numpy()
    for i, (t, w) in enumerate(zip(tokens, want)):
        print(i, kinds[i // len(u)], u[i % len(u)], t, w, flush=True)
        assert 0 <= t < v and got[i, t] > 2.0 ** -(bits(v) + 2), (i, t, w)
        assert t == w, (i, t, w)


@pytest.mark.parametrize("limits", ["none", "min_p"])
def test_largest_vocabulary_of_light_logits(K, limits):
    """2^20 logits of 0.45 units each are 2^-23 of all weights by their number: more
    than the last random number leaves."""
    v = 1 << 20
    x = torch.full((3, v), float(np.log(0.45 * 2.0 ** -bits(v))))
    x[:, 0], x[:, -1] = -INF, -INF
    x[:, 8000] = 0.0
    u = torch.tensor([0.0, LAST, 2.0 ** -24], device="cuda")
    kw = {} if limits == "none" else dict(min_p=torch.full((3,), 1e-30, device="cuda"))
    assert K.sample_tokens(x.cuda(), u, **kw).tolist() == [8000] * 3
