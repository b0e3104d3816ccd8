"""The selective state-space scan against a 64-bit token-by-token reference:
prompts, one token a request, runs of drafted tokens with a step cache; head
and group counts, dtypes, strided rows, ragged and empty sequences, strong and
weak decays."""
import math

import numpy as np
import pytest
import torch

import serve_ref as R

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
DTYPES = {"bf16": BF, "f32": F32}


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


def offsets(lens):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
    return cu.cuda()


class Layer:
    """Inputs of T tokens: x, B, C slices of one row, z and dt of another."""

    def __init__(self, seed, T, H, P, S, G, dtype, packed=True, opts=True, decay=1.0, shift=0.0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.dims = g, (H, P, S)
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        row = rand(T, H * P + 2 * G * S + 8).to(dtype).cuda()
        proj = (rand(T, H * P + (H + 7) // 8 * 8)).to(dtype).cuda()
        x = row[:, :H * P].unflatten(1, (H, P))
        B = row[:, H * P:H * P + G * S].unflatten(1, (G, S))
        C = row[:, H * P + G * S:H * P + 2 * G * S].unflatten(1, (G, S))
        z, dt = proj[:, :H * P].unflatten(1, (H, P)), proj[:, H * P:H * P + H]
        if not packed:
            x, B, C, z, dt = (t.contiguous() for t in (x, B, C, z, dt))
        self.args = (x, dt, torch.log((1 + 15 * torch.rand(H, generator=g)) * decay).cuda(), B, C)
        first = torch.exp(torch.rand(H, generator=g) * math.log(100.0) + math.log(1e-3))
        self.kw = dict(D=rand(H).cuda(), z=z, dt_bias=(first + torch.log(-torch.expm1(-first)) + shift).cuda()) if opts else {}

    def ref(self, lens, states):
        x, dt, A, B, C = self.args
        return R.scan(x, dt, A, B, C, lens, states, **self.kw)


def states(layer, n, dtype, size=0.5):
    return (torch.randn(n, *layer.dims, generator=layer.g) * size).to(dtype)


PROMPTS = [   # lens, H, P, S, G, io, state, packed, opts
    ([1], 1, 32, 32, 1, "bf16", "f32", True, True),
    ([64], 2, 128, 128, 1, "bf16", "f32", True, True),
    ([65, 63, 0, 1, 128, 2], 4, 64, 128, 2, "bf16", "f32", True, True),
    ([130, 0, 17], 8, 64, 64, 8, "bf16", "bf16", False, True),
    ([200, 300], 6, 32, 64, 3, "bf16", "f32", True, False),
    ([77, 5], 3, 128, 32, 1, "bf16", "f32", False, True),
    ([96, 33], 5, 32, 128, 5, "bf16", "f32", True, True),
    ([150], 12, 64, 32, 2, "bf16", "bf16", True, False),
    ([65, 63, 0, 1, 128, 2], 4, 64, 128, 2, "f32", "f32", True, True),
    ([200, 31], 3, 128, 64, 1, "f32", "bf16", False, True),
    ([129], 2, 32, 32, 2, "f32", "f32", True, False),
    ([100, 64], 2, 128, 128, 1, "f32", "f32", True, True),
    ([700], 2, 64, 128, 1, "bf16", "f32", True, True),
]


@pytest.mark.parametrize("lens,H,P,S,G,io,sd,packed,opts", PROMPTS, ids=[str(i) for i in range(len(PROMPTS))])
def test_prompts(K, lens, H, P, S, G, io, sd, packed, opts):
    dt, sd = DTYPES[io], DTYPES[sd]
    T, N = sum(lens), len(lens)
    m = Layer(sum(lens) + H, T, H, P, S, G, dt, packed, opts)
    first = states(m, N, sd)
    ref = m.ref(lens, first)
    cu = offsets(lens)
    y, last = K.ssm_prefill(*m.args, cu, initial_state=first.cuda(), **m.kw)
    R.check("y", y, ref["y"], ref["ytol"], dt)
    rel = R.check("states", last, ref["last"], ref["ltol"], sd)
    if sd == F32 and T:
        assert rel < 2e-6     # fp32 all through: far below one bf16 term's 2^-9
    # from nothing
    y0, last0 = K.ssm_prefill(*m.args, cu, state_dtype=sd, **m.kw)
    ref0 = m.ref(lens, torch.zeros_like(first))
    R.check("y from zeros", y0, ref0["y"], ref0["ytol"], dt)
    R.check("states from zeros", last0, ref0["last"], ref0["ltol"], sd)
    # the pool gives the dense form's bits and leaves its other rows alone
    slots = N + 4
    pool0 = states(m, slots, sd)
    idx = torch.randperm(slots - 1, generator=m.g)[:N].to(torch.int32)
    idx[0] = -1
    at = torch.from_numpy(R.slots_of(idx, slots)).long()
    pool0[at] = first
    pool = pool0.cuda()
    yp, same = K.ssm_prefill(*m.args, cu, initial_state=pool, state_indices=idx.cuda(), **m.kw)
    want = pool0.clone()
    want[at] = last.cpu()
    assert same is pool and torch.equal(yp, y) and torch.equal(pool.cpu(), want)
    yn, none = K.ssm_prefill(*m.args, cu, initial_state=first.cuda(), output_final_state=False, **m.kw)
    assert none is None and torch.equal(yn, y)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("decay,shift", [(40.0, 3.0), (1e-4, 0.0), (1.0, -12.0)], ids=["strong", "none", "small steps"])
def test_decays(K, io, decay, shift):
    """Log-decays of hundreds a token (a block's products underflow, its sums
    reach 1e5), nearly none over 300 tokens, and steps near 1e-7."""
    dt = DTYPES[io]
    m = Layer(7, 300, 4, 64, 64, 2, dt, decay=decay, shift=shift)
    first = states(m, 1, F32)
    y, last = K.ssm_prefill(*m.args, offsets([300]), initial_state=first.cuda(), **m.kw)
    ref = m.ref([300], first)
    R.check("y", y, ref["y"], ref["ytol"], dt)
    R.check("states", last, ref["last"], ref["ltol"], F32)


def test_magnitudes(K):
    """bf16's own range: inputs and states beyond fp16's."""
    m = Layer(8, 150, 2, 64, 64, 1, BF)
    x, dt, A, B, C = m.args
    m.args = (x * 1e6, dt, A, B * 1e-7, C)
    first = states(m, 1, F32, size=1e5)
    y, last = K.ssm_prefill(*m.args, offsets([150]), initial_state=first.cuda(), **m.kw)
    ref = m.ref([150], first)
    R.check("y", y, ref["y"], ref["ytol"], BF)
    R.check("states", last, ref["last"], ref["ltol"], F32)


TOKENS = [   # B, H, P, S, G, io, state, packed, opts
    (1, 2, 32, 32, 1, "bf16", "f32", True, True),
    (3, 4, 64, 128, 2, "bf16", "f32", True, True),
    (5, 3, 128, 64, 3, "f32", "f32", False, True),
    (2, 6, 128, 128, 2, "bf16", "bf16", True, False),
    (4, 2, 64, 32, 1, "f32", "bf16", True, True),
    (9, 1, 32, 64, 1, "bf16", "f32", False, True),
    (300, 32, 32, 32, 4, "bf16", "f32", True, True),
]


@pytest.mark.parametrize("B,H,P,S,G,io,sd,packed,opts", TOKENS, ids=[str(i) for i in range(len(TOKENS))])
def test_tokens(K, B, H, P, S, G, io, sd, packed, opts):
    dt, sd = DTYPES[io], DTYPES[sd]
    m = Layer(B + H, B, H, P, S, G, dt, packed, opts)
    slots = B + 3
    pool0 = states(m, slots, sd)
    idx = torch.randperm(slots - 1, generator=m.g)[:B].to(torch.int32)
    idx[-1] = -1
    at = torch.from_numpy(R.slots_of(idx, slots)).long()
    pool = pool0.cuda()
    y = K.ssm_decode(*m.args, pool, idx.cuda(), **m.kw)
    ref = m.ref([1] * B, pool0[at])
    R.check("y", y, ref["y"], ref["ytol"], dt)
    R.check("states", pool[at.cuda()], ref["last"], ref["ltol"], sd)
    other = np.setdiff1d(np.arange(slots), at.numpy())
    assert torch.equal(pool.cpu()[other], pool0[other])


@pytest.mark.parametrize("io,sd", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("steps,pitch", [(3, 5), (4, 4), (0, 0)])
def test_runs_of_tokens(K, io, sd, steps, pitch):
    dt, sd = DTYPES[io], DTYPES[sd]
    lens, H, P, S, G = [4, 0, 1, 6, 3], 4, 64, 128, 2
    N = len(lens)
    m = Layer(steps, sum(lens), H, P, S, G, dt)
    slots = N + 2
    pool0 = states(m, slots, sd)
    idx = torch.tensor([3, 5, -1, 0, 2], dtype=torch.int32)
    at = torch.from_numpy(R.slots_of(idx, slots)).long()
    whole = torch.full((N, pitch, H, P, S), 7.0, dtype=sd, device="cuda") if pitch else None
    cache = None if whole is None else whole[:, :steps]
    pool = pool0.cuda()
    y = K.ssm_decode_multi(*m.args, offsets(lens), pool, idx.cuda(), intermediate_states=cache, update_pool=False, **m.kw)
    ref = m.ref(lens, pool0[at])
    R.check("y", y, ref["y"], ref["ytol"], dt)
    assert torch.equal(pool.cpu(), pool0)
    for n, L in enumerate(lens):
        for j in range(pitch):
            if j < min(L, steps):
                R.check("step", whole[n, j], ref["steps"][n][j], ref["stol"][n][j], sd)
            else:      # steps a request has not, and rows beyond the view: as they were
                assert bool((whole[n, j] == 7.0).all())
    y2 = K.ssm_decode_multi(*m.args, offsets(lens), pool, idx.cuda(), **m.kw)
    assert torch.equal(y2, y)
    some = [n for n, L in enumerate(lens) if L]
    R.check("last", pool[at[some].cuda()], ref["last"][some], ref["ltol"][some], sd)
    rest = np.setdiff1d(np.arange(slots), at[some].numpy())
    assert torch.equal(pool.cpu()[rest], pool0[rest])


def test_prefill_then_tokens_continue(K):
    """A prompt and then tokens one by one give what the whole gives at once."""
    T, H, P, S = 150, 4, 64, 64
    m = Layer(11, T, H, P, S, 2, F32)
    pool = torch.zeros(3, H, P, S, device="cuda")
    idx = torch.tensor([1], dtype=torch.int32, device="cuda")
    whole = m.ref([T], torch.zeros(1, H, P, S))
    cut = lambda a, b: [t[a:b] if t.dim() > 1 else t for t in m.args]  # noqa: E731
    kw = lambda a, b: dict(m.kw, z=m.kw["z"][a:b])  # noqa: E731
    parts = [K.ssm_prefill(*cut(0, 140), offsets([140]), initial_state=pool, state_indices=idx, **kw(0, 140))[0]]
    for t in range(140, T):
        parts.append(K.ssm_decode(*cut(t, t + 1), pool, idx, **kw(t, t + 1)))
    R.check("y", torch.cat(parts), whole["y"], whole["ytol"] * 2, F32)
    R.check("state", pool[1:2], whole["last"], whole["ltol"] * 2, F32)


def test_empty_calls(K):
    m = Layer(1, 0, 4, 32, 32, 2, BF)
    first = torch.randn(2, 4, 32, 32, device="cuda")
    y, last = K.ssm_prefill(*m.args, offsets([0, 0]), initial_state=first, **m.kw)
    assert y.shape == (0, 4, 32) and torch.equal(last, first)
    y, last = K.ssm_prefill(*m.args, offsets([0, 0]), **m.kw)
    assert not last.any() and last.shape == first.shape
    y, last = K.ssm_prefill(*m.args, offsets([]), **m.kw)
    assert last.shape == (0, 4, 32, 32)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert K.ssm_decode(*m.args, first, none, **m.kw).shape == (0, 4, 32)
    assert K.ssm_decode_multi(*m.args, offsets([0]), first, none.new_zeros(1), **m.kw).shape == (0, 4, 32)
