"""Cases of the state-space and draft-verification operators: what is timed and compared.

Four operators of one serving path:

  conv     the short causal convolution in front of a recurrent layer (per channel, SiLU after it), for packed
           prompts and for one token a request, its last inputs kept in a pool of slots
  scan     the selective state space scan, S = exp(dt A) S + dt x B^T, y = S C + D x, for packed prompts, for one
           token a request and for a short run of drafted tokens with the state kept after every one
  drafts   verification of drafted tokens against the target's probabilities, from given random numbers
  commit   the accepted step's states (and the convolution's last inputs) written back to their pools

``own`` False computes them from elementary torch operations in 32 bits (64 for sums of decays and for the
sums a sampled token is found by); ``own`` True calls the package.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64   # tokens in a block of the plain scan


def listed():
    return [
        # the convolution in front of a layer of 32 heads x 128 with 8 groups of 128 states, 16 prompts at once
        dict(name="conv prompts", op="conv", n=16, lo=512, hi=4096, lens=4, d=6144, w=4, io="bf16", bias=True, pool=True),
        # the same step in a small batch of one-token requests, in 32 bits, an odd channel count, three taps
        dict(name="conv tokens f32", op="conv1", b=200, d=2051, w=3, io="f32", bias=False),
        # 16 prompts of 512 to 4096 tokens, 32 heads, states of 128 x 128 in a pool, inputs sliced from packed rows
        dict(name="scan prompts", op="scan", n=16, lo=512, hi=4096, lens=4, h=32, p=128, s=128, g=8, io="bf16", state="f32",
             pool=True, z=False, packed=True),
        # one long prompt, gated, all heads sharing one B and C
        dict(name="scan long", op="scan", n=1, lo=32768, hi=32768, lens=0, h=32, p=64, s=128, g=1, io="bf16", state="f32",
             pool=True, z=True, packed=True),
        # few short ragged prompts in 32 bits, states handed in and out densely
        dict(name="scan ragged f32", op="scan", n=7, lo=1, hi=300, lens=9, h=8, p=64, s=64, g=2, io="f32", state="f32",
             pool=False, z=False, packed=False),
        # one request: the latency of a token
        dict(name="scan token", op="scan1", b=1, slots=4, h=32, p=128, s=128, g=8, io="bf16", state="f32", z=False, packed=True),
        # 4096 requests: the pool streams through
        dict(name="scan tokens", op="scan1", b=4096, slots=4160, h=32, p=128, s=128, g=8, io="bf16", state="f32", z=True,
             packed=True),
        # the verify step of speculative decoding: 1024 requests x 4 tokens, the state kept after each
        dict(name="scan verify", op="scanm", n=1024, lo=4, hi=4, lens=0, slots=1088, pitch=4, h=32, p=64, s=128, g=8, io="bf16",
             state="f32", z=False, packed=True),
        # one request's three drafts against a large vocabulary
        dict(name="drafts one", op="drafts", n=1, lo=4, hi=4, lens=0, v=131072, io="f32", q=True),
        # 1024 requests at once
        dict(name="drafts many", op="drafts", n=1024, lo=4, hi=4, lens=0, v=65536, io="f32", q=True),
        # the accepted states of a few requests
        dict(name="commit few", op="commit", n=3, lo=2, hi=4, lens=2, slots=9, pitch=5, h=32, p=64, s=128, state="bf16", d=4096, w=4,
             io="bf16"),
        # and of 1024
        dict(name="commit many", op="commit", n=1024, lo=4, hi=4, lens=0, slots=1088, pitch=4, h=32, p=64, s=128, state="f32",
             d=4096, w=4, io="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["conv", "conv1", "scan", "scan", "scan1", "scanm", "drafts", "drafts", "commit"])
    io = rng.choice(["bf16", "bf16", "f32"])
    h = rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16, 24, 32])
    g = rng.choice([k for k in range(1, h + 1) if h % k == 0 and k <= 8])
    heads = dict(h=h, p=rng.choice([32, 64, 128]), s=rng.choice([32, 64, 128]), g=g, io=io, state=rng.choice(["f32", "f32", "bf16"]))
    lens = rng.randrange(1 << 30)
    if op == "conv":
        n = _log(rng, 1, 200)
        hi = _log(rng, 1, max(1, 32768 // n))
        return dict(op=op, n=n, lo=rng.randint(0, hi), hi=hi, lens=lens, d=_log(rng, 24, 6000), w=rng.choice([2, 3, 4]), io=io,
                    bias=rng.random() < 0.5, pool=rng.random() < 0.5)
    if op == "conv1":
        return dict(op=op, b=_log(rng, 1, 4096), d=_log(rng, 24, 6000), w=rng.choice([2, 3, 4]), io=io, bias=rng.random() < 0.5)
    if op == "scan":
        n = _log(rng, 1, 100)
        hi = _log(rng, 1, max(1, 32768 // n))
        return dict(op=op, n=n, lo=rng.randint(0, hi), hi=hi, lens=lens, pool=rng.random() < 0.6, z=rng.random() < 0.5,
                    packed=rng.random() < 0.5, **heads)
    if op == "scan1":
        b = _log(rng, 1, 2048)
        return dict(op=op, b=b, slots=b + rng.randint(2, 40), z=rng.random() < 0.5, packed=rng.random() < 0.5, **heads)
    if op == "scanm":
        n = _log(rng, 1, 512)
        hi = rng.randint(1, 8)
        return dict(op=op, n=n, lo=rng.randint(0, hi), hi=hi, lens=lens, slots=n + rng.randint(2, 40), pitch=rng.randint(1, hi),
                    z=rng.random() < 0.5, packed=rng.random() < 0.5, **heads)
    if op == "drafts":
        n = _log(rng, 1, 512)
        hi = rng.randint(1, 8)
        return dict(op=op, n=n, lo=rng.randint(1, hi), hi=hi, lens=lens, v=_log(rng, 30, min(150000, 150_000_000 // (n * hi))), io=io,
                    q=rng.random() < 0.7)
    n = _log(rng, 1, 512)
    hi = rng.randint(1, 8)
    heads.pop("g")
    return dict(op=op, n=n, lo=rng.randint(0, hi), hi=hi, lens=lens, slots=n + rng.randint(2, 40), pitch=hi, d=_log(rng, 24, 6000),
                w=rng.choice([2, 3, 4]), **heads)


def _lengths(c):
    r = random.Random(c["lens"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["n"])]


# ---- inputs ----------------------------------------------------------------------------------------------------


def _sequences(c, st, dev):
    lens = _lengths(c)
    st["lens"], st["longest"], st["T"] = lens, max(lens), sum(lens)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)


def _heads(c, st, T, gen, dev):
    """x, B, C (and z, dt) of a layer of h heads: slices of one row a token where they come packed."""
    h, p, s, g, dt = c["h"], c["p"], c["s"], c["g"], DT[c["io"]]
    rand = lambda *z: torch.randn(*z, generator=gen, device=dev)  # noqa: E731
    # what a convolution with SiLU after it gives: mostly small, a long positive tail
    row = torch.nn.functional.silu(rand(T, h * p + 2 * g * s)).to(dt)
    x, B, C = row[:, :h * p].unflatten(1, (h, p)), row[:, h * p:h * p + g * s].unflatten(1, (g, s)), row[:, h * p + g * s:].unflatten(1, (g, s))
    proj = rand(T, h * p + (h + 7) // 8 * 8).to(dt)   # the projection's width is a multiple of 8
    z, step = proj[:, :h * p].unflatten(1, (h, p)), proj[:, h * p:h * p + h]
    if not c["packed"]:
        x, B, C, z, step = (t.contiguous() for t in (x, B, C, z, step))
    st.update(x=x, B=B, C=C, z=z if c["z"] else None, dt=step)
    st["A_log"] = torch.log(1 + 15 * torch.rand(h, generator=gen, device=dev))
    first = torch.exp(torch.rand(h, generator=gen, device=dev) * math.log(100.0) + math.log(1e-3))
    st["dt_bias"] = first + torch.log(-torch.expm1(-first))
    st["D"] = rand(h)


def _slots(n, slots, seed, dev, pad):
    """Slots in the pool, each its own; the last of them padding, where that is asked for."""
    r = random.Random(seed)
    idx = r.sample(range(slots - 1), n)
    if pad:
        idx[-1] = -1
    return torch.tensor(idx, dtype=torch.int32, device=dev)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 1009 + 17)
    rand = lambda *z: torch.randn(*z, generator=gen, device=dev)  # noqa: E731
    st = dict(case=c)
    op = c["op"]
    if op in ("conv", "scan", "scanm", "drafts", "commit"):
        _sequences(c, st, dev)
    if op in ("conv", "conv1", "commit"):
        dt = DT[c["io"]]
        d, w = c["d"], c["w"]
        n = c["n"] if op != "conv1" else c["b"]
        st["cx"] = rand(st["T"] if op != "conv1" else n, d).to(dt)
        st["weight"] = ((torch.rand(d, w, generator=gen, device=dev) * 2 - 1) / math.sqrt(w)).to(dt)
        st["bias"] = (rand(d) * 0.1).to(dt) if c.get("bias") else None
        slots = c.get("slots", n + 7)
        if op == "conv" and not c["pool"]:
            st["cstate"], st["idx"] = rand(n, w - 1, d).to(dt), None
        else:
            st["cstate"] = rand(slots, w - 1, d).to(dt)
            st["idx"] = _slots(n, slots, seed, dev, pad=n > 2)
    if op in ("scan", "scan1", "scanm"):
        n = c["b"] if op == "scan1" else c["n"]
        _heads(c, st, n if op == "scan1" else st["T"], gen, dev)
        one = (c["h"], c["p"], c["s"])
        if op == "scan" and not c["pool"]:
            st["state"], st["idx"] = (rand(n, *one) * 0.3).to(DT[c["state"]]), None
        else:
            slots = c.get("slots", n + 5)
            st["state"] = (rand(slots, *one) * 0.3).to(DT[c["state"]])
            st["idx"] = _slots(n, slots, seed, dev, pad=n > 2)
        if op == "scanm":
            st["cache"] = torch.zeros(n, c["pitch"], *one, dtype=DT[c["state"]], device=dev)
    if op == "commit":
        one = (c["h"], c["p"], c["s"])
        st["state"] = rand(c["slots"], *one).to(DT[c["state"]])
        st["cache"] = rand(c["n"], c["pitch"], *one).to(DT[c["state"]])
        r = random.Random(seed)
        st["steps"] = torch.tensor([r.randint(0, x - 1) if x else -1 for x in st["lens"]], dtype=torch.int32, device=dev)
    if op == "drafts":
        T, v = st["T"], c["v"]
        logits = 2.5 * rand(T, v)
        st["probs"] = torch.softmax(logits, 1).to(DT[c["io"]])
        # a smaller model's: near the target's, and the drafts drawn from it (row t's gives token t + 1)
        logits += 0.7 * rand(T, v)
        near = torch.softmax(logits, 1)
        drawn = torch.multinomial(near, 1, generator=gen).flatten()
        st["tokens"] = torch.cat([drawn.new_zeros(1), drawn[:-1]]).int()
        st["near"] = near.to(DT[c["io"]]) if c["q"] else None
        st["u"] = torch.rand(T, generator=gen, device=dev)
        st["r"] = torch.rand(c["n"], generator=gen, device=dev)
    return st


# ---- plain forms -----------------------------------------------------------------------------------------------


def _rows_of(idx, slots):
    return torch.where(idx < 0, torch.full_like(idx, slots - 1), idx).long()


def _padded(cu, longest):
    """(rows of the packed tokens, which of them are there), each [sequences, longest]."""
    at = torch.arange(longest, device=cu.device)
    there = at[None] < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None].long() + at[None], 0), there


def _silu(x):
    return x / (1 + torch.exp(-x))


def _plain_conv(x, first, weight, bias):
    """x [N, L, D], first [N, W - 1, D]: the taps summed, then SiLU."""
    w = weight.shape[1]
    full = torch.cat([first.float(), x.float()], 1)
    y = sum(full[:, j:j + x.shape[1]] * weight[:, j].float() for j in range(w))
    return _silu(y if bias is None else y + bias.float()), full


def _last_inputs(full, lengths, w):
    """Rows lengths .. lengths + W - 2 of the inputs with the first state before them."""
    at = lengths.long()[:, None] + torch.arange(w - 1, device=full.device)
    return full.gather(1, at[:, :, None].expand(-1, -1, full.shape[2]))


def _steps_of(st, dt):
    z = dt.float() + st["dt_bias"]
    return z.clamp_min(0) + torch.log1p(torch.exp(-z.abs()))


def _finish(st, y, x, z):
    y = y + st["D"][:, None] * x
    return y if z is None else y * _silu(z.float())


def _plain_scan(st, first):
    """The scan in blocks of CHUNK tokens: products inside a block, and one product over the blocks' states."""
    c, cu = st["case"], st["cu"]
    n, h, p, s, g = c["n"], c["h"], c["p"], c["s"], c["g"]
    blocks = max(1, -(-st["longest"] // CHUNK))
    rows, there = _padded(cu, blocks * CHUNK)
    if not st["T"]:
        return st["x"].new_zeros(0, h, p), first
    pick = lambda t: torch.where(there.view(*there.shape, *(1,) * (t.dim() - 1)), t[rows].float(), 0).view(n, blocks, CHUNK, *t.shape[1:])  # noqa: E731
    step = torch.where(there[..., None], _steps_of(st, st["dt"])[rows], 0).view(n, blocks, CHUNK, h).permute(0, 1, 3, 2)
    x = pick(st["x"]).permute(0, 1, 3, 2, 4)                                              # [n, blocks, h, CHUNK, p]
    B, C = (pick(st[k]).permute(0, 1, 3, 2, 4) for k in ("B", "C"))                       # [n, blocks, g, CHUNK, s]
    a = step.double() * -torch.exp(st["A_log"].double())[:, None]
    far = a.cumsum(-1)                                                                    # [n, blocks, h, CHUNK]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp(torch.where(low, far[..., :, None] - far[..., None, :], -math.inf).float())
    near = torch.matmul(C, B.transpose(-1, -2)).repeat_interleave(h // g, 2)
    y = torch.matmul(near * decay * step[..., None, :], x)
    w = (step * torch.exp((far[..., -1:] - far).float()))[..., None] * x
    each = torch.matmul(w.transpose(-1, -2), B.repeat_interleave(h // g, 2))              # [n, blocks, h, p, s]
    total = torch.cat([a.new_zeros(n, 1, h), far[..., -1].cumsum(1)], 1).permute(0, 2, 1)  # [n, h, blocks + 1]
    low = torch.ones(blocks + 1, blocks + 1, dtype=torch.bool, device=x.device).tril()
    carry = torch.exp(torch.where(low, total[..., :, None] - total[..., None, :], -math.inf).float())
    each = torch.cat([first.float()[:, None], each], 1).permute(0, 2, 1, 3, 4).flatten(3)  # [n, h, blocks + 1, p s]
    each = torch.matmul(carry, each).view(n, h, blocks + 1, p, s)
    before = each[:, :, :-1].transpose(1, 2)                                              # [n, blocks, h, p, s]
    y = y + torch.matmul(C.repeat_interleave(h // g, 2), before.transpose(-1, -2)) * torch.exp(far.float())[..., None]
    y = y.permute(0, 1, 3, 2, 4).reshape(n, blocks * CHUNK, h, p)[there]
    return _finish(st, y, st["x"].float(), st["z"]).to(st["x"].dtype), each[:, :, -1]


def _plain_token(st, first):
    rep = st["case"]["h"] // st["case"]["g"]
    step, x = _steps_of(st, st["dt"]), st["x"].float()
    B, C = (st[k].float().repeat_interleave(rep, 1) for k in ("B", "C"))
    S = first.float() * torch.exp(-step * torch.exp(st["A_log"]))[..., None, None]
    S = S + (step[..., None] * x)[..., None] * B[:, :, None]
    y = (S * C[:, :, None]).sum(-1)
    return _finish(st, y, x, st["z"]).to(st["x"].dtype), S


def _plain_run_of_tokens(st, first):
    """States after every token of a short run: one product with the decays between the tokens."""
    c = st["case"]
    rows, there = _padded(st["cu"], max(1, st["longest"]))
    n, L = rows.shape
    h, p, s, rep = c["h"], c["p"], c["s"], c["h"] // c["g"]
    if not st["T"]:
        return st["x"].new_zeros(0, h, p), first.float()[:, None].expand(n, L, h, p, s), there
    step = torch.where(there[..., None], _steps_of(st, st["dt"])[rows], 0)                # [n, L, h]
    x = torch.where(there[..., None, None], st["x"][rows].float(), 0)
    B, C = (torch.where(there[..., None, None], st[k][rows].float(), 0).repeat_interleave(rep, 2) for k in ("B", "C"))
    a = torch.cat([step.new_zeros(n, 1, h).double(), step.double() * -torch.exp(st["A_log"].double())], 1).cumsum(1).permute(0, 2, 1)
    low = torch.ones(L + 1, L + 1, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp(torch.where(low, a[..., :, None] - a[..., None, :], -math.inf).float())   # [n, h, L + 1, L + 1]
    new = (step[..., None] * x)[..., None] * B[:, :, :, None]                             # [n, L, h, p, s]
    new = torch.cat([first.float()[:, None], new], 1).transpose(1, 2).flatten(3)
    S = torch.matmul(decay[:, :, 1:], new).view(n, h, L, p, s).transpose(1, 2)
    y = (S * C[:, :, :, None]).sum(-1)[there]
    return _finish(st, y, st["x"].float(), st["z"]).to(st["x"].dtype), S, there


def _plain_drafts(st):
    cu, v, T = st["cu"].long(), st["case"]["v"], st["T"]
    n, L = cu.numel() - 1, max(1, st["longest"])
    lens = cu[1:] - cu[:-1]
    rows, there = _padded(st["cu"], L)
    more = there[:, 1:]                                                                   # a draft after row j
    token = torch.where(more, st["tokens"][rows[:, 1:]].long(), 0)
    row = rows[:, :-1]
    p = st["probs"][row, token].float()
    q = st["near"][row, token].float() if st["near"] is not None else torch.ones_like(p)
    good = (st["u"][row] * q < p) & more
    accepted = good.long().cumprod(1).sum(1)
    last = cu[:-1] + accepted
    refused = accepted < lens - 1
    P = st["probs"][last].float()
    wrong = st["tokens"][torch.where(refused, last + 1, 0)].long()
    if st["near"] is not None:
        rest = (P - st["near"][last].float()).clamp_min(0)
    else:
        rest = P.scatter(1, wrong[:, None], 0.0)
    rest = torch.where(refused[:, None], rest, P).double()
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, P.double())
    cum = rest.cumsum(1)
    found = (cum <= st["r"].double()[:, None] * cum[:, -1:]).sum(1)
    biggest = (rest > 0).long().mul(torch.arange(1, v + 1, device=rest.device)).amax(1) - 1
    found = torch.minimum(found, biggest)
    at = torch.arange(L, device=cu.device)[None]
    after = torch.where(at + 1 < lens[:, None], st["tokens"][(rows + 1).clamp_max(T - 1)].long(), -1)
    emitted = torch.where(at < accepted[:, None], after, torch.where(at == accepted[:, None], found[:, None], -1))[there]
    return accepted.int(), found.int(), emitted.int()


# ---- one pass --------------------------------------------------------------------------------------------------


def _own_run(st):
    import gated_delta_rule_51_amd as kda
    op = st["case"]["op"]
    if op == "conv":
        return kda.conv_prefill(st["cx"], st["weight"], st["bias"], st["cu"], initial_state=st["cstate"], state_indices=st["idx"])
    if op == "conv1":
        return kda.conv_decode(st["cx"], st["weight"], st["bias"], st["cstate"], st["idx"]), st["cstate"]
    if op == "scan":
        return kda.ssm_prefill(st["x"], st["dt"], st["A_log"], st["B"], st["C"], st["cu"], D=st["D"], z=st["z"], dt_bias=st["dt_bias"],
                               initial_state=st["state"], state_indices=st["idx"])
    if op == "scan1":
        return kda.ssm_decode(st["x"], st["dt"], st["A_log"], st["B"], st["C"], st["state"], st["idx"], D=st["D"], z=st["z"],
                              dt_bias=st["dt_bias"]), st["state"]
    if op == "scanm":
        return kda.ssm_decode_multi(st["x"], st["dt"], st["A_log"], st["B"], st["C"], st["cu"], st["state"], st["idx"], D=st["D"], z=st["z"],
                                    dt_bias=st["dt_bias"], intermediate_states=st["cache"], update_pool=False), st["cache"]
    if op == "drafts":
        return kda.verify_drafts(st["tokens"], st["probs"], st["cu"], st["u"], st["r"], draft_probs=st["near"])
    kda.commit_states(st["state"], st["idx"], st["cache"], st["steps"])
    kda.conv_commit(st["cx"], st["cu"], st["steps"], st["cstate"], st["idx"])
    return st["state"], st["cstate"]


def run(state):
    if own:
        return _own_run(state)
    st, c = state, state["case"]
    op, idx = c["op"], state.get("idx")
    if op == "conv":
        rows, there = _padded(st["cu"], max(1, st["longest"]))
        first = st["cstate"] if idx is None else st["cstate"][_rows_of(idx, st["cstate"].shape[0])]
        x = st["cx"][rows] if st["T"] else st["cx"].new_zeros(*rows.shape, c["d"])
        y, full = _plain_conv(x, first, st["weight"], st["bias"])
        last = _last_inputs(full, st["cu"][1:] - st["cu"][:-1], c["w"]).to(st["cstate"].dtype)
        if idx is not None:
            last = st["cstate"].index_copy_(0, _rows_of(idx, st["cstate"].shape[0]), last)
        return y[there].to(st["cx"].dtype), last
    if op == "conv1":
        at = _rows_of(idx, st["cstate"].shape[0])
        y, full = _plain_conv(st["cx"][:, None], st["cstate"][at], st["weight"], st["bias"])
        st["cstate"].index_copy_(0, at, full[:, 1:].to(st["cstate"].dtype))
        return y[:, 0].to(st["cx"].dtype), st["cstate"]
    if op == "scan":
        first = st["state"] if idx is None else st["state"][_rows_of(idx, st["state"].shape[0])]
        y, last = _plain_scan(st, first)
        last = last.to(st["state"].dtype)
        if idx is not None:
            last = st["state"].index_copy_(0, _rows_of(idx, st["state"].shape[0]), last)
        return y, last
    if op == "scan1":
        at = _rows_of(idx, st["state"].shape[0])
        y, S = _plain_token(st, st["state"][at])
        st["state"].index_copy_(0, at, S.to(st["state"].dtype))
        return y, st["state"]
    if op == "scanm":
        y, S, there = _plain_run_of_tokens(st, st["state"][_rows_of(idx, st["state"].shape[0])])
        k = min(c["pitch"], S.shape[1])
        st["cache"][:, :k] = torch.where(there[:, :k, None, None, None], S[:, :k].to(st["cache"].dtype), st["cache"][:, :k])
        return y, st["cache"]
    if op == "drafts":
        return _plain_drafts(st)
    steps = st["steps"].long()
    at, some = _rows_of(idx, st["state"].shape[0]), steps >= 0
    there = torch.arange(c["n"], device=steps.device)
    shape = (-1, 1, 1, 1)
    st["state"].index_copy_(0, at, torch.where(some.view(shape), st["cache"][there, steps.clamp_min(0)], st["state"][at]))
    rows, _ = _padded(st["cu"], max(1, st["longest"]))
    x = st["cx"][rows] if st["T"] else st["cx"].new_zeros(*rows.shape, c["d"])
    last = _last_inputs(torch.cat([st["cstate"][at], x], 1), steps + 1, c["w"])
    st["cstate"].index_copy_(0, at, last)
    return st["state"], st["cstate"]


def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "f32": 4}
    if op in ("conv", "conv1"):
        e, d, w = size[c["io"]], c["d"], c["w"]
        T, n = (c["b"], c["b"]) if op == "conv1" else (sum(_lengths(c)), c["n"])
        return {"bytes": 2 * T * d * e + 2 * n * (w - 1) * d * e + d * w * e, "flops": (2 * w + 4) * T * d}
    if op in ("scan", "scan1", "scanm"):
        e, se = size[c["io"]], size[c["state"]]
        h, p, s, g = c["h"], c["p"], c["s"], c["g"]
        T, n = (c["b"], c["b"]) if op == "scan1" else (sum(_lengths(c)), c["n"])
        one = h * p * s * se
        states = n * one * 2 if op != "scanm" else n * one + sum(min(x, c["pitch"]) for x in _lengths(c)) * one
        return {"bytes": T * ((3 if c["z"] else 2) * h * p + 2 * g * s + h) * e + states, "flops": T * h * (4 * p * s + 4 * p)}
    if op == "drafts":
        # the row the next token is drawn from, of the target and, where a draft was refused, of the draft's model: about two
        # of three requests of several drafts have one refused
        e, v = size[c["io"]], c["v"]
        rows = c["n"] * (1 + (0.6 if c["q"] and c["hi"] > 1 else 0))
        return {"bytes": int(rows * v * e) + 20 * sum(_lengths(c)), "flops": 3 * c["n"] * v}
    there = sum(x > 0 for x in _lengths(c))
    return {"bytes": max(1, there * (c["h"] * c["p"] * c["s"] * size[c["state"]] * 2 + (c["w"] - 1) * c["d"] * size[c["io"]] * 2)), "flops": 0}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------


def exact(case, seed):
    """Token by token, in 64 bits."""
    c, op = case, case["op"]
    if op == "drafts":
        return None
    st = prepare(case, seed)
    f = lambda t: None if t is None else t.double()  # noqa: E731
    idx = st.get("idx")
    slot = lambda k, n: [j if j >= 0 else st[k].shape[0] - 1 for j in idx.tolist()] if idx is not None else list(range(n))  # noqa: E731
    if op in ("conv", "conv1"):
        n = c["b"] if op == "conv1" else c["n"]
        lens = [1] * n if op == "conv1" else st["lens"]
        x, w, b, pool = f(st["cx"]), f(st["weight"]), f(st["bias"]), f(st["cstate"])
        at, t, k, out = slot("cstate", n), 0, c["w"], []
        for j, L in enumerate(lens):
            win = torch.cat([pool[at[j]], x[t:t + L]])
            if L:
                y = (win.unfold(0, k, 1) * w).sum(-1) + (0 if b is None else b)
                out.append(y * torch.sigmoid(y))
            pool[at[j]] = win[L:L + k - 1]
            t += L
        return torch.cat(out) if out else x, pool
    if op == "commit":
        pool, cpool, x, t = f(st["state"]), f(st["cstate"]), f(st["cx"]), 0
        for j, (L, a, k) in enumerate(zip(st["lens"], slot("state", c["n"]), st["steps"].tolist())):
            if k >= 0:
                pool[a] = st["cache"][j, k].double()
                cpool[a] = torch.cat([cpool[a], x[t:t + k + 1]])[-(c["w"] - 1):]
            t += L
        return pool, cpool
    # every sequence's token j at once, the longest sequences first, so that those still running are a prefix
    n = c["b"] if op == "scan1" else c["n"]
    lens = [1] * n if op == "scan1" else st["lens"]
    if max(lens) > 40000:
        return None
    starts = [0]
    for L in lens:
        starts.append(starts[-1] + L)
    order = sorted(range(n), key=lambda j: -lens[j])
    dev = st["x"].device
    seq = torch.tensor(order, device=dev)
    begin = torch.tensor([starts[j] for j in order], device=dev)
    pool, rows = f(st["state"]), torch.tensor(slot("state", n), device=dev)
    S = pool[rows[seq]]
    of = torch.arange(c["h"], device=dev) // (c["h"] // c["g"])
    A, bias, D = -torch.exp(f(st["A_log"])), f(st["dt_bias"]), f(st["D"])
    y = torch.zeros(st["x"].shape, dtype=torch.float64, device=dev)
    cache = f(st["cache"]) if op == "scanm" else None
    live = n
    for j in range(max(lens)):
        while live and lens[order[live - 1]] <= j:
            live -= 1
        t = begin[:live] + j
        step = torch.logaddexp(torch.zeros((), dtype=torch.float64, device=dev), st["dt"][t].double() + bias)
        x, B, C = st["x"][t].double(), st["B"][t].double()[:, of], st["C"][t].double()[:, of]
        S[:live] = S[:live] * torch.exp(step * A)[:, :, None, None] + torch.einsum("bh,bhp,bhn->bhpn", step, x, B)
        out = torch.matmul(S[:live], C[..., None])[..., 0] + D[:, None] * x
        if st["z"] is not None:
            gate = st["z"][t].double()
            out = out * gate * torch.sigmoid(gate)
        y[t] = out
        if cache is not None and j < c["pitch"]:
            cache[seq[:live], j] = S[:live]
    if op == "scanm":
        return y, cache
    if idx is None:
        last = torch.empty_like(S)
        last[seq] = S
        return y, last
    pool[rows[seq]] = S
    return y, pool
