"""Cases of the paged-attention and sampling operators: what is timed and compared.

Four operators of one serving step of a model whose recurrent layers stand beside layers of attention:

  reserve  blocks for the tokens that are to come, out of a list of free ones: block tables and slot maps from
           the requests' lengths; and their return (a request cut back or ended)
  store    keys and values into their blocks in 8 bits (e4m3), one power-of-two scale a block and head each
  attend   causal attention over those blocks: one token a request, runs of drafted tokens, prompts
  sample   the next token of given random numbers under temperature, top-k, top-p and min-p, and the
           probabilities it is drawn from, which draft verification takes

``own`` False computes them from elementary torch operations in 32 bits (64 for sampling's weights and sums);
``own`` True calls the package.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
LEAST = -100   # the least exponent of a scale


def listed():
    return [
        # the step of a running batch: one token each of 256 requests, a few of them at a block's end; then cut back
        # to where they were, as after a step that is taken back
        dict(name="reserve step", op="reserve", n=256, lo=1, hi=1, held=2000, bs=16, pad=8),
        # prompts coming in and, ended again, giving all back: 96 of up to 2500 tokens
        dict(name="reserve prompts", op="reserve", n=96, lo=50, hi=2500, held=0, bs=64, pad=0),
        # one token each of 256 requests into blocks that are partly filled, 8 heads of 128
        dict(name="store step", op="store", n=256, lo=1, hi=1, held=250, hk=8, d=128, bs=16, io="bf16"),
        # 16 prompts of 512 to 4096 tokens, keys and values slices of one projection's rows
        dict(name="store prompts", op="store", n=16, lo=512, hi=4096, held=0, hk=8, d=128, bs=64, io="bf16"),
        # one token of one request, 8000 tokens behind it: latency
        dict(name="attend one", op="attend", n=1, lo=1, hi=1, clo=8000, chi=8000, hq=32, hk=8, d=128, bs=64, io="bf16"),
        # one token each of 64 requests of 100 to 16,000 tokens, groups of eight heads
        dict(name="attend tokens", op="attend", n=64, lo=1, hi=1, clo=100, chi=16000, hq=32, hk=4, d=128, bs=64, io="bf16"),
        # drafted tokens: four each of 128 requests, every query head with keys of its own, small blocks
        dict(name="attend drafts", op="attend", n=128, lo=4, hi=4, clo=200, chi=4000, hq=16, hk=16, d=64, bs=16, io="bf16"),
        # prompts behind contexts of other lengths (none to 2000 tokens): the largest
        dict(name="attend prompts", op="attend", n=4, lo=2000, hi=4096, clo=0, chi=2000, hq=32, hk=8, d=128, bs=64, io="bf16"),
        # short prompts in 32 bits, odd lengths, one of them empty, groups of three
        dict(name="attend short f32", op="attend", n=9, lo=0, hi=300, clo=0, chi=150, hq=12, hk=4, d=64, bs=32, io="f32"),
        # one request's next token, 131,072 logits in 32 bits: latency
        dict(name="sample one", op="sample", n=1, v=131072, io="f32", mix="p", probs=False),
        # 256 requests with settings of their own, bf16 logits
        dict(name="sample batch", op="sample", n=256, v=65536, io="bf16", mix="all", probs=False),
        # the probabilities of 32 requests' runs of four, for the verification of drafts; an odd vocabulary
        dict(name="sample probs", op="sample", n=128, v=50001, io="f32", mix="kp", probs=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["reserve", "store", "attend tokens", "attend prompts", "attend tokens", "attend prompts", "sample"])
    bs = rng.choice([16, 32, 64, 128])
    if op == "reserve":
        if rng.random() < 0.5:
            return dict(op="reserve", n=_spread(rng, 1, 1500), lo=1, hi=rng.choice([1, 1, 5]), held=_spread(rng, 10, 4000), bs=bs, pad=rng.randint(0, 5))
        return dict(op="reserve", n=_spread(rng, 1, 90), lo=rng.randint(0, 60), hi=_spread(rng, 70, 2500), held=_spread(rng, 1, 500), bs=bs, pad=rng.randint(0, 5))
    if op == "store":
        heads = dict(hk=rng.choice([1, 2, 3, 4, 8, 16]), d=rng.choice([64, 128]), bs=bs, io=rng.choice(["bf16", "bf16", "f32"]))
        if rng.random() < 0.5:
            return dict(op="store", n=_spread(rng, 1, 1000), lo=1, hi=rng.choice([1, 4]), held=_spread(rng, 10, 250), **heads)
        return dict(op="store", n=_spread(rng, 1, 12), lo=rng.randint(0, 60), hi=_spread(rng, 100, 3500), held=_spread(rng, 1, 200), **heads)
    if op == "sample":
        n = _spread(rng, 1, 250)
        return dict(op="sample", n=n, v=_spread(rng, 300, min(131072, 14000000 // n)), io=rng.choice(["bf16", "f32"]), mix=rng.choice(["t", "k", "p", "kp", "all"]),
                    probs=rng.random() < 0.4)
    hk = rng.choice([1, 2, 4, 8])
    heads = dict(hq=hk * rng.choice([1, 2, 4, 5, 8]), hk=hk, d=rng.choice([64, 128]), bs=bs, io=rng.choice(["bf16", "bf16", "f32"]))
    if op == "attend tokens":
        n = _spread(rng, 1, 200)
        most = max(300, min(16000, 250000 // n))
        run = rng.choice([1, 1, 2, 5])
        return dict(op="attend", n=n, lo=run, hi=run, clo=rng.randint(0, 200), chi=_spread(rng, 250, most), **heads)
    n = _spread(rng, 1, 12)
    most = 2048 if heads["io"] == "bf16" else 700
    return dict(op="attend", n=n, lo=rng.randint(0, 60), hi=_spread(rng, 100, most // (1 + n // 5)), clo=0, chi=_spread(rng, 10, 1500), **heads)


def _lengths(c):
    """Host lengths of the case's requests: new tokens and those held before."""
    r = random.Random(c["n"] * 31 + c["hi"])
    new = [r.randint(c["lo"], c["hi"]) for _ in range(c["n"])]
    if "held" in c:
        old = [r.randint(c["held"] // 2, c["held"]) for _ in range(c["n"])]
    else:
        old = [r.randint(c["clo"], c["chi"]) for _ in range(c["n"])]
    if c["op"] == "attend" and c["lo"] == 0 and c["n"] > 2:
        new[1], old[1] = 0, 0      # a request without anything
    return new, old


def _pages(c, s, seed, dev):
    """Requests on rows of a block table, their blocks scattered over the cache."""
    bs, n = c["bs"], c["n"]
    new, old = _lengths(c)
    gen = np.random.RandomState(seed % (1 << 31))
    s["T"], s["longest"], s["reach"] = sum(new), max(new), max(a + b for a, b in zip(new, old))
    rows = n + 5
    s["wide"] = wide = -(-max(s["reach"], 1) // bs) + 2
    have = [-(-(b if c["op"] == "reserve" else a + b) // bs) for a, b in zip(new, old)]
    more = sum(-(-(a + b) // bs) for a, b in zip(new, old)) - sum(have)
    s["blocks"] = blocks = sum(have) + max(more, 0) + 9
    order = gen.permutation(blocks).astype(np.int32)
    table = np.full((rows, wide), -1, np.int32)
    at = gen.permutation(rows - 1)[:n].astype(np.int32)
    used = 0
    for i in range(n):
        table[at[i], :have[i]] = order[used:used + have[i]]
        used += have[i]
    free = np.zeros(blocks, np.int32)
    free[:blocks - used] = order[used:]
    pad = c.get("pad", 0)      # a batch padded to a captured size: requests of row -1 without tokens
    up = lambda a: torch.as_tensor(np.ascontiguousarray(a), device=dev)  # noqa: E731
    s["cu"] = up(np.concatenate([[0], np.cumsum(new), np.full(pad, sum(new))]).astype(np.int32))
    s["idx"] = up(np.concatenate([at, np.full(pad, -1)]).astype(np.int32))
    s["table"] = up(table)
    lens, held = np.zeros(rows, np.int32), np.zeros(rows, np.int32)
    lens[at], held[at] = old, have
    s["lens"], s["held"], s["free"] = up(lens), up(held), up(free)
    s["count"] = up(np.array([blocks - used], np.int32))
    s["before"] = up(np.concatenate([old, np.zeros(pad)]).astype(np.int32))
    s["totals"] = up(np.array([a + b for a, b in zip(new, old)], np.int32))
    pos = np.concatenate([np.arange(b, a + b) for a, b in zip(new, old)] or [np.zeros(0)]).astype(np.int64)
    of = np.repeat(np.arange(n), new)
    s["slots"] = up((table[at[of], pos // bs].astype(np.int64) * bs + pos % bs).astype(np.int32)) if c["op"] == "store" else None


def _cache(c, s, gen, dev):
    """Blocks that hold keys and values of N(0, 1), their scales, as a store leaves them."""
    b, hk, bs, d = s["blocks"], c["hk"], c["bs"], c["d"]
    e = lambda: (-6 + (torch.rand(b, hk, generator=gen, device=dev) < 0.3).float())  # noqa: E731
    s["ks"], s["vs"] = torch.exp2(e()), torch.exp2(e())
    made = lambda *z: torch.randn(*z, generator=gen, device=dev, dtype=torch.bfloat16).clamp_(-5, 5)  # noqa: E731
    s["kc"] = (made(b, hk, bs, d) / s["ks"][:, :, None, None].bfloat16()).to(F8)
    s["vc"] = (made(b, hk, d, bs) / s["vs"][:, :, None, None].bfloat16()).to(F8)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 1009 + 17)
    rand = lambda *z: torch.randn(*z, generator=gen, device=dev)  # noqa: E731
    s = dict(case=c)
    if c["op"] != "sample":
        _pages(c, s, seed, dev)
    if c["op"] in ("store", "attend"):
        _cache(c, s, gen, dev)
    if c["op"] == "store":
        hk, d = c["hk"], c["d"]
        # some heads' keys are larger than the blocks' so far: their scales grow
        size = torch.exp(0.5 * rand(1, 2 * hk, 1))
        row = (rand(s["T"], 4 * hk, d) * torch.cat([size, size], 1)).to(DT[c["io"]])
        s["k"], s["v"] = row[:, 2 * hk:3 * hk], row[:, 3 * hk:]
    if c["op"] == "attend":
        s["q"] = (rand(s["T"], c["hq"], c["d"]) * 1.5).to(DT[c["io"]])
        s["scale"] = c["d"] ** -0.5
    if c["op"] == "sample":
        n, v = c["n"], c["v"]
        s["logits"] = (3.0 * rand(n, v)).to(DT[c["io"]])
        s["u"] = torch.rand(n, generator=gen, device=dev)
        pick = lambda *z: torch.tensor(z, device=dev)[torch.randint(len(z), (n,), generator=gen, device=dev)]  # noqa: E731
        mix = c["mix"]
        s["t"] = pick(0.7, 0.9, 1.0, 1.2) if mix != "all" else pick(0.0, 0.6, 0.8, 1.0, 1.3)
        s["k"] = pick(20, 50, 64).int() if mix in ("k", "kp") else pick(0, 1, 40, 200).int() if mix == "all" else None
        s["p"] = pick(0.9, 0.95) if mix in ("p", "kp") else pick(0.5, 0.9, 0.97, 1.0) if mix == "all" else None
        s["m"] = pick(0.0, 0.02, 0.1) if mix == "all" else None
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------


def _rows_of(s):
    idx = s["idx"].long()
    return torch.where(idx < 0, s["table"].shape[0] - 1, idx), idx >= 0


def _reserve(s):
    c = s["case"]
    bs, (rows, real), table, cu = c["bs"], _rows_of(s), s["table"], s["cu"].long()
    new = cu[1:] - cu[:-1]
    old, held, count = s["lens"][rows].long(), s["held"][rows].long(), s["count"].long()
    total = old + new
    want = (total + bs - 1) // bs
    fits = real & (want <= table.shape[1])
    need = torch.where(fits, (want - held).clamp(min=0), 0)
    upto = torch.cumsum(need, 0)
    given = fits & ((need == 0) | (upto <= count))
    j = torch.arange(table.shape[1], device=cu.device)[None]
    fresh = given[:, None] & (j >= held[:, None]) & (j < (held + need)[:, None])
    at = count - 1 - ((upto - need)[:, None] + j - held[:, None])
    table[rows] = torch.where(fresh, s["free"][at.clamp(0, s["free"].shape[0] - 1)], table[rows])
    taken = torch.where(given, need, 0)
    s["held"][rows] = (held + taken).int()
    s["count"].sub_(taken.sum().int())
    t = torch.arange(s["T"], device=cu.device)
    n = torch.searchsorted(cu[1:], t, right=True)
    pos = old[n] + t - cu[n]
    slots = torch.where(given[n], table[rows[n], pos // bs] * bs + (pos % bs).int(), -1)
    return slots.int(), torch.where(given, total, 0).int()


def _release(s):
    c = s["case"]
    bs, (rows, real), free = c["bs"], _rows_of(s), s["free"]
    held, keep = s["held"][rows].long(), torch.minimum(s["before"], s["lens"][rows])
    left = (keep.long() + bs - 1) // bs
    give = torch.where(real, (held - left).clamp(min=0), 0)
    upto = torch.cumsum(give, 0)
    j = torch.arange(s["table"].shape[1], device=free.device)[None]
    back = (j >= left[:, None]) & (j < (left + give)[:, None])
    at = s["count"].long() + upto[-1] - 1 - ((upto - give)[:, None] + j - left[:, None])
    wider = torch.cat([free, free.new_zeros(1)])
    wider[torch.where(back, at, free.shape[0])] = s["table"][rows]
    free.copy_(wider[:-1])
    s["held"][rows] = (held - give).int()
    s["lens"][rows] = torch.where(real, keep, s["lens"][rows])
    s["count"].add_(upto[-1].int())


def _store_one(x, slots, cache, scale, bs, tokens_last):
    """x [T, H, D] into cache [B, H, bs, D] (or [B, H, D, bs]) and scale [B, H]."""
    blocks, heads = scale.shape
    real = slots >= 0
    block = torch.where(real, slots // bs, blocks).long()
    off = torch.where(real, slots % bs, bs)
    first = off.new_full((blocks + 1,), bs).scatter_reduce_(0, block, off, "amin")[:blocks]
    most = x.float().abs().nan_to_num(nan=0.0, posinf=0.0).amax(2)
    most = most.new_zeros(blocks + 1, heads).scatter_reduce_(0, block[:, None].expand(-1, heads), most, "amax")[:blocks]
    m, e = torch.frexp(most)      # most = m 2^e, m in [1/2, 1): 448 = 7/8 2^9
    e = torch.where(most > 0, e - 9 + (m > 0.875).int(), LEAST).clamp(min=LEAST)
    wide = torch.ldexp(torch.ones_like(scale), e)
    touched, kept = (first < bs)[:, None], (first > 0)[:, None]
    after = torch.where(touched, torch.where(kept, torch.maximum(scale, wide), wide), scale)
    older = torch.arange(bs, device=off.device)[None] < torch.where(touched & kept, first[:, None], 0)
    older = older[:, None, None, :] if tokens_last else older[:, None, :, None]
    held = cache.float()      # a factor of one leaves what is stored as it is
    held = torch.where(older, (held * (scale / after)[:, :, None, None]).to(F8).float(), held)
    held = torch.cat([held, torch.zeros_like(held[:1])])
    y = (x.float() / torch.cat([after, after.new_ones(1, heads)])[block][:, :, None]).to(F8).float()
    if tokens_last:
        held[block, :, :, off % bs] = y
    else:
        held[block, :, off % bs] = y
    cache.copy_(held[:blocks].to(F8))
    scale.copy_(after)


def _attend(s):
    c = s["case"]
    hq, hk, d, bs, n = c["hq"], c["hk"], c["d"], c["bs"], c["n"]
    g, cu, rows = hq // hk, s["cu"].long(), s["idx"].long()
    pages = s["table"][rows][:, :-(-max(s["reach"], 1) // bs)].clamp(min=0).long()
    S = pages.shape[1] * bs
    k = s["kc"][pages].float() * s["ks"][pages][..., None, None]
    v = s["vc"][pages].float() * s["vs"][pages][..., None, None]
    k = k.permute(0, 2, 4, 1, 3).reshape(n, hk, d, S).contiguous()
    v = v.permute(0, 2, 1, 4, 3).reshape(n, hk, S, d).contiguous()
    L = s["longest"]
    j = torch.arange(L, device=cu.device)
    q = s["q"][(cu[:-1, None] + j).clamp(max=s["T"] - 1)].float()
    q = q.reshape(n, L, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * L, d).contiguous()
    x = torch.matmul(q, k).mul_(s["scale"]).view(n, hk, g, L, S)
    last = s["totals"].long()[:, None] - (cu[1:] - cu[:-1])[:, None] + j      # the last position that a token sees
    hidden = torch.arange(S, device=cu.device) > last[:, :, None]
    x.masked_fill_(hidden[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    x = x.view(n, hk, g * L, S)
    o = torch.matmul(x, v) / x.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(n, hk, g, L, d).permute(0, 3, 1, 2, 4).reshape(n, L, hq, d)
    t = torch.arange(s["T"], device=cu.device)
    of = torch.searchsorted(cu[1:], t, right=True)
    return o[of, t - cu[of]].to(s["q"].dtype)


def _sample(s):
    x = s["logits"].double()
    n, v = x.shape
    greedy = (s["t"] <= 0)[:, None]
    z, order = torch.sort(x / torch.where(greedy, 1.0, s["t"].double()[:, None]), dim=1, descending=True, stable=True)
    w = torch.exp(z - z[:, :1])
    rank = torch.arange(v, device=x.device)[None]
    keep = torch.where(greedy, rank < 1, rank >= 0)
    if s["k"] is not None:
        k = s["k"][:, None]
        keep &= (k <= 0) | (rank < k)
    if s["p"] is not None:
        cum = torch.cumsum(torch.where(keep, w, 0.0), 1)
        p = s["p"].double()[:, None]
        keep &= (p >= 1) | (rank < 1) | (cum - torch.where(keep, w, 0.0) < p * cum[:, -1:])
    if s["m"] is not None:
        keep &= w >= s["m"].double()[:, None]
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    cum = torch.cumsum(w, 1)
    past = (cum > s["u"].double()[:, None] * cum[:, -1:]) & (w > 0)
    token = past.to(torch.uint8).argmax(1).int()
    return (token, (w / cum[:, -1:]).float()) if s["case"]["probs"] else (token,)


def run(s):
    c = s["case"]
    op = c["op"]
    if op == "reserve":
        if own:
            import gated_delta_rule_51_amd as kda
            slots, totals = kda.kv_reserve(s["cu"], s["T"], s["idx"], s["lens"], s["held"], s["table"], s["free"], s["count"], block_size=c["bs"])
            kda.kv_release(s["idx"], s["lens"], s["held"], s["table"], s["free"], s["count"], block_size=c["bs"], keep_lens=s["before"])
        else:
            slots, totals = _reserve(s)
            _release(s)
        return slots, totals, s["table"], s["held"], s["free"], s["count"], s["lens"]
    if op == "store":
        if own:
            import gated_delta_rule_51_amd as kda
            kda.kv_store(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
        else:
            _store_one(s["k"], s["slots"], s["kc"], s["ks"], c["bs"], False)
            _store_one(s["v"], s["slots"], s["vc"], s["vs"], c["bs"], True)
        return s["kc"], s["vc"], s["ks"], s["vs"]
    if op == "attend":
        if own:
            import gated_delta_rule_51_amd as kda
            return kda.kv_attention(s["q"], s["cu"], s["totals"], s["idx"], s["table"], s["kc"], s["vc"], s["ks"], s["vs"], scale=s["scale"])
        return _attend(s)
    if own:
        import gated_delta_rule_51_amd as kda
        kw = dict(temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"])
        return kda.sample_tokens(s["logits"], s["u"], return_probs=c["probs"], **kw) if c["probs"] else (kda.sample_tokens(s["logits"], s["u"], **kw),)
    return _sample(s)


# ---- what a pass cannot do without -----------------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "sample":
        size = 2 if c["io"] == "bf16" else 4
        cells = c["n"] * c["v"]
        return {"bytes": cells * (size + (4 if c["probs"] else 0)), "flops": 2 * cells}
    new, old = _lengths(c)
    T, bs = sum(new), c["bs"]
    if c["op"] == "reserve":
        fresh = sum(max(0, -(-(a + b) // bs) - -(-b // bs)) for a, b in zip(new, old))
        return {"bytes": 4 * (T + 8 * c["n"] + 4 * fresh), "flops": T + 8 * c["n"]}
    row = c["hk"] * c["d"]
    if c["op"] == "store":
        size = 2 if c["io"] == "bf16" else 4
        return {"bytes": T * (2 * row * (size + 1) + 4), "flops": 4 * T * row}
    size = 2 if c["io"] == "bf16" else 4
    pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, old))
    reads = sum(a + b for a, b in zip(new, old) if a)
    return {"bytes": 2 * T * c["hq"] * c["d"] * size + reads * 2 * row, "flops": 4 * c["d"] * c["hq"] * pairs}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------


def _exact_attend(s):
    c = s["case"]
    hq, hk, d, bs = c["hq"], c["hk"], c["d"], c["bs"]
    out = torch.zeros(s["T"], hq, d, dtype=torch.float64, device=s["q"].device)
    cu, table, idx, totals = s["cu"].tolist(), s["table"].tolist(), s["idx"].tolist(), s["totals"].tolist()
    for n in range(c["n"]):
        a, b, total = cu[n], cu[n + 1], totals[n]
        if a == b:
            continue
        page = torch.tensor(table[idx[n]][:-(-total // bs)], device=out.device)
        keys = (s["kc"][page].double() * s["ks"][page].double()[:, :, None, None]).transpose(1, 2).reshape(-1, hk, d)[:total]
        vals = (s["vc"][page].double() * s["vs"][page].double()[:, :, None, None]).permute(0, 3, 1, 2).reshape(-1, hk, d)[:total]
        see = torch.arange(total, device=out.device)[None] <= torch.arange(total - (b - a), total, device=out.device)[:, None]
        for h in range(hq):
            z = (s["q"][a:b, h].double() * s["scale"]) @ keys[:, h // (hq // hk)].t().contiguous()
            out[a:b, h] = torch.softmax(torch.where(see, z, -math.inf), 1) @ vals[:, h // (hq // hk)].contiguous()
    return out


def _exact_store(x, slots, cache, scale, bs, tokens_last):
    """Block by block on the host: values [as cache], scales."""
    c, sc = cache.float().cpu().numpy().astype(np.float64), scale.cpu().numpy().astype(np.float64)
    if tokens_last:
        c = c.transpose(0, 1, 3, 2)
    x, slots = x.double().cpu().numpy(), slots.cpu().numpy()
    runs = np.flatnonzero(np.r_[True, (slots[1:] != slots[:-1] + 1) | (slots[1:] % bs == 0)]) if len(slots) else []
    for i, a in enumerate(runs):
        b = runs[i + 1] if i + 1 < len(runs) else len(slots)
        if slots[a] < 0:
            continue
        blk, off = slots[a] // bs, slots[a] % bs
        top = np.abs(x[a:b]).max((0, 2))
        need = np.where(top > 0, np.maximum(np.ceil(np.log2(np.maximum(top, 1e-300) / 448)), LEAST), LEAST)
        s1 = np.maximum(2.0 ** need, sc[blk] if off else 0)
        if off:
            c[blk, :, :off] = _e4m3(c[blk, :, :off] * (sc[blk] / s1)[:, None, None])
        c[blk, :, off:off + b - a] = _e4m3(x[a:b].transpose(1, 0, 2) / s1[:, None, None])
        sc[blk] = s1
    return (c.transpose(0, 1, 3, 2) if tokens_last else c), sc


def _e4m3(x):
    """To the nearest value of 4 exponent and 3 fraction bits, ties to the even one."""
    e = np.maximum(np.frexp(x)[1] - 1, -6)
    return np.ldexp(np.rint(np.ldexp(x, 3 - e)), e - 3)


def _exact_sample(s):
    """Row by row from the threshold that the three limits set."""
    x, u = s["logits"].double().cpu().numpy(), s["u"].double().cpu().numpy()
    get = lambda k: None if s[k] is None else s[k].double().cpu().numpy()  # noqa: E731
    t, k, p, m = get("t"), get("k"), get("p"), get("m")
    probs, tokens = np.zeros_like(x), []
    for n, row in enumerate(x):
        order = np.lexsort((np.arange(len(row)), -row))
        w = np.exp((row[order] - row[order[0]]) / (t[n] if t[n] > 0 else 1))
        last = 1 if t[n] <= 0 else len(row)
        if k is not None and k[n] > 0:
            last = min(last, int(k[n]))
        if p is not None and p[n] < 1:
            part = np.cumsum(w[:last])
            last = min(last, 1 + int(np.searchsorted(part, p[n] * part[-1])))
        if m is not None:
            last = min(last, int((w >= m[n]).sum()))
        probs[n, order[:last]] = w[:last]
        part = np.cumsum(probs[n])
        tokens.append(int(np.searchsorted(part, u[n] * part[-1], side="right")))
        probs[n] /= part[-1]
    return torch.tensor(tokens, dtype=torch.int32), torch.from_numpy(probs)


def exact(case, seed):
    c = case
    if c["op"] == "reserve":      # whole numbers: nothing is rounded
        return None
    s = prepare(case, seed)
    if c["op"] == "attend":
        return _exact_attend(s)
    if c["op"] == "store":
        if s["blocks"] * c["hk"] * c["bs"] * c["d"] > 200e6:
            return None
        kc, ks = _exact_store(s["k"], s["slots"], s["kc"], s["ks"], c["bs"], False)
        vc, vs = _exact_store(s["v"], s["slots"], s["vc"], s["vs"], c["bs"], True)
        return tuple(torch.from_numpy(np.ascontiguousarray(a)) for a in (kc, vc, ks, vs))
    if c["n"] * c["v"] > 20e6:
        return None
    return _exact_sample(s)
