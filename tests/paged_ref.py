"""Definitions of the paged cache, its attention and the choice of the next
token, in 64 bits on the host, with the error bounds the GPU tests hold the
kernels to.

Bounds of the attention.  e = 2^-23 for every fp32 operation (a matrix-core
accumulation may truncate).  A score is a sum of D exact products: it is off by
(D + 2) e A, A the largest scale * sum |q k| that a column has; the reference
subtracted is of that size too, and scaling, subtraction and the exponential's
argument round three times, exp2 by one step: a numerator is off by
ep = e ((D + 10) A + 8), relative.  fp32 io adds the operands' remainder after
three bf16 terms, below e.  Numerators rounded to bf16, p_i (1 + d_i) with |d_i| <=
2^-8, in the product and in its divisor alike move o by sum d_i p_i (v_i - o) / sum p
to first order: at most 2^-8 (sum p |v| / sum p + |o|).  Sums over n keys add (n +
64) e to the numerators' sum and to the product's.  All else goes with sum p |v| /
sum p, and the output's own rounding with |o|.
"""
import numpy as np
import torch

E32 = 2.0 ** -23
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
LEAST = -100


def e4m3(x):
    """To the nearest value of 4 exponent and 3 fraction bits, ties to even; not
    finite: NaN.  |x| <= 448."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    y = np.where(fine, x, 0)
    e = np.maximum(np.frexp(y)[1] - 1, -6)
    return np.where(fine, np.ldexp(np.rint(np.ldexp(y, 3 - e)), e - 3), np.nan)


def scale_for(top):
    """The least power of two s >= 2^LEAST with top <= 448 s, by trial."""
    s = 2.0 ** LEAST
    while top > 448 * s:
        s *= 2
    return s


class Pages:
    """Block tables on the host: the state and the calls of kv_reserve, kv_commit
    and kv_release, request by request."""

    def __init__(self, rows, max_blocks, block_size, free):
        self.bs = block_size
        self.lens, self.held = [0] * rows, [0] * rows
        self.table = [[-1] * max_blocks for _ in range(rows)]
        self.free, self.count = list(free), len(free)

    def reserve(self, cu, idx, T):
        slots, totals, full = [-1] * T, [], False
        for n, r in enumerate(idx):
            L = cu[n + 1] - cu[n]
            if not 0 <= r < len(self.lens):
                totals.append(0)
                continue
            total = self.lens[r] + L
            want = -(-total // self.bs)
            need = max(want - self.held[r], 0)
            if want > len(self.table[r]):
                totals.append(0)
                continue
            full = full or need > self.count
            if need and full:
                totals.append(0)
                continue
            for _ in range(need):
                self.count -= 1
                self.table[r][self.held[r]] = self.free[self.count]
                self.held[r] += 1
            totals.append(total)
            for j in range(L):
                p = self.lens[r] + j
                slots[cu[n] + j] = self.table[r][p // self.bs] * self.bs + p % self.bs
        return slots, totals

    def commit(self, cu, idx, steps=None):
        for n, r in enumerate(idx):
            L = cu[n + 1] - cu[n]
            s = L - 1 if steps is None else steps[n]
            if 0 <= r < len(self.lens) and 0 <= s < L and self.lens[r] + s + 1 <= self.held[r] * self.bs:
                self.lens[r] += s + 1

    def release(self, idx, keep=None):
        back = []
        for n, r in enumerate(idx):
            if not 0 <= r < len(self.lens):
                continue
            self.lens[r] = min(self.lens[r], 0 if keep is None else max(keep[n], 0))
            left = -(-self.lens[r] // self.bs)
            back += self.table[r][left:self.held[r]]
            self.held[r] = min(self.held[r], left) if self.held[r] > left else self.held[r]
        for b in reversed(back):
            if self.count < len(self.free):
                self.free[self.count] = b
                self.count += 1


def store(x, slots, cache, scale):
    """x [T, H, D] float64 into cache [B, H, bs, D] and scale [B, H], token runs one
    by one, in place."""
    B, H, bs, D = cache.shape
    t = 0
    while t < len(slots):
        s = slots[t]
        if not 0 <= s < B * bs:
            t += 1
            continue
        b, f, m = s // bs, s % bs, 1
        while t + m < len(slots) and slots[t + m] == s + m and f + m < bs:
            m += 1
        for h in range(H):
            run = x[t:t + m, h]
            fine = np.abs(run[np.isfinite(run)])
            new = max(scale_for(fine.max() if fine.size else 0.0), scale[b, h] if f else 0.0)
            if f and new > scale[b, h]:
                cache[b, h, :f] = e4m3(cache[b, h, :f] * (scale[b, h] / new))
            cache[b, h, f:f + m] = e4m3(run / new)
            scale[b, h] = new
        t += m


def attention(q, cu, totals, idx, table, k_cache, v_cache, k_scale, v_scale, scale, io):
    """(o, bound before rounding) [T, Hq, D]; k_cache [B, H, bs, D], v_cache [B, H, D,
    bs] of stored values, all float64."""
    T, Hq, D = q.shape
    B, H, bs, _ = k_cache.shape
    g = Hq // H
    o, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for n in range(len(cu) - 1):
        L, r = cu[n + 1] - cu[n], idx[n]
        if not L or not 0 <= r < len(table):
            continue
        total = min(max(totals[n], 0), len(table[r]) * bs)
        page = np.asarray(table[r][:-(-total // bs)], np.int64)
        there = (page >= 0) & (page < B)
        page = np.where(there, page, 0)
        real = np.repeat(there, bs)[:total]
        for h in range(H):
            k = (k_cache[page, h] * k_scale[page, h][:, None, None]).reshape(-1, D)[:total]
            v = (v_cache[page, h].transpose(0, 2, 1) * v_scale[page, h][:, None, None]).reshape(-1, D)[:total]
            for j in range(L):
                last = total - L + j
                see = np.flatnonzero(real & (np.arange(total) <= last))
                if not len(see):
                    continue
                for i in range(h * g, h * g + g):
                    x = q[cu[n] + j, i]
                    z = scale * (k[see] @ x)
                    A = scale * (np.abs(k[see]) @ np.abs(x)).max()
                    p = np.exp(z - z.max())
                    o[cu[n] + j, i] = p @ v[see] / p.sum()
                    ep = E32 * ((D + 10) * A + 8)
                    near = 2 * ep + (2.0 ** -8 if io == torch.bfloat16 else 4 * E32) + 2 * (len(see) + 64) * E32
                    tol[cu[n] + j, i] = near * (p @ np.abs(v[see])) / p.sum()
                    if io == torch.bfloat16:
                        tol[cu[n] + j, i] += 2.0 ** -8 * np.abs(o[cu[n] + j, i])
    return o, tol


def check(name, got, ref, tol, dtype):
    got = got.detach().cpu().double().numpy()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), name
    got, ref, tol = (np.where(np.isnan(ref), 0, a) for a in (got, ref, tol))
    assert np.isfinite(got).all(), name
    if not ref.size:
        return
    over = np.abs(got - ref) - (tol + HALF[dtype] * (np.abs(ref) + tol))
    rel = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300)
    print("%s: rel-L2 %.3e, worst past its bound %.3e" % (name, rel, over.max()), flush=True)
    assert over.max() <= 1e-30, (name, np.unravel_index(over.argmax(), over.shape))


def sample(logits, u=None, temperature=None, top_k=None, top_p=None, min_p=None):
    """(tokens, probabilities) of logits [N, V] float64; limits as lists or None."""
    N, V = logits.shape
    tokens, probs = [], np.zeros((N, V))
    for n in range(N):
        x = logits[n]
        get = lambda a, d: d if a is None else float(a[n])  # noqa: E731
        t, k, p, m = get(temperature, 1.0), int(get(top_k, 0)), get(top_p, 1.0), get(min_p, 0.0)
        order = [i for i in sorted(range(V), key=lambda i: (-x[i] if x[i] == x[i] else np.inf, i)) if x[i] == x[i]]
        if not order or x[order[0]] == -np.inf:
            tokens.append(-1)
            continue
        top = x[order[0]]
        if not t > 0:
            tokens.append(order[0])
            probs[n, order[0]] = 1
            continue
        with np.errstate(invalid="ignore"):
            w = np.array([1.0 if x[i] == top else np.exp((x[i] - top) / t) for i in order])
        if 0 < k < V:
            w = w[:k]
        if p < 1:
            part = np.cumsum(w)
            w = w[:1 + int(np.searchsorted(part, max(p, 0.0) * part[-1]))]
        w = w[w >= min(m, 1.0)]
        probs[n, order[:len(w)]] = w
        part = np.cumsum(probs[n])
        if u is not None:
            tokens.append(int(np.searchsorted(part, float(u[n]) * part[-1], side="right")))
        probs[n] /= part[-1]
    return tokens, probs
