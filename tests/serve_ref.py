"""64-bit references of the convolution, the state-space scan, draft
verification and commit, token by token, with the error bounds the GPU tests
hold the kernels to.

Bounds.  e = 2^-23 is taken for every fp32 operation (a correctly rounded one
is off by 2^-24, a matrix-core accumulation may truncate), and |.| sums go with
each value.  A rounding to the io or state dtype is off by eps / 2 relative
(bf16 2^-8, fp32 2^-24).

* Convolution: W + 1 sums and products of terms with magnitude m = |bias| +
  sum |w x| give (W + 2) e m; SiLU's slope is at most 1.1; its exponential has
  an argument error of |s| e and its hardware exp2 and reciprocal 1 ulp each:
  |y| (4 + 2 |s|) e.
* Scan.  M is the recursion of magnitudes.  One step multiplies by a decay
  whose relative error is (4 + 4 |a|) e (a = A dt: its own rounding and that of
  the exponential's argument, 1 ulp of exp2, A's exponential), and adds a term
  with 4 roundings, 3 ulp of softplus and its argument: 12 e.  E is the
  recursion of those errors.  Where products are summed 64 tokens at a time the
  sum adds at most 64 e M per block; decayed, over all blocks, at most
  128 e M stays where the decays halve a block's weight, and the recursion
  carries it in general (added once every 64 tokens).
* y adds S + 2 roundings of sum |state| |C|, and, where operands are carried as
  two bf16 terms, their remainder: 2^-16 of it (bf16 io only).
"""
import numpy as np
import torch

E32 = 2.0 ** -23
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def silu(x):
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def slots_of(idx, slots):
    idx = np.asarray(idx.cpu())
    return np.where(idx < 0, slots - 1, idx)


def conv(x, weight, bias, lens, states, activation=True):
    """(y, bound of y before rounding, final states): states [N, W - 1, D]."""
    x, weight, bias, states = f64(x), f64(weight), f64(bias), f64(states)
    D, W = weight.shape
    y, tol, last, t = [], [], states.copy(), 0
    for n, L in enumerate(lens):
        full = np.concatenate([states[n], x[t:t + L]])
        for j in range(L):
            win = full[j:j + W]
            s = (win * weight.T).sum(0) + (0 if bias is None else bias)
            m = (np.abs(win) * np.abs(weight.T)).sum(0) + (0 if bias is None else np.abs(bias))
            o = silu(s) if activation else s
            y.append(o)
            tol.append(E32 * (1.1 * (W + 2) * m + (np.abs(o) * (4 + 2 * np.abs(s)) if activation else 0)))
        last[n] = full[L:L + W - 1]
        t += L
    shape = (0, D)
    return (np.array(y) if y else np.zeros(shape)), (np.array(tol) if tol else np.zeros(shape)), last


def softplus(z):
    return np.logaddexp(0.0, z)


def scan(x, dt, A_log, B, C, lens, states, D=None, z=None, dt_bias=None):
    """Per sequence from states [N, H, P, S]: dict of y, its bound before
    rounding, the last states with their bound, and all steps' states
    (lists [L][H, P, S]) with bounds."""
    x, dt, A_log, B, C, D, z, dt_bias, states = (f64(t) for t in (x, dt, A_log, B, C, D, z, dt_bias, states))
    T, H, P = x.shape
    G, S = B.shape[1:]
    of = np.arange(H) // (H // G)
    A = -np.exp(A_log)
    y, ytol = np.zeros((T, H, P)), np.zeros((T, H, P))
    last, ltol = states.copy(), np.zeros_like(states)
    steps, stol = [], []
    t = 0
    for n, L in enumerate(lens):
        st, M, E = states[n].copy(), np.abs(states[n]), np.zeros_like(states[n])
        all_s, all_e = [], []
        for j in range(L):
            d = softplus(dt[t] + (0 if dt_bias is None else dt_bias))
            a = A * d
            dec = np.exp(a)[:, None, None]
            new = (d[:, None] * x[t])[:, :, None] * B[t][of][:, None, :]
            st = dec * st + new
            E = dec * (E + (4 + 4 * np.abs(a))[:, None, None] * E32 * M) + 12 * E32 * np.abs(new)
            M = dec * M + np.abs(new)
            if j % 64 == 63 or j == L - 1:
                E = E + 64 * E32 * M
            c = C[t][of]
            o = np.einsum("hps,hs->hp", st, c)
            mag = np.einsum("hps,hs->hp", M, np.abs(c))
            tol = np.einsum("hps,hs->hp", E + 64 * E32 * M, np.abs(c)) + (S + 2) * E32 * mag
            rest = mag
            if D is not None:
                o = o + D[:, None] * x[t]
                tol = tol + 2 * E32 * np.abs(D[:, None] * x[t])
                rest = rest + np.abs(D[:, None] * x[t])
            tol = tol + 2.0 ** -16 * rest
            if z is not None:
                zz = z[t]
                g = silu(zz)
                tol = tol * np.abs(g) + np.abs(o * g) * (6 + 2 * np.abs(zz)) * E32
                o = o * g
            y[t], ytol[t] = o, tol
            all_s.append(st.copy())
            all_e.append(E.copy())
            t += 1
        last[n], ltol[n] = st, E
        steps.append(all_s)
        stol.append(all_e)
    return dict(y=y, ytol=ytol, last=last, ltol=ltol, steps=steps, stol=stol)


def check(name, got, ref, tol, dtype):
    """Every value within tol and the rounding to dtype."""
    got = f64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), name
    if not ref.size:
        return
    over = np.abs(got - ref) - (tol + HALF[dtype] * (np.abs(ref) + tol))
    rel = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300)
    print("%s: rel-L2 %.3e, worst past its bound %.3e" % (name, rel, over.max()), flush=True)
    assert over.max() <= 1e-30, (name, np.unravel_index(over.argmax(), over.shape))
    return rel


def verify(tokens, p, cu, u, r, q=None):
    """(accepted, next, emitted) by the definition, in 64 bits but for the
    acceptance test and p - q, which are defined in 32."""
    tokens, cu = tokens.cpu().numpy(), cu.cpu().numpy()
    p = p.detach().cpu().float().numpy()
    q = None if q is None else q.detach().cpu().float().numpy()
    u, r = u.cpu().numpy(), r.cpu().numpy()
    V = p.shape[1]
    acc, nxt = [], []
    emitted = np.full(len(tokens), -7, np.int64)
    for n in range(len(cu) - 1):
        t0, L = cu[n], cu[n + 1] - cu[n]
        if L <= 0:
            acc.append(-1)
            nxt.append(-1)
            continue
        a, wrong = L - 1, None
        for j in range(L - 1):
            d = tokens[t0 + j + 1]
            if not (0 <= d < V and np.float32(u[t0 + j]) * (np.float32(1) if q is None else q[t0 + j, d]) < p[t0 + j, d]):
                a, wrong = j, d
                break
        row = p[t0 + a]
        own = np.where(row > 0, row, 0).astype(np.float64)
        w = own.copy()
        if wrong is not None:
            if q is not None:
                diff = row - q[t0 + a]
                w = np.where(diff > 0, diff, 0).astype(np.float64)
            elif 0 <= wrong < V:
                w[wrong] = 0
        if not w.sum() > 0:
            w = own
        cum = np.cumsum(w)
        past = np.nonzero((cum > np.float64(r[n]) * cum[-1]) & (w > 0))[0]
        some = np.nonzero(w > 0)[0]
        k = int(past[0]) if len(past) else int(some[-1]) if len(some) else -1
        acc.append(a)
        nxt.append(k)
        emitted[t0:t0 + L] = -1
        emitted[t0:t0 + a] = tokens[t0 + 1:t0 + a + 1]
        emitted[t0 + a] = k
    return np.array(acc), np.array(nxt), emitted
