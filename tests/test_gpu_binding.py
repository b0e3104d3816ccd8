"""The native call and the Python checks that name its refusals accept the same
calls: every accepted call runs natively, and with the native module out of the
way the Python checks find nothing wrong with it."""
import pytest
import torch

import gated_delta_rule_51_amd as kda

pytestmark = pytest.mark.gpu
F32, BF, I32 = torch.float32, torch.bfloat16, torch.int32


def zeros(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def ints(*values):
    return torch.tensor(values, dtype=I32, device="cuda")


def conv_calls():
    for io in (BF, F32):
        for T, D, W in ((0, 16, 4), (1, 7, 2), (5, 24, 3), (9, 1, 4)):
            x, w, cu = zeros(T, D + 8, dtype=io)[:, :D], zeros(D, W, dtype=io), ints(0, T)
            pool = zeros(3, W - 1, D, dtype=io)
            steps = ints(*([0] * T)) if T else zeros(0, dtype=I32)
            yield "conv_prefill", (x, w, None, cu), {}
            yield "conv_prefill", (x, w, zeros(D, dtype=io), cu), dict(initial_state=pool, output_final_state=False, activation=None)
            yield "conv_prefill", (x, w, None, cu), dict(initial_state=pool, state_indices=ints(0, 0), update_pool=False)
            yield "conv_decode", (x[:2], w, None, pool, ints(0, 1, 0)), {}
            yield "conv_commit", (x, cu, ints(0, 0), pool, ints(1)), {}
            if T:
                yield "conv_decode", (x[:1].t().contiguous().t(), w, None, pool, steps), {}
        yield "conv_prefill", (zeros(0, 8, dtype=io), zeros(8, 2, dtype=io), None, ints(0)), {}


def scan_calls():
    for io in (BF, F32):
        for T, H, P, G, S in ((0, 2, 32, 1, 32), (1, 1, 64, 1, 128), (6, 4, 128, 2, 64), (3, 10, 32, 5, 32)):
            row, proj = zeros(T, H * P + 2 * G * S + 8, dtype=io), zeros(T, H * P + H + (-(H * P + H)) % 2, dtype=io)
            x, B = row[:, :H * P].unflatten(1, (H, P)), row[:, H * P:H * P + G * S].unflatten(1, (G, S))
            C = row[:, H * P + G * S:H * P + 2 * G * S].unflatten(1, (G, S))
            z, dt, A = proj[:, :H * P].unflatten(1, (H, P)), proj[:, H * P:H * P + H], zeros(H)
            cu, pool, idx = ints(0, T), zeros(max(3, T + 1), H, P, S), zeros(T + 2, dtype=I32)
            idx[:T] = torch.arange(T, dtype=I32)
            args = (x, dt, A, B, C)
            more = dict(D=A, z=z, dt_bias=A)
            long = tuple(torch.cat([t, t[:1]]) if t.dim() > 1 and T else t for t in args)    # rows behind the last token
            yield "ssm_prefill", (*args, cu), {}
            yield "ssm_prefill", (*args, cu), dict(more, initial_state=pool, state_indices=idx)
            yield "ssm_prefill", (*args, cu), dict(initial_state=pool.to(BF), output_final_state=False, state_dtype=BF)
            yield "ssm_prefill", (x, *long[1:], cu), dict(more, state_dtype=BF)
            yield "ssm_decode", (*args, pool, idx), more
            yield "ssm_decode", (x, *long[1:], pool.to(BF), idx), {}
            yield "ssm_decode_multi", (*args, cu, pool, idx), more
            for cache in (zeros(1, 4, H, P, S), zeros(3, 4, H, P, S)[:, :1], zeros(3, H, P, S)[:, None], zeros(2, 0, H, P, S)):
                yield "ssm_decode_multi", (*args, cu, pool, idx), dict(more, intermediate_states=cache, update_pool=False)
                yield "commit_states", (pool, idx, cache, ints(0)), {}


def verify_calls():
    for io in (BF, F32):
        for T, V in ((0, 5), (1, 1), (4, 33), (4, 64)):
            p, u, r, cu = zeros(T + 1, V + 3, dtype=io)[:, :V], zeros(T + 2), zeros(2), ints(0, T)
            yield "verify_drafts", (zeros(T, dtype=I32), p, cu, u, r), {}
            yield "verify_drafts", (zeros(T, dtype=I32), p, cu, u, r), dict(draft_probs=zeros(T, V, dtype=io))


CALLS = [c for calls in (conv_calls, scan_calls, verify_calls) for c in (calls,)]


@pytest.mark.parametrize("calls", CALLS, ids=[c.__name__ for c in CALLS])
def test_accepted_by_both(calls, monkeypatch):
    for n, (name, args, kw) in enumerate(calls()):
        print(n, name, [None if a is None else (tuple(a.shape), a.stride()) for a in args], sorted(kw), flush=True)
        with monkeypatch.context() as m:
            m.setattr(kda, "_run", lambda *a: None)
            with pytest.raises(kda.KdaError, match="plain strided"):
                getattr(kda, name)(*args, **kw)
        getattr(kda, name)(*args, **kw)
    torch.cuda.synchronize()


def test_refused_by_both():
    """Calls that the native module declines and the Python checks name."""
    x, w, cu, idx = zeros(4, 16), zeros(16, 4), ints(0, 4), ints(0, 1, 2, 3)
    pool = zeros(5, 3, 16)
    X, dt, A, B, S = zeros(4, 2, 32), zeros(4, 2), zeros(2), zeros(4, 1, 32), zeros(5, 2, 32, 32)
    p, tok, u, r = zeros(4, 9), zeros(4, dtype=I32), zeros(4), zeros(1)
    refused = [
        ("conv_prefill", (x, w[:8], None, cu), {}), ("conv_prefill", (x.double(), w.double(), None, cu), {}),
        ("conv_prefill", (x, w, None, cu.long()), {}), ("conv_prefill", (x, w, None, cu), dict(state_indices=idx)),
        ("conv_prefill", (x, w, zeros(8), cu), {}), ("conv_prefill", (x, w, None, zeros(0, dtype=I32)), {}),
        ("conv_decode", (x, w, None, pool, idx[:3]), {}), ("conv_decode", (x, w, None, pool[:, :2], idx), {}),
        ("conv_commit", (x, cu, zeros(0, dtype=I32), pool, idx), {}), ("conv_commit", (x[:, :8], cu, idx, pool, idx), {}),
        ("ssm_prefill", (X, dt[:3], A, B, B, cu), {}), ("ssm_prefill", (X, dt, A, B, B[:, :, :16], cu), {}),
        ("ssm_prefill", (X, dt, A.double(), B, B, cu), {}), ("ssm_prefill", (X, dt, A, B, B, cu), dict(z=X[:, :1])),
        ("ssm_prefill", (X, dt, A, B, B, cu), dict(initial_state=S[0:0])), ("ssm_prefill", (X.transpose(1, 2), dt, A, B, B, cu), {}),
        ("ssm_decode", (X, dt, A, B, B, S, idx[:1]), {}), ("ssm_decode", (X, dt, A, B, B, S.transpose(2, 3)[:, :, :, :16], idx), {}),
        ("ssm_decode_multi", (X, dt, A, B, B, cu, S, idx), dict(intermediate_states=S[None, :, :1])),
        ("ssm_decode_multi", (X, dt, A, B, B, cu, S, idx), dict(intermediate_states=S.to(BF)[None])),
        ("verify_drafts", (tok, p[:2], cu, u, r), {}), ("verify_drafts", (tok, p, cu, u, r), dict(draft_probs=p.to(BF))),
        ("verify_drafts", (tok, p, cu, u, zeros(0)), {}), ("verify_drafts", (tok, p.t().contiguous().t(), cu, u, r), {}),
        ("commit_states", (S, idx, S[None, :, :1], ints(0)), {}), ("commit_states", (S, idx[:1], S[None], ints(0, 0)), {}),
    ]
    for name, args, kw in refused:
        with pytest.raises(ValueError):
            getattr(kda, name)(*args, **kw)
            print("accepted:", name, [tuple(a.shape) for a in args if a is not None], kw.keys(), flush=True)
