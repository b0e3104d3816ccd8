"""Variants that only large calls reach: whole heads of 128 rows a workgroup in
the scan's and the delta rule's decodes (bit by bit against the same requests in
small batches, whose workgroups take 32 rows), and vocabularies whose parts are
searched in several steps."""
import pytest
import torch

import gated_delta_rule_51_amd as kda
import kda_workloads as W
import serve_ref as R
from test_gpu_drafts import check, make
from test_gpu_ssm import Layer, offsets, states

pytestmark = pytest.mark.gpu
F32, BF, I32 = torch.float32, torch.bfloat16, torch.int32


def cut(t, a, b):
    return None if t is None else t[a:b]


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("sd", [F32, BF], ids=["states-f32", "states-bf16"])
@pytest.mark.parametrize("S", [32, 64, 128])
def test_runs_of_whole_heads(io, sd, S):
    """72 requests x 16 heads of 128 rows: more than 1024 heads."""
    P, H, G, B, L = 128, 16, 4, 72, [1, 3, 2, 0, 4, 2] * 12
    m = Layer(S, sum(L), H, P, S, G, io)
    first = states(m, B + 1, sd)
    idx = torch.randperm(B, generator=m.g).to(I32)
    x, dt, A, Bm, C = m.args

    def run(a, b):
        t0, t1 = sum(L[:a]), sum(L[:b])
        pool, cache = first.cuda(), torch.full((b - a, 3, H, P, S), 5.0, dtype=sd, device="cuda")
        y = kda.ssm_decode_multi(x[t0:t1], dt[t0:t1], A, Bm[t0:t1], C[t0:t1], offsets(L[a:b]), pool, idx[a:b].cuda(),
                                 intermediate_states=cache, **dict(m.kw, z=cut(m.kw["z"], t0, t1)))
        return y, pool[idx[a:b].long().cuda()], cache

    whole = run(0, B)
    few = [run(a, a + 6) for a in range(0, B, 6)]
    for k in range(3):
        assert torch.equal(whole[k], torch.cat([f[k] for f in few])), k
    ref = m.ref(L[:6], first[idx[:6].long()])
    T = sum(L[:6])
    R.check("y", whole[0][:T], ref["y"][:T], ref["ytol"][:T], io)
    R.check("states", whole[1][:6], ref["last"], ref["ltol"], sd)
    for n in range(6):
        for j in range(3):
            if j < L[n]:
                R.check("step", whole[2][n, j], ref["steps"][n][j], ref["stol"][n][j], sd)
            else:
                assert bool((whole[2][n, j] == 5.0).all())


@pytest.mark.parametrize("io,sd,S", [(BF, F32, 128), (BF, BF, 128), (F32, F32, 64), (BF, F32, 32), (F32, BF, 32), (BF, BF, 64)])
def test_tokens_of_whole_heads(io, sd, S):
    """540 requests x 16 heads of 128 rows: more than 8192 heads."""
    P, H, G, B = 128, 16, 2, 540
    m = Layer(S + 1, B, H, P, S, G, io)
    first = (torch.randn(B + 1, H, P, S, generator=torch.Generator("cuda").manual_seed(S), device="cuda") * 0.5).to(sd)
    idx = torch.randperm(B, generator=m.g).to(I32).cuda()
    idx[7] = -1
    x, dt, A, Bm, C = m.args

    def run(pool, a, b):
        return kda.ssm_decode(x[a:b], dt[a:b], A, Bm[a:b], C[a:b], pool, idx[a:b], **dict(m.kw, z=cut(m.kw["z"], a, b)))

    pool, small = first.clone(), first.clone()
    y = run(pool, 0, B)
    assert torch.equal(y, torch.cat([run(small, a, a + 60) for a in range(0, B, 60)])) and torch.equal(pool, small)
    at = torch.where(idx[:9] < 0, B, idx[:9]).long()
    ref = m.ref([1] * 9, first[at].cpu())
    R.check("y", y[:9], ref["y"][:9], ref["ytol"][:9], io)
    R.check("states", pool[at], ref["last"], ref["ltol"], sd)


@pytest.mark.parametrize("cache", [BF, F32], ids=["cache-bf16", "cache-f32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (32, 128), (128, 64), (32, 64)])
def test_delta_rule_runs(cache, dk, dv):
    """The delta rule's verify decode with step caches: a large batch gives the
    bits of small ones, state by state."""
    B, H, L = 144, 16, [1, 3, 2, 0, 4, 2] * 24
    d = W.make_multi_decode(dk + dv, L, H, H, dk, dv, num_slots=B + 1, cache_pitch=4)
    q, k, v, g, beta = (getattr(d.tok, name).cuda() for name in ("q", "k", "v", "g", "beta"))
    pool0, idx = d.pool.to(cache).cuda(), torch.randperm(B).to(I32).cuda()

    def run(a, b):
        t0, t1 = sum(L[:a]), sum(L[:b])
        steps = torch.full((b - a, 4, H, dv, dk), 5.0, dtype=cache, device="cuda")
        pool = pool0.clone()
        o = kda.recurrent_decode_multi(*(t[t0:t1] for t in (q, k, v, g, beta)), offsets(L[a:b]), pool, idx[a:b].clone(),
                                       intermediate_states=steps, update_pool=True)
        return o, steps, pool[idx[a:b].long()]

    whole, few = run(0, B), [run(a, a + 6) for a in range(0, B, 6)]
    for n in range(3):
        assert torch.equal(whole[n], torch.cat([f[n] for f in few])), n
    last = [n for n in range(B) if L[n]]
    assert torch.equal(whole[2][last], torch.stack([whole[1][n, L[n] - 1] for n in last]))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("V", [262145, 300000, 524289, 600001])
def test_parts_of_several_steps(V, with_q, dtype):
    """Parts of more than 1024 tokens, and of more than the 2048 that a step of
    the search for the token takes."""
    lens = [3, 2, 1, 0, 1, 2, 1, 1, 3, 1, 1, 1]
    p, q, tokens, u, r = make(V, lens, V, dtype)
    r[-1], r[-2] = 1 - 2.0 ** -24, 0.0
    check(kda, lens, p, q if with_q else None, tokens, u, r)


@pytest.mark.parametrize("V", [20001, 40001])
def test_token_whatever_the_batch(V):
    """Random numbers on and next to the borders of the running sums: a request
    among 300 (rows summed by one workgroup at the smaller V) finds the token that
    it finds alone (by several, with a second launch)."""
    g = torch.Generator().manual_seed(V)
    p = torch.softmax(2.5 * torch.randn(1, V, generator=g), 1)
    cum = p.double().cumsum(1)[0]
    r = (cum[torch.randint(0, V - 1, (100,), generator=g)] / cum[-1]).float()
    r = torch.cat([r, torch.nextafter(r, torch.zeros(())), torch.nextafter(r, torch.ones(()))]).clamp(0, 1 - 2.0 ** -24)
    n = len(r)
    tokens, u = torch.zeros(n, dtype=I32, device="cuda"), torch.zeros(n, device="cuda")
    many = kda.verify_drafts(tokens, p.expand(n, V).contiguous().cuda(), offsets([1] * n), u, r.cuda())[1]
    one = p.cuda()
    alone = [kda.verify_drafts(tokens[:1], one, offsets([1]), u[:1], x.clone())[1] for x in r.cuda().split(1)]
    assert torch.equal(many, torch.cat(alone))
