"""Verification of drafted tokens against the 64-bit definition (whole numbers:
equal), the commit of accepted states, and a speculative step of a recurrent
layer run end to end: verify decode, verification, commits, next step."""
import pytest
import torch

import kda_workloads as W
import serve_ref as R

pytestmark = pytest.mark.gpu
F32, BF, I32 = torch.float32, torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


def offsets(lens):
    cu = torch.zeros(len(lens) + 1, dtype=I32)
    cu[1:] = torch.tensor(lens, dtype=I32).cumsum(0)
    return cu


def make(seed, lens, V, dtype, noise=0.7, wide=0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    logits = 2.5 * torch.randn(T, V, generator=g)
    p = torch.zeros(T, V + wide, dtype=dtype)
    p[:, :V] = torch.softmax(logits, 1).to(dtype)
    q = torch.softmax(logits + noise * torch.randn(T, V, generator=g), 1)
    d = torch.multinomial(q, 1, generator=g).flatten() if T else torch.zeros(0, dtype=torch.long)
    tokens = torch.cat([torch.zeros(1, dtype=torch.long), d])[:T].to(I32)
    return p[:, :V], q.to(dtype), tokens, torch.rand(T, generator=g), torch.rand(len(lens), generator=g)


def check(K, lens, p, q, tokens, u, r):
    dev = lambda t: None if t is None else t.cuda() if t.is_contiguous() else t._base.cuda()[:, :t.shape[1]]  # noqa: E731
    got = K.verify_drafts(dev(tokens), dev(p), offsets(lens).cuda(), dev(u), dev(r), draft_probs=dev(q))
    want = R.verify(tokens, p, offsets(lens), u, r, q)
    for name, a, b in zip(("accepted", "next", "emitted"), got, want):
        assert a.cpu().tolist() == b.tolist(), name
    return got


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("V,wide", [(1, 0), (2, 0), (63, 0), (512, 8), (513, 3), (4097, 0), (33333, 0), (150001, 0)])
def test_verify(K, dtype, with_q, V, wide):
    lens = [4, 1, 0, 3, 8, 2, 1, 5]
    p, q, tokens, u, r = make(V, lens, V, dtype, wide=wide)
    check(K, lens, p, q if with_q else None, tokens, u, r)


def test_many_requests_and_long_runs(K):
    lens = [4] * 700 + [1, 0, 130, 65, 66]
    p, q, tokens, u, r = make(5, lens, 300, F32, noise=0.05)
    u[-261:] *= 0.2      # long runs that mostly stand
    acc, _, _ = check(K, lens, p, q, tokens, u, r)
    assert int(acc.max()) > 8


def test_borders(K):
    """Certain drafts, refusals at each place, random numbers at 0 and just
    below 1, rows with no weight left, drafts out of range."""
    V, lens = 6, [3] * 9
    T = 27
    p, q = torch.zeros(T, V), torch.zeros(T, V)
    tokens = torch.zeros(T, dtype=I32)
    u, r = torch.full((T,), 0.5), torch.full((9,), 0.5)

    def req(n, d, prow, qrow, uu, rr):
        for j in range(2):
            tokens[3 * n + j + 1] = d[j]
        for j in range(3):
            p[3 * n + j], q[3 * n + j] = torch.tensor(prow[j]), torch.tensor(qrow[j])
            u[3 * n + j] = uu[j] if j < 2 else 0.0
        r[n] = rr

    one = lambda k: [1.0 if i == k else 0.0 for i in range(V)]  # noqa: E731
    half = [0.0, 0.5, 0.0, 0.5, 0.0, 0.0]
    last = 1 - 2.0 ** -24
    req(0, (1, 3), (half, half, half), (half, half, one(0)), (last, last), 0.0)        # equal rows: stand
    req(1, (0, 3), (half, half, half), (one(0), half, half), (0.0, 0.0), 0.5)          # p = 0: refused at u = 0; r on a border
    req(2, (1, 2), (half, half, half), (half, one(2), half), (0.9, 0.1), last)         # refused at the second
    req(3, (1, 1), (half, half, half), (half, half, half), (last, last), last)         # the last row's own
    req(4, (-1, 1), (half, half, half), (half, half, half), (0.1, 0.1), 0.2)           # outside, below; p - q leaves nothing
    req(5, (1, 6), (half, half, half), (half, half, half), (0.1, 0.1), 0.7)            # outside, above
    req(6, (1, 2), ([0.0] * V,) * 3, (half, half, half), (0.1, 0.1), 0.7)              # no probability anywhere
    nan = float("nan")
    req(7, (1, 2), ([nan] * V, half, half), (half, half, half), (0.1, 0.1), 0.7)       # NaN: refused, weighs nothing
    req(8, (3, 2), ([nan, 0.2, nan, 0.1, 0.0, 0.0],) * 3, ([0.5, 0.1, 0.0, 0.4, 0.0, 0.0],) * 3, (0.5, 0.1), 0.0)
    acc, nxt, _ = check(K, lens, p, q, tokens, u, r)
    assert acc.tolist() == [2, 0, 1, 2, 0, 1, 0, 0, 0]
    assert nxt.tolist() == [1, 3, 3, 3, 1, 3, -1, -1, 1]
    check(K, lens, p, None, tokens, u, r)


@pytest.mark.parametrize("V", [20001, 40001])
def test_many_requests_long_rows(K, V):
    """Rows summed by one workgroup, and by several with a second launch."""
    lens = [1, 3, 2, 0, 1] * 52
    p, q, tokens, u, r = make(V, lens, V, F32)
    check(K, lens, p, q, tokens, u, r)


def test_verify_empty(K):
    z = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    acc, nxt, out = K.verify_drafts(z(0, dtype=I32), z(0, 9), offsets([0, 0]).cuda(), z(0), z(2))
    assert acc.tolist() == [-1, -1] and nxt.tolist() == [-1, -1] and out.numel() == 0
    acc, nxt, out = K.verify_drafts(z(0, dtype=I32), z(0, 9), offsets([]).cuda(), z(0), z(0))
    assert acc.numel() == 0


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 32, 32), (3, 64, 32), (8, 128, 128)])
def test_commit(K, dtype, shape):
    g = torch.Generator().manual_seed(3)
    pool0 = torch.randn(9, *shape, generator=g).to(dtype)
    whole = torch.randn(6, 5, *shape, generator=g).to(dtype)
    steps = torch.tensor([0, 3, -1, 2, 4, 1], dtype=I32)
    idx = torch.tensor([4, 0, 2, -1, 6, 7], dtype=I32)
    for cache, there in ((whole, 5), (whole[:, :4], 4)):
        pool = pool0.cuda()
        c = whole.cuda()[:, :there]
        K.commit_states(pool, idx.cuda(), c, steps.cuda())
        want = pool0.clone()
        for n in range(6):
            if 0 <= int(steps[n]) < there:
                want[int(R.slots_of(idx, 9)[n])] = whole[n, int(steps[n])]
        assert torch.equal(pool.cpu(), want)


def layer(seed, T, H, P, S, G):
    g = torch.Generator().manual_seed(seed)
    D = H * P + 2 * G * S
    return dict(x=torch.randn(T, D, generator=g).cuda(), dt=torch.randn(T, H, generator=g).cuda(), A=torch.randn(H, generator=g).cuda(),
                w=torch.randn(D, 4, generator=g).mul(0.4).cuda(), b=torch.randn(D, generator=g).cuda())


def test_speculative_step(K):
    """Prompt, drafted tokens through convolution and scan with the pools only
    read, verification, commits: the pools then hold what a run over the
    accepted tokens alone gives."""
    H, P, S, G, V = 4, 32, 64, 2, 500
    lens, drafted = [40, 3, 70], [4, 1, 3]
    m = layer(1, sum(lens) + sum(drafted), H, P, S, G)
    N, T0 = 3, sum(lens)
    idx = torch.tensor([2, 0, 4], dtype=I32, device="cuda")
    D = H * P + 2 * G * S

    def parts(y):
        return (y[:, :H * P].unflatten(1, (H, P)), y[:, H * P:H * P + G * S].unflatten(1, (G, S)),
                y[:, H * P + G * S:].unflatten(1, (G, S)))

    conv, pool = torch.zeros(6, 3, D, device="cuda"), torch.zeros(6, H, P, S, device="cuda")
    cu = offsets(lens).cuda()
    y, _ = K.conv_prefill(m["x"][:T0], m["w"], m["b"], cu, initial_state=conv, state_indices=idx)
    x, B, C = parts(y)
    K.ssm_prefill(x, m["dt"][:T0], m["A"], B, C, cu, initial_state=pool, state_indices=idx)
    conv1, pool1 = conv.clone(), pool.clone()

    p, q, tokens, u, r = (t.cuda() for t in make(2, drafted, V, F32))
    cd = offsets(drafted).cuda()
    y, _ = K.conv_prefill(m["x"][T0:], m["w"], m["b"], cd, initial_state=conv, state_indices=idx, update_pool=False)
    x, B, C = parts(y)
    cache = torch.zeros(N, 4, H, P, S, device="cuda")
    out = K.ssm_decode_multi(x, m["dt"][T0:], m["A"], B, C, cd, pool, idx, intermediate_states=cache, update_pool=False)
    accepted, _, _ = K.verify_drafts(tokens, p, cd, u, r, draft_probs=q)
    K.commit_states(pool, idx, cache, accepted)
    K.conv_commit(m["x"][T0:], cd, accepted, conv, idx)

    keep = accepted.tolist()
    rows = [T0 + int(cd[n]) + j for n in range(N) for j in range(keep[n] + 1)]
    cut = offsets([k + 1 for k in keep]).cuda()
    y, _ = K.conv_prefill(m["x"][rows], m["w"], m["b"], cut, initial_state=conv1, state_indices=idx)
    x, B, C = parts(y)
    again = K.ssm_decode_multi(x, m["dt"][rows], m["A"], B, C, cut, pool1, idx)
    assert torch.equal(conv, conv1) and torch.equal(pool, pool1)
    assert torch.equal(again, out[[i - T0 for i in rows]])


def test_delta_rule_speculative_step(K):
    """The delta rule's own verify decode, its step cache committed."""
    d = W.make_multi_decode(31, [4, 2, 0, 3], 2, 4, 64, 64, num_slots=9, cache_pitch=4)
    t = {k: getattr(d.tok, k).cuda() for k in ("q", "k", "v", "g", "beta", "cu_seqlens")}
    pool0, idx = d.pool.cuda(), d.indices.cuda()
    cache = torch.zeros(4, 4, 4, 64, 64, device="cuda")
    args = (t["q"], t["k"], t["v"], t["g"], t["beta"])
    pool = pool0.clone()
    K.recurrent_decode_multi(*args, t["cu_seqlens"], pool, idx, intermediate_states=cache, update_pool=False)
    p, q, tokens, u, r = (x.cuda() for x in make(4, [4, 2, 0, 3], 1000, F32))
    accepted, _, _ = K.verify_drafts(tokens, p, t["cu_seqlens"], u, r, draft_probs=q)
    K.commit_states(pool, idx, cache, accepted)
    lens = [a + 1 for a in accepted.tolist()]
    rows = [int(t["cu_seqlens"][n]) + j for n in range(4) for j in range(lens[n])]
    want = pool0.clone()
    K.recurrent_decode_multi(*(x[rows].contiguous() for x in args), offsets(lens).cuda(), want, idx, update_pool=True)
    assert lens[2] == 0 and torch.equal(pool, want)


def test_graph_replays(K):
    """A whole step (two graphs on one stream, replayed in turn) against the
    eager calls."""
    H, P, S, G, V = 4, 64, 64, 2, 40000
    drafted = [4, 2, 3]
    m = layer(5, sum(drafted), H, P, S, G)
    cd, idx = offsets(drafted).cuda(), torch.tensor([2, 0, 4], dtype=I32, device="cuda")
    p, q, tokens, u, r = (t.cuda() for t in make(6, drafted, V, F32))
    conv0, pool0 = torch.randn(6, 3, H * P + 2 * G * S, device="cuda"), torch.randn(6, H, P, S, device="cuda")
    conv, pool, cache = conv0.clone(), pool0.clone(), torch.zeros(3, 4, H, P, S, device="cuda")

    def step():
        y, _ = K.conv_prefill(m["x"], m["w"], m["b"], cd, initial_state=conv, state_indices=idx, update_pool=False)
        x, B, C = (y[:, :H * P].unflatten(1, (H, P)), y[:, H * P:H * P + G * S].unflatten(1, (G, S)),
                   y[:, H * P + G * S:].unflatten(1, (G, S)))
        o = K.ssm_decode_multi(x, m["dt"], m["A"], B, C, cd, pool, idx, intermediate_states=cache, update_pool=False)
        acc, nxt, out = K.verify_drafts(tokens, p, cd, u, r, draft_probs=q)
        K.commit_states(pool, idx, cache, acc)
        K.conv_commit(m["x"], cd, acc, conv, idx)
        o2, _ = K.ssm_prefill(x, m["dt"], m["A"], B, C, cd, initial_state=pool, state_indices=idx)
        return o, acc, nxt, out, o2

    def only():
        return K.verify_drafts(tokens, p, cd, u, r, draft_probs=q)

    want = [t.clone() for t in step()]
    conv_e, pool_e = conv.clone(), pool.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graphs = []
    for f in (step, only):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs = f()
        graphs.append((g, outs))
    for _ in range(3):
        conv.copy_(conv0)
        pool.copy_(pool0)
        torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], want))
        assert all(torch.equal(a, b) for a, b in zip(graphs[1][1], want[1:4]))
        assert torch.equal(conv, conv_e) and torch.equal(pool, pool_e)


def test_two_streams(K):
    """Verifications on two streams at once match the lone calls."""
    lens = [4] * 3
    sets = [[t.cuda() for t in make(s, lens, 120000, F32)] for s in (8, 9)]
    cu = offsets(lens).cuda()
    run = lambda a: K.verify_drafts(a[2], a[0], cu, a[3], a[4], draft_probs=a[1])  # noqa: E731
    want = [run(a) for a in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for s, a in zip(streams, sets):
        with torch.cuda.stream(s):
            got.append([run(a) for _ in range(5)])
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for g in gs:
            assert all(torch.equal(x, y) for x, y in zip(w, g))
