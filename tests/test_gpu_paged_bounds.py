"""The paged cache's calls through the C ABI, every array inside a larger one: nothing
in front of or behind what a call describes is written, rows of o behind the last
request stay as they were, and a workspace of just the size asked for is enough."""
import ctypes
import random

import numpy as np
import pytest
import torch

from test_gpu_kv import Cache, layout, up

pytestmark = pytest.mark.gpu
F32, BF, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
PAD = 4096


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


class Guarded:
    """n bytes with PAD bytes of a pattern on either side."""

    def __init__(self, n, like=None):
        self.n = n
        self.all = torch.full((n + 2 * PAD,), 0xa5, dtype=U8, device="cuda")
        if like is not None:
            self.all[PAD:PAD + n] = like.contiguous().view(-1).view(U8)

    def ptr(self):
        return ctypes.c_void_p(self.all.data_ptr() + PAD)

    def view(self, dtype, *shape):
        return self.all[PAD:PAD + self.n].view(dtype).view(*shape)

    def intact(self):
        return bool((self.all[:PAD] == 0xa5).all()) and bool((self.all[PAD + self.n:] == 0xa5).all())


def guarded(t):
    return Guarded(t.numel() * t.element_size(), t)


def stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


ATTEND = [   # lengths, held, Hq, H, D, bs, io
    ([1] * 5, [3000, 0, 17, 700, 64], 8, 2, 128, 64, BF),
    ([4, 1, 0, 5], [600, 3, 2, 900], 16, 4, 64, 16, BF),
    ([4] * 300, [40] * 300, 4, 1, 64, 16, F32),
    ([150, 33, 0, 90], [700, 0, 5, 90], 8, 2, 128, 32, BF),
    ([150, 33, 0, 90], [700, 0, 5, 90], 6, 2, 64, 32, F32),
    ([1300, 0, 801], [30, 2, 0], 64, 8, 64, 64, BF),
    ([45] * 270, [0] * 270, 6, 2, 128, 128, F32),
]


@pytest.mark.parametrize("lens,old,Hq,H,D,bs,io", ATTEND, ids=[str(i) for i in range(len(ATTEND))])
def test_attention(K, lens, old, Hq, H, D, bs, io):
    L, g = K.lib(), torch.Generator().manual_seed(len(lens))
    blocks = sum(-(-(a + b) // bs) for a, b in zip(lens, old)) + 2
    table, at, cu = layout(lens, old, bs, blocks, 2)
    kc, vc = (torch.randint(0, 0x70, s, dtype=U8, generator=g).cuda() for s in ((blocks, H, bs, D), (blocks, H, D, bs)))
    ks = vs = torch.full((blocks, H), 2.0 ** -6, device="cuda")
    T, N = int(cu[-1]) + 7, len(lens)
    q = torch.randn(T, Hq, D, generator=g).to(io).cuda()
    d = K.KvDesc(num_seqs=N, total_tokens=T, q_heads=Hq, kv_heads=H, head_dim=D, block_size=bs, num_blocks=blocks, rows=len(table),
                 max_blocks=table.shape[1], io_dtype=int(io == BF), scale=D ** -0.5, q_stride=Hq * D, k_stride=H * D, v_stride=H * D)
    need = L.kda_kv_attention_workspace_size(ctypes.byref(d))
    ws, o = Guarded(need), guarded(torch.full((T, Hq, D), 7.0, dtype=io))
    ins = [guarded(x) for x in (q, up(cu), up([a + b for a, b in zip(lens, old)]), up(at), up(table), kc, vc, ks, vs)]
    for _ in range(2):
        assert L.kda_kv_attention(ctypes.byref(d), *[x.ptr() for x in ins], o.ptr(), ws.ptr() if need else None, need, stream()) == 0
    torch.cuda.synchronize()
    assert ws.intact() and o.intact() and all(x.intact() for x in ins)
    got = o.view(io, T, Hq, D)
    assert bool((got[T - 7:] == 7.0).all()) and not bool((got[:T - 7] == 7.0).all(2).any())
    assert bool(got.isfinite().all())


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,v,stride", [(1, 70001, 70001), (5, 4099, 4200), (300, 257, 261), (3, 1, 1), (2, 131072, 131077)])
def test_sample(K, n, v, stride, io):
    L, g = K.lib(), torch.Generator().manual_seed(v)
    x = torch.randn(n, stride, generator=g).to(io)
    d = K.SampleDesc(num_rows=n, vocab=v, logits_dtype=int(io == BF), stride=stride)
    need = L.kda_sample_tokens_workspace_size(ctypes.byref(d))
    r = random.Random(v)
    ins = [guarded(y.cuda()) for y in (x, torch.rand(n, generator=g), torch.tensor([r.choice([0.0, 0.7, 5.0]) for _ in range(n)]),
                                       torch.tensor([r.choice([0, 50, 2000, v]) for _ in range(n)], dtype=I32),
                                       torch.tensor([r.choice([0.5, 0.9, 1.0]) for _ in range(n)]), torch.tensor([r.choice([0.0, 0.01]) for _ in range(n)]))]
    ws, tokens, probs = Guarded(need), Guarded(n * 4), Guarded(n * v * 4)
    assert L.kda_sample_tokens(ctypes.byref(d), *[y.ptr() for y in ins], tokens.ptr(), probs.ptr(), ws.ptr(), need, stream()) == 0
    torch.cuda.synchronize()
    assert ws.intact() and tokens.intact() and probs.intact() and all(y.intact() for y in ins)
    t, p = tokens.view(I32, n), probs.view(F32, n, v)
    assert bool(((t >= 0) & (t < v)).all()) and bool((p.gather(1, t[:, None].long()) > 0).all())
    assert float((p.double().sum(1) - 1).abs().max()) < 2.0 ** -20


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,D,bs", [(1, 64, 16), (3, 128, 64), (8, 64, 128)])
def test_store(K, H, D, bs, io):
    L, g, blocks = K.lib(), torch.Generator().manual_seed(bs), 7
    slots = list(range(0, 3)) + list(range(bs, 3 * bs)) + [-1, blocks * bs, (1 << 31) - 1] + list(range(blocks * bs - bs + 1, blocks * bs)) + [4 * bs + 5]
    c = Cache(blocks, H, bs, D)
    c.ks.fill_(1.0), c.vs.fill_(1.0)
    d = K.KvDesc(total_tokens=len(slots), kv_heads=H, head_dim=D, block_size=bs, num_blocks=blocks, io_dtype=int(io == BF), k_stride=H * D, v_stride=H * D)
    k, v = (guarded(torch.randn(len(slots), H, D, generator=g).to(io).cuda()) for _ in range(2))
    s, caches = guarded(up(slots)), [guarded(x) for x in c.all()]
    before = [x.all.clone() for x in caches]
    assert L.kda_kv_store(ctypes.byref(d), k.ptr(), v.ptr(), s.ptr(), *[x.ptr() for x in caches], stream()) == 0
    torch.cuda.synchronize()
    assert all(x.intact() for x in (k, v, s, *caches))
    # blocks without a token stay as they are, whole
    for x, b in zip(caches, before):
        per = x.n // blocks
        for i in (3, 5):
            assert torch.equal(x.all[PAD + i * per:PAD + (i + 1) * per], b[PAD + i * per:PAD + (i + 1) * per])


@pytest.mark.parametrize("n,most", [(1, 1), (3, 200), (1500, 3), (40, 900)])
def test_pages(K, n, most):
    """The list runs out on the way; what is given goes back."""
    L, bs, r = K.lib(), 16, random.Random(n)
    lens = [r.randint(0, most) for _ in range(n)]
    cu = np.concatenate([[0], np.cumsum(lens)])
    T, wide, rows = int(cu[-1]) + 5, -(-most // bs) + 1, n + 3
    num_free = max(1, sum(-(-x // bs) for x in lens) * 2 // 3)
    d = K.PagesDesc(num_seqs=n, total_tokens=T, rows=rows, max_blocks=wide, block_size=bs, num_free=num_free)
    at = r.sample(range(rows), n)
    cu, at, held, lens_, table = (guarded(up(x)) for x in (cu, at, [0] * rows, [0] * rows, [[-1] * wide] * rows))
    free, count = guarded(up(r.sample(range(5 * num_free), num_free))), guarded(up([num_free]))
    slots, totals = Guarded(T * 4), Guarded(n * 4)
    every = (cu, at, held, lens_, table, free, count, slots, totals)
    listed = free.view(I32, num_free).tolist()
    ptr = lambda *a: [x.ptr() for x in a]  # noqa: E731
    assert L.kda_kv_reserve(ctypes.byref(d), *ptr(cu, at, lens_, held, table, free, count, slots, totals), stream()) == 0
    assert L.kda_kv_commit(ctypes.byref(d), cu.ptr(), None, *ptr(at, lens_, held), stream()) == 0
    torch.cuda.synchronize()
    assert all(x.intact() for x in every) and int(held.view(I32, rows).sum()) == num_free - int(count.view(I32, 1))
    assert sorted(lens_.view(I32, rows).tolist()) == sorted(totals.view(I32, n).tolist() + [0] * 3)
    assert L.kda_kv_release(ctypes.byref(d), None, *ptr(at, lens_, held, table, free, count), stream()) == 0
    torch.cuda.synchronize()
    assert all(x.intact() for x in every) and free.view(I32, num_free).tolist() == listed and int(count.view(I32, 1)) == num_free
