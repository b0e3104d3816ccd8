"""Paged cache, attention and next-token entry points without a GPU: descriptors'
layouts and every refusal that host-visible values decide, through the C ABI (fake,
never dereferenced addresses) and through the binding (host tensors)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import gated_delta_rule_51_amd as kda
from test_serve_abi import ALIAS, ALIGN, NULL, OK, SHAPE, UNSUP, WS, L, fake  # noqa: F401  (L: fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_descriptor_layouts(tmp_path):
    structs = {"kda_pages_desc": kda.PagesDesc, "kda_kv_desc": kda.KvDesc, "kda_sample_desc": kda.SampleDesc}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "kda.h"', "int main(void) {"]
    for c, ct in structs.items():
        lines.append('    printf("%s %%zu\\n", sizeof(%s));' % (c, c))
        lines += ['    printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (c, f, c, f) for f, _ in ct._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["    return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(line.rsplit(" ", 1) for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for c, ct in structs.items():
        assert int(got[c]) == ctypes.sizeof(ct)
        for f, _ in ct._fields_:
            assert int(got["%s.%s" % (c, f)]) == getattr(ct, f).offset, (c, f)


def call(fn, d, args, given, tail=()):
    """fn with fake addresses for the names in args, those in `given` replaced."""
    a = {n: fake(i + 1) for i, n in enumerate(args)}
    assert not set(given) - set(a)
    a.update(given)
    return fn(ctypes.byref(d) if d is not None else None, *a.values(), *tail, None)


def pages(**kw):
    d = dict(num_seqs=3, total_tokens=40, rows=8, max_blocks=10, block_size=16, num_free=100)
    d.update(kw)
    return kda.PagesDesc(**d)


RESERVE = ("cu", "idx", "lens", "held", "table", "free", "count", "slots", "totals")
COMMIT = ("cu", "steps", "idx", "lens", "held")
RELEASE = ("keep", "idx", "lens", "held", "table", "free", "count")


def test_pages_refusals(L):  # noqa: F811
    every = ((L.kda_kv_reserve, RESERVE), (L.kda_kv_commit, COMMIT), (L.kda_kv_release, RELEASE))
    for fn, args in every:
        assert call(fn, None, args, {}) == NULL
        for kw, want in ((dict(num_seqs=-1), SHAPE), (dict(total_tokens=-1), SHAPE), (dict(rows=0), SHAPE), (dict(block_size=8), UNSUP),
                         (dict(block_size=48), UNSUP), (dict(block_size=256), UNSUP), (dict(block_size=0), UNSUP), (dict(block_size=-16), UNSUP)):
            assert call(fn, pages(**kw), args, {}) == want, kw
        for n in args:
            if n not in ("steps", "keep"):
                assert call(fn, pages(), args, {n: None}) == NULL, n
            assert call(fn, pages(), args, {n: fake(50, 2)}) == ALIGN, n
    for fn, args in (every[0], every[2]):
        for kw, want in ((dict(max_blocks=0), SHAPE), (dict(num_free=-1), SHAPE), (dict(max_blocks=(1 << 26) + 1), UNSUP)):
            assert call(fn, pages(**kw), args, {}) == want, kw
        assert call(fn, pages(num_free=0), args, {"free": None, args[0]: fake(1, 2)}) == ALIGN     # an empty list may be NULL
    outs = {"held", "table", "count", "slots", "totals"}
    for o in outs:
        for n in set(RESERVE) - {o}:
            assert call(L.kda_kv_reserve, pages(), RESERVE, {n: fake(60), o: fake(60)}) == ALIAS, (o, n)
    for n in set(COMMIT) - {"lens"}:
        assert call(L.kda_kv_commit, pages(), COMMIT, {n: fake(60), "lens": fake(60, 28)} if n == "held" else {n: fake(60, 8), "lens": fake(60)}) == ALIAS, n
    for o in ("lens", "held", "free", "count"):
        for n in set(RELEASE) - {o}:
            assert call(L.kda_kv_release, pages(), RELEASE, {n: fake(60), o: fake(60)}) == ALIAS, (o, n)
    # nothing to do: nothing is looked at
    none = {n: None for n in RESERVE}
    assert call(L.kda_kv_reserve, pages(num_seqs=0, total_tokens=0), RESERVE, none) == OK
    assert call(L.kda_kv_commit, pages(num_seqs=0), COMMIT, {n: None for n in COMMIT}) == OK
    assert call(L.kda_kv_release, pages(num_seqs=0), RELEASE, {n: None for n in RELEASE}) == OK


def kv(**kw):
    d = dict(num_seqs=3, total_tokens=40, q_heads=8, kv_heads=2, head_dim=64, block_size=16, num_blocks=50, rows=8, max_blocks=10, io_dtype=1,
             scale=0.125, q_stride=512, k_stride=128, v_stride=128)
    d.update(kw)
    return kda.KvDesc(**d)


STORE = ("k", "v", "slots", "kc", "vc", "ks", "vs")
ATTEND = ("q", "cu", "totals", "idx", "table", "kc", "vc", "ks", "vs", "o", "ws")
F32 = dict(io_dtype=0)


def test_store_refusals(L):  # noqa: F811
    fn = L.kda_kv_store
    assert call(fn, None, STORE, {}) == NULL
    for kw, want in ((dict(total_tokens=-1), SHAPE), (dict(kv_heads=0), SHAPE), (dict(num_blocks=0), SHAPE), (dict(head_dim=32), UNSUP),
                     (dict(head_dim=96), UNSUP), (dict(block_size=8), UNSUP), (dict(io_dtype=2), UNSUP), (dict(num_blocks=1 << 27), UNSUP),
                     (dict(k_stride=127), SHAPE), (dict(v_stride=120), SHAPE), (dict(k_stride=132), ALIGN), (dict(v_stride=129), ALIGN),
                     (dict(F32, k_stride=130), ALIGN), (dict(F32, k_stride=132, v_stride=129), ALIGN)):
        assert call(fn, kv(**kw), STORE, {}) == want, kw
    for n in STORE:
        assert call(fn, kv(), STORE, {n: None}) == NULL, n
        off = 2 if n in ("slots", "ks", "vs") else 8
        assert call(fn, kv(), STORE, {n: fake(50, off)}) == ALIGN, n
    for o in ("kc", "vc", "ks", "vs"):
        for n in set(STORE) - {o}:
            assert call(fn, kv(), STORE, {n: fake(60), o: fake(60)}) == ALIAS, (o, n)
    assert call(fn, kv(total_tokens=0), STORE, {n: None for n in STORE}) == OK


def test_attention_refusals(L):  # noqa: F811
    fn, d = L.kda_kv_attention, kv()
    need = L.kda_kv_attention_workspace_size(ctypes.byref(d))
    assert need > 0
    run = lambda d, given: call(fn, d, ATTEND, given, (need,))  # noqa: E731
    assert run(None, {}) == NULL
    for kw, want in ((dict(num_seqs=-1), SHAPE), (dict(total_tokens=-1), SHAPE), (dict(q_heads=0), SHAPE), (dict(q_heads=7), SHAPE),
                     (dict(kv_heads=3), SHAPE), (dict(rows=0), SHAPE), (dict(max_blocks=0), SHAPE), (dict(q_stride=511), SHAPE),
                     (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=2.0 ** 21), UNSUP),
                     (dict(scale=float("inf")), UNSUP), (dict(head_dim=256), UNSUP), (dict(block_size=24), UNSUP), (dict(io_dtype=-1), UNSUP),
                     (dict(max_blocks=(1 << 26) + 1), UNSUP), (dict(total_tokens=1 << 29), UNSUP), (dict(q_stride=516), ALIGN),
                     (dict(F32, q_stride=514), ALIGN)):
        assert run(kv(**kw), {}) == want, kw
        if want != ALIGN:
            assert L.kda_kv_attention_workspace_size(ctypes.byref(kv(**kw))) == 0
    for n in set(ATTEND) - {"ws"}:
        assert run(d, {n: None}) == NULL, n
        off = 8 if n in ("q", "kc", "vc", "o") else 2
        assert run(d, {n: fake(50, off)}) == ALIGN, n
    assert run(d, {"ws": None}) == WS and call(fn, d, ATTEND, {}, (need - 1,)) == WS
    assert run(d, {"ws": fake(50, 8)}) == ALIGN
    for o in ("o", "ws"):
        for n in set(ATTEND) - {o}:
            assert run(d, {n: fake(60), o: fake(60)}) == ALIAS, (o, n)
    for kw in (dict(total_tokens=0), dict(num_seqs=0)):
        assert call(fn, kv(**kw), ATTEND, {n: None for n in ATTEND}, (0,)) == OK


SAMPLE = ("x", "u", "t", "k", "p", "m", "tokens", "probs", "ws")


def test_sample_refusals(L):  # noqa: F811
    make = lambda **kw: kda.SampleDesc(**dict(dict(num_rows=4, vocab=1000, logits_dtype=1, stride=1001), **kw))  # noqa: E731
    fn, d = L.kda_sample_tokens, make()
    need = L.kda_sample_tokens_workspace_size(ctypes.byref(d))
    assert need > 0
    run = lambda d, given: call(fn, d, SAMPLE, given, (need,))  # noqa: E731
    assert run(None, {}) == NULL
    for kw, want in ((dict(num_rows=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(stride=999), SHAPE), (dict(logits_dtype=2), UNSUP),
                     (dict(vocab=(1 << 20) + 1, stride=1 << 21), UNSUP), (dict(num_rows=1 << 23), UNSUP),
                     (dict(num_rows=1 << 20, vocab=1 << 20, stride=1 << 20), UNSUP)):
        assert run(make(**kw), {}) == want, kw
        assert L.kda_sample_tokens_workspace_size(ctypes.byref(make(**kw))) == 0
    assert run(d, {"x": None}) == NULL and run(d, {"u": None}) == NULL and run(d, {"tokens": None, "probs": None}) == NULL
    assert run(d, {"ws": None}) == WS and call(fn, d, SAMPLE, {}, (need - 1,)) == WS
    for n in SAMPLE:
        assert run(d, {n: fake(50, 1)}) == ALIGN, n
    assert run(make(logits_dtype=0), {"x": fake(50, 2)}) == ALIGN
    for o in ("tokens", "probs", "ws"):
        for n in set(SAMPLE) - {o}:
            assert run(d, {n: fake(60), o: fake(60)}) == ALIAS, (o, n)
    assert call(fn, make(num_rows=0), SAMPLE, {n: None for n in SAMPLE}, (0,)) == OK


I32, F8 = torch.int32, torch.float8_e4m3fn


def z(*s, dtype=I32):
    return torch.zeros(*s, dtype=dtype)


def refuses(call, msg):
    with pytest.raises(ValueError, match=msg):
        call()


def test_binding_pages():
    ok = dict(cu=z(4), idx=z(3), lens=z(8), held=z(8), table=z(8, 10), free=z(100), count=z(1))

    def reserve(total=40, bs=16, **kw):
        a = dict(ok, **kw)
        return kda.kv_reserve(a["cu"], total, a["idx"], a["lens"], a["held"], a["table"], a["free"], a["count"], block_size=bs)

    def release(bs=16, keep=None, **kw):
        a = dict(ok, **kw)
        return kda.kv_release(a["idx"], a["lens"], a["held"], a["table"], a["free"], a["count"], block_size=bs, keep_lens=keep)

    def commit(bs=16, steps=None, **kw):
        a = dict(ok, **kw)
        return kda.kv_commit(a["cu"], a["idx"], a["lens"], a["held"], block_size=bs, steps=steps)

    refuses(reserve, "GPU")
    refuses(release, "GPU")
    refuses(commit, "GPU")
    for f in (reserve, release, commit):
        refuses(lambda: f(bs=17), "block_size")
    refuses(lambda: reserve(total=-1), "total_tokens")
    refuses(lambda: reserve(cu=z(0)), "cu_seqlens")
    refuses(lambda: reserve(cu=z(4, dtype=torch.int64)), "cu_seqlens")
    for f in (reserve, release):
        refuses(lambda: f(table=z(8, 0)), "rows and entries")
        refuses(lambda: f(table=z(8, 20)[:, ::2]), "contiguous")
        refuses(lambda: f(lens=z(7)), "kv_lens")
        refuses(lambda: f(held=z(9)), "blocks_held")
        refuses(lambda: f(free=z(10, 10)), "free_blocks")
        refuses(lambda: f(count=z(2)), "free_count")
        refuses(lambda: f(lens=z(8, dtype=torch.int64)), "kv_lens")
    refuses(lambda: reserve(idx=z(2)), "state_indices")
    refuses(lambda: release(keep=z(2)), "keep_lens")
    refuses(lambda: commit(steps=z(2)), "steps")
    refuses(lambda: commit(held=z(7)), "blocks_held")


def test_binding_cache_and_attention():
    B, H, bs, D, T = 6, 2, 16, 64, 5
    f = torch.float32
    cache = dict(kc=z(B, H, bs, D, dtype=F8), vc=z(B, H, D, bs, dtype=F8), ks=z(B, H, dtype=f), vs=z(B, H, dtype=f))
    ok = dict(k=z(T, H, D, dtype=f), v=z(T, H, D, dtype=f), slots=z(T), q=z(T, 4, D, dtype=f), cu=z(3), totals=z(2), idx=z(2), table=z(3, 4), **cache)

    def store(**kw):
        a = dict(ok, **kw)
        return kda.kv_store(a["k"], a["v"], a["slots"], a["kc"], a["vc"], a["ks"], a["vs"])

    def attend(scale=None, **kw):
        a = dict(ok, **kw)
        return kda.kv_attention(a["q"], a["cu"], a["totals"], a["idx"], a["table"], a["kc"], a["vc"], a["ks"], a["vs"], scale=scale)

    for fn in (store, attend):
        refuses(fn, "GPU")
        refuses(lambda: fn(kc=z(B, H, bs, D, dtype=torch.uint8)), "k_cache")
        refuses(lambda: fn(vc=z(B, H, bs, D, dtype=F8)), "v_cache")
        refuses(lambda: fn(ks=z(B, H + 1, dtype=f)), "k_scale")
        refuses(lambda: fn(vs=z(B, H, dtype=torch.bfloat16)), "v_scale")
        refuses(lambda: fn(kc=z(B, H, 8, D, dtype=F8), vc=z(B, H, D, 8, dtype=F8)), "block_size")
        refuses(lambda: fn(kc=z(B, H, bs, 96, dtype=F8), vc=z(B, H, 96, bs, dtype=F8)), "head dim")
        refuses(lambda: fn(kc=z(0, H, bs, D, dtype=F8)), "blocks and heads")
    refuses(lambda: store(k=z(T, H, D, dtype=torch.float16)), "float32 or bfloat16")
    refuses(lambda: store(v=z(T, H, D, dtype=torch.bfloat16)), "v must be")
    refuses(lambda: store(k=z(T - 1, H, D, dtype=f)), "k must")
    refuses(lambda: store(k=z(T, D, H, dtype=f).transpose(1, 2)), "contiguous within")
    refuses(lambda: store(slots=z(T, dtype=torch.int64)), "slots")
    refuses(lambda: attend(q=z(T, 3, D, dtype=f)), "query heads")
    refuses(lambda: attend(q=z(T, 4, 128, dtype=f)), "q must")
    refuses(lambda: attend(q=z(T, 4 * D, dtype=f)), "q must")
    refuses(lambda: attend(totals=z(1)), "kv_totals")
    refuses(lambda: attend(idx=z(1)), "state_indices")
    refuses(lambda: attend(table=z(12)), "block_table")
    refuses(lambda: attend(table=z(0, 4)), "rows and entries")
    for s in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** 20 + 1):
        refuses(lambda: attend(scale=s), "scale")


def test_binding_sample():
    f = torch.float32
    x, u = z(4, 50, dtype=f), z(4, dtype=f)
    refuses(lambda: kda.sample_tokens(x, u), "GPU")
    refuses(lambda: kda.token_probs(x), "GPU")
    refuses(lambda: kda.sample_tokens(x[0], u), "logits")
    refuses(lambda: kda.sample_tokens(z(4, 0, dtype=f), u), "vocabulary")
    refuses(lambda: kda.sample_tokens(x.half(), u), "float32 or bfloat16")
    refuses(lambda: kda.sample_tokens(x.t().contiguous().t(), u), "contiguous within")
    refuses(lambda: kda.sample_tokens(x, None), "uniform")
    refuses(lambda: kda.sample_tokens(x, u[:3]), "uniform")
    refuses(lambda: kda.sample_tokens(x, u.double()), "uniform")
    for name in ("temperature", "top_p", "min_p"):
        refuses(lambda: kda.sample_tokens(x, u, **{name: z(3, dtype=f)}), name)
        refuses(lambda: kda.token_probs(x, **{name: z(4)}), name)
    refuses(lambda: kda.sample_tokens(x, u, top_k=z(4, dtype=f)), "top_k")
