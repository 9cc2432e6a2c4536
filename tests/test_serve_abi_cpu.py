"""The entry points of include/flint_serve.h: exported, and their refusals (no GPU is needed: every
call here fails validation or is a no-op, so no kernel is launched)."""
import ctypes
import os
import re
import subprocess

import pytest

import sparse_moe_transformer_wave_amd as fm
from sparse_moe_transformer_wave_amd import ops, serve

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B16, MIS = 1 << 20, 1 << 21, (1 << 20) + 8  # aligned and misaligned addresses, never dereferenced
BIG = 1 << 40


def test_library_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "flint_serve.h")).read()
    names = set(re.findall(r"^(?:int|size_t) (flint_\w+)\s*\(", src, re.M))
    assert names == set(fm.EXPORTED_SERVE)
    L = ctypes.CDLL(fm.LIB_PATH)
    for n in names:
        assert hasattr(L, n), n


def _cache(Hq=32, Hkv=4, D=128, page=64, pages=100, stride=0, data=A):
    return serve._KV4Cache(Hq, Hkv, D, page, pages, stride, data)


BLOCK = 2 * 4 * 64 * (64 + 4)
BAD_CACHES = (dict(D=32), dict(D=256), dict(D=96), dict(page=8), dict(page=48), dict(page=256), dict(Hkv=0), dict(Hkv=65, Hq=65),
              dict(Hq=0), dict(Hq=30), dict(Hq=132), dict(pages=0), dict(pages=1 << 31), dict(stride=BLOCK - 16),
              dict(stride=BLOCK + 8), dict(stride=1 << 61))


def _append(c=None, T=1, t=True, qn=None, kn=None, eps=0.0, rot=0, style=0, max_pos=0, cos=None, sin=None, qkv=A, ld=5120,
            pos=None, slots=A, q=A, ldq=4096, k=None, ldk=0, v=None, ldv=0):
    c = _cache() if c is None else c
    tr = ops._QKTransform(qn, kn, eps, rot, style, max_pos, cos, sin)
    return serve._serve().flint_kv4_append(ctypes.byref(c), ctypes.byref(tr) if t else None, T, qkv, ld, pos, slots, q, ldq, k, ldk,
                                           v, ldv, None)


def test_append_refusals():
    assert serve._serve().flint_kv4_append(None, None, 1, A, 1, A, A, A, 1, None, 0, None, 0, None) == fm.ERR_NULL
    assert _append(t=False) == fm.ERR_NULL
    for kw in BAD_CACHES:
        assert _append(_cache(**kw)) == fm.ERR_SHAPE, kw
    rope = dict(rot=128, max_pos=10, cos=A, sin=A, pos=A)
    for kw in (dict(rot=-2), dict(rot=3), dict(rot=130), dict(rope, max_pos=0), dict(eps=-1.0), dict(eps=float("nan")), dict(T=-1),
               dict(T=(1 << 20) + 1), dict(ld=5112), dict(ld=5121), dict(ldq=4088), dict(ldq=4100), dict(k=A, ldk=504),
               dict(k=A, ldk=516), dict(v=A, ldv=504), dict(v=A, ldv=513)):
        assert _append(**kw) == fm.ERR_SHAPE, kw
    assert _append(style=2) == fm.ERR_FORMAT
    for kw in (dict(qkv=None), dict(slots=None), dict(q=None), dict(rope, cos=None), dict(rope, sin=None), dict(rope, pos=None)):
        assert _append(**kw) == fm.ERR_NULL, kw
    assert _append(_cache(data=None)) == fm.ERR_NULL
    assert _append(_cache(data=MIS)) == fm.ERR_ALIGN
    for kw in (dict(qkv=MIS), dict(q=MIS), dict(qn=MIS), dict(kn=MIS), dict(rope, cos=MIS), dict(rope, sin=MIS),
               dict(rope, pos=A + 2), dict(slots=A + 4), dict(k=MIS, ldk=512), dict(v=MIS, ldv=512)):
        assert _append(**kw) == fm.ERR_ALIGN, kw
    assert _append(T=0, qkv=None, slots=None, q=None) == fm.OK


def _attn(c=None, B=2, window=0, sinks=None, q=A, ldq=4096, table=A, ldt=10, lens=A, prefix=0, out=A, ldo=4096, ws=A, nb=BIG, a=True):
    c = _cache() if c is None else c
    at = ops._Attn(0.1, window, sinks)
    return serve._serve().flint_kv4_attn_decode(ctypes.byref(c), ctypes.byref(at) if a else None, B, q, ldq, table, ldt, lens,
                                                prefix, out, ldo, ws, nb, None)


def test_attn_refusals():
    L = serve._serve()
    assert _attn(a=False) == fm.ERR_NULL
    for kw in BAD_CACHES:
        assert _attn(_cache(**kw)) == fm.ERR_SHAPE, kw
        assert L.flint_kv4_attn_decode_workspace_bytes(ctypes.byref(_cache(**kw)), 1) == 0
    for kw in (dict(B=-1), dict(B=1025), dict(window=-1), dict(prefix=-1), dict(prefix=641), dict(ldq=4088), dict(ldq=4100),
               dict(ldo=4088), dict(ldo=4100), dict(ldt=0), dict(ldt=1 << 30)):
        assert _attn(**kw) == fm.ERR_SHAPE, kw
    for kw in (dict(q=None), dict(table=None), dict(lens=None), dict(out=None), dict(ws=None)):
        assert _attn(**kw) == fm.ERR_NULL, kw
        assert _attn(B=0, **kw) == fm.OK
    for kw in (dict(q=MIS), dict(out=MIS), dict(ws=MIS), dict(table=A + 2), dict(lens=A + 1), dict(sinks=A + 2)):
        assert _attn(**kw) == fm.ERR_ALIGN, kw
    need = [L.flint_kv4_attn_decode_workspace_bytes(ctypes.byref(_cache()), b) for b in (1, 2, 3, 31, 33, 128, 1024)]
    assert need == sorted(need) and need[0] > 0
    for b in (-1, 1025):
        assert L.flint_kv4_attn_decode_workspace_bytes(ctypes.byref(_cache()), b) == 0
    assert _attn(nb=15) == fm.ERR_WORKSPACE


def _pages(n=100, page=64, arrays=((A, 1024, 1024), (B16, 2048, 4096))):
    arr = (serve._KVArray * max(len(arrays), 1))(*arrays)
    p = serve._KVPages(page, len(arrays), n, ctypes.addressof(arr) if arrays else None)
    p.keep = arr
    return p


def _state(base=A, **kw):
    names = ("refs", "free_list", "n_free", "table", "kv_len")
    return serve._KVState(*[kw.get(n, base + 4096 * i) for i, n in enumerate(names)])


BAD_PAGES = (dict(n=0), dict(n=(1 << 24) + 1), dict(page=8), dict(page=100), dict(arrays=((A, 0, 16),)), dict(arrays=((A, 24, 32),)),
             dict(arrays=((A, 32, 16),)), dict(arrays=((A, 16, 24),)), dict(arrays=((A, 16, 1 << 61),)),
             dict(arrays=((A, (1 << 30) + 16, 1 << 31),)))


def _advance(p=None, ldt=8, ro=2, old=None, r=3, new=None, parent=A, grow=A, slots=None, lds=0, ws=A, nb=BIG):
    p = _pages() if p is None else p
    old, new = _state() if old is None else old, _state(B16) if new is None else new
    return serve._serve().flint_kv_advance(ctypes.byref(p), ldt, ro, ctypes.byref(old), r, ctypes.byref(new), parent, grow, slots, lds,
                                           ws, nb, None)


def _compact(p=None, ldt=8, r=3, old=None, new=None, moved=A, ws=A, nb=BIG):
    p = _pages() if p is None else p
    old, new = _state() if old is None else old, _state(B16) if new is None else new
    return serve._serve().flint_kv_compact(ctypes.byref(p), ldt, r, ctypes.byref(old), ctypes.byref(new), moved, ws, nb, None)


def test_pages_refusals():
    L = serve._serve()
    assert L.flint_kv_advance(None, 1, 0, None, 0, None, None, None, None, 0, A, 0, None) == fm.ERR_NULL
    assert L.flint_kv_compact(None, 1, 0, None, None, A, A, 0, None) == fm.ERR_NULL
    for kw in BAD_PAGES:
        assert _advance(_pages(**kw)) == fm.ERR_SHAPE and _compact(_pages(**kw)) == fm.ERR_SHAPE, kw
        assert L.flint_kv_pages_workspace_bytes(ctypes.byref(_pages(**kw)), 1) == 0, kw
    many = _pages()
    many.n_arrays = 1025
    assert _advance(many) == fm.ERR_SHAPE
    none = _pages()
    none.arrays = None
    assert _advance(none) == fm.ERR_NULL and _compact(none) == fm.ERR_NULL
    for kw in (dict(ldt=0), dict(ldt=(1 << 25) // 64 + 1), dict(r=-1), dict(r=1025)):
        assert _advance(**kw) == fm.ERR_SHAPE and _compact(**kw) == fm.ERR_SHAPE, kw
    for kw in (dict(ro=-1), dict(ro=1025), dict(slots=A, lds=0), dict(slots=A, lds=(1 << 25) + 1)):
        assert _advance(**kw) == fm.ERR_SHAPE, kw
    for kw in (dict(parent=None), dict(grow=None), dict(ws=None)):
        assert _advance(**kw) == fm.ERR_NULL, kw
    for kw in (dict(moved=None), dict(ws=None)):
        assert _compact(**kw) == fm.ERR_NULL, kw
    for kw in (dict(parent=A + 2), dict(grow=A + 1), dict(slots=A + 4, lds=1), dict(ws=MIS)):
        assert _advance(**kw) == fm.ERR_ALIGN, kw
    assert _compact(moved=A + 2) == fm.ERR_ALIGN and _compact(ws=MIS) == fm.ERR_ALIGN
    for n in ("refs", "free_list", "n_free", "table", "kv_len"):
        for call in (_advance, _compact):
            assert call(old=_state(**{n: None})) == fm.ERR_NULL and call(new=_state(B16, **{n: None})) == fm.ERR_NULL
            assert call(old=_state(**{n: A + 2})) == fm.ERR_ALIGN
            # a state's array that is also the other's
            assert call(new=_state(B16, **{n: A + 4096 * 3})) == fm.ERR_SHAPE
    for bad in ((0, 16, 16), ):
        assert _advance(_pages(arrays=(bad,))) == fm.ERR_NULL
    assert _advance(_pages(arrays=((MIS, 16, 16),))) == fm.ERR_ALIGN
    need = L.flint_kv_pages_workspace_bytes(ctypes.byref(_pages()), 3)
    assert need > 0 and _advance(nb=need - 1) == fm.ERR_WORKSPACE and _compact(nb=need - 1) == fm.ERR_WORKSPACE
    for rows in (-1, 1025):
        assert L.flint_kv_pages_workspace_bytes(ctypes.byref(_pages()), rows) == 0


def test_pages_refuse_states_that_overlap():
    """An array of one state that begins or ends inside one of the other's; side by side they are taken (and
    the workspace is what is refused)."""
    at = {n: A + 4096 * i for i, n in enumerate(("refs", "free_list", "n_free", "table", "kv_len"))}
    size = dict(refs=400, free_list=400, n_free=4, table=3 * 8 * 4, kv_len=3 * 4)
    for n, start in at.items():
        for m in at:
            for call in (lambda **kw: _advance(ro=3, nb=0, **kw), lambda **kw: _compact(nb=0, **kw)):
                for to in (start + size[n] - 4, start - size[m] + 4):
                    assert call(new=_state(B16, **{m: to})) == fm.ERR_SHAPE, (n, m, to)
                for to in (start + size[n], start - size[m]):
                    assert call(new=_state(B16, **{m: to})) == fm.ERR_WORKSPACE, (n, m, to)
    # tables without rows take no memory
    assert _advance(ro=0, nb=0, old=_state(table=B16, kv_len=B16)) == fm.ERR_WORKSPACE


def _lora(T=2, K=256, N=8, R=16, n=4, a=A, b=A, ranks=None, scales=None, x=A, ldx=None, ids=A, base=None, ldb=0, bt=0, y=A, ldy=None,
          yt=0, ws=A, nb=BIG, l=True):
    c = serve._Lora(K, N, R, n, a, b, ranks, scales)
    return serve._serve().flint_lora(ctypes.byref(c) if l else None, T, x, K if ldx is None else ldx, ids, base, ldb, bt, y,
                                     N if ldy is None else ldy, yt, ws, nb, None)


def test_lora_refusals():
    L = serve._serve()
    assert _lora(l=False) == fm.ERR_NULL
    bad = (dict(K=0), dict(K=12), dict(K=32776), dict(N=0), dict(N=(1 << 24) + 1), dict(R=0), dict(R=4), dict(R=12), dict(R=136),
           dict(n=0), dict(n=(1 << 20) + 1))
    for kw in bad:
        assert _lora(**kw) == fm.ERR_SHAPE, kw
        c = dict(K=256, N=8, R=16, n=4)
        c.update(kw)
        assert L.flint_lora_workspace_bytes(ctypes.byref(serve._Lora(c["K"], c["N"], c["R"], c["n"], A, A, None, None)), 1) == 0
    for kw in (dict(T=-1), dict(T=65537), dict(ldx=248), dict(ldx=260), dict(ldy=7), dict(base=A, ldb=7)):
        assert _lora(**kw) == fm.ERR_SHAPE, kw
    assert _lora(yt=2) == fm.ERR_FORMAT and _lora(base=A, ldb=8, bt=-1) == fm.ERR_FORMAT
    for kw in (dict(a=None), dict(b=None), dict(x=None), dict(ids=None), dict(y=None), dict(ws=None)):
        assert _lora(**kw) == fm.ERR_NULL, kw
        assert _lora(T=0, **kw) == fm.OK
    for kw in (dict(a=MIS), dict(b=MIS), dict(ranks=A + 2), dict(scales=A + 2), dict(x=MIS), dict(ids=A + 2), dict(y=A + 1),
               dict(y=A + 2, yt=1), dict(base=A + 2, ldb=8, bt=1), dict(base=A + 1, ldb=8), dict(ws=MIS)):
        assert _lora(**kw) == fm.ERR_ALIGN, kw


def test_lora_in_place_is_the_same_rows():
    for kw in (dict(ldb=16), dict(ldb=8, bt=1), dict(ldb=8, yt=1)):
        assert _lora(base=A, T=0, **kw) == fm.ERR_SHAPE, kw
    assert _lora(base=A, ldb=8, T=0) == fm.OK and _lora(base=A, ldb=8, bt=1, yt=1, T=0) == fm.OK


@pytest.mark.parametrize("K,R", [(8, 8), (2048, 16), (32768, 128)])
def test_lora_workspace_covers_smaller_batches(K, R):
    L = serve._serve()
    c = serve._Lora(K, 8, R, 4, A, A, None, None)
    most = 0
    for T in (0, 1, 2, 15, 16, 17, 33, 100, 1023, 1024, 1025, 1041, 4095, 4096, 4097, 5000, 65535, 65536):
        need = L.flint_lora_workspace_bytes(ctypes.byref(c), T)
        assert need >= most > -1
        most = need
        if T:  # what the smaller batches need: a call with as much is not refused for it
            for t in {1, T // 2 + 1, T}:
                assert _lora(T=t, K=K, R=R, ws=A, nb=need, x=MIS) == fm.ERR_ALIGN
                assert _lora(T=t, K=K, R=R, nb=15) == fm.ERR_WORKSPACE
    for T in (-1, 65537):
        assert L.flint_lora_workspace_bytes(ctypes.byref(c), T) == 0


def _logits(T=2, V=1000, x=A, ld=None, out=B16, ldo=None, dt=0, rules=True, **kw):
    r = serve._LogitRules(**dict(dict(history=A, ldh=7), **kw))
    return serve._serve().flint_logits_adjust(ctypes.byref(r) if rules else None, T, V, x, V if ld is None else ld, out,
                                              V if ldo is None else ldo, dt, None)


def test_logits_refusals():
    assert _logits(rules=False) == fm.ERR_NULL and _logits(dt=2) == fm.ERR_FORMAT
    for kw in (dict(T=-1), dict(T=65537), dict(V=0), dict(V=(1 << 20) + 1), dict(ld=999), dict(ldo=999), dict(ldh=-1),
               dict(ldh=1 << 31), dict(bias_start=A, n_bias=-1), dict(masks=A, ldm=31, n_masks=1), dict(masks=A, ldm=32, n_masks=-1),
               dict(masks=A, ldm=1 << 60, n_masks=1 << 60), dict(out=A, ldo=1008)):
        assert _logits(**kw) == fm.ERR_SHAPE, kw
    for kw in (dict(x=None), dict(out=None), dict(bias_start=A, n_bias=1, bias_ids=A), dict(bias_start=A, n_bias=1, bias=A)):
        assert _logits(**kw) == fm.ERR_NULL, kw
        assert _logits(T=0, **kw) == fm.OK
    for kw in (dict(x=A + 1), dict(x=A + 2, dt=1), dict(out=A + 1), dict(history=A + 2), dict(prompt_len=A + 2), dict(total_len=A + 1),
               dict(repetition=A + 2), dict(frequency=A + 2), dict(presence=A + 2), dict(bias_start=A + 2), dict(mask_rows=A + 2),
               dict(bias_start=A, n_bias=1, bias_ids=A + 2, bias=A), dict(bias_start=A, n_bias=1, bias_ids=A, bias=A + 2),
               dict(masks=A + 2, ldm=32, n_masks=1)):
        assert _logits(**kw) == fm.ERR_ALIGN, kw


torch = pytest.importorskip("torch")


class _Gpu(torch.Tensor):
    is_cuda = True


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_Gpu)


def test_binding_refuses_what_does_not_fit():
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    raises = lambda: pytest.raises(ValueError)  # noqa: E731
    block = fm.KV4Cache.page_bytes(2, 64, 16)
    with raises():
        fm.KV4Cache(torch.zeros(3, block, dtype=u8), 4, 2, 64, 16)  # host
    with raises():
        fm.KV4Cache(_t(3, block + 1, dtype=u8), 4, 2, 64, 16)
    with raises():
        fm.KV4Cache(_t(1, block, dtype=u8).expand(5, block), 4, 2, 64, 16)  # pages that are the same memory
    with raises():
        fm.KV4Cache(_t(3, block, dtype=torch.int8), 4, 2, 64, 16)
    cache = fm.KV4Cache(_t(3, block, dtype=u8), 4, 2, 64, 16)
    assert cache.k_codes.shape == (3, 2, 16, 32) and cache.v_scales.shape == (3, 2, 2, 16)
    wide = fm.KV4Cache(_t(3, 3, block, dtype=u8)[:, 1], 4, 2, 64, 16)  # a layer's slice
    assert wide.c.page_stride == 3 * block
    tr = fm.QKTransform()
    with raises():
        fm.kv4_append(cache, tr, _t(2, 512), None, _t(2, dtype=i32), _t(2, 256), stream=0)  # slots of 32 bits
    with raises():
        fm.kv4_append(cache, tr, _t(2, 512), None, _t(2, dtype=torch.int64), _t(2, 256), _t(3, 128), stream=0)
    ws = _t(1 << 20, dtype=u8)
    for bad in (torch.zeros(1, dtype=u8).expand(1 << 20).as_subclass(_Gpu), ws[::2]):  # a size that is not the memory's
        with raises():
            fm.kv4_attn_decode(cache, fm.AttnDecode(1.0), _t(1, 256), _t(1, 3, dtype=i32), _t(1, dtype=i32), 0, _t(1, 256), bad, stream=0)
    with raises():
        fm.KVPages([])
    with raises():
        fm.KVPages([cache, fm.KV4Cache(_t(4, block, dtype=u8), 4, 2, 64, 16)])
    pages = fm.KVPages([cache, wide, fm.KVCache(_t(3, 2, 16, 64), _t(3, 2, 64, 16), 4)])
    assert [(a.bytes, a.stride) for a in pages.arrays] == [(block, block), (block, 3 * block), (4096, 4096), (4096, 4096)]

    def state(n=3, rows=2, width=5):
        z = lambda *s: _t(*s, dtype=i32)  # noqa: E731
        return fm.KVState(z(n), z(n), z(1), z(rows, width), z(rows))

    with raises():
        fm.KVState(_t(3, dtype=i32), _t(2, dtype=i32), _t(1, dtype=i32), _t(2, 5, dtype=i32), _t(2, dtype=i32))
    i2 = _t(2, dtype=i32)
    for old, new in ((state(), state(4)), (state(), state(width=6)), (state(4), state(4))):
        with raises():
            fm.kv_advance(pages, old, new, i2, i2, None, ws, stream=0)
    with raises():
        fm.kv_advance(pages, state(), state(), _t(3, dtype=i32), i2, None, ws, stream=0)
    with raises():
        fm.kv_advance(pages, state(), state(), i2, i2, _t(3, 4, dtype=torch.int64), ws, stream=0)
    with raises():
        fm.kv_compact(pages, state(), state(rows=3), _t(3, dtype=i32), ws, stream=0)
    with raises():
        fm.LoraAdapters(_t(2, 8, 64), _t(2, 32, 16))
    ad = fm.LoraAdapters(_t(2, 8, 64), _t(2, 32, 8))
    for kw in (dict(ids=_t(3, dtype=i32)), dict(x=_t(2, 72)), dict(y=_t(2, 32, dtype=torch.float16)), dict(base=_t(2, 31)), dict(x=_t(2, 64, dtype=f32))):
        a = dict(dict(x=_t(2, 64), ids=i2, base=None, y=_t(2, 32)), **kw)
        with raises():
            fm.lora(ad, a["x"], a["ids"], a["base"], a["y"], ws, stream=0)
    with raises():
        fm.LogitRules(repetition=_t(2, dtype=f32))
    with raises():
        fm.LogitRules(history=_t(2, 5, dtype=i32), total_len=_t(3, dtype=i32))
    with raises():
        fm.LogitRules(bias_start=_t(3, dtype=i32), bias_ids=_t(4, dtype=i32))
    with raises():
        fm.LogitRules(bias_start=_t(3, dtype=i32), bias_ids=_t(4, dtype=i32), bias=_t(5, dtype=f32))
    with raises():
        fm.LogitRules(mask_rows=i2)
    rules = fm.LogitRules(history=_t(2, 5, dtype=i32))
    for x, y in ((_t(3, 9), _t(3, 9)), (_t(2, 9), _t(2, 9, dtype=f32)), (_t(2, 9), _t(2, 8))):
        with raises():
            fm.logits_adjust(rules, x, y, stream=0)


@pytest.mark.parametrize("cc,std", [("gcc", "c11"), ("g++", "c++14")])
def test_header_compiles_alone(cc, std, tmp_path):
    src = tmp_path / ("use.c" if cc == "gcc" else "use.cpp")
    src.write_text('#include "flint_serve.h"\n'
                   "int use(void) { flint_lora_adapters l = {128, 1, 8, 1, 0, 0, 0, 0};\n"
                   "    return flint_lora(&l, 0, 0, 128, 0, 0, 0, 0, 0, 1, FLINT_DT_BF16, 0, 0, 0); }\n")
    subprocess.run([cc, "-std=" + std, "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"), "-c",
                    str(src), "-o", str(tmp_path / "use.o")], check=True)
