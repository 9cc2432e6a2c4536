"""The entry points of include/flint_ops.h: exported, and their refusals (no GPU is needed:
every call here fails validation or is a no-op, so no kernel is launched)."""
import ctypes
import os
import re
import subprocess

import pytest

import sparse_moe_transformer_wave_amd as fm
from sparse_moe_transformer_wave_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, MIS = 1 << 20, (1 << 20) + 8  # an aligned and a misaligned address, never dereferenced
BIG = 1 << 40


def test_library_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "flint_ops.h")).read()
    names = set(re.findall(r"^(?:int|size_t) (flint_\w+)\s*\(", src, re.M))
    assert names == set(fm.EXPORTED_OPS)
    L = ctypes.CDLL(fm.LIB_PATH)
    for n in names:
        assert hasattr(L, n), n


def _linear(T=1, K=256, N=8, group=128, codes=A, scales=A, x=A, ldx=None, res=None, ldr=0, y=A, ldy=None, ty=0, w=True):
    c = ops._Int4Linear(K, N, group, codes, scales)
    return ops._ops().flint_linear_int4(ctypes.byref(c) if w else None, T, x, K if ldx is None else ldx, res, ldr, y,
                                        N if ldy is None else ldy, ty, None)


def test_linear_refusals():
    assert _linear(w=False) == fm.ERR_NULL
    for kw in (dict(K=0), dict(K=64), dict(K=200), dict(K=32896), dict(N=0), dict(N=(1 << 24) + 1), dict(group=16),
               dict(group=256), dict(T=-1), dict(T=65), dict(ldx=128), dict(ldx=260), dict(ldy=7), dict(res=A, ldr=7)):
        assert _linear(**kw) == fm.ERR_SHAPE, kw
    assert _linear(ty=2) == fm.ERR_FORMAT
    for kw in (dict(codes=None), dict(scales=None), dict(x=None), dict(y=None)):
        assert _linear(**kw) == fm.ERR_NULL, kw
        assert _linear(T=0, **kw) == fm.OK
    for kw in (dict(codes=MIS), dict(scales=MIS), dict(x=MIS), dict(y=A + 1), dict(y=A + 2, ty=1), dict(res=A + 1, ldr=8)):
        assert _linear(**kw) == fm.ERR_ALIGN, kw


def _cache(Hq=32, Hkv=4, D=128, page=64, pages=100, stride=0, k=A, v=A):
    return ops._KVCache(Hq, Hkv, D, page, pages, stride, k, v)


BAD_CACHES = (dict(D=32), dict(D=256), dict(D=96), dict(page=8), dict(page=48), dict(page=256), dict(Hkv=0), dict(Hkv=65, Hq=65),
              dict(Hq=0), dict(Hq=30), dict(Hq=132), dict(pages=0), dict(pages=1 << 31), dict(stride=4 * 64 * 128 - 8),
              dict(stride=4 * 64 * 128 + 4), dict(stride=1 << 60))


def _append(c=None, T=1, t=True, qn=None, kn=None, eps=0.0, rot=0, style=0, max_pos=0, cos=None, sin=None, qkv=A, ld=5120,
            pos=None, slots=A, q=A, ldq=4096):
    c = _cache() if c is None else c
    tr = ops._QKTransform(qn, kn, eps, rot, style, max_pos, cos, sin)
    return ops._ops().flint_kv_append(ctypes.byref(c), ctypes.byref(tr) if t else None, T, qkv, ld, pos, slots, q, ldq, None)


def test_append_refusals():
    L = ops._ops()
    assert L.flint_kv_append(None, None, 1, A, 1, A, A, A, 1, None) == fm.ERR_NULL
    assert _append(t=False) == fm.ERR_NULL
    for kw in BAD_CACHES:
        assert _append(_cache(**kw)) == fm.ERR_SHAPE, kw
    rope = dict(rot=128, max_pos=10, cos=A, sin=A, pos=A)
    for kw in (dict(rot=-2), dict(rot=3), dict(rot=130), dict(rope, max_pos=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(T=-1), dict(T=(1 << 20) + 1), dict(ld=5112), dict(ld=5121), dict(ldq=4088), dict(ldq=4100)):
        assert _append(**kw) == fm.ERR_SHAPE, kw
    assert _append(style=2) == fm.ERR_FORMAT
    for kw in (dict(qkv=None), dict(slots=None), dict(q=None), dict(rope, cos=None), dict(rope, sin=None), dict(rope, pos=None)):
        assert _append(**kw) == fm.ERR_NULL, kw
    assert _append(_cache(k=None)) == fm.ERR_NULL and _append(_cache(v=None)) == fm.ERR_NULL
    assert _append(_cache(k=MIS)) == fm.ERR_ALIGN and _append(_cache(v=MIS)) == fm.ERR_ALIGN
    for kw in (dict(qkv=MIS), dict(q=MIS), dict(qn=MIS), dict(kn=MIS), dict(rope, cos=MIS), dict(rope, sin=MIS),
               dict(rope, pos=A + 2), dict(slots=A + 4)):
        assert _append(**kw) == fm.ERR_ALIGN, kw
    assert _append(T=0, qkv=None, slots=None, q=None) == fm.OK


def _attn(c=None, B=2, window=0, sinks=None, q=A, ldq=4096, table=A, ldt=10, lens=A, prefix=0, out=A, ldo=4096, ws=A, nb=BIG, a=True):
    c = _cache() if c is None else c
    at = ops._Attn(0.1, window, sinks)
    return ops._ops().flint_attn_decode(ctypes.byref(c), ctypes.byref(at) if a else None, B, q, ldq, table, ldt, lens, prefix,
                                        out, ldo, ws, nb, None)


def test_attn_refusals():
    L = ops._ops()
    assert L.flint_attn_decode(None, None, 1, A, 1, A, 1, A, 0, A, 1, A, 0, None) == fm.ERR_NULL
    assert _attn(a=False) == fm.ERR_NULL
    for kw in BAD_CACHES:
        assert _attn(_cache(**kw)) == fm.ERR_SHAPE, kw
        assert L.flint_attn_decode_workspace_bytes(ctypes.byref(_cache(**kw)), 1) == 0
    for kw in (dict(B=-1), dict(B=1025), dict(window=-1), dict(prefix=-1), dict(prefix=641), dict(ldq=4088), dict(ldq=4100),
               dict(ldo=4088), dict(ldo=4100), dict(ldt=0), dict(ldt=1 << 30)):
        assert _attn(**kw) == fm.ERR_SHAPE, kw
    for kw in (dict(q=None), dict(table=None), dict(lens=None), dict(out=None), dict(ws=None)):
        assert _attn(**kw) == fm.ERR_NULL, kw
        assert _attn(B=0, **kw) == fm.OK
    assert _attn(_cache(k=None)) == fm.ERR_NULL and _attn(_cache(v=MIS)) == fm.ERR_ALIGN
    for kw in (dict(q=MIS), dict(out=MIS), dict(ws=MIS), dict(table=A + 2), dict(lens=A + 1), dict(sinks=A + 2)):
        assert _attn(**kw) == fm.ERR_ALIGN, kw
    need = [L.flint_attn_decode_workspace_bytes(ctypes.byref(_cache()), b) for b in (1, 2, 1024)]
    assert 0 < need[0] <= need[1] <= need[2]
    assert L.flint_attn_decode_workspace_bytes(ctypes.byref(_cache()), -1) == 0
    assert L.flint_attn_decode_workspace_bytes(ctypes.byref(_cache()), 1025) == 0
    assert _attn(nb=need[1] - 1) == fm.ERR_WORKSPACE


def _logprobs(T=2, V=1000, x=A, ld=None, dt=0, tok=A, lp=A, h=A, n=3, ids=A, tl=A, ws=A, nb=BIG):
    return ops._ops().flint_token_logprobs(T, V, x, V if ld is None else ld, dt, tok, lp, h, n, ids, tl, ws, nb, None)


def test_logprobs_refusals():
    L = ops._ops()
    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(V=0, n=0), dict(V=(1 << 20) + 1), dict(ld=999), dict(n=-1), dict(n=33), dict(V=2)):
        assert _logprobs(**kw) == fm.ERR_SHAPE, kw
    assert _logprobs(dt=2) == fm.ERR_FORMAT
    for kw in (dict(x=None), dict(tok=None), dict(ws=None), dict(ids=None), dict(tl=None)):
        assert _logprobs(**kw) == fm.ERR_NULL, kw
        assert _logprobs(T=0, **kw) == fm.OK
    for kw in (dict(x=A + 1), dict(x=A + 2, dt=1), dict(tok=A + 2), dict(lp=A + 2), dict(h=A + 1), dict(ids=A + 2), dict(tl=A + 2), dict(ws=MIS)):
        assert _logprobs(**kw) == fm.ERR_ALIGN, kw
    for args in ((-1, 10, 0), (1 << 21, 10, 0), (1, 0, 0), (1, 1 << 21, 0), (1, 10, 11), (1, 100, 33), (1, 100, -1)):
        assert L.flint_token_logprobs_workspace_bytes(*args) == 0, args
    need = [L.flint_token_logprobs_workspace_bytes(t, 131072, 20) for t in (1, 8, 512, 4096)]
    assert 0 < need[0] <= need[1] <= need[2] <= need[3]
    assert _logprobs(T=1, V=131072, n=20, nb=need[0] - 1) == fm.ERR_WORKSPACE


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    with pytest.raises(ValueError):
        fm.Int4Linear(torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 1, dtype=bf))
    with pytest.raises(ValueError):
        fm.KVCache(torch.zeros(2, 1, 16, 64, dtype=bf), torch.zeros(2, 1, 64, 16, dtype=bf), 4)
    with pytest.raises(ValueError):
        fm.AttnDecode(1.0, 0, torch.zeros(4))
    x = torch.zeros(2, 100)
    with pytest.raises(ValueError):
        fm.token_logprobs(x, None, None, torch.zeros(2), None, None, x)
    with pytest.raises(AttributeError):
        fm.no_such_operator


@pytest.mark.parametrize("cc,std", [("gcc", "c11"), ("g++", "c++14")])
def test_header_compiles_alone(cc, std, tmp_path):
    src = tmp_path / ("use.c" if cc == "gcc" else "use.cpp")
    src.write_text('#include "flint_ops.h"\n'
                   "int use(void) { flint_int4_linear w = {128, 1, 128, 0, 0};\n"
                   "    return flint_linear_int4(&w, 0, 0, 128, 0, 0, 0, 1, FLINT_DT_BF16, 0); }\n")
    subprocess.run([cc, "-std=" + std, "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"), "-c",
                    str(src), "-o", str(tmp_path / "use.o")], check=True)


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 4, 128), (1, 1, 64), (64, 8, 64), (17, 1, 128), (40, 8, 64)])
def test_attention_workspace_covers_smaller_batches(Hq, Hkv, D):
    """The workspace of B_max sequences is enough for every smaller batch, and a byte less than a
    batch's own need is refused."""
    c = _cache(Hq, Hkv, D)
    L = ops._ops()
    sizes = [L.flint_attn_decode_workspace_bytes(ctypes.byref(c), b) for b in (1, 2, 3, 7, 31, 32, 33, 128, 1024)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    at = ops._Attn(1.0, 0, None)
    w = Hq * D
    for b in (1, 2, 33):
        few = L.flint_attn_decode(ctypes.byref(c), ctypes.byref(at), b, A, w, A, 4, A, 0, A, w, A, 15, None)
        assert few == fm.ERR_WORKSPACE
