"""Python binding of the decode-step operators (include/flint_ops.h) over torch tensors.

  Int4Linear(codes, scales)                              a linear layer's 4-bit weights
  linear_int4(w, x, y, residual=None)
  KVCache(k, v, n_q_heads)                               one layer's paged cache
  QKTransform(q_norm, k_norm, eps, cos, sin, pairs)      norm and rotation of queries and keys
  kv_append(cache, transform, qkv, positions, slots, q)
  AttnDecode(scale, window, sinks)                       attention parameters
  attn_decode_workspace(cache, B_max)
  attn_decode(cache, attn, q, table, kv_len, prefix_len, out, ws)
  token_logprobs_workspace(T_max, vocab, top_n)
  token_logprobs(logits, tokens, logprob, entropy, top_ids, top_logprobs, ws)

The descriptor classes are made once and hold their tensors; a call passes pointers, shapes
and strides to the C entry point of the same name, which checks their ranges (FlintError).
What the C side cannot see (a tensor's type, device or a shape that does not fit the
others) raises ValueError here.  bf16 tensors may be torch.bfloat16 or int16 / uint16 bits.
"""
from __future__ import annotations

import ctypes

import torch

from . import FlintError, _ptr, lib

DT_BF16, DT_FP32 = 0, 1
ROPE_HALF, ROPE_PAIRS = 0, 1

EXPORTED_OPS = ("flint_linear_int4", "flint_kv_append", "flint_attn_decode_workspace_bytes",
                "flint_attn_decode", "flint_token_logprobs_workspace_bytes", "flint_token_logprobs")

_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


class _Int4Linear(ctypes.Structure):
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32), ("group", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class _KVCache(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class _QKTransform(ctypes.Structure):
    _fields_ = [("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("rot_dim", ctypes.c_int32), ("rope_style", ctypes.c_int32), ("max_position", ctypes.c_int32),
                ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p)]


class _Attn(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("window", ctypes.c_int32), ("sinks", ctypes.c_void_p)]


_fns = None


def _ops():
    """The entry points with their argument types, set once."""
    global _fns
    if _fns is None:
        L = lib()
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        L.flint_linear_int4.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, i32, vp]
        L.flint_kv_append.argtypes = [vp, vp, i64, vp, i64, vp, vp, vp, i64, vp]
        L.flint_attn_decode_workspace_bytes.argtypes = [vp, i64]
        L.flint_attn_decode.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp, i32, vp, i64, vp, sz, vp]
        L.flint_token_logprobs_workspace_bytes.argtypes = [i64, i32, i32]
        L.flint_token_logprobs.argtypes = [i64, i32, vp, i64, i32, vp, vp, vp, i32, vp, vp, vp, sz, vp]
        for n in EXPORTED_OPS:
            getattr(L, n).restype = sz if n.endswith("_bytes") else ctypes.c_int
        _fns = L
    return _fns


def _current_stream():
    return torch.cuda.current_stream().cuda_stream


# a call's checks and its stream are most of a small call's cost on the host: torch's raw
# accessor gives the same stream without an object (2.5 us less)
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    _raw, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice

    def _current_stream():  # noqa: F811
        return _raw(_device())


def _fail(what):
    raise ValueError(what)


def _dense(t, dtypes, what):
    if not (t.is_cuda and t.dtype in dtypes and t.is_contiguous()):
        _fail("%s: a contiguous GPU tensor of %s" % (what, "/".join(map(str, dtypes))))


def _vector(t, dtype, n, what):
    """The address of n contiguous values on the GPU."""
    if t.dtype != dtype or t.numel() != n or not t.is_cuda or not t.is_contiguous():
        _fail("%s: %d contiguous %s on the GPU" % (what, n, dtype))
    return t.data_ptr()


def _rows(t, T, width, what):
    """Row stride in elements of a GPU tensor [T][...] whose rows are `width` dense elements."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        ok = shape[1] == width and (stride[1] == 1 or width == 1)
    else:
        ok = len(shape) == 3 and shape[1] * shape[2] == width and stride[2] == 1 and stride[1] == shape[2]
    if not ok or shape[0] != T or not t.is_cuda:
        _fail("%s: %d rows of %d dense elements on the GPU" % (what, T, width))
    # one row has no stride of its own: torch may report any
    return stride[0] if T > 1 or stride[0] > width else width


class Int4Linear:
    """codes: uint8 [out][in / 2]; scales: bf16 [out][in / group] (layouts in flint_ops.h)."""

    def __init__(self, codes, scales):
        _dense(codes, (torch.uint8,), "codes")
        _dense(scales, _BF16, "scales")
        if codes.dim() != 2 or scales.dim() != 2 or codes.shape[0] != scales.shape[0]:
            _fail("codes [N][K/2], scales [N][K/group]")
        self.codes, self.scales = codes, scales
        self.out_features, self.in_features = codes.shape[0], 2 * codes.shape[1]
        groups = scales.shape[1]
        if groups == 0 or self.in_features % groups:
            _fail("in_features is a multiple of the number of scales")
        self.c = _Int4Linear(self.in_features, self.out_features, self.in_features // groups, _ptr(codes), _ptr(scales))
        self.ref = ctypes.addressof(self.c)


def linear_int4(w: Int4Linear, x, y, residual=None, stream=None):
    """y = x W^T (+ residual): x bf16 [T][in], y bf16 or fp32 [T][out], rows may be strided."""
    T, N, dt = x.shape[0], w.out_features, y.dtype
    fp32 = dt is torch.float32
    if x.dtype not in _BF16 or not (fp32 or dt in _BF16):
        _fail("x: bf16, y: bf16 or fp32")
    res, ldr = None, 0
    if residual is not None:
        if residual.dtype not in _BF16:
            _fail("residual: bf16")
        res, ldr = residual.data_ptr(), _rows(residual, T, N, "residual")
    rc = (_fns or _ops()).flint_linear_int4(
        w.ref, T, x.data_ptr(), _rows(x, T, w.in_features, "x"), res, ldr, y.data_ptr(), _rows(y, T, N, "y"),
        DT_FP32 if fp32 else DT_BF16, _current_stream() if stream is None else stream)
    if rc:
        raise FlintError(rc, "flint_linear_int4")


class KVCache:
    """k: bf16 [n_pages][n_kv_heads][page][head_dim]; v: bf16 [n_pages][n_kv_heads][head_dim][page].
    The pages may be strided (a layer's slice of a larger allocation), the rest is dense."""

    def __init__(self, k, v, n_q_heads: int):
        if not (k.dtype in _BF16 and v.dtype in _BF16 and k.dim() == 4 and v.dim() == 4 and k.is_cuda and v.is_cuda):
            _fail("k and v: 4-dimensional bf16 GPU tensors")
        pages, heads, page, dim = k.shape
        if tuple(v.shape) != (pages, heads, dim, page):
            _fail("v: [n_pages][n_kv_heads][head_dim][page]")
        if any(t.stride()[1:] != (page * dim, t.shape[3], 1) for t in (k, v)):
            _fail("a page of k and of v is dense")
        if pages > 1 and k.stride(0) != v.stride(0):
            _fail("k and v have the same page stride")
        if pages > 1 and k.stride(0) < heads * page * dim:  # 0 would mean dense pages to the C side
            _fail("the pages of k and of v lie apart")
        self.k, self.v = k, v
        self.n_q_heads, self.n_kv_heads, self.head_dim, self.page_size = n_q_heads, heads, dim, page
        self.c = _KVCache(n_q_heads, heads, dim, page, pages, k.stride(0) if pages > 1 else 0, _ptr(k), _ptr(v))
        self.ref = ctypes.addressof(self.c)


class QKTransform:
    """q_norm, k_norm: bf16 [head_dim] or None; cos, sin: fp32 [max_position][rot_dim / 2] or
    None (no rotation); pairs: channels (2 i, 2 i + 1) are rotated together, else (i, i + rot_dim / 2)."""

    def __init__(self, q_norm=None, k_norm=None, eps=1e-6, cos=None, sin=None, pairs=False):
        for t in (q_norm, k_norm):
            if t is not None:
                _dense(t, _BF16, "norm weights")
        if (cos is None) != (sin is None):
            _fail("cos and sin together")
        if cos is not None:
            _dense(cos, (torch.float32,), "cos")
            _dense(sin, (torch.float32,), "sin")
            if cos.dim() != 2 or cos.shape != sin.shape:
                _fail("cos, sin: [max_position][rot_dim / 2]")
        self.norm_dims = {t.numel() for t in (q_norm, k_norm) if t is not None}
        self.q_norm, self.k_norm, self.cos, self.sin = q_norm, k_norm, cos, sin
        self.c = _QKTransform(_ptr(q_norm), _ptr(k_norm), eps, 0 if cos is None else 2 * cos.shape[1],
                              ROPE_PAIRS if pairs else ROPE_HALF, 0 if cos is None else cos.shape[0],
                              _ptr(cos), _ptr(sin))
        self.ref = ctypes.addressof(self.c)


def kv_append(cache: KVCache, transform: QKTransform, qkv, positions, slots, q, stream=None):
    """qkv: bf16 [T][(n_q_heads + 2 n_kv_heads) head_dim]; positions int32 [T] (None without
    rotation); slots int64 [T]; q: bf16 [T][n_q_heads head_dim], the transformed queries."""
    T, D, Hq = qkv.shape[0], cache.head_dim, cache.n_q_heads
    if qkv.dtype not in _BF16 or q.dtype not in _BF16:
        _fail("qkv and q: bf16")
    if transform.norm_dims and transform.norm_dims != {D}:
        _fail("norm weights: [head_dim]")
    rc = (_fns or _ops()).flint_kv_append(
        cache.ref, transform.ref, T, qkv.data_ptr(), _rows(qkv, T, (Hq + 2 * cache.n_kv_heads) * D, "qkv"),
        None if positions is None else _vector(positions, torch.int32, T, "positions"),
        _vector(slots, torch.int64, T, "slots"), q.data_ptr(), _rows(q, T, Hq * D, "q"),
        _current_stream() if stream is None else stream)
    if rc:
        raise FlintError(rc, "flint_kv_append")


class AttnDecode:
    """scale multiplies q . k; window 0: every token is seen; sinks: fp32 [n_q_heads] or None."""

    def __init__(self, scale: float, window: int = 0, sinks=None):
        if sinks is not None:
            _dense(sinks, (torch.float32,), "sinks")
        self.sinks = sinks
        self.c = _Attn(scale, window, _ptr(sinks))
        self.ref = ctypes.addressof(self.c)


def attn_decode_workspace_bytes(cache: KVCache, B_max: int) -> int:
    return int(_ops().flint_attn_decode_workspace_bytes(cache.ref, B_max))


def attn_decode_workspace(cache: KVCache, B_max: int):
    """A workspace for batches of up to B_max sequences, beside the cache."""
    return torch.empty(max(attn_decode_workspace_bytes(cache, B_max), 16), dtype=torch.uint8, device=cache.k.device)


def attn_decode(cache: KVCache, attn: AttnDecode, q, table, kv_len, prefix_len: int, out, ws, stream=None):
    """One query per sequence: q, out bf16 [B][n_q_heads head_dim]; table int32 [B][pages];
    kv_len int32 [B]; prefix_len: tokens at the start that all sequences share (0: none)."""
    B, width = q.shape[0], cache.n_q_heads * cache.head_dim
    if q.dtype not in _BF16 or out.dtype not in _BF16:
        _fail("q and out: bf16")
    if table.dim() != 2 or table.shape[0] != B:
        _fail("table: [B][pages]")
    if attn.sinks is not None and attn.sinks.numel() != cache.n_q_heads:
        _fail("sinks: fp32 [n_q_heads]")
    if not ws.is_cuda or not ws.is_contiguous():
        _fail("ws: a contiguous GPU tensor")
    rc = (_fns or _ops()).flint_attn_decode(
        cache.ref, attn.ref, B, q.data_ptr(), _rows(q, B, width, "q"),
        _vector(table, torch.int32, B * table.shape[1], "table"), table.shape[1], _vector(kv_len, torch.int32, B, "kv_len"),
        prefix_len, out.data_ptr(), _rows(out, B, width, "out"), ws.data_ptr(), ws.nbytes,
        _current_stream() if stream is None else stream)
    if rc:
        raise FlintError(rc, "flint_attn_decode")


def token_logprobs_workspace_bytes(T_max: int, vocab: int, top_n: int = 0) -> int:
    return int(_ops().flint_token_logprobs_workspace_bytes(T_max, vocab, top_n))


def token_logprobs_workspace(T_max: int, vocab: int, top_n: int = 0, device="cuda"):
    return torch.empty(max(token_logprobs_workspace_bytes(T_max, vocab, top_n), 16), dtype=torch.uint8, device=device)


def token_logprobs(logits, tokens, logprob, entropy, top_ids, top_logprobs, ws, stream=None):
    """logits: bf16 or fp32 [T][vocab], rows may be strided; tokens int32 [T]; logprob, entropy
    fp32 [T]; top_ids int32 and top_logprobs fp32 [T][n].  tokens with logprob, entropy, and
    top_ids with top_logprobs may be None."""
    T, V = logits.shape
    dt = logits.dtype
    fp32 = dt is torch.float32
    if not fp32 and dt not in _BF16:
        _fail("logits: bf16 or fp32 [T][vocab]")
    tok = None if tokens is None else _vector(tokens, torch.int32, T, "tokens")
    lp = None if logprob is None else _vector(logprob, torch.float32, T, "logprob")
    ent = None if entropy is None else _vector(entropy, torch.float32, T, "entropy")
    n, ids, top = 0, None, None
    if (top_ids is None) != (top_logprobs is None):
        _fail("top_ids and top_logprobs together")
    if top_ids is not None and top_ids.shape[-1]:
        n = top_ids.shape[-1]
        ids, top = _vector(top_ids, torch.int32, T * n, "top_ids"), _vector(top_logprobs, torch.float32, T * n, "top_logprobs")
    if not ws.is_cuda or not ws.is_contiguous():
        _fail("ws: a contiguous GPU tensor")
    rc = (_fns or _ops()).flint_token_logprobs(
        T, V, logits.data_ptr(), _rows(logits, T, V, "logits"), DT_FP32 if fp32 else DT_BF16, tok, lp, ent, n, ids, top,
        ws.data_ptr(), ws.nbytes, _current_stream() if stream is None else stream)
    if rc:
        raise FlintError(rc, "flint_token_logprobs")
