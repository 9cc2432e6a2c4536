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

from . import _check, _ptr, _stream, lib

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


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _dense(t, dtypes, what):
    _need(t.is_cuda and t.dtype in dtypes and t.is_contiguous(),
          "%s: a contiguous GPU tensor of %s" % (what, "/".join(map(str, dtypes))))


def _vector(t, dtype, n, what):
    _need(t.is_cuda and t.dtype == dtype and t.numel() == n and t.is_contiguous(), "%s: %d contiguous %s on the GPU" % (what, n, dtype))


def _row_stride(t, width, what):
    """Row stride in elements of a [T][...] tensor whose rows are `width` dense elements."""
    shape, stride = t.shape, t.stride()
    _need(t.is_cuda, "%s: a GPU tensor" % what)
    if len(shape) == 2:
        ok = shape[1] == width and (stride[1] == 1 or width == 1)
    else:
        ok = len(shape) == 3 and shape[1] * shape[2] == width and stride[2] == 1 and stride[1] == shape[2]
    _need(ok, "%s: rows of %d dense elements" % (what, width))
    # one row has no stride of its own: torch may report any
    return stride[0] if shape[0] > 1 else max(stride[0], width)


class Int4Linear:
    """codes: uint8 [out][in / 2]; scales: bf16 [out][in / group] (layouts in flint_ops.h)."""

    def __init__(self, codes, scales):
        _dense(codes, (torch.uint8,), "codes")
        _dense(scales, _BF16, "scales")
        _need(codes.dim() == 2 and scales.dim() == 2 and codes.shape[0] == scales.shape[0], "codes [N][K/2], scales [N][K/group]")
        self.codes, self.scales = codes, scales
        self.out_features, self.in_features = codes.shape[0], 2 * codes.shape[1]
        groups = scales.shape[1]
        _need(groups > 0 and self.in_features % groups == 0, "in_features is a multiple of the number of scales")
        self.c = _Int4Linear(self.in_features, self.out_features, self.in_features // groups, _ptr(codes), _ptr(scales))
        self.ref = ctypes.addressof(self.c)


def linear_int4(w: Int4Linear, x, y, residual=None, stream=None):
    """y = x W^T (+ residual): x bf16 [T][in], y bf16 or fp32 [T][out], rows may be strided."""
    T, N = x.shape[0], w.out_features
    _need(x.dtype in _BF16 and y.shape[0] == T, "x: bf16 [T][in], y: [T][out]")
    fp32 = y.dtype == torch.float32
    _need(fp32 or y.dtype in _BF16, "y: bf16 or fp32")
    ldr = 0
    if residual is not None:
        _need(residual.dtype in _BF16 and residual.shape[0] == T, "residual: bf16 [T][out]")
        ldr = _row_stride(residual, N, "residual")
    rc = _ops().flint_linear_int4(w.ref, T, x.data_ptr(), _row_stride(x, w.in_features, "x"), _ptr(residual), ldr,
                                  y.data_ptr(), _row_stride(y, N, "y"), DT_FP32 if fp32 else DT_BF16, _stream(stream))
    _check(rc, "flint_linear_int4")


class KVCache:
    """k: bf16 [n_pages][n_kv_heads][page][head_dim]; v: bf16 [n_pages][n_kv_heads][head_dim][page].
    The pages may be strided (a layer's slice of a larger allocation), the rest is dense."""

    def __init__(self, k, v, n_q_heads: int):
        _need(k.dtype in _BF16 and v.dtype in _BF16 and k.dim() == 4 and v.dim() == 4 and k.is_cuda and v.is_cuda,
              "k and v: 4-dimensional bf16 GPU tensors")
        pages, heads, page, dim = k.shape
        _need(tuple(v.shape) == (pages, heads, dim, page), "v: [n_pages][n_kv_heads][head_dim][page]")
        for t in (k, v):
            _need(t.stride()[1:] == (page * dim, t.shape[3], 1), "a page of k and of v is dense")
        _need(pages < 2 or k.stride(0) == v.stride(0), "k and v have the same page stride")
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
        _need((cos is None) == (sin is None), "cos and sin together")
        if cos is not None:
            _dense(cos, (torch.float32,), "cos")
            _dense(sin, (torch.float32,), "sin")
            _need(cos.dim() == 2 and cos.shape == sin.shape, "cos, sin: [max_position][rot_dim / 2]")
        self.q_norm, self.k_norm, self.cos, self.sin = q_norm, k_norm, cos, sin
        self.c = _QKTransform(_ptr(q_norm), _ptr(k_norm), eps, 0 if cos is None else 2 * cos.shape[1],
                              ROPE_PAIRS if pairs else ROPE_HALF, 0 if cos is None else cos.shape[0],
                              _ptr(cos), _ptr(sin))
        self.ref = ctypes.addressof(self.c)


def kv_append(cache: KVCache, transform: QKTransform, qkv, positions, slots, q, stream=None):
    """qkv: bf16 [T][(n_q_heads + 2 n_kv_heads) head_dim]; positions int32 [T] (None without
    rotation); slots int64 [T]; q: bf16 [T][n_q_heads head_dim], the transformed queries."""
    T, D, Hq = qkv.shape[0], cache.head_dim, cache.n_q_heads
    _need(qkv.dtype in _BF16 and q.dtype in _BF16 and q.shape[0] == T, "qkv and q: bf16 [T][...]")
    _vector(slots, torch.int64, T, "slots")
    if positions is not None:
        _vector(positions, torch.int32, T, "positions")
    for t in (transform.q_norm, transform.k_norm):
        _need(t is None or t.numel() == D, "norm weights: [head_dim]")
    rc = _ops().flint_kv_append(cache.ref, transform.ref, T, qkv.data_ptr(),
                                _row_stride(qkv, (Hq + 2 * cache.n_kv_heads) * D, "qkv"), _ptr(positions),
                                slots.data_ptr(), q.data_ptr(), _row_stride(q, Hq * D, "q"), _stream(stream))
    _check(rc, "flint_kv_append")


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
    _need(q.dtype in _BF16 and out.dtype in _BF16 and out.shape[0] == B, "q and out: bf16 [B][...]")
    _need(table.is_cuda and table.dtype == torch.int32 and table.dim() == 2 and table.shape[0] == B
          and table.is_contiguous(), "table: contiguous int32 [B][pages]")
    _vector(kv_len, torch.int32, B, "kv_len")
    _need(ws.is_cuda, "ws: a GPU tensor")
    _need(attn.sinks is None or attn.sinks.numel() == cache.n_q_heads, "sinks: fp32 [n_q_heads]")
    rc = _ops().flint_attn_decode(cache.ref, attn.ref, B, q.data_ptr(), _row_stride(q, width, "q"), table.data_ptr(),
                                  table.shape[1], kv_len.data_ptr(), prefix_len, out.data_ptr(),
                                  _row_stride(out, width, "out"), ws.data_ptr(), ws.numel() * ws.element_size(),
                                  _stream(stream))
    _check(rc, "flint_attn_decode")


def token_logprobs_workspace_bytes(T_max: int, vocab: int, top_n: int = 0) -> int:
    return int(_ops().flint_token_logprobs_workspace_bytes(T_max, vocab, top_n))


def token_logprobs_workspace(T_max: int, vocab: int, top_n: int = 0, device="cuda"):
    return torch.empty(max(token_logprobs_workspace_bytes(T_max, vocab, top_n), 16), dtype=torch.uint8, device=device)


def token_logprobs(logits, tokens, logprob, entropy, top_ids, top_logprobs, ws, stream=None):
    """logits: bf16 or fp32 [T][vocab], rows may be strided; tokens int32 [T]; logprob, entropy
    fp32 [T]; top_ids int32 and top_logprobs fp32 [T][n].  tokens with logprob, entropy, and
    top_ids with top_logprobs may be None."""
    T, V = logits.shape
    fp32 = logits.dtype == torch.float32
    _need(fp32 or logits.dtype in _BF16, "logits: bf16 or fp32 [T][vocab]")
    for t, dt, what in ((tokens, torch.int32, "tokens"), (logprob, torch.float32, "logprob"),
                        (entropy, torch.float32, "entropy")):
        if t is not None:
            _vector(t, dt, T, what)
    _need(ws.is_cuda, "ws: a GPU tensor")
    n = 0
    if top_ids is not None:
        n = top_ids.shape[1]
        _vector(top_ids, torch.int32, T * n, "top_ids")
        _need(top_logprobs is not None and top_logprobs.shape == top_ids.shape, "top_logprobs: fp32 [T][n], like top_ids")
        _vector(top_logprobs, torch.float32, T * n, "top_logprobs")
    else:
        _need(top_logprobs is None, "top_ids and top_logprobs together")
    rc = _ops().flint_token_logprobs(T, V, logits.data_ptr(), _row_stride(logits, V, "logits"), DT_FP32 if fp32 else DT_BF16,
                                     _ptr(tokens), _ptr(logprob), _ptr(entropy), n, _ptr(top_ids) if n else None,
                                     _ptr(top_logprobs) if n else None, ws.data_ptr(), ws.numel() * ws.element_size(),
                                     _stream(stream))
    _check(rc, "flint_token_logprobs")
