"""Python binding of the operators of a server of many requests (include/flint_serve.h) over torch
tensors.

  KV4Cache(data, n_q_heads, n_kv_heads, head_dim, page_size)   one layer's paged cache in 4 bits
  kv4_append(cache, transform, qkv, positions, slots, q, k=None, v=None)
  kv4_attn_decode_workspace(cache, B_max)
  kv4_attn_decode(cache, attn, q, table, kv_len, prefix_len, out, ws)
  KVPages(caches)                                              the memory of a pool's pages
  KVState(refs, free_list, n_free, table, kv_len), kv_state(n_pages, rows, width)   who holds them
  kv_pages_workspace(pages, rows_max)
  kv_advance(pages, old, new, parent, grow, slots, ws)         fork, free, reorder, grow, copy on write
  kv_compact(pages, old, new, moved, ws)                       live pages to the front
  LoraAdapters(a, b, ranks=None, scales=None)                  low-rank adapters of one linear layer
  lora_workspace(adapters, T_max)
  lora(adapters, x, ids, base, y, ws)
  LogitRules(history=..., bias_start=..., masks=..., ...)      penalties, biases, grammar masks
  logits_adjust(rules, logits, out)

As in ops.py: descriptors are made once and hold their tensors, a call passes pointers, shapes and
strides to the C entry point of the same name, which checks their ranges (FlintError); a tensor's
type, device or a shape that does not fit the others raises ValueError here.
"""
from __future__ import annotations

import ctypes

import torch

from . import FlintError, _ptr, lib
from .ops import _BF16, DT_BF16, DT_FP32, AttnDecode, KVCache, QKTransform, _current_stream, _dense, _fail, _rows, _vector

EXPORTED_SERVE = ("flint_kv4_append", "flint_kv4_attn_decode_workspace_bytes", "flint_kv4_attn_decode",
                  "flint_kv_pages_workspace_bytes", "flint_kv_advance", "flint_kv_compact",
                  "flint_lora_workspace_bytes", "flint_lora", "flint_logits_adjust")

_I32 = torch.int32


class _KV4Cache(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("data", ctypes.c_void_p)]


class _KVArray(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("bytes", ctypes.c_int64), ("stride", ctypes.c_int64)]


class _KVPages(ctypes.Structure):
    _fields_ = [("page_size", ctypes.c_int32), ("n_arrays", ctypes.c_int32), ("n_pages", ctypes.c_int64),
                ("arrays", ctypes.c_void_p)]


class _KVState(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("refs", "free_list", "n_free", "table", "kv_len")]


class _Lora(ctypes.Structure):
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32), ("max_rank", ctypes.c_int32),
                ("n_adapters", ctypes.c_int32), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class _LogitRules(ctypes.Structure):
    _fields_ = [("history", ctypes.c_void_p), ("ldh", ctypes.c_int64)] + [
        (n, ctypes.c_void_p) for n in ("prompt_len", "total_len", "repetition", "frequency", "presence",
                                       "bias_start", "bias_ids", "bias")] + [
        ("n_bias", ctypes.c_int64), ("masks", ctypes.c_void_p), ("ldm", ctypes.c_int64), ("n_masks", ctypes.c_int64),
        ("mask_rows", ctypes.c_void_p)]


_fns = None


def _serve():
    """The entry points with their argument types, set once."""
    global _fns
    if _fns is None:
        L = lib()
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        L.flint_kv4_append.argtypes = [vp, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, i64, vp]
        L.flint_kv4_attn_decode_workspace_bytes.argtypes = [vp, i64]
        L.flint_kv4_attn_decode.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp, i32, vp, i64, vp, sz, vp]
        L.flint_kv_pages_workspace_bytes.argtypes = [vp, i64]
        L.flint_kv_advance.argtypes = [vp, i64, i64, vp, i64, vp, vp, vp, vp, i64, vp, sz, vp]
        L.flint_kv_compact.argtypes = [vp, i64, i64, vp, vp, vp, vp, sz, vp]
        L.flint_lora_workspace_bytes.argtypes = [vp, i64]
        L.flint_lora.argtypes = [vp, i64, vp, i64, vp, vp, i64, i32, vp, i64, i32, vp, sz, vp]
        L.flint_logits_adjust.argtypes = [vp, i64, i32, vp, i64, vp, i64, i32, vp]
        for n in EXPORTED_SERVE:
            getattr(L, n).restype = sz if n.endswith("_bytes") else ctypes.c_int
        _fns = L
    return _fns


def _dense_ws(ws):
    if not ws.is_cuda or not ws.is_contiguous():
        _fail("ws: a contiguous GPU tensor")
    return ws.data_ptr()


# ---- 4-bit cache -------------------------------------------------------------------------
class KV4Cache:
    """data: uint8 [n_pages][bytes of a page], a page's block as in flint_serve.h: key codes, value
    codes, key scales, value scales.  The pages may be strided (a layer's slice of a larger
    allocation), the rest is dense.  k_codes, v_codes [page][head][token][dim / 2] and k_scales,
    v_scales [page][head][dim / 32][token] are views of it."""

    @staticmethod
    def page_bytes(n_kv_heads: int, head_dim: int, page_size: int) -> int:
        return 2 * n_kv_heads * page_size * (head_dim // 2 + head_dim // 32)

    def __init__(self, data, n_q_heads: int, n_kv_heads: int, head_dim: int, page_size: int):
        if data.dtype != torch.uint8 or data.dim() != 2 or not data.is_cuda:
            _fail("data: a uint8 GPU tensor [n_pages][bytes of a page]")
        if head_dim not in (64, 128):
            _fail("head_dim: 64 or 128")
        pages, block = data.shape
        if block != self.page_bytes(n_kv_heads, head_dim, page_size) or data.stride(1) != 1:
            _fail("data: %d dense bytes to a page" % self.page_bytes(n_kv_heads, head_dim, page_size))
        if pages > 1 and data.stride(0) < block:  # 0 would mean dense pages to the C side
            _fail("the pages lie apart")
        self.data = data
        self.n_q_heads, self.n_kv_heads, self.head_dim, self.page_size = n_q_heads, n_kv_heads, head_dim, page_size
        c, z = n_kv_heads * page_size * head_dim // 2, n_kv_heads * page_size * head_dim // 32
        codes, scales = (n_kv_heads, page_size, head_dim // 2), (n_kv_heads, head_dim // 32, page_size)
        self.k_codes, self.v_codes = data[:, :c].unflatten(1, codes), data[:, c:2 * c].unflatten(1, codes)
        self.k_scales, self.v_scales = data[:, 2 * c:2 * c + z].unflatten(1, scales), data[:, 2 * c + z:].unflatten(1, scales)
        self.c = _KV4Cache(n_q_heads, n_kv_heads, head_dim, page_size, pages, data.stride(0) if pages > 1 else 0, _ptr(data))
        self.ref = ctypes.addressof(self.c)


def kv4_append(cache: KV4Cache, transform: QKTransform, qkv, positions, slots, q, k=None, v=None, stream=None):
    """As kv_append; k, v: bf16 [T][n_kv_heads head_dim] or None, the values of the new codes."""
    T, D, Hq, Hkv = qkv.shape[0], cache.head_dim, cache.n_q_heads, cache.n_kv_heads
    if qkv.dtype not in _BF16 or q.dtype not in _BF16 or (k is not None and k.dtype not in _BF16) or (
            v is not None and v.dtype not in _BF16):
        _fail("qkv, q, k and v: bf16")
    if transform.norm_dims and transform.norm_dims != {D}:
        _fail("norm weights: [head_dim]")
    rc = (_fns or _serve()).flint_kv4_append(
        cache.ref, transform.ref, T, qkv.data_ptr(), _rows(qkv, T, (Hq + 2 * Hkv) * D, "qkv"),
        None if positions is None else _vector(positions, _I32, T, "positions"),
        _vector(slots, torch.int64, T, "slots"), q.data_ptr(), _rows(q, T, Hq * D, "q"),
        None if k is None else k.data_ptr(), 0 if k is None else _rows(k, T, Hkv * D, "k"),
        None if v is None else v.data_ptr(), 0 if v is None else _rows(v, T, Hkv * D, "v"),
        _current_stream() if stream is None else stream)
    if rc:
        raise FlintError(rc, "flint_kv4_append")


def kv4_attn_decode_workspace_bytes(cache: KV4Cache, B_max: int) -> int:
    return int(_serve().flint_kv4_attn_decode_workspace_bytes(cache.ref, B_max))


def kv4_attn_decode_workspace(cache: KV4Cache, B_max: int):
    """A workspace for batches of up to B_max sequences, beside the cache."""
    return torch.empty(max(kv4_attn_decode_workspace_bytes(cache, B_max), 16), dtype=torch.uint8, device=cache.data.device)


def kv4_attn_decode(cache: KV4Cache, attn: AttnDecode, q, table, kv_len, prefix_len: int, out, ws, stream=None):
    """As attn_decode, over a 4-bit cache."""
    B, width = q.shape[0], cache.n_q_heads * cache.head_dim
    if q.dtype not in _BF16 or out.dtype not in _BF16:
        _fail("q and out: bf16")
    if table.dim() != 2 or table.shape[0] != B:
        _fail("table: [B][pages]")
    if attn.sinks is not None and attn.sinks.numel() != cache.n_q_heads:
        _fail("sinks: fp32 [n_q_heads]")
    rc = (_fns or _serve()).flint_kv4_attn_decode(
        cache.ref, attn.ref, B, q.data_ptr(), _rows(q, B, width, "q"),
        _vector(table, _I32, B * table.shape[1], "table"), table.shape[1], _vector(kv_len, _I32, B, "kv_len"),
        prefix_len, out.data_ptr(), _rows(out, B, width, "out"), _dense_ws(ws), ws.nbytes,
        _current_stream() if stream is None else stream)
    if rc:
        raise FlintError(rc, "flint_kv4_attn_decode")


# ---- pages -------------------------------------------------------------------------------
class KVPages:
    """The memory behind the page numbers of a pool: the caches (KVCache or KV4Cache) of all layers,
    with the same number of pages of the same size."""

    def __init__(self, caches):
        self.caches = list(caches)
        if not self.caches:
            _fail("at least one cache")
        arrays = []
        for c in self.caches:
            for t in (c.data,) if isinstance(c, KV4Cache) else (c.k, c.v):
                size = t[0].numel() * t.element_size()
                arrays.append((t.data_ptr(), size, t.stride(0) * t.element_size() if t.shape[0] > 1 else size))
        self.n_pages, self.page_size = self.caches[0].c.n_pages, self.caches[0].page_size
        if any(c.c.n_pages != self.n_pages or c.page_size != self.page_size for c in self.caches):
            _fail("caches of the same number of pages of the same size")
        first = self.caches[0]
        self.device = (first.data if isinstance(first, KV4Cache) else first.k).device
        self.arrays = (_KVArray * len(arrays))(*arrays)
        self.c = _KVPages(self.page_size, len(arrays), self.n_pages, ctypes.addressof(self.arrays))
        self.ref = ctypes.addressof(self.c)


class KVState:
    """Who holds which page, int32 tensors: refs and free_list [n_pages], n_free [1], table
    [rows][width], kv_len [rows]."""

    def __init__(self, refs, free_list, n_free, table, kv_len):
        n = refs.numel()
        if table.dim() != 2:
            _fail("table: [rows][pages]")
        self.n_pages, (self.rows, self.width) = n, table.shape
        self.refs, self.free_list, self.n_free, self.table, self.kv_len = refs, free_list, n_free, table, kv_len
        self.c = _KVState(_vector(refs, _I32, n, "refs"), _vector(free_list, _I32, n, "free_list"), _vector(n_free, _I32, 1, "n_free"),
                          _vector(table, _I32, self.rows * self.width, "table"), _vector(kv_len, _I32, self.rows, "kv_len"))
        self.ref = ctypes.addressof(self.c)


def kv_state(n_pages: int, rows: int, width: int, device="cuda") -> KVState:
    """A state of empty rows and free pages, of which page 0 is taken first."""
    z = lambda *s: torch.zeros(*s, dtype=_I32, device=device)  # noqa: E731
    free = torch.arange(n_pages - 1, -1, -1, dtype=_I32, device=device)
    return KVState(z(n_pages), free, z(1) + n_pages, z(rows, width) - 1, z(rows))


def kv_pages_workspace_bytes(pages: KVPages, rows_max: int) -> int:
    return int(_serve().flint_kv_pages_workspace_bytes(pages.ref, rows_max))


def kv_pages_workspace(pages: KVPages, rows_max: int):
    return torch.empty(max(kv_pages_workspace_bytes(pages, rows_max), 16), dtype=torch.uint8, device=pages.device)


def _states(pages, old, new):
    if old.n_pages != pages.n_pages or new.n_pages != pages.n_pages or old.width != new.width:
        _fail("states of the pool's pages with tables of the same width")


def kv_advance(pages: KVPages, old: KVState, new: KVState, parent, grow, slots, ws, stream=None):
    """parent, grow: int32 [rows of new]; slots: int64 [rows of new][n] or None."""
    R, lds = new.rows, 0
    _states(pages, old, new)
    if slots is not None:
        if slots.dim() != 2 or slots.shape[0] != R:
            _fail("slots: [rows][tokens]")
        lds = slots.shape[1]
        slots = _vector(slots, torch.int64, R * lds, "slots") if lds else None
    rc = (_fns or _serve()).flint_kv_advance(
        pages.ref, old.width, old.rows, old.ref, R, new.ref, _vector(parent, _I32, R, "parent"), _vector(grow, _I32, R, "grow"),
        slots, lds, _dense_ws(ws), ws.nbytes, _current_stream() if stream is None else stream)
    if rc:
        raise FlintError(rc, "flint_kv_advance")


def kv_compact(pages: KVPages, old: KVState, new: KVState, moved, ws, stream=None):
    """moved: int32 [n_pages], the new number of each page."""
    _states(pages, old, new)
    if old.rows != new.rows:
        _fail("states of the same rows")
    rc = (_fns or _serve()).flint_kv_compact(
        pages.ref, old.width, old.rows, old.ref, new.ref, _vector(moved, _I32, pages.n_pages, "moved"), _dense_ws(ws), ws.nbytes,
        _current_stream() if stream is None else stream)
    if rc:
        raise FlintError(rc, "flint_kv_compact")


# ---- adapters ----------------------------------------------------------------------------
class LoraAdapters:
    """a: bf16 [n][max_rank][in]; b: bf16 [n][out][max_rank]; ranks int32 [n], scales fp32 [n] or None."""

    def __init__(self, a, b, ranks=None, scales=None):
        _dense(a, _BF16, "a")
        _dense(b, _BF16, "b")
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            _fail("a [n][max_rank][in], b [n][out][max_rank]")
        n, rank, self.in_features = a.shape
        self.out_features = b.shape[1]
        self.a, self.b, self.ranks, self.scales = a, b, ranks, scales
        self.c = _Lora(self.in_features, self.out_features, rank, n, _ptr(a), _ptr(b),
                       None if ranks is None else _vector(ranks, _I32, n, "ranks"),
                       None if scales is None else _vector(scales, torch.float32, n, "scales"))
        self.ref = ctypes.addressof(self.c)


def lora_workspace_bytes(adapters: LoraAdapters, T_max: int) -> int:
    return int(_serve().flint_lora_workspace_bytes(adapters.ref, T_max))


def lora_workspace(adapters: LoraAdapters, T_max: int):
    return torch.empty(max(lora_workspace_bytes(adapters, T_max), 16), dtype=torch.uint8, device=adapters.a.device)


def lora(adapters: LoraAdapters, x, ids, base, y, ws, stream=None):
    """y = base + the adapters' part: x bf16 [T][in]; ids int32 [T] (-1: none); base bf16 or fp32
    [T][out] or None, may be y; y bf16 or fp32 [T][out]; rows may be strided."""
    T, N = x.shape[0], adapters.out_features
    if x.dtype not in _BF16:
        _fail("x: bf16")
    for t in (y,) if base is None else (y, base):
        if t.dtype is not torch.float32 and t.dtype not in _BF16:
            _fail("base and y: bf16 or fp32")
    rc = (_fns or _serve()).flint_lora(
        adapters.ref, T, x.data_ptr(), _rows(x, T, adapters.in_features, "x"), _vector(ids, _I32, T, "ids"),
        _ptr(base), 0 if base is None else _rows(base, T, N, "base"),
        DT_FP32 if base is not None and base.dtype is torch.float32 else DT_BF16, y.data_ptr(), _rows(y, T, N, "y"),
        DT_FP32 if y.dtype is torch.float32 else DT_BF16, _dense_ws(ws), ws.nbytes, _current_stream() if stream is None else stream)
    if rc:
        raise FlintError(rc, "flint_lora")


# ---- logits ------------------------------------------------------------------------------
class LogitRules:
    """Per-row rules of a batch of T rows; any of them may be None.
    history int32 [T][n] with total_len and prompt_len int32 [T]; repetition, frequency, presence
    fp32 [T]; bias_start int32 [T + 1], bias_ids int32 and bias fp32 [entries]; masks int32 or
    uint32 [n_masks][words], mask_rows int32 [T].  The tensors are read at each call."""

    def __init__(self, history=None, prompt_len=None, total_len=None, repetition=None, frequency=None, presence=None,
                 bias_start=None, bias_ids=None, bias=None, masks=None, mask_rows=None):
        self.held = (history, prompt_len, total_len, repetition, frequency, presence, bias_start, bias_ids, bias, masks, mask_rows)
        f32 = torch.float32
        self.rows = None
        if history is None and any(t is not None for t in (prompt_len, total_len, repetition, frequency, presence)):
            _fail("penalties need a history")
        if (bias_start is None) != (bias_ids is None) or (bias_ids is None) != (bias is None):
            _fail("bias_start, bias_ids and bias together")
        if mask_rows is not None and masks is None:
            _fail("mask_rows need masks")

        def rows(t, dtype, what, more=0):
            if t is None:
                return None
            n = t.numel() - more
            if self.rows is None:
                self.rows = n
            return _vector(t, dtype, self.rows + more, what)

        ldh = 0
        if history is not None:
            if history.dim() != 2:
                _fail("history: [T][tokens]")
            self.rows, ldh = history.shape
            _vector(history, _I32, history.numel(), "history")
        pl, tl = rows(prompt_len, _I32, "prompt_len"), rows(total_len, _I32, "total_len")
        rep, freq, pres = rows(repetition, f32, "repetition"), rows(frequency, f32, "frequency"), rows(presence, f32, "presence")
        bs = rows(bias_start, _I32, "bias_start", 1)
        n_bias = 0 if bias is None else bias.numel()
        bi = None if bias_ids is None else _vector(bias_ids, _I32, n_bias, "bias_ids")
        bv = None if bias is None else _vector(bias, f32, n_bias, "bias")
        ldm = n_masks = 0
        if masks is not None:
            if masks.dim() != 2 or masks.dtype not in (_I32, torch.uint32):
                _fail("masks: int32 or uint32 [n_masks][words]")
            _vector(masks, masks.dtype, masks.numel(), "masks")
            n_masks, ldm = masks.shape
        mr = rows(mask_rows, _I32, "mask_rows")
        self.c = _LogitRules(_ptr(history), ldh, pl, tl, rep, freq, pres, bs, bi, bv, n_bias, _ptr(masks), ldm, n_masks, mr)
        self.ref = ctypes.addressof(self.c)


def logits_adjust(rules: LogitRules, logits, out, stream=None):
    """logits, out: bf16 or fp32 [T][vocab] of the same type, rows may be strided; out may be logits."""
    T, V = logits.shape
    fp32 = logits.dtype is torch.float32
    if not (fp32 and out.dtype is torch.float32) and not (logits.dtype in _BF16 and out.dtype in _BF16):
        _fail("logits and out: bf16 or fp32 [T][vocab], the same")
    if rules.rows is not None and rules.rows != T:
        _fail("rules of %d rows" % rules.rows)
    rc = (_fns or _serve()).flint_logits_adjust(
        rules.ref, T, V, logits.data_ptr(), _rows(logits, T, V, "logits"), out.data_ptr(), _rows(out, T, V, "out"),
        DT_FP32 if fp32 else DT_BF16, _current_stream() if stream is None else stream)
    if rc:
        raise FlintError(rc, "flint_logits_adjust")
