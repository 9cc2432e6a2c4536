"""Plain 64-bit forms of the decode-step operators on the CPU, with the a-priori error bounds
that the GPU tests hold the kernels to.  u = 2^-24 is the fp32 rounding unit, and a result
rounded to bf16 once is within 2^-9 of its value (2^-8 allows for a value on the other side
of a rounding boundary).
"""
import math

import torch

U = 2.0 ** -24
F64 = torch.float64


def int4_weights(codes, scales):
    c = codes.to(torch.int32)
    q = torch.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)
    q = torch.where(q > 7, q - 16, q).to(F64)
    g = q.shape[1] // scales.shape[1]
    return q * scales.to(F64).repeat_interleave(g, 1)


def linear(codes, scales, x, residual=None, bf16=True):
    """(y, bound): K exact products, their sum in fp32 in any order, a scale and a residual."""
    w, x = int4_weights(codes, scales), x.to(F64)
    y, mag = x @ w.t(), x.abs() @ w.abs().t()
    if residual is not None:
        y, mag = y + residual.to(F64), mag + residual.to(F64).abs()
    return y, (w.shape[1] + 8) * U * mag + (2.0 ** -8 * y.abs() if bf16 else 0)


def transform(x, w, eps, cos, sin, pairs):
    """(x', bound) of heads [..., D]: x' rounded to bf16 once; cos, sin: [..., rot / 2]."""
    D = x.shape[-1]
    x = x.to(F64)
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(F64)
    mag = x.abs()
    if cos is not None and cos.shape[-1]:
        h = cos.shape[-1]
        i = torch.arange(h)
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + h)
        c, s = cos.to(F64), sin.to(F64)
        xa, xb = x[..., a], x[..., b]
        x, mag = x.clone(), mag.clone()
        x[..., a], x[..., b] = xa * c - xb * s, xb * c + xa * s
        mag[..., a], mag[..., b] = xa.abs() + xb.abs(), xa.abs() + xb.abs()
    # the mean of squares: D products and sums; sqrt, division, weight, rotation: 16 more
    return x, 2.0 ** -8 * x.abs() + (D + 16) * U * mag


def attn(q, k_cache, v_cache, table, lens, scale, window=0, sinks=None):
    """(out, bound): q [B][Hq][D] on the CPU, caches as the kernels see them."""
    B, Hq, D = q.shape
    n_pages, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    out, bound = torch.zeros(B, Hq, D, dtype=F64), torch.zeros(B, Hq, D, dtype=F64)
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        j = torch.arange(max(0, n - window) if window else 0, n)
        pg = table[b, j // page].long()
        ok = (pg >= 0) & (pg < n_pages)
        j, pg = j[ok], pg[ok]
        if len(j) == 0:
            continue
        k = k_cache[pg, :, j % page].to(F64).transpose(0, 1)       # [Hkv][n][D]
        v = v_cache[pg, :, :, j % page].to(F64).transpose(0, 1)
        qq = q[b].to(F64).view(Hkv, G, D)
        s = qq @ k.transpose(1, 2) * scale
        mag = (qq.abs() @ k.abs().transpose(1, 2) * abs(scale)).amax(-1, keepdim=True)
        m = s.amax(-1, keepdim=True)
        if sinks is not None:
            m = torch.maximum(m, sinks.to(F64).view(Hkv, G, 1))
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        if sinks is not None:
            l = l + torch.exp(sinks.to(F64).view(Hkv, G, 1) - m)
        o, w = p @ v / l, p @ v.abs() / l
        # a score is off by (D + 4) u of its terms' magnitudes, its scaled exponent by 4 u more
        # and the exponential by 2^-22; the weights are relative to their own sum (twice), are
        # rounded to bf16 (2^-9) and summed over n tokens in fp32
        d = (D + 8) * U * mag + 4 * U * (s - m).abs().clamp(max=100).amax(-1, keepdim=True) + 2.0 ** -22
        err = (2 * d + 2.0 ** -9 + (len(j) + 64) * U) * w
        out[b], bound[b] = o.reshape(Hq, D), (err + 2.0 ** -8 * o.abs()).reshape(Hq, D)
    return out, bound


def logprobs(x, tokens, n):
    """(logprob, entropy, top_ids, top_logprobs, bound of the log probabilities, of the entropy)."""
    x = x.to(F64)
    T, V = x.shape
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    lp = x - m - torch.log(z)
    p = e / z
    plogp = torch.where(p > 0, p * lp.clamp(min=-1e6), torch.zeros_like(p))
    ids = torch.sort(torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x), dim=-1, descending=True, stable=True).indices
    # a sum of V terms in fp32, each an exponential of a difference off by 2 u of its size (at
    # most 100 before it vanishes) and by 2^-22 itself
    eps = (V / 8 + 256) * U + 2.0 ** -21
    fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    b_lp = eps + 4 * U * (fin + 32)
    b_h = eps * (4 + 2 * -plogp.sum(-1)) + 4 * U * 32
    t = tokens.long().clamp(0, V - 1)
    lt = lp.gather(1, t[:, None])[:, 0]
    return lt, -plogp.sum(-1), ids[:, :n], lp.gather(1, ids[:, :n]), b_lp, b_h
