"""Decode-step operators on inputs where rounding on the way would show in the result: sums whose
large terms must leave nothing behind, probabilities that cancel, logits with a large common
offset.  U = 2^-24 is the fp32 rounding unit; each bound counts the roundings of the path."""
import math
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(__file__))

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import ops_ref as ref  # noqa: E402
import sparse_moe_transformer_wave_amd as fm  # noqa: E402

BF = torch.bfloat16
F64 = torch.float64
U = 2.0 ** -24


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---- attention ---------------------------------------------------------------------------
def _fine_probabilities(n, D, seed):
    """One head whose scores are the bf16 numbers t (0 for tokens 0 and 1, then -2 .. 0), exact in
    fp32, and values that leave of channel d's result only what bf16 twice over leaves of
    token j(d)'s probability: o = (p_j - a - b) / sum p, a = bf16(p_j), b = bf16(p_j - a)."""
    g = _gen(seed)
    t = -2 * torch.rand(n, generator=g, dtype=F64)
    t[:2] = 0
    t = t.to(BF).to(F64)
    p = t.exp()
    j = 2 + torch.randperm(n - 2, generator=g)[:D]
    k, v = torch.zeros(n, D, dtype=BF), torch.zeros(n, D, dtype=BF)
    k[:, 0] = t.to(BF)
    a = p[j].to(BF)
    b = (p[j] - a.to(F64)).to(BF)
    d = torch.arange(len(j))
    v[j, d], v[0, d], v[1, d] = 1.0, -a, -b
    out = torch.zeros(D, dtype=F64)
    out[d] = (p[j] - a.to(F64) - b.to(F64)) / p.sum()
    # The weight of token j: two bf16 parts, each rounded to nearest, hold it to 2^-17.  Its
    # exponent (two roundings, at most 3 in size), the exponential (4 U) and the factors that join a
    # part's maximum with the call's (two more exponentials): 32 U.  The sums: 16 U.
    bound = torch.zeros(D, dtype=F64)
    bound[d] = (2.0 ** -17 + 48 * U) * p[j] / p.sum()
    return k, v, out, bound


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,n,prefix", [(1, 200, 0), (1, 3000, 0), (20, 4133, 4096), (3, 4133, 4096)])
def test_attn_probabilities(B, n, prefix, D):
    """A short sequence (one launch), a long one in parts, a shared prefix with enough rows for the
    32-row tiles and with few."""
    page = 64
    k, v, want, bound = _fine_probabilities(n, D, n)
    pages = -(-n // page)
    kc, vc = torch.zeros(pages, 1, page, D, dtype=BF), torch.zeros(pages, 1, D, page, dtype=BF)
    at = torch.arange(n)
    kc[at // page, 0, at % page], vc[at // page, 0, :, at % page] = k, v
    cache = fm.KVCache(kc.cuda(), vc.cuda(), 1)
    q = torch.zeros(B, D, dtype=BF)
    q[:, 0] = 1
    table = torch.arange(pages, dtype=torch.int32).expand(B, pages).contiguous()
    out = torch.empty(B, D, dtype=BF, device="cuda")
    fm.attn_decode(cache, fm.AttnDecode(1.0), q.cuda(), table.cuda(), torch.full((B,), n, dtype=torch.int32).cuda(), prefix, out,
                   fm.attn_decode_workspace(cache, B))
    over = (out.cpu().to(F64) - want).abs() - bound - 2.0 ** -8 * want.abs()
    assert (over <= 0).all(), "over the bound in %d of %d, by %g of it" % ((over > 0).sum(), over.numel(), (over / bound).max())
