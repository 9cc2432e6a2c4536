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


# ---- linear ------------------------------------------------------------------------------
def _outliers(g, T, K):
    """Activations of size 1 with some of several thousand, all of one sign in the last token."""
    x = torch.randn(T, K, generator=g)
    x = torch.where(torch.rand(T, K, generator=g) < 0.02, x * 3000, x)
    x[-1] = x[-1].abs() + 1
    return x.to(BF)


# both kernels, one and two row tiles to a workgroup or a wave, K split and whole
LINEAR = [(1, 640, 100), (3, 1152, 5000), (8, 640, 16400), (1, 1152, 33000), (20, 640, 33000), (16, 256, 17003), (40, 384, 65601),
          (64, 1280, 50), (33, 640, 6000)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear_zero_codes(T, K, N, group):
    """What meets a code of zero adds nothing: rows of zeros are zero, and a row of one code is the
    product itself (q x s has 20 bits: exact in fp32), whatever else is in x."""
    g = _gen(K + N)
    codes = torch.zeros(N, K // 2, dtype=torch.uint8)
    q = torch.randint(-8, 8, (N,), generator=g)
    q[::3] = 0
    col = torch.randint(0, K, (N,), generator=g)
    nib = ((q & 15) << (4 * (col % 2))).to(torch.uint8)
    codes[torch.arange(N), col // 2] = nib
    scales = ((torch.rand(N, K // group, generator=g) + 0.5) * 0.01).to(BF)
    x = _outliers(g, T, K)
    y = torch.full((T, N), 7.0, device="cuda")
    fm.linear_int4(fm.Int4Linear(codes.cuda(), scales.cuda()), x.cuda(), y)
    want = x.to(F64)[:, col] * (q.to(F64) * scales.to(F64)[torch.arange(N), col // group])
    assert torch.equal(y.cpu().to(F64), want), "off by %g" % (y.cpu().to(F64) - want).abs().max()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear_few_codes(T, K, N, group):
    """Mostly zero codes under outliers, within the bound of the products that are there."""
    g = _gen(K + N + 1)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    codes[torch.rand(N, K // 2, generator=g) < 0.95] = 0
    scales = ((torch.rand(N, K // group, generator=g) + 0.5) * 0.01).to(BF)
    x = _outliers(g, T, K)
    y = torch.full((T, N), 7.0, device="cuda")
    fm.linear_int4(fm.Int4Linear(codes.cuda(), scales.cuda()), x.cuda(), y)
    want, bound = ref.linear(codes, scales, x, bf16=False)
    over = (y.cpu().to(F64) - want).abs() - bound
    assert (over <= 0).all(), "over the bound by %g" % over.max()


def test_linear_infinity_signs():
    """An infinity times a code is an infinity of their sign, times a code of zero NaN."""
    K = 256
    codes = torch.zeros(3, K // 2, dtype=torch.uint8)
    codes[0, 5], codes[1, 5] = 0x03, 0x0d  # column 10: 3 and -3
    scales = torch.full((3, 2), 0.5, dtype=BF)
    x = torch.zeros(2, K, dtype=BF)
    x[1, 10] = math.inf
    y = torch.zeros(2, 3, device="cuda")
    fm.linear_int4(fm.Int4Linear(codes.cuda(), scales.cuda()), x.cuda(), y)
    y = y.cpu()
    assert (y[0] == 0).all() and y[1, 0] == math.inf and y[1, 1] == -math.inf and torch.isnan(y[1, 2])


# ---- log probabilities -------------------------------------------------------------------
def _logprob_bounds(x, lp):
    """Bounds of a row's log probabilities and entropy from the order of the sums: 256 lanes at
    least take a row, 16 bytes of a time and four such to a step.  A lane's sum has V / 256 terms
    (a rounding of the sum each, and of its own U t, 2^-22 of its exponential) and takes a factor
    at each step whose values are its largest yet (6 U); 128 U for the joins, the logarithm and what
    is left.  Nothing grows with a common offset of the logits: the sums and the results are
    formed against the same number."""
    V = x.shape[-1]
    steps = -(-V // (256 * 16))
    rel = (V / 256 + 6 * steps + 128) * U
    p = lp.exp()
    spread = (p * (x.amax(-1, keepdim=True) - x)).sum(-1)  # of the exponents that matter
    base = rel + 4 * U * spread
    h = -(p * lp.clamp(min=-1e6)).sum(-1)
    return base[:, None] + 4 * U * (lp.clamp(min=-1e6).abs() + 8), base * (4 + 2 * spread + 2 * h) + 32 * U


@pytest.mark.parametrize("T,V", [(1, 24576), (3, 20011), (600, 131072), (1, 200000), (40, 32001)])
@pytest.mark.parametrize("offset,peak", [(0.0, 30.0), (100.0, 20.0), (-1000.0, 20.0), (3000.0, 20.0)])
def test_logprobs_offsets(T, V, offset, peak):
    """Logits with a large common offset and one that dominates: one launch and rows in parts."""
    g = _gen(V)
    rows = min(T, 3)
    x = torch.randn(rows, V, generator=g) * 3
    x[:, V // 3] = peak
    x += offset
    _check_rows(x, T, V // 3)


@pytest.mark.parametrize("T,V", [(1, 24576), (600, 65536), (1, 200000)])
def test_logprobs_rising(T, V):
    """A lane that rises at every step beside lanes whose maximum comes first: a factor of one is one."""
    x = torch.randn(1, V, generator=_gen(1)) + 1000
    x[0, ::256] = 1000 + torch.arange(-(-V // 256)) * (12.0 / (V // 256))
    x[0, :4096] += 8
    _check_rows(x, T, 5)


def _check_rows(x, T, token):
    """The rows of x, repeated to T, against 64 bits."""
    rows, V = x.shape
    x64 = x.to(F64)
    lp = x64 - torch.logsumexp(x64, -1, keepdim=True)
    b_lp, b_h = _logprob_bounds(x64, lp)
    d = x.cuda()[torch.arange(T) % rows]
    got, h = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    ids, tops = torch.empty(T, 3, dtype=torch.int32, device="cuda"), torch.empty(T, 3, device="cuda")
    fm.token_logprobs(d, torch.full((T,), token, dtype=torch.int32, device="cuda"), got, h, ids, tops,
                      fm.token_logprobs_workspace(T, V, 3))
    for r in range(min(rows, T)):
        same = torch.arange(r, T, rows)
        ent = -(lp[r].exp() * lp[r]).sum()
        for v, want, bound, what in ((got, lp[r, token], b_lp[r, token], "logprob"), (h, ent, b_h[r], "entropy")):
            off = (v.cpu().to(F64)[same] - want).abs().max()
            assert off <= bound, "%s: off by %g, bound %g" % (what, off, bound)
        order = torch.sort(x[r], descending=True, stable=True).indices[:3]
        assert torch.equal(ids[r].cpu().long(), order)
        off = (tops[r].cpu().to(F64) - lp[r, order]).abs() - b_lp[r, order]
        assert (off <= 0).all(), "top: over the bound by %g" % off.max()
