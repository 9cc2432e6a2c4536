"""Decode attention over batches and lengths that take its paths as far as they go, against the plain
64-bit form (ops_ref.py) with the bounds derived there."""
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


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF)


def _run(q, k, v, table, lens, prefix, scale, window=0, sinks=None):
    B, Hq, D = q.shape
    cache = fm.KVCache(k.cuda(), v.cuda(), Hq)
    out = torch.full((B, Hq * D), math.nan, dtype=BF, device="cuda")
    fm.attn_decode(cache, fm.AttnDecode(scale, window, None if sinks is None else sinks.cuda()), q.reshape(B, -1).cuda(),
                   table.cuda(), lens.to(torch.int32).cuda(), prefix, out, fm.attn_decode_workspace(cache, B))
    return out.view(B, Hq, D).cpu()


def _within(got, want, bound):
    got = got.to(torch.float64)
    assert torch.isfinite(got).all()
    over = (got - want).abs() - bound
    assert (over <= 0).all(), "over the bound by %g" % over.max()


@pytest.mark.parametrize("n,prefix", [(100, 0), (3000, 0), (300, 256)])
def test_attn_infinite_sink(n, prefix):
    """A sink of +infinity takes everything, one launch, parts and a shared prefix; the heads beside it
    have theirs, and a NaN score stays a NaN."""
    B, Hq, Hkv, D, page = 3, 12, 2, 64, 32
    g = _gen(n)
    pages = -(-n // page)
    k, v = _randn(g, pages, Hkv, page, D), _randn(g, pages, Hkv, D, page)
    q = _randn(g, B, Hq, D)
    table = torch.arange(pages, dtype=torch.int32).expand(B, pages).contiguous()
    lens = torch.full((B,), n)
    sinks = torch.randn(Hq, generator=g)
    want, bound = ref.attn(q, k, v, table, lens, 0.125, 0, sinks)
    sinks[1], sinks[7] = math.inf, 3e38
    want[:, [1, 7]], bound[:, [1, 7]] = 0, 0
    _within(_run(q, k, v, table, lens, prefix, 0.125, 0, sinks), want, bound)
    q[:, 1, 0] = math.nan
    out = _run(q, k, v, table, lens, prefix, 0.125, 0, sinks)
    assert torch.isnan(out[:, 1]).all() and (out[:, 7] == 0).all() and torch.isfinite(out[:, 2:]).all()


@pytest.mark.parametrize("D,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("window", [0, 650])
@pytest.mark.parametrize("B,Hq,Hkv,first", [(5, 16, 2, 3), (3, 4, 1, 2), (90, 8, 2, 77), (70, 1, 1, 64), (6, 8, 1, 6)])
def test_attn_prefix_first_rows(B, Hq, Hkv, first, window, D, page):
    """The rows ahead of the first sequence that takes part name other pages or none: empty places of
    a batch, sequences shorter than the prefix, windows that have left it.  `first` == B: all."""
    prefix = 512
    g = _gen(B + D)
    lens = [prefix + (13 * b) % 100 for b in range(B)]
    for b in range(first):
        lens[b] = (0, 40, prefix - 1, 700 if window else 300)[b % 4]
    width = -(-800 // page)
    pages = prefix // page + B * width
    k, v = _randn(g, pages, Hkv, page, D), _randn(g, pages, Hkv, D, page)
    q = _randn(g, B, Hq, D, std=2.0)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = order[prefix // page:].view(B, width).clone()
    table[first:, :prefix // page] = order[:prefix // page]
    table[0] = -1  # nothing there at all
    n = torch.tensor(lens)
    want, bound = ref.attn(q, k, v, table, n, 0.1, window)
    _within(_run(q, k, v, table, n, prefix, 0.1, window), want, bound)


def _repeated_pages(q, k, v, shared, table, lens, prefix, scale):
    """The 64-bit form where the prefix repeats a few pages many times: a page that is there c times
    has c times the weight.  shared: the prefix's pages (negative: masked).  Returns (out, bound)."""
    B, Hq, D = q.shape
    P, Hkv, page, _ = k.shape
    G = Hq // Hkv
    F64 = torch.float64
    times = torch.bincount(shared[shared >= 0].long(), minlength=P).to(F64).repeat_interleave(page)
    kk = k.transpose(0, 1).reshape(Hkv, P * page, D).to(F64)
    vv = v.permute(1, 0, 3, 2).reshape(Hkv, P * page, D).to(F64)
    qq = q.view(B, Hkv, G, D).to(F64)
    out, bound = torch.zeros(B, Hkv, G, D, dtype=F64), torch.zeros(B, Hkv, G, D, dtype=F64)
    # Sums: 64 tokens a stage, at most 70 stages an item, 256 items a row, 128 parts of own tokens.
    depth = (64 * 70 + 256 + 128 + 64) * 2.0 ** -24
    U = 2.0 ** -24
    for b in range(B):
        j = torch.arange(prefix, int(lens[b]))
        own = table[b, j // page].long() * page + j % page
        weight = times + torch.bincount(own, minlength=P * page)
        s = qq[b] @ kk.transpose(1, 2) * scale
        mag = (qq[b].abs() @ kk.abs().transpose(1, 2) * abs(scale)).amax(-1, keepdim=True)
        m = torch.where(weight > 0, s, torch.full_like(s, -math.inf)).amax(-1, keepdim=True)
        p = weight * torch.exp(torch.where(weight > 0, s - m, torch.zeros_like(s)))
        l = p.sum(-1, keepdim=True)
        out[b], w = p @ vv / l, p @ vv.abs() / l
        # scores, their exponents (at most 100 below the maximum count), exponentials; the weights in
        # two bf16 parts; sums; the result rounded once
        d = (D + 8) * U * mag + 400 * U + 2.0 ** -22
        bound[b] = (2 * d + 2.0 ** -17 + depth) * w + 2.0 ** -8 * out[b].abs()
    return out.view(B, Hq, D), bound.view(B, Hq, D)


# (stages of 64 tokens to an item)
DEEP = [(32, 32, 4, 128, 64, 32832),    # 17: odd, items that start at either slot
        (32, 32, 4, 128, 16, 32832),
        (32, 32, 4, 128, 128, 32896),   # 17, from the middle of a page
        (9, 32, 4, 64, 64, 24576),      # 3, rows of one workgroup that are not all there
        (8, 32, 4, 128, 32, 24576),     # 3
        (32, 32, 4, 64, 32, 70400),     # 18, two workgroups to a CU with 128 rows each
        (256, 32, 1, 64, 16, 32832),    # 65: the page list is filled again
        (256, 32, 1, 128, 128, 32896),  # 65
        (2, 16, 1, 64, 64, 1049600)]    # 65 for the join's sake


@pytest.mark.parametrize("order", ["mixed", "rising", "holes"])
@pytest.mark.parametrize("B,Hq,Hkv,D,page,prefix", DEEP)
def test_attn_prefix_deep(B, Hq, Hkv, D, page, prefix, order):
    """Items of many stages: every slot used again and again, sums carried and rescaled, lists filled
    again.  rising: later pages have larger scores; holes: masked pages, one of them in the last
    quarter alone for the first half's items to run unmasked."""
    print("deep", B, Hq, Hkv, D, page, prefix, order, flush=True)
    g = _gen(prefix + B)
    P, tail = 640 // page + 3, 200
    k, v = _randn(g, P, Hkv, page, D), _randn(g, P, Hkv, D, page)
    q = _randn(g, B, Hq, D, std=2.0)
    shared = torch.randint(0, P, (prefix // page,), generator=g, dtype=torch.int32)
    if order == "rising":
        shared = shared.sort().values
        k = (k.float() * torch.linspace(0.1, 2.0, P).view(P, 1, 1, 1)).to(BF)
    if order == "holes":
        shared[7 * len(shared) // 8] = -1
        shared[3 * len(shared) // 4:][torch.rand(len(shared) - 3 * len(shared) // 4, generator=g) < 0.02] = 2 ** 30
    table = torch.randint(0, P, (B, prefix // page + -(-tail // page)), generator=g, dtype=torch.int32)
    table[:, :len(shared)] = shared
    lens = prefix + torch.randint(0, tail + 1, (B,), generator=g)
    shared = torch.where(shared < P, shared, torch.full_like(shared, -1))
    scale = D ** -0.5
    want, bound = _repeated_pages(q, k, v, shared, table, lens, prefix, scale)
    _within(_run(q, k, v, table, lens, prefix, scale), want, bound)


def test_attn_many_sequences_shared():
    """As many sequences as a call takes, one query row each, a prefix of a few pages."""
    B, page, prefix = 1024, 16, 256
    g = _gen(3)
    k, v = _randn(g, 60, 1, page, 64), _randn(g, 60, 1, 64, page)
    q = _randn(g, B, 1, 64, std=2.0)
    table = torch.randint(0, 60, (B, 20), generator=g, dtype=torch.int32)
    table[:, :16] = table[0, :16]
    n = prefix + torch.arange(B) % 40
    want, bound = ref.attn(q, k, v, table, n, 0.125)
    _within(_run(q, k, v, table, n, prefix, 0.125), want, bound)
