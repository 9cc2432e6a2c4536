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
