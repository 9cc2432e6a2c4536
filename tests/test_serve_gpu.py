"""GPU tests of the operators of include/flint_serve.h against their plain 64-bit forms (serve_ref.py),
with the bounds derived there, at the sizes, strides and masks where such kernels go wrong."""
import math
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(__file__))

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import ops_ref  # noqa: E402
import serve_ref as ref  # noqa: E402
import sparse_moe_transformer_wave_amd as fm  # noqa: E402

BF, U8, I32, I64, F32, F64 = torch.bfloat16, torch.uint8, torch.int32, torch.int64, torch.float32, torch.float64
INF, NAN = math.inf, math.nan


def _say(*a):
    print(*a, flush=True)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _close(got, want, bound, what):
    got = got.detach().cpu().to(F64)
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    assert (over <= 0).all(), "%s: over its bound by %g" % (what, over.max())


def _cache(pages, Hq, Hkv, D, page, g, gap=0, scales=(120, 134)):
    """Random codes of all kinds and scales; pages `gap` blocks apart."""
    block = fm.KV4Cache.page_bytes(Hkv, D, page)
    data = torch.randint(0, 256, (pages, block * (gap + 1)), generator=g, dtype=U8).cuda()
    c = fm.KV4Cache(data[:, gap * block:], Hq, Hkv, D, page)
    for s in (c.k_scales, c.v_scales):
        s.copy_(torch.randint(*scales, s.shape, generator=g, dtype=U8))
    return c


def _values(c):
    """Keys [page][head][token][D] and values [page][head][D][token], in 64 bits."""
    k = ref.values(c.k_codes.cpu(), c.k_scales.cpu())
    return k, ref.values(c.v_codes.cpu(), c.v_scales.cpu()).transpose(-1, -2).contiguous()


# ---- append ------------------------------------------------------------------------------
def _append(T, Hq, Hkv, D, page, rot, pairs, norm, slots, n_pages, positions=None, seed=0, gap=0, qkv=None, in_place=False,
            outs=True):
    g = _gen(seed)
    W = (Hq + 2 * Hkv) * D
    qkv = _randn(g, T, W) if qkv is None else qkv
    max_pos = 300
    positions = (torch.randint(0, max_pos, (T,), generator=g) if positions is None else positions).to(I32)
    ang = torch.rand(max_pos, rot // 2, generator=g) * 6.3
    cos, sin = ang.cos(), ang.sin()
    qn, kn = (_randn(g, D, std=0.2) + 1, _randn(g, D, std=0.2) + 1) if norm else (None, None)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    tr = fm.QKTransform(cu(qn), cu(kn), 1e-6, cu(cos) if rot else None, cu(sin) if rot else None, pairs)
    c = _cache(n_pages, Hq, Hkv, D, page, g, gap)
    before = c.data.cpu().clone()
    slots = torch.as_tensor(slots, dtype=I64)
    dq = qkv.cuda()
    q = dq[:, :Hq * D] if in_place else torch.full((T, Hq * D), 7.0, dtype=BF, device="cuda")
    k, v = (torch.full((T, Hkv * D + 8), 7.0, dtype=BF, device="cuda") for _ in range(2))
    fm.kv4_append(c, tr, dq, positions.cuda() if rot else None, slots.cuda(), q, k[:, :Hkv * D] if outs else None,
                  v[:, :Hkv * D] if outs else None)
    # the oracle
    x = qkv.view(T, Hq + 2 * Hkv, D)
    ok = (positions >= 0) & (positions < max_pos) if rot else torch.ones(T, dtype=torch.bool)
    at = positions.long().clamp(0, max_pos - 1)
    cs, sn = (cos[at][:, None], sin[at][:, None]) if rot else (None, None)
    wq, bq = ops_ref.transform(x[:, :Hq], qn, 1e-6, cs, sn, pairs)
    kk, _ = ops_ref.transform(x[:, Hq:Hq + Hkv], kn, float(torch.tensor(1e-6)), cs, sn, pairs)
    want_q = torch.where(ok[:, None, None], wq, torch.zeros_like(wq))
    _close(q.reshape(T, Hq, D), want_q, bq, "q")
    want = before.clone()
    w = fm.KV4Cache(want.cuda(), Hq, Hkv, D, page)
    for kind, vals, out, codes, scales in (("k", kk, k, w.k_codes, w.k_scales), ("v", x[:, Hq + Hkv:], v, w.v_codes, w.v_scales)):
        qc, qs, qv = ref.quantise(vals)
        packed = (qc[..., 0::2] | qc[..., 1::2] << 4).cuda()
        for t, s in enumerate(slots.tolist()):
            if ok[t] and 0 <= s < n_pages * page:
                codes[s // page, :, s % page] = packed[t]
                scales[s // page, :, :, s % page] = qs[t].cuda()
        if outs:
            qv = torch.where(ok[:, None, None], qv, torch.zeros_like(qv)).reshape(T, -1)
            assert torch.equal(out[:, :Hkv * D].cpu().to(F64).nan_to_num(12345.0), qv.nan_to_num(12345.0)), kind
        assert (out[:, Hkv * D if outs else 0:] == 7).all()
    assert torch.equal(c.data, w.data), "the cache"
    return c


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,page,rot,norm", [
    (1, 32, 4, 128, 64, 128, True), (7, 8, 1, 64, 16, 64, True), (3, 6, 2, 128, 32, 64, False), (9, 4, 4, 64, 128, 0, True),
    (33, 10, 2, 128, 16, 10, True), (5, 1, 1, 64, 16, 6, False), (2, 40, 8, 64, 64, 62, True), (18, 20, 4, 128, 16, 126, False),
    (4, 3, 3, 64, 32, 2, True), (300, 5, 5, 64, 16, 32, True)])
def test_append(T, Hq, Hkv, D, page, rot, norm, pairs):
    _say("append4", T, Hq, Hkv, D, page, rot, norm, pairs)
    g = _gen(T)
    n_pages = T // page + 5
    slots = torch.randperm(n_pages * page, generator=g)[:T]
    _append(T, Hq, Hkv, D, page, rot, pairs, norm, slots, n_pages)


def test_append_prompt_in_place_and_strided_pages():
    for page in (16, 64):
        order = torch.randperm(40, generator=_gen(1))
        at = 7 + torch.arange(200)
        _append(200, 4, 2, 64, page, 64, False, True, order[at // page] * page + at % page, 40, gap=2, in_place=True)
    _append(3, 4, 2, 128, 16, 0, False, False, [5, 40, 2], 4, outs=False)


def test_append_skips():
    """Slots outside the cache and positions outside the table."""
    pos = torch.tensor([0, -1, 300, 299, 5, 2 ** 31 - 1])
    _append(6, 4, 2, 64, 16, 32, False, True, [3, 4, 5, 6, -1, 7], 2, positions=pos)
    _append(5, 2, 1, 128, 16, 0, False, False, [32, -5, 2 ** 40, 31, -2 ** 63], 2)


def test_append_ties_zeros_and_extremes():
    """Values on the borders between codes, blocks of zeros, of the type's extremes and of non-finite values."""
    D, rows = 64, []
    for e in (-130, -126, -125, -20, 0, 3, 100, 124, 125):
        top = 2.0 ** e
        borders = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.0, 6.9375, 0.24902, 1.2578, 5.03125, 3.484375, 4.96875]
        rows.append([b * top if abs(b * top) < 3e38 else 3e38 for b in borders + [-b for b in borders]])
    rows.append([0.0] * 32)
    rows.append([-0.0] * 32)
    rows.append([0.0] * 31 + [7.03125])
    rows.append([0.0] * 31 + [-3.5])
    for bad in (INF, -INF, NAN):
        rows.append([1.0] * 15 + [bad] + [2.0] * 16)
    rows.append([3.38e38] * 32)
    rows.append([9.2e-41, -9.2e-41] * 16)
    if len(rows) % 2:
        rows.append([1.0] * 32)
    kv = torch.tensor(rows, dtype=F32).to(BF).view(-1, D)
    T = kv.shape[0]
    qkv = torch.cat([torch.ones(T, D, dtype=BF), kv, kv.flip(0)], 1)
    _append(T, 1, 1, D, 16, 0, False, False, torch.arange(T), 2, qkv=qkv)


@pytest.mark.parametrize("D,rot,pairs,norm", [(128, 128, False, True), (128, 64, True, True), (64, 0, False, True), (64, 20, False, True),
                                              (128, 128, False, False), (64, 6, True, True)])
def test_append_queries_are_those_of_the_bf16_cache(D, rot, pairs, norm):
    """Bit for bit, for few tokens and for many."""
    g = _gen(D + rot)
    Hq, Hkv, page, n = 12, 2, 16, 80
    angle = torch.rand(500, max(rot // 2, 1), generator=g) * 6.28
    w = [(_randn(g, D, std=0.3) + 1).cuda() if norm else None for _ in range(2)]
    tr = fm.QKTransform(*w, 1e-6, *((angle.cos().cuda(), angle.sin().cuda()) if rot else (None, None)), pairs=pairs)
    c4 = _cache(n, Hq, Hkv, D, page, g)
    c16 = fm.KVCache(torch.zeros(n, Hkv, page, D, dtype=BF, device="cuda"), torch.zeros(n, Hkv, D, page, dtype=BF, device="cuda"), Hq)
    for T in (1, 9, 1200):
        qkv = (_randn(g, T, (Hq + 2 * Hkv) * D).float() * torch.exp2(torch.randint(-9, 9, (T, 1), generator=g).float())).to(BF).cuda()
        pos, slots = torch.randint(0, 500, (T,), generator=g).to(I32).cuda(), torch.randperm(n * page, generator=g)[:T].cuda()
        q = [torch.zeros(T, Hq * D, dtype=BF, device="cuda") for _ in range(2)]
        fm.kv_append(c16, tr, qkv, pos if rot else None, slots, q[0])
        fm.kv4_append(c4, tr, qkv, pos if rot else None, slots, q[1])
        assert torch.equal(q[0].view(torch.int16), q[1].view(torch.int16)), T


def test_append_beyond_32_bits():
    """The last page of more than 2^32 bytes."""
    Hq, Hkv, D, page = 8, 8, 128, 128
    block = fm.KV4Cache.page_bytes(Hkv, D, page)
    n = 2 ** 32 // block + 3
    data = torch.zeros(n, block, dtype=U8, device="cuda")
    c = fm.KV4Cache(data, Hq, Hkv, D, page)
    g = _gen(3)
    qkv = _randn(g, 2, 3 * Hkv * D)
    q = torch.empty(2, Hq * D, dtype=BF, device="cuda")
    slots = torch.tensor([n * page - 1, (n - 1) * page])
    fm.kv4_append(c, fm.QKTransform(), qkv.cuda(), None, slots.cuda(), q)
    for i, (codes, scales) in enumerate(((c.k_codes, c.k_scales), (c.v_codes, c.v_scales))):
        qc, qs, _ = ref.quantise(qkv.view(2, 3 * Hkv, D)[:, (i + 1) * Hkv:(i + 2) * Hkv])
        for t, off in enumerate((page - 1, 0)):
            assert torch.equal(codes[-1, :, off].cpu(), qc[t, :, 0::2] | qc[t, :, 1::2] << 4)
            assert torch.equal(scales[-1, :, :, off].cpu(), qs[t])
    assert int(data[:-1].max()) == 0
    # and attention over it: one sequence of one page, the last
    kq = _randn(g, 1, Hq * D)
    out = torch.empty(1, Hq * D, dtype=BF, device="cuda")
    table, lens = torch.tensor([[n - 1]], dtype=I32), torch.tensor([page], dtype=I32)
    fm.kv4_attn_decode(c, fm.AttnDecode(0.1), kq.cuda(), table.cuda(), lens.cuda(), 0, out, fm.kv4_attn_decode_workspace(c, 1))
    one = fm.KV4Cache(data[-1:], Hq, Hkv, D, page)
    k, v = _values(one)
    want, bound = _oracle(kq.view(1, Hq, D), k, v, torch.zeros(1, 1, dtype=I32), lens, 0.1)
    _close(out.view(1, Hq, D), want, bound, "attention")


# ---- attention -----------------------------------------------------------------------------
def _oracle(q, k, v, table, lens, *args):
    """ops_ref.attn, and in its bound what an underflow leaves: against the largest, a probability or a
    part of one below 2^-126 vanishes, and so does the factor of a part of the tokens, whose sum is at
    most n 2^8 max |v| (a reference lags 8 behind at most): n 2^-116 max |v| in all."""
    want, bound = ops_ref.attn(q, k, v, table, lens, *args)
    n = torch.as_tensor(lens).to(F64).clamp(min=0).view(-1, 1, 1)
    return want, bound + torch.where(want != 0, n * 2.0 ** -116 * v.abs().nan_to_num(0).max(), torch.zeros_like(bound))


def _attn(lens, Hq, Hkv, D, page, window=0, sinks=False, prefix=0, seed=0, gap=0, holes=False, scale=None, std=1.0, stride=False,
          table=None, n_pages=None, tame=None):
    if tame is None:  # keys of all sizes, and scores of a few units
        for tame in (False, True):
            _attn(lens, Hq, Hkv, D, page, window, sinks, prefix, seed, gap, holes, scale, std, stride, table, n_pages, tame)
        return
    g = _gen(seed)
    B = len(lens)
    lens = torch.tensor(lens, dtype=I32)
    width = max(1, -(-max(int(lens.max()), 1) // page))
    shared = prefix // page
    n_pages = n_pages or B * width + 3
    c = _cache(n_pages, Hq, Hkv, D, page, g, gap)
    if tame:
        c.k_scales.copy_(torch.randint(124, 127, c.k_scales.shape, generator=g, dtype=U8))
    if table is None:
        order = torch.randperm(n_pages, generator=g, dtype=I32)
        table = order[:B * width].view(B, width).clone()
        if holes:
            bad = torch.rand(B, width, generator=g) < 0.3
            table = torch.where(bad, torch.tensor([-1, n_pages, 2 ** 31 - 1, -2 ** 31])[torch.randint(0, 4, (B, width), generator=g)].to(I32), table)
        table[:, :shared] = table[0, :shared]  # the same tokens: holes are shared too
    q = _randn(g, B, Hq * D, std=std)
    sk = _randn(g, Hq, dtype=F32, std=2.0) if sinks else None
    scale = D ** -0.5 if scale is None else scale
    if stride:
        dq = torch.full((B, Hq * D + 16), NAN, dtype=BF, device="cuda")
        dq[:, 8:-8] = q.cuda()
        dq, out = dq[:, 8:-8], torch.full((B, Hq * D + 8), 7.0, dtype=BF, device="cuda")
        res = out[:, 8:]
    else:
        dq, res = q.cuda(), torch.full((B, Hq * D), NAN, dtype=BF, device="cuda")
    ws = fm.kv4_attn_decode_workspace(c, B)
    ws.fill_(255)
    fm.kv4_attn_decode(c, fm.AttnDecode(scale, window, None if sk is None else sk.cuda()), dq, table.cuda(), lens.cuda(), prefix, res, ws)
    k, v = _values(c)
    want, bound = _oracle(q.view(B, Hq, D), k, v, table, lens, scale, window, sk)
    _close(res.reshape(B, Hq, D), want, bound, "out")
    if stride:
        assert (out[:, :8] == 7).all()


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (8, 1, 128), (6, 2, 64), (10, 2, 128), (4, 4, 128), (32, 4, 128), (40, 8, 64), (17, 1, 64),
                                      (64, 2, 128)])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attn_ragged(Hq, Hkv, D, page):
    _say("attn4", Hq, Hkv, D, page)
    _attn([0, 1, 15, 33, 64, 129, 300, 7], Hq, Hkv, D, page, sinks=page == 32)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 257, 700, 2049, 5000])
def test_attn_single(n):
    """One sequence, alone: one workgroup a head, and split over many."""
    for D in (64, 128):
        _say("single", n, D)
        _attn([n], 8, 2, D, 64, seed=n)
        _attn([n], 8, 2, D, 16, window=100, sinks=True, seed=n)


@pytest.mark.parametrize("window", [1, 31, 513])
def test_attn_window(window):
    _attn([0, 1, 40, 600, 1300], 12, 3, 64, 16, window=window, sinks=True)
    _attn([2000] * 3, 8, 1, 128, 64, window=window)


@pytest.mark.parametrize("B,Hq,Hkv,D,page,prefix", [
    (2, 8, 1, 128, 64, 1024), (5, 32, 4, 128, 64, 960), (33, 8, 2, 64, 16, 640), (9, 16, 1, 64, 128, 1408), (40, 8, 2, 128, 32, 512),
    (3, 64, 2, 128, 16, 4992)])
def test_attn_shared_prefix(B, Hq, Hkv, D, page, prefix):
    """Own suffixes of 1 token and more, a sequence that is shorter than the prefix, an empty one."""
    _say("prefix", B, Hq, Hkv, D, page, prefix)
    lens = [prefix + 1 + 37 * b % 211 for b in range(B)]
    if B > 3:
        lens[2], lens[3] = 0, prefix // 2
    _attn(lens, Hq, Hkv, D, page, prefix=prefix, sinks=True)
    _attn(lens, Hq, Hkv, D, page, prefix=prefix, window=prefix + 20, seed=1)


def test_attn_prefix_stages():
    """Prefix items of many stages, pages many times over in the table."""
    g = _gen(7)
    for B, Hkv, prefix, page in ((20, 1, 40000, 64), (6, 2, 9000, 16), (130, 1, 6400, 128)):
        prefix = prefix // page * page
        width, n_pages = prefix // page + 1, 61
        row = torch.randint(0, n_pages, (width,), generator=g, dtype=I32)
        table = row.expand(B, width).clone()
        _say("stages", B, prefix, page)
        _attn([prefix + 1 + b % page for b in range(B)], 8 * Hkv, Hkv, 64, page, prefix=prefix, table=table, n_pages=n_pages)


@pytest.mark.parametrize("B,Hq,Hkv,D,page,prefix", [(33, 8, 2, 128, 16, 64 * 15), (9, 16, 1, 64, 32, 64 * 7), (12, 16, 2, 128, 128, 128 * 5),
                                                    (40, 16, 1, 64, 64, 64 * 77), (5, 8, 1, 128, 64, 64 * 21)])
def test_attn_prefix_holes_of_many_rows(B, Hq, Hkv, D, page, prefix):
    """Missing pages in a prefix of 32 to 128 rows an item, and an odd number of stages: whole items
    masked, and items beside them that are not."""
    _say("prefix holes", B, Hq, Hkv, D, page, prefix)
    lens = [prefix + 1 + 29 * b % 150 for b in range(B)]
    _attn(lens, Hq, Hkv, D, page, prefix=prefix, holes=True, seed=B)
    g = _gen(B)
    width, n_pages = prefix // page + 150 // page + 2, 50
    table = torch.randint(0, n_pages, (B, width), generator=g, dtype=I32)
    table[:, :prefix // page] = table[0, :prefix // page]
    table[:, prefix // page // 2] = -1  # one
    _attn(lens, Hq, Hkv, D, page, prefix=prefix, sinks=True, table=table, n_pages=n_pages)


def test_attn_prefix_of_several_page_lists():
    """Items of more stages than the page list in LDS holds."""
    prefix, page, n_pages = 64 * 259, 64, 40
    g = _gen(3)
    row = torch.randint(0, n_pages, (prefix // page + 1,), generator=g, dtype=I32)
    for hole in (False, True):
        if hole:
            row[[5, 100, 200]] = n_pages
        _attn([prefix + 1 + b for b in range(17)], 64, 64, 64, page, prefix=prefix, table=row.expand(17, -1).clone(), n_pages=n_pages)


def test_attn_holes_strides_scales():
    _attn([100, 300, 64, 1], 8, 2, 128, 16, holes=True, seed=3)
    _attn([700, 700, 700, 650], 8, 2, 64, 32, holes=True, prefix=640, seed=4)
    _attn([100, 300], 6, 2, 64, 16, gap=1, stride=True)
    for scale in (-0.2, 0.0, 3.0):
        _attn([100, 333, 40], 8, 2, 64, 16, scale=scale, sinks=True)
        _attn([500, 500, 480], 24, 2, 128, 64, scale=scale, prefix=448)


def test_attn_all_holes():
    """Sequences whose pages are all missing see nothing, with a sink and without."""
    table = torch.full((3, 40), -1, dtype=I32)
    for prefix in (0, 512):
        _attn([600, 640, 1], 8, 2, 64, 16, table=table, n_pages=4, prefix=prefix)
        _attn([600, 640, 1], 32, 2, 64, 16, table=table, n_pages=4, prefix=prefix, sinks=True)


@pytest.mark.parametrize("prefix", [0, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_nan_blocks(D, prefix):
    """A NaN block that a query sees makes what it reaches NaN; unseen ones, in masked tokens, behind the
    end of a sequence or on pages of nobody, nothing."""
    Hq, Hkv, page = 16, 2, 16
    g = _gen(11)
    lens = torch.tensor([201, 190, 222, 0], dtype=I32)
    width = 14
    c = _cache(4 * width + 2, Hq, Hkv, D, page, g)
    table = torch.randperm(4 * width, generator=g, dtype=I32).view(4, width)
    table[:, :prefix // page] = table[0, :prefix // page]
    for b, n in enumerate(lens.tolist()):  # all behind the end
        for j in range(max(n, prefix), width * page):  # (the shared pages are seen by others)
            c.k_scales[table[b, j // page], :, :, j % page] = 255
            c.v_scales[table[b, j // page], :, :, j % page] = 255
    c.k_scales[-2:], c.v_scales[-2:] = 255, 255
    q = _randn(g, 4, Hq * D)
    run = lambda out: fm.kv4_attn_decode(c, fm.AttnDecode(D ** -0.5), q.cuda(), table.cuda(), lens.cuda(), prefix, out,  # noqa: E731
                                         fm.kv4_attn_decode_workspace(c, 4))
    out = torch.full((4, Hq * D), 7.0, dtype=BF, device="cuda")
    run(out)
    k, v = _values(c)
    want, bound = _oracle(q.view(4, Hq, D), k, v, table, lens, D ** -0.5)
    _close(out.view(4, Hq, D), want, bound, "out")
    clean = out.clone()
    # a value block of head 1 of sequence 0, channels 32 .. 63
    c.v_scales[table[0, 150 // page], 1, 1, 150 % page] = 255
    run(out)
    got = out.view(4, Hkv, Hq // Hkv, D).clone()
    assert torch.isnan(got[0, 1, :, 32:64]).all()
    got[0, 1, :, 32:64] = clean.view_as(got)[0, 1, :, 32:64]
    assert torch.equal(got, clean.view_as(got))
    # a key block of head 0 of sequence 2
    c.v_scales[table[0, 150 // page], 1, 1, 150 % page] = 127
    c.k_scales[table[2, 140 // page], 0, 0, 140 % page] = 255
    run(out)
    got = out.view(4, Hkv, Hq // Hkv, D)
    assert torch.isnan(got[2, 0]).all() and torch.isfinite(got[2, 1]).all() and torch.isfinite(got[[0, 1, 3]]).all()


def test_attn_extreme_scales():
    """Blocks at both ends of the range, and queries that make large scores."""
    _attn([90, 40], 8, 2, 64, 16, std=20.0)
    g = _gen(5)
    c = _cache(8, 4, 1, 64, 16, g)
    # sums before the division are in fp32: 100 tokens of up to 6 2^109 times 2^8 stay in range (of
    # 2^125 they would not, which the documentation says)
    c.k_scales.fill_(2), c.v_scales.fill_(236)
    q = _randn(g, 1, 256)
    lens, table = torch.tensor([100], dtype=I32), torch.arange(8, dtype=I32)[None]
    out = torch.empty(1, 256, dtype=BF, device="cuda")
    fm.kv4_attn_decode(c, fm.AttnDecode(1.0), q.cuda(), table.cuda(), lens.cuda(), 0, out, fm.kv4_attn_decode_workspace(c, 1))
    k, v = _values(c)
    want, bound = _oracle(q.view(1, 4, 64), k, v, table, lens, 1.0)
    _close(out.view(1, 4, 64), want, bound, "out")


# ---- pages ---------------------------------------------------------------------------------
def _pool(n_pages, page, layers, g, mixed=False):
    """Caches of small pages with random contents."""
    caches = []
    for i in range(layers):
        if i % 2 and mixed:
            bits = lambda *s: torch.randint(-2 ** 15, 2 ** 15, s, generator=g, dtype=torch.int16).cuda()  # noqa: E731
            caches.append(fm.KVCache(bits(n_pages, 1, page, 64), bits(n_pages, 1, 64, page), 1))
        else:
            block = fm.KV4Cache.page_bytes(1, 64, page)
            data = torch.randint(0, 256, (n_pages, 2 * block), generator=g, dtype=U8).cuda()
            caches.append(fm.KV4Cache(data[:, block:] if i % 3 == 2 else data[:, :block], 1, 1, 64, page))
    return fm.KVPages(caches)


def _contents(pages):
    return [t.clone() for c in pages.caches for t in ((c.data,) if isinstance(c, fm.KV4Cache) else (c.k, c.v))]


def _dev(n_pages, s):
    """A state on the GPU from lists (free: the stack's entries)."""
    i = lambda v, *shape: torch.tensor(v, dtype=I32).view(*shape).cuda()  # noqa: E731
    rows = len(s["table"])
    width = len(s["table"][0]) if rows else s["width"]
    return fm.KVState(i(s["refs"], n_pages), i(s["free"] + [-7] * (n_pages - len(s["free"])), n_pages), i([len(s["free"])], 1),
                      i(s["table"], rows, width), i(s["lens"], rows))


def _blank(n_pages, rows, width):
    f = lambda *s: torch.full(s, 12345, dtype=I32, device="cuda")  # noqa: E731
    return fm.KVState(f(n_pages), f(n_pages), f(1), f(rows, width), f(rows))


def _same_state(got, want, n_pages):
    assert got.refs.tolist() == want["refs"]
    assert got.n_free.item() == len(want["free"])
    assert got.free_list.tolist() == want["free"] + [-1] * (n_pages - len(want["free"]))
    assert got.table.tolist() == want["table"]
    assert got.kv_len.tolist() == want["lens"]


def _advance(pages, s, parent, grow, lds):
    """One step on the GPU and on the lists; the new state of the lists."""
    n, R = pages.n_pages, len(parent)
    width = len(s["table"][0]) if s["table"] else s["width"]
    old, new = _dev(n, s), _blank(n, R, width)
    kept = [t.clone() for t in (old.refs, old.free_list, old.n_free, old.table, old.kv_len)]
    slots = torch.full((R, max(lds, 1)), 9, dtype=I64, device="cuda") if lds else None
    before = _contents(pages)
    ws = fm.kv_pages_workspace(pages, max(R, old.rows))
    ws.fill_(255)
    i32 = lambda v: torch.tensor(v, dtype=I32).cuda()  # noqa: E731
    fm.kv_advance(pages, old, new, i32(parent), i32(grow), slots, ws)
    want = ref.advance(pages.page_size, s, parent, grow, lds)
    _same_state(new, want, n)
    if lds:
        assert slots.tolist() == want["slots"]
    for now, was in zip(_contents(pages), before):
        for src, dst in want["copied"]:
            was[dst] = was[src]
        assert torch.equal(now, was)
    for a, b in zip(kept, (old.refs, old.free_list, old.n_free, old.table, old.kv_len)):
        assert torch.equal(a, b)
    return want


def _in_use(g, n_pages, page, rows, width, shares=0.5):
    """A pool in use: rows of random lengths that share whole pages (and sometimes the last) of rows ahead."""
    import random
    r = random.Random(int(torch.randint(0, 2 ** 30, (1,), generator=g)))
    order = list(range(n_pages))
    r.shuffle(order)
    table, lens = [], []
    for i in range(rows):
        n = r.randrange(0, min((width - 1) * page, len(order) * page // 2 + 1) + 1)
        used = -(-n // page)
        row = []
        if i and r.random() < shares:
            o = r.randrange(i)
            whole = min(lens[o] // page, used) if r.random() < 0.7 else used
            if whole == used and r.random() < 0.5:
                n, used = lens[o], -(-lens[o] // page)  # the whole of it, a partial last page too
                whole = used
            row = table[o][:min(whole, -(-lens[o] // page), used)]
        while len(row) < used and order:
            row.append(order.pop())
        n = min(n, len(row) * page)
        row = row[:-(-n // page)]
        table.append(row + [-1] * (width - len(row)))
        lens.append(n)
    refs = [0] * n_pages
    for row, n in zip(table, lens):
        for p in row[:-(-n // page)]:
            refs[p] += 1
    return dict(refs=refs, free=[p for p in order if refs[p] == 0], table=table, lens=lens)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("n_pages,page,rows,width", [(40, 16, 5, 6), (300, 32, 33, 12), (5000, 16, 70, 40), (70, 128, 300, 5)])
def test_advance(n_pages, page, rows, width, seed):
    """A chain of steps: forks, ends, new sequences, batches that grow and shrink, until pages run out."""
    import random
    _say("advance", n_pages, page, rows, width, seed)
    g, r = _gen(seed), random.Random(seed)
    pages = _pool(n_pages, page, 3, g, mixed=True)
    s = _in_use(g, n_pages, page, rows, width)
    for step in range(4):
        R = r.choice([rows, max(1, rows // 2), min(1024, rows + 3)])
        parent = [r.choice([r.randrange(-1, len(s["lens"])), r.randrange(0, min(3, len(s["lens"]))), i if i < len(s["lens"]) else -1])
                  for i in range(R)]
        if r.random() < 0.3:
            parent = [r.choice([-5, 10 ** 6, p]) for p in parent]
        top = r.choice([1, 1, 3, page + 1, 3 * page])
        grow = [r.choice([0, 1, r.randrange(-1, top + 1)]) for _ in range(R)]
        s = _advance(pages, s, parent, grow, r.choice([0, 1, top, top + 5]))


def test_advance_one_step_beam_and_out_of_pages():
    pages = _pool(6, 16, 1, _gen(0))
    s = dict(refs=[3, 3, 0, 0, 0, 0], free=[5, 4, 3, 2], table=[[0, 1, -1]] * 3, lens=[20, 20, 20])
    # three rows on one partial page, all grow: two copies, the last keeps it
    a = _advance(pages, s, [0, 1, 2], [1, 1, 1], 1)
    assert a["table"] == [[0, 2, -1], [0, 3, -1], [0, 1, -1]] and a["refs"] == [3, 1, 1, 1, 0, 0]
    # all beams continue the second: the others' pages return and are taken again
    _advance(pages, a, [1, 1, 1], [1, 1, 1], 1)
    # one page short: the second row may not grow, and the last may not write to the page that both hold
    b = _advance(pages, dict(s, refs=[3, 3, 1, 1, 1, 0], free=[5]), [0, 1, 2], [1, 1, 1], 2)
    assert b["lens"] == [21, 20, 20] and b["slots"][2] == [-1, -1]
    # growth beyond the table; and none at all
    c = _advance(pages, s, [0, 1, 2], [100, 28, 0], 30)
    assert c["lens"] == [20, 48, 20]
    # nobody goes on: everything is free
    d = _advance(pages, s, [-1, -1], [0, 0], 0)
    assert sorted(d["free"]) == list(range(6))
    # an empty batch, and a new one
    e = _advance(pages, s, [], [], 0)
    f = dict(e, width=3)
    assert sorted(e["free"]) == list(range(6))
    _advance(pages, dict(f, table=[], lens=[]), [-1, -1, 0], [17, 1, 0], 17)


def test_advance_strange_tables():
    """Entries that are no pages, lengths out of range, a page that the free list names too: nothing
    outside is touched."""
    pages = _pool(8, 16, 1, _gen(1))
    s = dict(refs=[1, 1, 0, 1, 0, 0, 0, 0], free=[7, 6, 5, 4, 2], table=[[0, -1, 1], [99, 3, -9], [-2 ** 31, 2 ** 31 - 1, 8]],
             lens=[48, 20, 10 ** 9])
    _advance(pages, s, [0, 1, 2], [0, 1, 0], 1)
    _advance(pages, dict(s, lens=[-5, 33, 40]), [0, 1, 2, 2], [2, 1, 1, 1], 1)
    _advance(pages, s, [2, -1, 0], [1, 5, 0], 6)


@pytest.mark.parametrize("rows", [1, 257, 1024])
def test_advance_many_rows_many_arrays(rows):
    """Every place of a batch, and more arrays than a launch's arguments hold."""
    g = _gen(rows)
    n_pages, page, width = 3000, 16, 3
    block = fm.KV4Cache.page_bytes(1, 64, page)
    data = torch.randint(0, 256, (n_pages, 140, block), generator=g, dtype=U8).cuda()
    pages = fm.KVPages([fm.KV4Cache(data[:, i], 1, 1, 64, page) for i in range(140)])
    s = dict(refs=[0] * n_pages, free=list(range(n_pages)), table=[[-1] * width] * rows, lens=[0] * rows)
    s = _advance(pages, s, [-1] * rows, [i % 40 for i in range(rows)], 40)
    s = _advance(pages, s, [i // 2 for i in range(rows)], [1] * rows, 1)
    _advance(pages, s, [rows - 1 - i for i in range(rows)], [i % 3 for i in range(rows)], 2)


def test_advance_of_needs_that_add_up_to_2_to_the_31_pages():
    """As many rows, entries and tokens as there may be: the rows' needs come to 2^31 pages, and none is served
    beyond the first, where that is a small one."""
    rows, width, page = 1024, 2 ** 21, 16
    pages = fm.KVPages([fm.KV4Cache(torch.zeros(64, fm.KV4Cache.page_bytes(1, 64, page), dtype=U8, device="cuda"), 1, 1, 64, page)])
    old, ws = fm.kv_state(64, 0, width), fm.kv_pages_workspace(pages, rows)
    new = fm.KVState(*(torch.full(s, 7, dtype=I32, device="cuda") for s in ((64,), (64,), (1,), (rows, width), (rows,))))
    parent, grow = torch.full((rows,), -1, dtype=I32, device="cuda"), torch.full((rows,), 2 ** 25, dtype=I32, device="cuda")
    slots = torch.zeros(rows, 40, dtype=I64, device="cuda")
    for first in (2 ** 25, 40):
        grow[0] = first
        took = 3 if first == 40 else 0
        _say("needs", first)
        fm.kv_advance(pages, old, new, parent, grow, slots, ws)
        assert new.n_free.item() == 64 - took
        assert new.refs.tolist() == [1] * took + [0] * (64 - took)
        assert new.free_list.tolist() == list(range(63, took - 1, -1)) + [-1] * took
        assert new.kv_len.tolist() == [40 if took else 0] + [0] * (rows - 1)
        assert new.table[0, :took].tolist() == list(range(took)) and (new.table[0, took:] == -1).all() and (new.table[1:] == -1).all()
        assert slots[0].tolist() == (list(range(40)) if took else [-1] * 40) and (slots[1:] == -1).all()


def _compact(pages, s):
    n, width = pages.n_pages, len(s["table"][0]) if s["table"] else s["width"]
    old, new = _dev(n, s), _blank(n, len(s["table"]), width)
    moved = torch.full((n,), 9, dtype=I32, device="cuda")
    before = _contents(pages)
    ws = fm.kv_pages_workspace(pages, max(1, old.rows))
    ws.fill_(255)
    fm.kv_compact(pages, old, new, moved, ws)
    want = ref.compact(pages.page_size, s)
    assert moved.tolist() == want["moved"]
    _same_state(new, want, n)
    for now, was in zip(_contents(pages), before):
        w = was.clone()
        for p, to in enumerate(want["moved"]):
            if to >= 0:
                w[to] = was[p]
        assert torch.equal(now, w)
    return want


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("n_pages,page,rows,width", [(40, 16, 5, 6), (300, 32, 33, 12), (9000, 16, 70, 40), (70, 128, 300, 5)])
def test_compact(n_pages, page, rows, width, seed):
    _say("compact", n_pages, page, rows, width, seed)
    g = _gen(seed)
    pages = _pool(n_pages, page, 3, g, mixed=True)
    s = _compact(pages, _in_use(g, n_pages, page, rows, width))
    t = _compact(pages, s)  # nothing is left to move
    assert t["moved"][:n_pages - len(s["free"])] == list(range(n_pages - len(s["free"])))


def test_compact_edges():
    pages = _pool(5, 16, 1, _gen(0))
    full = dict(refs=[1] * 5, free=[], table=[[0, 1, 2, 3, 4]], lens=[80])
    _compact(pages, full)
    _compact(pages, dict(refs=[0] * 5, free=[0, 1, 2, 3, 4], table=[[-1] * 5], lens=[0]))
    _compact(pages, dict(refs=[0, 0, 0, 0, 2], free=[0, 1, 2, 3], table=[[4, -1, 0, 99, -1]] * 2, lens=[16, 80]))
    _compact(pages, dict(refs=[0, 3, 0, 1, 0], free=[0, 2, 4], table=[], lens=[], width=2))
    _compact(pages, dict(refs=[-1, 1, 0, 0, 1], free=[2, 3], table=[[1, 4]], lens=[10 ** 9]))


def test_pages_of_ranges_beyond_4096_times_1024():
    """So many pages that a workgroup takes 16384 of them."""
    n, page = 2 ** 22 + 12345, 16
    block = fm.KV4Cache.page_bytes(1, 64, page)
    data = torch.zeros(1, block, dtype=U8, device="cuda")
    pages = fm.KVPages([fm.KV4Cache(data, 1, 1, 64, page)])
    pages.c.n_pages = pages.n_pages = n  # no arrays: the bookkeeping alone
    pages.c.n_arrays = 0
    rows, width = 4, 9
    old, new = fm.kv_state(n, rows, width), fm.kv_state(n, rows, width)
    live = [n - 1, n - 2, 3, 2 ** 22, 70000, 16384, 16383]
    old.refs[live] = 1
    old.table[0, :7] = torch.tensor(live, dtype=I32).cuda()
    old.kv_len[0] = 7 * page - 3
    free = torch.ones(n, dtype=torch.bool, device="cuda")
    free[live] = False
    old.free_list[:n - 7] = free.nonzero()[:, 0].to(I32)
    old.n_free.fill_(n - 7)
    ws = fm.kv_pages_workspace(pages, rows)
    moved = torch.empty(n, dtype=I32, device="cuda")
    fm.kv_compact(pages, old, new, moved, ws)
    order = sorted(live)  # 3 stays; the others take 0, 1, 2, 4, 5, 6 in order
    to = {p: d for p, d in zip([p for p in order if p >= 7], [0, 1, 2, 4, 5, 6])}
    assert new.table[0].tolist() == [to.get(p, p) for p in live] + [-1, -1]
    assert new.n_free.item() == n - 7 and new.refs[:7].tolist() == [1] * 7 and int(new.refs.sum()) == 7
    assert torch.equal(new.free_list[:n - 7], torch.arange(n - 1, 6, -1, dtype=I32, device="cuda"))
    assert {p: int(moved[p]) for p in live} == {p: to.get(p, p) for p in live} and int((moved >= 0).sum()) == 7
    # the row ends: its pages come back in ascending order, on top
    fm.kv_advance(pages, old, new, torch.full((rows,), -1, dtype=I32, device="cuda"), torch.zeros(rows, dtype=I32, device="cuda"), None, ws)
    assert new.n_free.item() == n and new.free_list[-7:].tolist() == order and int(new.refs.abs().sum()) == 0


@pytest.mark.parametrize("n", [262143, 262145, 2 ** 20 + 7])
def test_pages_of_middle_ranges(n):
    """The sizes where a workgroup's range of pages changes: the bookkeeping alone, against the lists."""
    page, rows, width = 16, 5, 1500
    g = _gen(n)
    pages = fm.KVPages([fm.KV4Cache(torch.zeros(1, fm.KV4Cache.page_bytes(1, 64, page), dtype=U8, device="cuda"), 1, 1, 64, page)])
    pages.c.n_pages = pages.n_pages = n
    pages.c.n_arrays = 0
    order = torch.randperm(n, generator=g).tolist()
    lens = [page * width, 7001, 0, 123 * page, 20000]
    table, refs, at = [], [0] * n, 0
    for m in lens:
        used = -(-m // page)
        row = order[at:at + used]
        at += used
        if row:  # pages at the borders of ranges, and some that rows share
            row[0] = [0, n - 1, 1024, 4095, 16384][len(table)]
        for p in set(row):
            refs[p] += row.count(p)
        table.append(row + [-1] * (width - used))
    s = dict(refs=refs, free=[p for p in order if refs[p] == 0], table=table, lens=lens)
    ws = fm.kv_pages_workspace(pages, 6)
    ws.fill_(255)
    old, new = _dev(n, s), _blank(n, rows, width)
    moved = torch.empty(n, dtype=I32, device="cuda")
    fm.kv_compact(pages, old, new, moved, ws)
    want = ref.compact(page, s)
    _same_state(new, want, n)
    assert moved.tolist() == want["moved"]
    parent, grow = [0, 1, 1, 4, -1, 3], [0, 5, 40, 1, 33, 0]
    new = _blank(n, 6, width)
    i32 = lambda v: torch.tensor(v, dtype=I32).cuda()  # noqa: E731
    slots = torch.empty(6, 40, dtype=I64, device="cuda")
    fm.kv_advance(pages, old, new, i32(parent), i32(grow), slots, ws)
    want = ref.advance(page, s, parent, grow, 40)
    _same_state(new, want, n)
    assert slots.tolist() == want["slots"]


# ---- adapters ------------------------------------------------------------------------------
def _lora(T, K, N, R, n, ids=None, ranks=None, scales=True, base=BF, out=BF, seed=0, stride=False, x=None, in_place=False):
    g = _gen(seed)
    ids = torch.randint(-1, n, (T,), generator=g) if ids is None else torch.as_tensor(ids)
    ids = ids.to(I32)
    a, b = _randn(g, n, R, K, std=K ** -0.5), _randn(g, n, N, R)
    x = _randn(g, T, K) if x is None else x
    sc = torch.randn(n, generator=g) if scales else None
    rk = None if ranks is None else torch.tensor(ranks, dtype=I32)
    bs = None if base is None else _randn(g, T, N, dtype=base)
    if rk is not None:  # what does not count may hold anything
        for i in range(n):
            r = min(max(int(rk[i]), 0), R)
            a[i, r:], b[i, :, r:] = NAN, INF
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    ad = fm.LoraAdapters(a.cuda(), b.cuda(), cu(rk), cu(sc))
    if stride:
        wide = torch.full((T, K + 16), NAN, dtype=BF, device="cuda")
        wide[:, 8:-8] = x.cuda()
        whole = torch.full((T, N + 5), 7.0, dtype=out, device="cuda")
        dx, y = wide[:, 8:-8], whole[:, 3:N + 3]
        db = None
        if bs is not None:
            db = torch.full((T, N + 1), NAN, dtype=base, device="cuda")
            db[:, 1:] = bs.cuda()
            db = db[:, 1:]
    else:
        dx, db, y = x.cuda(), cu(bs), torch.full((T, N), NAN, dtype=out, device="cuda")
    if in_place:
        y = db
    ws = fm.lora_workspace(ad, T)
    ws.fill_(255)
    fm.lora(ad, dx, ids.cuda(), db, y, ws)
    want, bound = ref.lora(x, ids, a, b, rk, sc, bs, bf16=out == BF)
    _close(y, want, bound, "y")
    if stride and not in_place:
        assert (whole[:, :3] == 7).all() and (whole[:, N + 3:] == 7).all()
    return y


@pytest.mark.parametrize("R", [8, 16, 24, 64, 128])
@pytest.mark.parametrize("T,K,N,n", [(1, 8, 1, 1), (1, 2048, 5120, 3), (3, 264, 17, 2), (16, 1000, 64, 5), (17, 96, 130, 40), (33, 2056, 65, 4),
                                     (64, 128, 1000, 64), (130, 512, 48, 7)])
def test_lora(T, K, N, R, n):
    _say("lora", T, K, N, R, n)
    _lora(T, K, N, R, n, base=F32)
    _lora(T, K, N, R, n, base=None, out=F32, scales=False, seed=1)


@pytest.mark.parametrize("base,out", [(BF, BF), (F32, F32), (BF, F32)])
def test_lora_types_strides_in_place(base, out):
    for T, N in ((5, 67), (40, 128)):
        _lora(T, 72, N, 16, 3, base=base, out=out, stride=True)
        if base == out:
            _lora(T, 72, N, 16, 3, base=base, out=out, in_place=True)
            _lora(T, 72, N, 16, 3, base=base, out=out, stride=True, in_place=True)


def test_lora_ids_and_ranks():
    """No adapter at all, ids outside, every order in a tile, ranks of 0 and out of range."""
    _lora(20, 64, 40, 16, 2, ids=[-1] * 20)
    _lora(20, 64, 40, 16, 2, ids=[5, -7, 2 ** 31 - 1, -2 ** 31] * 5)
    _lora(20, 64, 40, 16, 2, ids=[-1] * 20, base=None)
    _lora(48, 64, 40, 16, 16, ids=list(range(16)) + [3] * 16 + [i % 2 for i in range(16)])
    _lora(40, 136, 50, 32, 6, ranks=[0, 1, 7, 8, 31, 32])
    _lora(40, 136, 50, 64, 6, ranks=[33, 64, 99, -3, 40, 9], out=F32, base=F32)
    _lora(9, 4096, 33, 128, 4, ranks=[127, 100, 65, 3])


@pytest.mark.parametrize("T", [512, 2049, 4096, 4111])
def test_lora_prompts(T):
    """Runs of tokens with one adapter, and mixed ones, in tiles of 16 and of 64 tokens."""
    g = _gen(T)
    runs = torch.randint(-1, 5, (T // 50 + 1,), generator=g).repeat_interleave(50)[:T]
    _lora(T, 256, 96, 16, 5, ids=runs)
    _lora(T, 520, 33, 40, 40, seed=2, out=F32)


def test_lora_long_rows():
    _lora(2, 32768, 70, 16, 2)
    _lora(1, 64, 200003, 8, 1)


def test_lora_tokens_are_apart():
    """A token's infinities and NaN, or its adapter's, reach no other token; its result does not depend on
    the batch."""
    T, K, N = 20, 128, 50
    g = _gen(2)
    x = _randn(g, T, K)
    a, b = _randn(g, 3, 8, K, std=0.1), _randn(g, 3, N, 8)
    ids = torch.arange(T, dtype=I32) % 3
    b[2] = NAN
    x[4] = INF
    base = _randn(g, T, N, dtype=F32)
    ad = fm.LoraAdapters(a.cuda(), b.cuda())
    y = torch.empty(T, N, device="cuda")
    ws = fm.lora_workspace(ad, T)
    fm.lora(ad, x.cuda(), ids.cuda(), base.cuda(), y, ws)
    bad = (ids == 2) | (torch.arange(T) == 4)
    assert torch.isnan(y.cpu()[bad]).all()
    want, bound = ref.lora(x[~bad], ids[~bad], a, b, base=base[~bad], bf16=False)
    _close(y.cpu()[~bad], want, bound, "others")
    for t in (0, 7, 19):
        one = torch.empty(1, N, device="cuda")
        if not bad[t]:
            fm.lora(ad, x[t:t + 1].cuda(), ids[t:t + 1].cuda(), base[t:t + 1].cuda(), one, ws)
            _close(one, *[v[(~bad).nonzero()[:, 0].tolist().index(t)][None] for v in (want, bound)], "alone")


def test_lora_beyond_32_bits():
    """The last adapter of more than 2^32 bytes of weights, and rows of y far apart."""
    n, R, K, N = 70000, 8, 4096, 4096
    a = torch.zeros(n, R, K, dtype=BF, device="cuda")
    b = torch.zeros(n, N, R, dtype=BF, device="cuda")
    g = _gen(9)
    wa, wb, x = _randn(g, 1, R, K, std=0.02), _randn(g, 1, N, R), _randn(g, 3, K)
    a[-1], b[-1] = wa[0].cuda(), wb[0].cuda()
    ad = fm.LoraAdapters(a, b)
    y = torch.empty(3, N, device="cuda")
    fm.lora(ad, x.cuda(), torch.tensor([n - 1, 0, n - 1], dtype=I32).cuda(), None, y, fm.lora_workspace(ad, 3))
    want, bound = ref.lora(x, torch.tensor([0, 5, 0]), wa, wb, bf16=False)
    _close(y, want, bound, "y")


# ---- logits --------------------------------------------------------------------------------
def _rules(T, V, g, history=50, bias=5, masks=True, ld_extra=0):
    hist = torch.where(torch.rand(T, history, generator=g) < 0.4, torch.randint(0, min(4, V), (T, history), generator=g),
                       torch.randint(-2, V + 2, (T, history), generator=g)).to(I32)
    total = torch.randint(0, history + 1, (T,), generator=g).to(I32)
    total[0] = history
    prompt = (total * torch.rand(T, generator=g)).to(I32)
    n = torch.randint(0, bias + 1, (T,), generator=g)
    start = torch.cat([torch.zeros(1, dtype=I64), n.cumsum(0)]).to(I32)
    e = int(start[-1])
    r = dict(history=hist, prompt_len=prompt, total_len=total, repetition=0.5 + torch.rand(T, generator=g),
             presence=torch.randn(T, generator=g), frequency=torch.rand(T, generator=g),
             bias_start=start, bias_ids=torch.randint(-1, V + 1, (e,), generator=g).to(I32), bias=torch.randn(e, generator=g) * 5)
    if masks:
        r["masks"] = torch.randint(-2 ** 31, 2 ** 31, (3, -(-V // 32) + 1), generator=g).to(I32)
        r["mask_rows"] = torch.randint(-1, 4, (T,), generator=g).to(I32)
    return r


def _check_logits(x, rules, what, in_place=False, off=0, skew=0):
    """off: elements ahead of the rows; skew: more of them in out than in logits."""
    T, V = x.shape
    bf = x.dtype == BF
    wide = torch.full((T, V + 9 + off), NAN, dtype=x.dtype, device="cuda")
    src = wide[:, off:off + V]
    src.copy_(x)
    if in_place:
        whole, out, pos = wide, src, off
    else:
        whole = torch.full((T, V + 9 + off + skew), 7.0, dtype=x.dtype, device="cuda")
        pos = off + skew
        out = whole[:, pos:pos + V]
    cu = {k: v.cuda() for k, v in rules.items()}
    fm.logits_adjust(fm.LogitRules(**cu), src, out)
    want, bound = ref.logits(x, **rules, bf16=bf)
    got = out.cpu().to(F64)
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin].nan_to_num(5.0, 1e300, -1e300), want[~fin].nan_to_num(5.0, 1e300, -1e300)), what
    over = (got - want)[fin].abs() - bound[fin]
    assert (over <= 0).all(), "%s: over its bound by %g" % (what, over.max())
    edge = torch.cat([whole[:, :pos], whole[:, pos + V:]], 1)
    assert (torch.isnan(edge) if in_place else edge == 7).all(), what
    if not in_place:
        assert torch.equal(src.cpu().nan_to_num(5.0), x.nan_to_num(5.0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V", [(1, 1), (2, 7), (3, 33), (5, 1000), (4, 4099), (2, 20001), (1, 70003), (33, 300)])
def test_logits(T, V, dtype):
    for i, kw in enumerate((dict(), dict(masks=False), dict(bias=0), dict(history=3000, bias=200))):
        g = _gen(V + i)
        x = _randn(g, T, V, std=3.0, dtype=dtype)
        rules = _rules(T, V, g, **kw)
        for off, skew in ((0, 0), (3, 0), (1, 2)):
            _say("logits", T, V, dtype, kw, off, skew)
            _check_logits(x, rules, "apart", off=off, skew=skew)
        _check_logits(x, rules, "in place", in_place=True, off=i)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_logits_many_rows(dtype):
    """So many rows that a workgroup takes 16384 values."""
    g = _gen(3)
    for T, V in ((512, 1003), (190, 40001)):
        x = _randn(g, T, V, std=3.0, dtype=dtype)
        rules = _rules(T, V, g)
        _check_logits(x, rules, "apart", off=1)
        _check_logits(x, rules, "in place", in_place=True)


def test_logits_each_rule_alone():
    g = _gen(4)
    T, V = 3, 500
    x = _randn(g, T, V, std=3.0, dtype=F32)
    all_rules = _rules(T, V, g)
    groups = [dict(), dict(history=all_rules["history"])]
    groups += [{k: all_rules[k] for k in ("history", name)} for name in ("repetition", "presence", "frequency", "total_len", "prompt_len")]
    groups += [{k: all_rules[k] for k in ("bias_start", "bias_ids", "bias")}, dict(masks=all_rules["masks"]),
               {k: all_rules[k] for k in ("masks", "mask_rows")}, dict(masks=all_rules["masks"][:1])]
    for rules in groups:
        _say(sorted(rules))
        _check_logits(x, rules, str(sorted(rules)))
        _check_logits(x, rules, str(sorted(rules)), in_place=True)


def test_logits_special_values():
    """Infinities, NaN, the type's lowest value and zeros under every rule; a mask that leaves nothing; a
    token that is biased twice, said many times, listed in prompt and answer."""
    V = 64
    for dtype in (BF, F32):
        low = torch.finfo(dtype).min
        x = torch.tensor([INF, -INF, NAN, low, -low, 0.0, -0.0, 1.0] * 8).to(dtype).repeat(3, 1)
        h = torch.arange(8, dtype=I32).repeat(3, 1)
        rules = dict(history=h, prompt_len=torch.tensor([0, 8, 4], dtype=I32), repetition=torch.tensor([1.5, 0.5, 2.0]),
                     presence=torch.tensor([1.0, 1.0, 0.0]), frequency=torch.tensor([0.5, 0.5, 0.0]),
                     bias_start=torch.tensor([0, 3, 3, 4], dtype=I32), bias_ids=torch.tensor([9, 20, 9, 1], dtype=I32),
                     bias=torch.tensor([100.0, -INF, 3.0, 5.0]))
        _check_logits(x, rules, "special")
        rules["masks"] = torch.zeros(3, 2, dtype=I32)
        _check_logits(x, rules, "nothing left")
        _check_logits(x, rules, "nothing left", in_place=True)
    x = torch.zeros(1, V)
    hist = torch.full((1, 100000), 7, dtype=I32)
    _check_logits(x, dict(history=hist, frequency=torch.tensor([0.25])), "said many times")
    rules = dict(bias_start=torch.tensor([-5, 900], dtype=I32), bias_ids=torch.tensor([3] * 400, dtype=I32), bias=torch.arange(400.0))
    _check_logits(x, rules, "one token 400 times")


def test_logits_beyond_32_bits():
    """The last of rows that lie more than 2^32 bytes behind the first."""
    T, V = 4300, 1000
    buf = torch.zeros(T, 262144, dtype=F32, device="cuda")[:, :V]
    x = _randn(_gen(1), 1, V, dtype=F32)
    buf[-1] = x[0].cuda()
    mask = torch.zeros(T, 32, dtype=I32, device="cuda")
    mask[-1] = 0x55555555
    fm.logits_adjust(fm.LogitRules(masks=mask), buf, buf)
    want = x[0].clone()
    want[1::2] = -INF
    assert torch.equal(buf[-1].cpu(), want) and (buf[:-1] == -INF).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_logits_long_history_and_a_bias_for_every_token(dtype):
    """More entries than fit beside the counts of a long history.  The biases take all but 2^-9 of the
    penalised values away, so that those, rounded to bf16 before the biases are added, would be far off."""
    V, n = 131072, 16384
    g = _gen(8)
    x = _randn(g, 3, V, std=3.0, dtype=dtype)
    h = torch.randint(-1, V, (3, n), generator=g)
    h[:, :500] = torch.arange(500)
    h[0, 600:1100] = torch.arange(500)
    rules = dict(history=h.to(I32), prompt_len=torch.tensor([550, n, 0], dtype=I32), total_len=torch.tensor([n, n, 0], dtype=I32),
                 repetition=torch.tensor([1.3, 0.7, 2.0]), frequency=torch.tensor([0.013, 0.2, 0.5]),
                 presence=torch.tensor([0.0048828125, 0.3, 1.0]))
    y, _ = ref.logits(x, **rules, bf16=False)
    ids = [torch.randperm(V, generator=g), torch.randperm(V, generator=g)]
    rules["bias_start"] = torch.tensor([0, V, V, 2 * V], dtype=I32)
    rules["bias_ids"] = torch.cat(ids).to(I32)
    rules["bias"] = torch.cat([y[0][ids[0]], y[2][ids[1]]]).mul(2.0 ** -9 - 1).float()
    for kw in (dict(), dict(off=1, skew=2), dict(in_place=True)):
        _say(dtype, kw)
        _check_logits(x, rules, str(kw), **kw)
    rules["masks"] = torch.randint(-2 ** 31, 2 ** 31, (2, V // 32), generator=g).to(I32)
    rules["mask_rows"] = torch.tensor([1, -1, 0], dtype=I32)
    _check_logits(x, rules, "masked")
    _check_logits(x, rules, "masked, in place", in_place=True, off=3)


def test_logits_lists_of_2_to_the_31_less_one():
    """The longest history and list of biases that there may be, whose tokens are their first and last entries."""
    n = 2 ** 31 - 1
    x = _randn(_gen(2), 1, 40, std=3.0, dtype=F32)
    ids = torch.full((1, n), -1, dtype=I32, device="cuda")
    ids[0, 0] = 3
    ids[0, -4:] = torch.tensor([7, 8, 7, 9], dtype=I32)
    rules = dict(repetition=torch.tensor([1.25]), frequency=torch.tensor([0.25]), presence=torch.tensor([0.5]))
    prompt = torch.tensor([n - 3], dtype=I32)
    short = dict(rules, history=torch.tensor([[3, 7, 8, 7, 9]], dtype=I32), prompt_len=torch.tensor([2], dtype=I32))
    out = torch.zeros(1, 40, device="cuda")
    cu = {k: v.cuda() for k, v in rules.items()}
    fm.logits_adjust(fm.LogitRules(history=ids, prompt_len=prompt.cuda(), **cu), x.cuda(), out)
    want, bound = ref.logits(x, **short, bf16=False)
    _close(out, want, bound, "history")
    _say("history")
    bias = torch.zeros(n, device="cuda")
    bias[0] = 2.0
    bias[-4:] = torch.tensor([5.0, -3.0, 4.0, 1.5])
    fm.logits_adjust(fm.LogitRules(history=ids, prompt_len=prompt.cuda(), bias_start=torch.tensor([0, n], dtype=I32).cuda(),
                                   bias_ids=ids.view(-1), bias=bias, **cu), x.cuda(), out)
    short.update(bias_start=torch.tensor([0, 5], dtype=I32), bias_ids=torch.tensor([3, 7, 8, 7, 9], dtype=I32),
                 bias=torch.tensor([2.0, 5.0, -3.0, 4.0, 1.5]))
    want, bound = ref.logits(x, **short, bf16=False)
    _close(out, want, bound, "biases")


def test_logits_repetition_is_a_division():
    """x / r rounded once, so bit for bit fp32's quotient: also where 1 / r is out of fp32's range or among
    its smallest numbers."""
    V = 5000
    r = torch.tensor([1.1, 1.3, 0.7, 3.0, 1.0, 2.0 ** -130, 1.7e38, 0.9999999, 1e-3])
    x = (_randn(_gen(6), 1, V, std=3.0, dtype=F32).abs() * 2.0 ** -10).repeat(len(r), 1)
    x[:, ::7] *= -1
    rules = fm.LogitRules(history=torch.arange(V, dtype=I32).repeat(len(r), 1).cuda(), repetition=r.cuda())
    out = torch.zeros(len(r), V, device="cuda")
    fm.logits_adjust(rules, x.cuda(), out)
    want = torch.where(x > 0, x / r[:, None], x * r[:, None])
    assert torch.isfinite(want).all() and torch.equal(out.cpu(), want)


# ---- streams and graphs ----------------------------------------------------------------------
def _all_ops(seed=0):
    """Every operator as (call, outputs, inputs that a program changes between steps)."""
    g = _gen(seed)
    made = []
    c = _cache(60, 16, 2, 128, 16, g)
    tr = fm.QKTransform((_randn(g, 128) + 1).cuda(), (_randn(g, 128) + 1).cuda())
    qkv, slots = _randn(g, 5, 20 * 128).cuda(), torch.randperm(900, generator=g)[:5].cuda()
    q, k, v = (torch.zeros(5, h * 128, dtype=BF, device="cuda") for h in (16, 2, 2))
    made.append((lambda s=None: fm.kv4_append(c, tr, qkv, None, slots, q, k, v, stream=s), [q, k, v, c.data], [qkv]))
    c2 = _cache(300, 16, 2, 128, 16, g)
    aq, out = _randn(g, 5, 16 * 128).cuda(), torch.zeros(5, 16 * 128, dtype=BF, device="cuda")
    table = torch.randperm(300, generator=g, dtype=I32)[:295].view(5, 59).cuda()
    table[:, :32] = table[0, :32]
    lens, ws = torch.tensor([900, 700, 944, 512, 0], dtype=I32).cuda(), fm.kv4_attn_decode_workspace(c2, 5)
    at = fm.AttnDecode(0.1, 0, torch.randn(16, generator=g).cuda())
    made.append((lambda s=None: fm.kv4_attn_decode(c2, at, aq, table, lens, 512, out, ws, stream=s), [out], [aq]))
    pages = _pool(64, 16, 2, g, mixed=True)
    s = _in_use(g, 64, 16, 6, 8)
    old, new, other = _dev(64, s), _blank(64, 6, 8), _blank(64, 6, 8)
    parent, grow = torch.tensor([0, 0, 2, 2, -1, 5], dtype=I32).cuda(), torch.tensor([1, 1, 0, 3, 20, 1], dtype=I32).cuda()
    sl, pw, moved = torch.zeros(6, 20, dtype=I64, device="cuda"), fm.kv_pages_workspace(pages, 6), torch.zeros(64, dtype=I32, device="cuda")
    state = lambda t: [t.refs, t.free_list, t.n_free, t.table, t.kv_len]  # noqa: E731
    data = [t for x in pages.caches for t in ((x.data,) if isinstance(x, fm.KV4Cache) else (x.k, x.v))]
    made.append((lambda s=None: fm.kv_advance(pages, old, new, parent, grow, sl, pw, stream=s), state(new) + [sl], [parent]))
    cp, cw = _pool(64, 16, 2, g), fm.kv_pages_workspace(pages, 6)
    made.append((lambda s=None: fm.kv_compact(cp, old, other, moved, cw, stream=s), state(other) + [moved], [old.table]))
    del data
    ad = fm.LoraAdapters(_randn(g, 4, 16, 256).cuda(), _randn(g, 4, 100, 16).cuda())
    x, ids, y = _randn(g, 40, 256).cuda(), torch.randint(-1, 4, (40,), generator=g).to(I32).cuda(), torch.zeros(40, 100, device="cuda")
    lw = fm.lora_workspace(ad, 40)
    made.append((lambda s=None: fm.lora(ad, x, ids, None, y, lw, stream=s), [y], [x, ids]))
    lo = _randn(g, 6, 5000, dtype=F32).cuda()
    adj = torch.zeros_like(lo)
    rules = fm.LogitRules(**{k: v.cuda() for k, v in _rules(6, 5000, g).items()})
    made.append((lambda s=None: fm.logits_adjust(rules, lo, adj, stream=s), [adj], [lo]))
    return made


def _perturb(t, i):
    if t.dtype == I32:
        t.copy_(t.roll(i, 0))
    else:
        t.copy_(t.roll(i, -1))


def test_other_stream():
    """Calls on a stream of their own, behind work that is still running there."""
    made = _all_ops()
    want = []
    for call, outs, _ in made:
        call()
        want.append([o.clone() for o in outs])
    torch.cuda.synchronize()
    made = _all_ops()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        busy = torch.randn(2048, 2048, device="cuda")
        for _ in range(5):
            busy = busy @ busy
        for call, _, _ in made:
            call()
    st.synchronize()
    for (_, outs, _), w in zip(made, want):
        for a, b in zip(outs, w):
            assert torch.equal(a, b)


def test_graph_replays():
    """All operators captured into one graph, replayed with changed inputs and eager work between."""
    eager, made = _all_ops(), _all_ops()
    for call, _, _ in made:
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call, _, _ in made:
            call()
    for i in range(4):
        for (_, _, ei), (_, _, gi) in zip(eager, made):
            for a, b in zip(ei, gi):
                _perturb(a, i)
                _perturb(b, i)
        for call, _, _ in eager:
            call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, ((_, eo, _), (_, go, _)) in enumerate(zip(eager, made)):
            for a, b in zip(eo, go):
                assert torch.equal(a, b), (i, n)


def test_same_bits_twice():
    made = _all_ops(5)
    for call, outs, _ in made:
        call()
        first = [o.clone() for o in outs]
        for o in outs[:1]:
            pass
        call()
        for a, b in zip(first, outs):
            assert torch.equal(a.view(U8) if a.dtype == BF else a, b.view(U8) if b.dtype == BF else b)


def test_empty_batches():
    g = _gen(0)
    c = _cache(2, 4, 2, 64, 16, g)
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    fm.kv4_append(c, fm.QKTransform(), z(0, 512), None, z(0, dtype=I64), z(0, 256))
    ws = fm.kv4_attn_decode_workspace(c, 0)
    fm.kv4_attn_decode(c, fm.AttnDecode(1.0), z(0, 256), z(0, 3, dtype=I32), z(0, dtype=I32), 0, z(0, 256), ws)
    ad = fm.LoraAdapters(z(1, 8, 8), z(1, 4, 8))
    fm.lora(ad, z(0, 8), z(0, dtype=I32), None, z(0, 4), fm.lora_workspace(ad, 0))
    fm.logits_adjust(fm.LogitRules(), z(0, 9), z(0, 9))
    y = z(2, 9)
    fm.logits_adjust(fm.LogitRules(history=z(2, 0, dtype=I32)), y + 1, y)
    assert (y == 1).all()


def _poison(t):
    """Values that change every result: nobody's rows and pages, NaN."""
    t.fill_(-1 if t.dtype == I32 else NAN)


@pytest.mark.parametrize("explicit", [False, True])
def test_inputs_that_come_late_on_another_stream(explicit):
    """Inputs that are written on a stream, behind work that is still running there, and the calls behind
    them: on the current stream, or on one that is passed.  Nothing else waits for that stream."""
    made, want = _all_ops(3), []
    for call, outs, _ in made:
        start = [o.clone() for o in outs]
        call()
        want.append([o.clone() for o in outs])
        for o, a in zip(outs, start):
            o.copy_(a)
    real = [[t.clone() for t in ins] for _, _, ins in made]
    for (call, outs, ins), w in zip(made, want):  # the inputs matter: without them the outputs are others
        start = [o.clone() for o in outs]
        for t in ins:
            _poison(t)
        call()
        assert not all(torch.equal(o.view(U8), a.view(U8)) for o, a in zip(outs, w))
        for o, a in zip(outs, start):
            o.copy_(a)
    busy = torch.randn(4096, 4096, device="cuda") / 64
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(20):
            busy = busy @ busy
        for (_, _, ins), values in zip(made, real):
            for t, v in zip(ins, values):
                t.copy_(v)
        if not explicit:
            for call, _, _ in made:
                call()
    if explicit:
        for call, _, _ in made:
            call(st.cuda_stream)
    st.synchronize()
    for n, ((_, outs, _), w) in enumerate(zip(made, want)):
        for a, b in zip(outs, w):
            assert torch.equal(a.view(U8), b.view(U8)), n


def test_same_bits_into_cleared_outputs():
    for call, outs, _ in _all_ops(6):
        start = [o.clone() for o in outs]
        call()
        first = [o.clone() for o in outs]
        for o, a in zip(outs, start):
            if o.dtype == U8:
                o.copy_(a)  # a cache, of which a call writes its tokens
            else:
                o.view(U8).fill_(0xA5)
        call()
        for a, b in zip(first, outs):
            assert torch.equal(a.view(U8), b.view(U8))


def _page_ops(seed):
    """kv_advance and kv_compact as (call, everything they write, the pools' memory among it), and what
    the pages hold at first."""
    g = _gen(seed)
    n, page, rows, width = 90, 16, 7, 9
    s = _in_use(g, n, page, rows, width)
    ws, made = None, []
    for kind in ("advance", "compact"):
        pool = _pool(n, page, 2, g, mixed=True)
        ws = fm.kv_pages_workspace(pool, rows) if ws is None else ws
        old, new = _dev(n, s), _blank(n, rows, width)
        data = [t for x in pool.caches for t in ((x.data,) if isinstance(x, fm.KV4Cache) else (x.k, x.v))]
        outs = [new.refs, new.free_list, new.n_free, new.table, new.kv_len]
        if kind == "advance":
            parent, grow = torch.tensor([1, 0, 0, 0, 3, 5, 6], dtype=I32).cuda(), torch.tensor([1, 1, 1, 1, 2, 0, 20], dtype=I32).cuda()
            outs.append(torch.zeros(rows, 20, dtype=I64, device="cuda"))
            call = lambda p=pool, o=old, w=new, pa=parent, gr=grow, sl=outs[-1]: fm.kv_advance(p, o, w, pa, gr, sl, ws)  # noqa: E731
        else:
            outs.append(torch.zeros(n, dtype=I32, device="cuda"))
            call = lambda p=pool, o=old, w=new, m=outs[-1]: fm.kv_compact(p, o, w, m, ws)  # noqa: E731
        made.append((call, outs, data, [t.clone() for t in data]))
    return made


def _clear_pages(outs, data, start):
    for o in outs:
        o.view(U8).fill_(0xA5)
    for t, a in zip(data, start):
        t.copy_(a)


@pytest.mark.parametrize("seed", range(3))
def test_pages_hold_the_same_twice_and_replayed(seed):
    """Tables, and what the copied and moved pages hold: called twice, on another stream, and captured and
    replayed with eager work between; outputs and pages are cleared before each."""
    made = _page_ops(seed)
    want = []
    for call, outs, data, start in made:
        call()
        want.append([t.clone() for t in outs + data])
        assert any(not torch.equal(t, a) for t, a in zip(data, start)), "no page was copied"
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call, _, _, _ in made:
            call()

    def check(what):
        torch.cuda.synchronize()
        for (_, outs, data, start), w in zip(made, want):
            for a, b in zip(outs + data, w):
                assert torch.equal(a, b), what
            _clear_pages(outs, data, start)
        torch.cuda.synchronize()

    check("once")
    st = torch.cuda.Stream()
    for i in range(3):
        for call, _, _, _ in made:
            call()
        check("eager")
        graph.replay()
        check("replayed")
        with torch.cuda.stream(st):
            for call, _, _, _ in made:
                call()
        check("another stream")
