"""GPU tests of the decode-step operators (include/flint_ops.h) against their plain 64-bit
forms (ops_ref.py), with the bounds derived there, at the sizes, strides and masks where such
kernels go wrong."""
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
INF, NAN = math.inf, math.nan


def _say(*a):
    print(*a, flush=True)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _close(got, want, bound, what):
    got = got.detach().cpu().to(torch.float64)
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    assert (over <= 0).all(), "%s: over its bound by %g" % (what, over.max())


# ---- linear ------------------------------------------------------------------------------
def _linear_case(T, K, N, group, seed=0, std=1.0):
    g = _gen(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scales = ((torch.rand(N, K // group, generator=g) + 0.5) * 0.01).to(BF)
    return codes, scales, _randn(g, T, K, std=std)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,K,N", [(1, 128, 1), (1, 384, 15), (2, 2048, 17), (5, 640, 4097), (16, 2048, 48),
                                   (17, 1152, 33), (33, 256, 130), (64, 2176, 100), (3, 8320, 16), (64, 32768, 5),
                                   (1, 1024, 70001)])
def test_linear(T, K, N, group):
    _say("linear", T, K, N, group)
    codes, scales, x = _linear_case(T, K, N, group)
    w = fm.Int4Linear(codes.cuda(), scales.cuda())
    for dt in (torch.float32, BF):
        y = torch.full((T, N), NAN, dtype=dt, device="cuda")
        fm.linear_int4(w, x.cuda(), y)
        want, bound = ref.linear(codes, scales, x, bf16=dt == BF)
        _close(y, want, bound, "y")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,K,N", [(1, 384, 16385), (3, 1280, 17003), (8, 256, 20001), (16, 3200, 16400), (17, 1152, 33000),
                                   (40, 2560, 16399), (64, 384, 65601), (30, 256, 66000), (9, 2304, 5120), (50, 1408, 4200)])
def test_linear_many_rows(T, K, N, group):
    """Rows that are shared out over whole workgroups, K in several chunks, two row tiles to a wave."""
    codes, scales, x = _linear_case(T, K, N, group)
    w = fm.Int4Linear(codes.cuda(), scales.cuda())
    y = torch.full((T, N), 7.0, device="cuda")
    fm.linear_int4(w, x.cuda(), y)
    want, bound = ref.linear(codes, scales, x, bf16=False)
    _close(y, want, bound, "y")


@pytest.mark.parametrize("T,N", [(1, 513), (20, 64)])
def test_linear_strides_and_residual(T, N):
    """Slices of wider matrices, a residual, and the residual's own memory as y."""
    codes, scales, x = _linear_case(T, 512, N, 128, seed=3)
    g = _gen(4)
    wide = torch.full((T, 1024), NAN, dtype=BF)
    wide[:, 256:768] = x
    res = _randn(g, T, N + 3)
    dx, dr = wide.cuda()[:, 256:768], res.cuda()
    w = fm.Int4Linear(codes.cuda(), scales.cuda())
    want, bound = ref.linear(codes, scales, x, res[:, 1:N + 1])
    out = torch.full((T, N + 5), 7.0, dtype=BF, device="cuda")
    fm.linear_int4(w, dx, out[:, 2:N + 2], dr[:, 1:N + 1])
    _close(out[:, 2:N + 2], want, bound, "y")
    assert (out[:, :2] == 7).all() and (out[:, N + 2:] == 7).all()
    fm.linear_int4(w, dx, dr[:, 1:N + 1], dr[:, 1:N + 1])
    assert torch.equal(dr[:, 1:N + 1], out[:, 2:N + 2])
    assert torch.equal(dr[:, 0].cpu(), res[:, 0])


def test_linear_codes_and_infinities():
    """Every code at every nibble place, and a token's infinities and NaN stay in its row."""
    K, N = 256, 16
    codes = torch.empty(N, K // 2, dtype=torch.uint8)
    for n in range(N):
        codes[n] = n * 16 + (15 - n)
    scales = torch.full((N, K // 32), -0.5, dtype=BF)
    x = torch.zeros(4, K, dtype=BF)
    x[0, 37], x[1, 255], x[2, 0], x[3] = 2.0, INF, NAN, 1.0
    w = fm.Int4Linear(codes.cuda(), scales.cuda())
    y = torch.zeros(4, N, device="cuda")
    fm.linear_int4(w, x.cuda(), y)
    want = x.to(torch.float64) @ ref.int4_weights(codes, scales).t()
    y = y.cpu().to(torch.float64)
    assert torch.equal(y[0], want[0]) and torch.equal(y[3], want[3])
    assert not torch.isfinite(y[1]).any() and torch.isnan(y[2]).all()


def test_linear_beyond_32_bits():
    """The last rows of a matrix of more than 2^32 code bytes."""
    K, N = 32768, 262160
    g = _gen(5)
    codes, scales = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda"), torch.zeros(N, K // 128, dtype=BF, device="cuda")
    tail = torch.randint(0, 256, (20, K // 2), generator=g, dtype=torch.uint8)
    ts = (torch.rand(20, K // 128, generator=g) * 0.01).to(BF)
    codes[-20:], scales[-20:] = tail.cuda(), ts.cuda()
    x = _randn(g, 2, K)
    y = torch.full((2, N), NAN, device="cuda")
    fm.linear_int4(fm.Int4Linear(codes, scales), x.cuda(), y)
    want, bound = ref.linear(tail, ts, x, bf16=False)
    _close(y[:, -20:], want, bound, "tail")
    assert (y[:, :-20] == 0).all()


# ---- append ------------------------------------------------------------------------------
def _append(T, Hq, Hkv, D, page, rot, pairs, norm, slots, n_pages, positions=None, seed=0, in_place=False, stride_pages=False):
    g = _gen(seed)
    W = (Hq + 2 * Hkv) * D
    qkv = _randn(g, T, W)
    max_pos = 5000
    if positions is None:
        positions = torch.randint(0, max_pos, (T,), generator=g)
    positions = positions.to(torch.int32)
    ang = torch.rand(max_pos, rot // 2, generator=g) * 6.3
    cos, sin = ang.cos(), ang.sin()
    qn = _randn(g, D, std=0.2) + 1 if norm else None
    kn = _randn(g, D, std=0.2) + 1 if norm else None
    k0, v0 = _randn(g, n_pages, Hkv, page, D), _randn(g, n_pages, Hkv, D, page)
    if stride_pages:  # two layers' pages interleaved in one allocation
        kd = torch.zeros(n_pages, 2, Hkv, page, D, dtype=BF, device="cuda")[:, 1]
        vd = torch.zeros(n_pages, 2, Hkv, D, page, dtype=BF, device="cuda")[:, 1]
        kd.copy_(k0)
        vd.copy_(v0)
    else:
        kd, vd = k0.cuda(), v0.cuda()
    tr = fm.QKTransform(None if qn is None else qn.cuda(), None if kn is None else kn.cuda(), 1e-5,
                        cos.cuda() if rot else None, sin.cuda() if rot else None, pairs)
    cache = fm.KVCache(kd, vd, Hq)
    dq = qkv.cuda()
    if in_place:
        q = dq[:, :Hq * D]
    else:
        q = torch.full((T, Hq * D + 8), 7.0, dtype=BF, device="cuda")[:, :Hq * D]
    fm.kv_append(cache, tr, dq, positions.cuda() if rot else None, slots.cuda(), q)
    x = qkv.view(T, -1, D)
    ok = (positions >= 0) & (positions < max_pos) if rot else torch.ones(T, dtype=torch.bool)
    p = torch.where(ok, positions, torch.zeros_like(positions)).long()
    c, s = cos[p][:, None], sin[p][:, None]
    wq, bq = ref.transform(x[:, :Hq], qn, 1e-5, c, s, pairs)
    wk, bk = ref.transform(x[:, Hq:Hq + Hkv], kn, 1e-5, c, s, pairs)
    wq[~ok], bq[~ok] = 0, 0
    _close(q.view(T, Hq, D) if q.is_contiguous() else q.reshape(T, Hq, D), wq, bq, "q")
    wkc, bkc, wv = k0.to(torch.float64), torch.zeros(k0.shape, dtype=torch.float64), v0.clone()
    for t in range(T):
        sl = int(slots[t])
        if ok[t] and 0 <= sl < n_pages * page:
            wkc[sl // page, :, sl % page], bkc[sl // page, :, sl % page] = wk[t], bk[t]
            wv[sl // page, :, :, sl % page] = x[t, Hq + Hkv:]
    _close(kd, wkc, bkc, "k")
    assert torch.equal(vd.cpu(), wv), "v"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,page,rot,pairs,norm", [
    (32, 4, 64, 64, False, True), (32, 4, 16, 64, True, True), (3, 3, 32, 2, False, False), (5, 1, 128, 6, True, True),
    (8, 8, 16, 0, False, True), (2, 1, 64, 20, False, True), (12, 2, 32, 32, False, False)])
@pytest.mark.parametrize("T", [1, 7])
def test_append_decode(T, Hq, Hkv, D, page, rot, pairs, norm):
    g = _gen(T)
    slots = torch.randperm(9 * page, generator=g)[:T].to(torch.int64)
    _say("append", T, Hq, Hkv, D, page, rot, pairs, norm)
    _append(T, Hq, Hkv, D, page, rot * D // 64, pairs, norm, slots, 9)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("T,start", [(64, 0), (200, 5), (129, 63), (65, 8), (73, 120)])
def test_append_prompt(T, start, page):
    """Consecutive tokens on shuffled pages from any place of one, across tiles and pages."""
    n_pages = (start + T) // page + 2
    order = torch.randperm(n_pages, generator=_gen(page))
    at = start + torch.arange(T)
    _append(T, 4, 2, 64, page, 64, False, True, order[at // page] * page + at % page, n_pages, at)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("T,start", [(513, 0), (700, 13), (1030, 8)])
def test_append_long_prompt(T, start, page):
    n_pages = (start + T) // page + 2
    order = torch.randperm(n_pages, generator=_gen(page))
    at = start + torch.arange(T)
    _append(T, 2, 2, 64, page, 64, False, True, order[at // page] * page + at % page, n_pages, at)


@pytest.mark.parametrize("T", [90, 600])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_append_runs(T, seed):
    """Runs of consecutive slots of every length from every place, pieces of 8 that are not aligned,
    tokens that are skipped between them."""
    g = _gen(seed)
    slots = []
    for block in torch.randperm(200, generator=g).tolist():  # 24 slots of their own each
        n, first = int(torch.randint(1, 18, (1,), generator=g)), int(torch.randint(0, 8, (1,), generator=g))
        slots += [24 * block + first + i for i in range(n)]
        if block % 5 == 0:
            slots.append(-1)
    slots = torch.tensor(slots[:T], dtype=torch.int64)
    assert len(slots) == T
    _append(T, 2, 1, 64, 32, 64, False, False, slots, 200 * 24 // 32, torch.arange(T) % 64)


def test_append_skips():
    """Slots of -1 and beyond the cache, positions outside the table, a hole in a run of slots."""
    T, page, n_pages = 90, 16, 8
    slots = torch.arange(T, dtype=torch.int64) + 3
    slots[5], slots[40], slots[41], slots[77] = -1, n_pages * page, 2 ** 40, -(2 ** 40)
    pos = torch.arange(T)
    pos[20], pos[21] = -1, 5000
    _append(T, 6, 2, 128, page, 128, False, True, slots, n_pages, pos)


def test_append_in_place_and_strided_pages():
    slots = torch.tensor([31, 4, 90], dtype=torch.int64)
    _append(3, 8, 2, 128, 32, 64, True, True, slots, 4, in_place=True, stride_pages=True)


# ---- attention -----------------------------------------------------------------------------
def _attn_case(B, Hq, Hkv, D, page, lens, prefix=0, seed=0, std=2.0, ldt=None, extra=2):
    g = _gen(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    shared = prefix // page
    ldt = ldt or max(max(need), shared, 1)
    n_pages = shared + sum(max(n - shared, 0) for n in need) + extra
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((B, ldt), -1, dtype=torch.int32)
    table[:, :shared] = order[:shared]
    at = shared
    for b, n in enumerate(need):
        own = max(n - shared, 0)
        table[b, shared:shared + own] = order[at:at + own]
        at += own
    k, v = _randn(g, n_pages, Hkv, page, D), _randn(g, n_pages, Hkv, D, page)
    return dict(q=_randn(g, B, Hq, D, std=std), k=k, v=v, table=table, lens=torch.tensor(lens, dtype=torch.int32))


def _attn_run(c, Hq, prefix, scale, window, sinks, out=None):
    k, v = c["k"].cuda(), c["v"].cuda()
    cache = fm.KVCache(k, v, Hq)
    B, _, D = c["q"].shape
    if out is None:
        out = torch.full((B, Hq * D), NAN, dtype=BF, device="cuda")
    ws = torch.full((fm.attn_decode_workspace_bytes(cache, B),), 0xff, dtype=torch.uint8, device="cuda")
    fm.attn_decode(cache, fm.AttnDecode(scale, window, None if sinks is None else sinks.cuda()), c["q"].cuda(),
                   c["table"].cuda(), c["lens"].cuda(), prefix, out, ws)
    return out


def _attn(B, Hq, Hkv, D, page, lens, prefix=0, window=0, sinks=False, seed=0, edit=None, **kw):
    _say("attn", B, Hq, Hkv, D, page, lens[:8], prefix, window, sinks)
    c = _attn_case(B, Hq, Hkv, D, page, lens, prefix, seed, **kw)
    if edit:
        edit(c)
    scale = D ** -0.5
    sk = _randn(_gen(seed + 1), Hq, dtype=torch.float32) if sinks else None
    out = _attn_run(c, Hq, prefix, scale, window, sk)
    want, bound = ref.attn(c["q"], c["k"], c["v"], c["table"], c["lens"], scale, window, sk)
    _close(out.view(B, Hq, D), want, bound, "out")
    return out, want


@pytest.mark.parametrize("D,page", [(128, 64), (64, 16), (128, 16), (64, 128)])
@pytest.mark.parametrize("Hq,Hkv", [(32, 4), (1, 1), (6, 2), (20, 1), (32, 1), (17, 1)])
def test_attn_lengths(D, page, Hq, Hkv):
    """Ragged lengths around tile and page edges, an empty sequence among them."""
    _attn(7, Hq, Hkv, D, page, [1, 0, 31, 32, 33, page + 1, 700], sinks=Hq == 32)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 513, 2050])
def test_attn_single(n):
    _attn(1, 8, 1, 128, 64, [n])


@pytest.mark.parametrize("window", [1, 5, 32, 33, 513])
@pytest.mark.parametrize("page", [16, 64])
def test_attn_window(window, page):
    _attn(5, 16, 2, 128, page, [1, 4, 33, 600, 1400], window=window, sinks=True)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,prefix", [(3, 8, 1, 256), (5, 12, 2, 1024), (40, 32, 4, 512), (33, 16, 2, 640), (2, 4, 4, 128)])
def test_attn_prefix(B, Hq, Hkv, prefix, page):
    """A shared prefix with suffixes from nothing to several tiles, at row counts that fill row
    tiles and that do not; the same result as the call that shares nothing."""
    lens = [prefix + (17 * b) % 150 for b in range(B)]
    c = _attn_case(B, Hq, Hkv, 128, page, lens, prefix)
    want, bound = ref.attn(c["q"], c["k"], c["v"], c["table"], c["lens"], 0.09)
    for p in (prefix, 0, prefix - 1):
        _close(_attn_run(c, Hq, p, 0.09, 0, None).view(B, Hq, 128), want, bound, "prefix %d" % p)


@pytest.mark.parametrize("D", [64, 128])
def test_attn_prefix_partly_shared(D):
    """Sequences shorter than the prefix (an empty one too) and windows that have left it do not
    take part; their table rows name the pages they use."""
    page, prefix = 32, 256
    c = _attn_case(6, 8, 2, D, page, [300, 100, 0, 256, 700, 290], prefix)
    for window in (0, 280):
        want, bound = ref.attn(c["q"], c["k"], c["v"], c["table"], c["lens"], 0.1, window)
        _close(_attn_run(c, 8, prefix, 0.1, window, None).view(6, 8, D), want, bound, "window %d" % window)


@pytest.mark.parametrize("prefix", [0, 128])
def test_attn_unseen_places(prefix):
    """NaN and infinities behind a sequence's end, before its window and in pages that a table
    entry out of range masks."""
    def edit(c):
        for b, n in enumerate(c["lens"].tolist()):
            page = int(c["table"][b, (n - 1) // 16])
            c["k"][page, :, (n - 1) % 16 + 1:] = NAN
            c["v"][page, :, :, (n - 1) % 16 + 1:] = INF
    _attn(3, 8, 2, 64, 16, [130, 145, 253], prefix=prefix, edit=edit)

    def before(c):
        edit(c)
        for b, n in enumerate(c["lens"].tolist()):
            for j in range(n - 40):
                c["k"][int(c["table"][b, j // 16]), :, j % 16] = -INF
                c["v"][int(c["table"][b, j // 16]), :, :, j % 16] = NAN
    if not prefix:
        _attn(3, 8, 2, 64, 16, [130, 145, 253], window=40, edit=before)

    def holes(c):
        c["table"][0, 3], c["table"][1, 8], c["table"][2, 9] = -1, 10 ** 6, -(2 ** 31)
    _attn(3, 8, 2, 64, 16, [130, 145, 253], prefix=0, edit=holes)


@pytest.mark.parametrize("D,page", [(128, 16), (64, 64), (128, 128)])
def test_attn_prefix_holes(D, page):
    """Table entries out of range inside the shared prefix, pages of NaN behind them, and all of
    the prefix masked for one head count that fills row tiles unevenly."""
    prefix, B, Hq = 768, 9, 8
    lens = [prefix + 5 * b for b in range(B)]
    for holes in ([1, 3], list(range(prefix // page))):
        c = _attn_case(B, Hq, 2, D, page, lens, prefix)
        c["k"][0], c["v"][0] = NAN, NAN  # what an entry out of range must not reach
        c["table"][c["table"] == 0] = -1
        for e in holes:
            c["table"][:, e] = -1 if e % 2 else 2 ** 30
        want, bound = ref.attn(c["q"], c["k"], c["v"], c["table"], c["lens"], 0.1)
        for p in (prefix, 0):
            _close(_attn_run(c, Hq, p, 0.1, 0, None).view(B, Hq, D), want, bound, "prefix %d" % p)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.7])
def test_attn_scales(scale):
    """A negative scale, none, and a large one, with and without a shared prefix."""
    c = _attn_case(4, 12, 2, 128, 64, [300, 257, 400, 256], 256)
    want, bound = ref.attn(c["q"], c["k"], c["v"], c["table"], c["lens"], scale)
    for p in (256, 0):
        _close(_attn_run(c, 12, p, scale, 0, None).view(4, 12, 128), want, bound, "prefix %d" % p)


def test_attn_prefix_visible_nan():
    """A NaN inside the shared prefix reaches the queries of its head, all of the batch."""
    c = _attn_case(5, 8, 2, 64, 16, [200 + b for b in range(5)], 192)
    c["v"][int(c["table"][0, 2]), 1, 7, 3] = NAN
    out = _attn_run(c, 8, 192, 0.125, 0, None).view(5, 8, 64).cpu()
    bad = torch.isnan(out)
    assert bad[:, 4:, 7].all() and bad.sum() == 5 * 4


def test_attn_masked_out_and_extremes():
    """No valid page at all gives zeros, with and without sinks; one large score takes all; an
    infinite sink takes everything; lengths below 0 and beyond the table are clamped."""
    def none(c):
        c["table"][:] = -1
    for sinks in (False, True):
        out, _ = _attn(2, 8, 2, 128, 64, [70, 3], sinks=sinks, edit=none)
        assert (out == 0).all()
    _attn(2, 8, 2, 128, 64, [500, 90], std=60.0)
    c = _attn_case(3, 4, 1, 64, 16, [50, 10, 20])
    c["lens"] = torch.tensor([1000, -5, 20], dtype=torch.int32)
    want, bound = ref.attn(c["q"], c["k"], c["v"], c["table"], c["lens"], 0.125)
    _close(_attn_run(c, 4, 0, 0.125, 0, None).view(3, 4, 64), want, bound, "clamped")
    sk = torch.tensor([INF, 0.0, -INF, 1e30])
    out = _attn_run(c, 4, 0, 0.125, 0, sk).view(3, 4, 64).cpu()
    want, bound = ref.attn(c["q"], c["k"], c["v"], c["table"], c["lens"], 0.125, 0, torch.tensor([0.0, 0.0, -INF, 1e30]))
    _close(out[:, 1:], want[:, 1:], bound[:, 1:], "sinks")
    assert (out[1] == 0).all()


def test_attn_visible_nan():
    """A NaN that a query sees reaches its own heads only."""
    c = _attn_case(2, 4, 2, 64, 16, [40, 40])
    c["k"][int(c["table"][0, 1]), 1, 3] = NAN
    out = _attn_run(c, 4, 0, 0.125, 0, None).view(2, 4, 64).cpu()
    assert torch.isnan(out[0, 2:]).all() and torch.isfinite(out[0, :2]).all() and torch.isfinite(out[1]).all()


def test_attn_long_and_many():
    _attn(1, 8, 1, 64, 128, [70001])
    _attn(300, 2, 1, 64, 16, [(37 * b) % 90 for b in range(300)])
    _attn(1024, 1, 1, 64, 16, [b % 40 for b in range(1024)], prefix=16 * 16 * 0)


def test_attn_strides():
    """Query and output rows inside wider ones, pages of two layers in one allocation."""
    B, Hq, Hkv, D, page = 3, 4, 2, 64, 32
    c = _attn_case(B, Hq, Hkv, D, page, [70, 5, 33])
    n_pages = c["k"].shape[0]
    kd = torch.zeros(n_pages, 3, Hkv, page, D, dtype=BF, device="cuda")[:, 2]
    vd = torch.zeros(n_pages, 3, Hkv, D, page, dtype=BF, device="cuda")[:, 2]
    kd.copy_(c["k"])
    vd.copy_(c["v"])
    cache = fm.KVCache(kd, vd, Hq)
    q = torch.full((B, Hq * D + 64), NAN, dtype=BF, device="cuda")
    q[:, 64:] = c["q"].view(B, -1).cuda()
    out = torch.full((B, Hq * D + 32), 7.0, dtype=BF, device="cuda")
    ws = fm.attn_decode_workspace(cache, 8)
    fm.attn_decode(cache, fm.AttnDecode(0.125), q[:, 64:], c["table"].cuda(), c["lens"].cuda(), 0, out[:, :Hq * D], ws)
    want, bound = ref.attn(c["q"], c["k"], c["v"], c["table"], c["lens"], 0.125)
    _close(out[:, :Hq * D].reshape(B, Hq, D), want, bound, "out")
    assert (out[:, Hq * D:] == 7).all()


def test_cache_beyond_32_bits():
    """Append to and attention over pages more than 2^31 elements into the cache."""
    Hq, Hkv, D, page, n_pages = 4, 2, 64, 16, 40
    stride = 2 ** 26  # elements between pages: 40 pages span 2.7e9
    big = [torch.zeros(n_pages, stride, dtype=BF, device="cuda") for _ in range(2)]
    k = big[0].as_strided((n_pages, Hkv, page, D), (stride, page * D, D, 1))
    v = big[1].as_strided((n_pages, Hkv, D, page), (stride, page * D, page, 1))
    cache = fm.KVCache(k, v, Hq)
    T = 40
    g = _gen(1)
    qkv = _randn(g, T, (Hq + 2 * Hkv) * D)
    pages = torch.tensor([39, 33, 35])
    at = torch.arange(T)
    q = torch.empty(T, Hq * D, dtype=BF, device="cuda")
    fm.kv_append(cache, fm.QKTransform(), qkv.cuda(), None, (pages[at // page] * page + at % page).cuda(), q)
    x = qkv.view(T, -1, D)
    assert torch.equal(k[39, :, 5].cpu(), x[5, Hq:Hq + Hkv]) and torch.equal(v[35, :, :, 7].cpu(), x[39, Hq + Hkv:])
    table = pages[None].to(torch.int32)
    lens = torch.tensor([T], dtype=torch.int32)
    out = torch.empty(1, Hq * D, dtype=BF, device="cuda")
    fm.attn_decode(cache, fm.AttnDecode(0.125), q[-1:], table.cuda(), lens.cuda(), 0, out, fm.attn_decode_workspace(cache, 1))
    ks, vs = torch.zeros(n_pages, Hkv, page, D, dtype=BF), torch.zeros(n_pages, Hkv, D, page, dtype=BF)
    for p in pages.tolist():
        ks[p], vs[p] = k[p].cpu(), v[p].cpu()
    want, bound = ref.attn(q[-1:].cpu().view(1, Hq, D), ks, vs, table, lens, 0.125)
    _close(out.view(1, Hq, D), want, bound, "out")


# ---- log probabilities ---------------------------------------------------------------------
def _logprobs(x, n, tokens=None, ld=None, what=""):
    T, V = x.shape
    g = _gen(T + V)
    if tokens is None:
        tokens = torch.randint(0, V, (T,), generator=g)
    tokens = tokens.to(torch.int32)
    d = x.cuda()
    if ld:
        wide = torch.full((T, ld), NAN, dtype=x.dtype, device="cuda")
        wide[:, 1:V + 1] = d
        d = wide[:, 1:V + 1]
    lp, h = (torch.full((T,), 7.0, device="cuda") for _ in range(2))
    ids, tl = torch.full((T, n), -7, dtype=torch.int32, device="cuda"), torch.full((T, n), 7.0, device="cuda")
    ws = torch.full((max(16, fm.token_logprobs_workspace_bytes(T, V, n)),), 0xff, dtype=torch.uint8, device="cuda")
    fm.token_logprobs(d, tokens.cuda(), lp, h, ids, tl, ws)
    return lp.cpu().double(), h.cpu().double(), ids.cpu().long(), tl.cpu().double(), tokens


def _check_logprobs(x, n, **kw):
    _say("logprobs", tuple(x.shape), x.dtype, n)
    lp, h, ids, tl, tokens = _logprobs(x, n, **kw)
    wl, wh, wi, wt, bl, bh = ref.logprobs(x, tokens, n)
    assert torch.equal(ids, wi), "top ids"
    for got, want, bound, name in ((lp, wl, bl, "logprob"), (h, wh, bh, "entropy"), (tl, wt, bl[:, None], "top")):
        fin = torch.isfinite(want)
        assert torch.equal(got[~fin], want[~fin]), name
        over = ((got - want).abs() - bound.expand_as(want))[fin]
        assert (over <= 0).all(), "%s: over its bound by %g" % (name, over.max())


@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("T,V,n", [(1, 1, 1), (2, 7, 3), (3, 32, 32), (5, 33, 32), (1, 1000, 0), (9, 4099, 5), (2, 16385, 20),
                                   (1, 130953, 20), (3, 131072, 1), (700, 333, 2)])
def test_logprobs(T, V, n, dt):
    _check_logprobs(_randn(_gen(V), T, V, std=3.0, dtype=dt), n)


@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("ld", [5003, 5008])
def test_logprobs_strides(dt, ld):
    _check_logprobs(_randn(_gen(1), 5, 5001, std=3.0, dtype=dt), 4, ld=ld)


@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("order", ["up", "down", "equal", "zeros", "few"])
def test_logprobs_orders(dt, order):
    """Rows whose order is the worst for a running selection, and ties: the lowest index wins."""
    V = 40001
    if order == "up":
        x = torch.arange(V).float()[None] / 1000
    elif order == "down":
        x = -torch.arange(V).float()[None] / 1000
    elif order == "equal":
        x = torch.full((2, V), -3.0)
    elif order == "zeros":
        x = torch.where(torch.rand(2, V, generator=_gen(0)) < 0.5, 0.0, -0.0)
    else:  # a handful of values, all tied many times over
        x = torch.randint(0, 3, (3, V), generator=_gen(2)).float()
    _check_logprobs(x.to(dt), 32)


@pytest.mark.parametrize("dt", [BF, torch.float32])
def test_logprobs_masks(dt):
    """Masked logits: -inf, the type's lowest value, all but one, fewer left than asked for, and
    rows with nothing left (every log probability -inf, entropy 0)."""
    V = 20001
    lowest = torch.finfo(dt).min
    x = _randn(_gen(3), 5, V, std=3.0, dtype=dt)
    x[0, torch.rand(V, generator=_gen(4)) < 0.999] = -INF
    x[1, torch.rand(V, generator=_gen(5)) < 0.9] = lowest
    x[2], x[2, 12345] = -INF, 2.0
    x[3] = lowest
    x[4, :19000] = -INF
    _check_logprobs(x, 32, tokens=torch.tensor([0, 1, 12345, 7, 20000]))
    none = torch.full((2, V), -INF, dtype=dt)
    lp, h, ids, tl, _ = _logprobs(none, 3)
    assert (lp == -INF).all() and (h == 0).all() and (tl == -INF).all() and ids.tolist() == [[0, 1, 2]] * 2


@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("V", [32769, 65535, 150001])
def test_logprobs_masks_in_parts(V, dt):
    """Rows in parts: whole parts masked, values in one part alone, NaN in one part."""
    x = _randn(_gen(8), 6, V, std=3.0, dtype=dt)
    x[0, torch.rand(V, generator=_gen(9)) < 0.9995] = -INF
    x[1, :V - 40] = -INF
    x[2, 40:] = torch.finfo(dt).min
    x[3], x[3, V // 2] = -INF, -5.0
    x[4] = -INF
    x[5, V // 3] = NAN
    tokens = torch.tensor([0, V - 1, 41, V // 2, 3, 5])
    lp, h, ids, tl, _ = _logprobs(x, 32, tokens=tokens)
    wl, wh, wi, wt, bl, bh = ref.logprobs(x[:4], tokens[:4], 32)
    for got, want, bound in ((lp[:4], wl, bl), (h[:4], wh, bh), (tl[:4], wt, bl[:, None])):
        fin = torch.isfinite(want)
        assert torch.equal(got[~fin], want[~fin]) and ((got - want).abs() <= bound.expand_as(want))[fin].all()
    assert torch.equal(ids[:4], wi)
    assert lp[4] == -INF and h[4] == 0 and (tl[4] == -INF).all() and ids[4].tolist() == list(range(32))
    assert torch.isnan(lp[5]) and torch.isnan(h[5]) and torch.isnan(tl[5]).all()


@pytest.mark.parametrize("dt", [BF, torch.float32])
def test_logprobs_not_finite(dt):
    """NaN and +inf: NaN log probabilities and entropy in that row alone, ids still ordered."""
    x = _randn(_gen(6), 4, 5000, std=3.0, dtype=dt)
    x[1, 77], x[2, 4444] = NAN, INF
    x[3] = NAN
    x[3, 10], x[3, 4000] = 1.0, 2.0
    lp, h, ids, tl, tokens = _logprobs(x, 4)
    wl, wh, wi, wt, bl, bh = ref.logprobs(x, tokens, 4)
    assert torch.isnan(lp[1:]).all() and torch.isnan(h[1:]).all() and torch.isnan(tl[1:]).all()
    assert abs(lp[0] - wl[0]) <= bl[0] and abs(h[0] - wh[0]) <= bh[0]
    assert torch.equal(ids[:3], wi[:3]) and ids[3].tolist() == [4000, 10, 0, 1]


@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("V", [40, 300, 2500, 9001])
def test_logprobs_fewer_numbers_than_asked(V, dt):
    """Rows with fewer numbers than alternatives, the rest NaN or -inf: the numbers first, then
    -inf, then NaN, each by index."""
    n = 32
    for fill in (NAN, -INF):
        x = torch.full((3, V), fill, dtype=dt)
        x[0, V - 1], x[0, 5] = 1.0, 1.0
        x[1, ::V // 10] = -2.0
        x[2, V // 2:V // 2 + 15] = -INF
        x[2, 3] = 0.5
        lp, h, ids, tl, tokens = _logprobs(x, n)
        rank = torch.where(torch.isnan(x), torch.full_like(x, 2), torch.where(x == -INF, torch.ones_like(x), torch.zeros_like(x)))
        key = torch.where(rank == 0, x, torch.zeros_like(x)).double() - 1000.0 * rank.double()
        want = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :n]
        assert torch.equal(ids, want)
        if fill == -INF:
            wl, wh, _, wt, bl, bh = ref.logprobs(x, tokens, n)
            _close(h, wh, bh, "entropy")
            fin = torch.isfinite(wt)
            assert torch.equal(tl[~fin], wt[~fin]) and ((tl - wt).abs() <= bl[:, None])[fin].all()


def test_logprobs_tokens_outside_and_optional():
    x = _randn(_gen(7), 3, 100, dtype=torch.float32)
    lp, _, _, _, _ = _logprobs(x, 0, tokens=torch.tensor([-1, 100, 5]))
    assert lp[0] == -INF and lp[1] == -INF and torch.isfinite(lp[2])
    h = torch.empty(3, device="cuda")
    ws = fm.token_logprobs_workspace(3, 100, 0)
    fm.token_logprobs(x.cuda(), None, None, h, None, None, ws)
    _, wh, _, _, _, bh = ref.logprobs(x, torch.zeros(3), 0)
    _close(h, wh, bh, "entropy")


def test_logprobs_beyond_32_bits():
    """The last row of more than 2^31 logits."""
    T, V = 16500, 131073
    x = torch.zeros(T, V, dtype=BF, device="cuda")
    last = _randn(_gen(8), 1, V, std=3.0)
    x[-1] = last[0].cuda()
    lp, h = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    ids, tl = torch.empty(T, 3, dtype=torch.int32, device="cuda"), torch.empty(T, 3, device="cuda")
    fm.token_logprobs(x, torch.full((T,), 9, dtype=torch.int32, device="cuda"), lp, h, ids, tl, fm.token_logprobs_workspace(T, V, 3))
    wl, wh, wi, wt, bl, bh = ref.logprobs(last, torch.tensor([9]), 3)
    assert torch.equal(ids[-1:].cpu().long(), wi) and ids[-2].tolist() == [0, 1, 2]
    _close(lp[-1:], wl, bl, "logprob")
    _close(h[-1:], wh, bh, "entropy")


# ---- all together --------------------------------------------------------------------------
def _all_ops(seed=0):
    """One state of each operator and a function that runs them all on the current stream."""
    c = _attn_case(5, 8, 2, 128, 64, [500, 320, 0, 321, 900], 256, seed)
    cache = fm.KVCache(c["k"].cuda(), c["v"].cuda(), 8)
    codes, scales, x = _linear_case(5, 512, 1000, 128, seed)
    w, dx = fm.Int4Linear(codes.cuda(), scales.cuda()), x.cuda()
    g = _gen(seed + 9)
    qkv, slots = _randn(g, 5, 12 * 128).cuda(), torch.tensor([1, 70, 131, -1, 300]).cuda()
    q, dq, table, lens = torch.empty(5, 1024, dtype=BF, device="cuda"), c["q"].cuda(), c["table"].cuda(), c["lens"].cuda()
    out, y = torch.empty(5, 1024, dtype=BF, device="cuda"), torch.empty(5, 1000, device="cuda")
    lp, h = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    ids, tl = torch.empty(5, 7, dtype=torch.int32, device="cuda"), torch.empty(5, 7, device="cuda")
    tokens = torch.arange(5, dtype=torch.int32, device="cuda")
    ws, ws2 = fm.attn_decode_workspace(cache, 5), fm.token_logprobs_workspace(5, 1000, 7)
    tr, at = fm.QKTransform(), fm.AttnDecode(0.09)

    def run(stream=None):
        fm.kv_append(cache, tr, qkv, None, slots, q, stream=stream)
        fm.attn_decode(cache, at, dq, table, lens, 256, out, ws, stream=stream)
        fm.linear_int4(w, dx, y, stream=stream)
        fm.token_logprobs(y, tokens, lp, h, ids, tl, ws2, stream=stream)

    return run, (q, cache.k, cache.v, out, y, lp, h, ids, tl)


def test_ops_repeat_bitwise_and_streams():
    """The same bits on a second call and on another stream."""
    run, outs = _all_ops()
    run()
    first = [o.clone() for o in outs]
    for o in outs[3:]:
        o.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    for a, b in zip(first, outs):
        assert torch.equal(a, b)


def test_ops_graph_replays():
    """Captured once, replayed with the program's own work between: every replay is the eager result."""
    run, outs = _all_ops(1)
    run()
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(4):
        for o in outs[3:]:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, outs):
            assert torch.equal(a, b)
        run()
        torch.cuda.synchronize()
        for a, b in zip(first, outs):
            assert torch.equal(a, b)


def test_ops_empty_batches():
    """T = 0 and B = 0 are no-ops."""
    codes, scales, _ = _linear_case(1, 128, 8, 128)
    w = fm.Int4Linear(codes.cuda(), scales.cuda())
    e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device="cuda")
    fm.linear_int4(w, e(0, 128), e(0, 8))
    cache = fm.KVCache(e(2, 1, 16, 64), e(2, 1, 64, 16), 1)
    fm.kv_append(cache, fm.QKTransform(), e(0, 192), None, e(0, dt=torch.int64), e(0, 64))
    fm.attn_decode(cache, fm.AttnDecode(1.0), e(0, 64), e(0, 1, dt=torch.int32), e(0, dt=torch.int32), 0, e(0, 64),
                   fm.attn_decode_workspace(cache, 1))
    fm.token_logprobs(e(0, 10), None, None, e(0, dt=torch.float32), None, None, fm.token_logprobs_workspace(1, 10))
    torch.cuda.synchronize()
