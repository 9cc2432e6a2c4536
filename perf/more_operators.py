"""Timed and compared cases of the operators of a server with many requests.

  lora      flint_lora             low-rank adapters of many requests beside a shared projection
  logits    flint_logits_adjust    penalties for repeated tokens, biases and grammar masks
  append4   flint_kv4_append       norm, rotation and new keys and values into a cache of 4 bits
  attn4     flint_kv4_attn_decode  one query per sequence over that cache, shared prefix read once
  advance   flint_kv_advance       the next step's page tables: fork, free, reorder, grow, copy on write
  compact   flint_kv_compact       live pages moved to the front of the pool

`own` selects the side: False runs the plain form (elementary torch operations in 32 bits,
rounded once), True the library's entry points.  Both sides get the same inputs.
"""
import math

import torch

own = False

HEADS, KV_HEADS, HEAD_DIM = 32, 4, 128  # the Flint model's attention heads
# (query heads, key heads) of the drawn cases: one head, shared by odd and even numbers of queries, wide
GROUPS = ((1, 1), (8, 1), (6, 2), (10, 2), (4, 4), (20, 4), (32, 4), (40, 8), (64, 8))
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # what the low three bits of a code stand for


# ---- cases ---------------------------------------------------------------------------
def listed():
    lora = dict(op="lora", rank=16, runs=False, base="fp32", out="bf16")
    lg = dict(op="logits", dtype="bf16", history=2000, bias=20, masked=0.0)
    app = dict(op="append4", heads=HEADS, kv_heads=KV_HEADS, dim=HEAD_DIM, page=64, rot=128, style="half", norm=True)
    att = dict(op="attn4", heads=HEADS, kv_heads=KV_HEADS, dim=HEAD_DIM, page=64, window=0, sinks=True)
    adv = dict(op="advance", kv_heads=KV_HEADS, dim=HEAD_DIM, page=64, bits=4, layers=4, group=1, grow=1)
    return [
        # eight requests with six adapters through the fused query, key and value projection
        dict(lora, name="lora_t8_qkv", T=8, K=2048, N=5120, adapters=6),
        # the prompts of several requests through the attention output projection, a larger rank
        dict(lora, name="lora_t4099_out_proj", T=4099, K=4096, N=2048, adapters=8, rank=64, runs=True, base="bf16"),
        # one request's next token after a long dialogue: an odd vocabulary
        dict(lg, name="logits_t1", T=1, V=130953, dtype="fp32", history=20000),
        # a large decode batch, half of it under a grammar that masks most of the vocabulary
        dict(lg, name="logits_t128_grammar", T=128, V=131072, masked=0.9),
        # the new token of eight requests
        dict(app, name="append4_t8", T=8, pages=1024),
        # an 8192-token prompt
        dict(app, name="append4_t8192", T=8192, pages=1024),
        # one request at 100K tokens
        dict(att, name="attn4_b1_100k", B=1, prefix=0, suffix=100003),
        # thirty-two requests that share a 32768-token prefix
        dict(att, name="attn4_b32_shared_32k", B=32, prefix=32768, suffix=1000),
        # a beam search of eight beams: survivors fork, the others' pages return
        dict(adv, name="advance_b8_beams", rows=8, tokens=2000, pages=1024, group=8),
        # a decode step of 256 requests in groups of four samples, one in eight finished
        dict(adv, name="advance_b256_samples", rows=256, tokens=4000, pages=16384, layers=1, group=4),
        # a small pool after its first requests have ended
        dict(adv, name="compact_512", op="compact", rows=16, tokens=900, pages=512, layers=2, bits=16),
        # a pool of 4096 bf16 pages, half of them live and scattered
        dict(adv, name="compact_4096", op="compact", rows=64, tokens=3500, pages=4096, layers=2, bits=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "logits", "append4", "attn4", "advance", "compact"])
    if op == "lora":
        rank = rng.choice([8, 16, 32, 64])
        adapters = _log(rng, 1, 32)
        K = 8 * _log(rng, 16, 1024)
        T = _log(rng, 1, 4096)
        N = _log(rng, 16, min(16384, 9000000 // T))
        return dict(op=op, T=T, K=K, N=N, rank=rank, adapters=adapters, runs=rng.random() < 0.6,
                    base=rng.choice(["fp32", "bf16", "none"]), out=rng.choice(["bf16", "fp32"]))
    if op == "logits":
        T = _log(rng, 1, 128)
        V = _log(rng, 1000, min(200000, 16000000 // T))
        return dict(op=op, T=T, V=V, dtype=rng.choice(["bf16", "fp32"]), history=_log(rng, 1, 20000),
                    bias=rng.choice([0, 1, 20, 300]), masked=rng.choice([0.0, 0.5, 0.9]))
    if op == "append4":
        (heads, kv), dim = rng.choice(GROUPS), rng.choice([64, 128])
        page = rng.choice([16, 32, 64, 128])
        T = _log(rng, 1, min(8192, 8192 * 40 * 128 // ((heads + 2 * kv) * dim)))
        return dict(op=op, T=T, heads=heads, kv_heads=kv, dim=dim, page=page,
                    pages=max((2 * T + 4096) // page + 8, 260), rot=rng.choice([0, dim // 2, dim]),
                    style=rng.choice(["half", "pairs"]), norm=rng.random() < 0.6)
    if op == "attn4":
        (heads, kv), dim = rng.choice(GROUPS), rng.choice([64, 128])
        page = rng.choice([16, 32, 64, 128])
        B = _log(rng, 1, 128)
        most = 3200000 // (B * kv)  # keys of one sequence: the plain form gathers them all
        prefix = rng.choice([0, 1]) * _log(rng, 256, 98304)
        prefix = min(prefix, most // 2) // page * page
        return dict(op=op, B=B, heads=heads, kv_heads=kv, dim=dim, page=page, prefix=prefix,
                    suffix=min(_log(rng, 1, 16384), most // 2), window=rng.choice([0, 0, 513]),
                    sinks=rng.random() < 0.5)
    page, dim, kv = rng.choice([16, 32, 64, 128]), rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    bits, layers = rng.choice([4, 16]), rng.choice([1, 2, 3])
    room = 400000000 // (kv * dim * 4 * layers)  # tokens that fit 400 MB of a bf16 pool
    rows = _log(rng, 1, 256)
    tokens = _log(rng, 1, max(2, min(8000, room // (2 * rows) - 2 * page)))
    pages = rows * (tokens // page + 2) * 2 + rng.randrange(64)
    return dict(op=op, rows=rows, tokens=tokens, pages=pages, kv_heads=kv, dim=dim, page=page, bits=bits, layers=layers,
                group=rng.choice([1, 2, 4, 5]), grow=rng.choice([1, 1, 7, 65]))


# ---- inputs --------------------------------------------------------------------------
def _lengths(case, seed):
    """Tokens of each sequence: the shared prefix and a suffix of 1 ... suffix, ragged; the
    first has the longest."""
    g = torch.Generator().manual_seed(seed)
    own_part = torch.randint(1, case["suffix"] + 1, (case["B"],), generator=g)
    own_part[0] = case["suffix"]
    return case["prefix"] + own_part


def _block(case):
    """Bytes of a page of the 4-bit cache: codes of keys and values, then their scales."""
    return 2 * case["kv_heads"] * case["page"] * (case["dim"] // 2 + case["dim"] // 32)


def _fill4(case, pages, g):
    """A 4-bit cache of pages of random codes, with scales of 2^-2 ... 2^1."""
    d = torch.randint(0, 256, (pages, _block(case)), generator=g, device="cuda", dtype=torch.uint8)
    codes = case["kv_heads"] * case["page"] * case["dim"]
    d[:, codes:] = d[:, codes:] % 4 + 125
    return d


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    types = dict(bf16=torch.bfloat16, fp32=torch.float32)
    op = case["op"]
    if op == "lora":
        T, K, N, r, n = case["T"], case["K"], case["N"], case["rank"], case["adapters"]
        ids = torch.randint(-1, n, (T,), generator=host, dtype=torch.int32)  # -1: a request without an adapter
        if case["runs"]:  # prompts: a request's tokens lie together
            ids = ids[torch.sort(torch.randint(0, max(1, T // 64), (T,), generator=host)).values]
        return dict(x=normal(T, K), ids=ids.cuda(), a=normal(n, r, K, std=K ** -0.5), b=normal(n, N, r, std=0.5),
                    scales=torch.rand(n, generator=g, device="cuda") * 2,
                    base=None if case["base"] == "none" else normal(T, N, dtype=types[case["base"]]),
                    y=torch.empty(T, N, device="cuda", dtype=types[case["out"]]))
    if op == "logits":
        T, V, L, nb = case["T"], case["V"], case["history"], min(case["bias"], case["V"])
        total = ints(0, L + 1, T)
        total[0] = L
        # words recur: a third of the history comes from 64 tokens
        hist = torch.where(torch.rand(T, L, generator=g, device="cuda") < 0.33, ints(0, 64, T, L), ints(0, V, T, L)) % V
        start = torch.arange(T + 1, device="cuda", dtype=torch.int32) * nb
        bias_ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:nb] for _ in range(T)]).to(torch.int32).view(-1)
        masks = rows = None
        if case["masked"]:  # one grammar state for every second request
            n, words = T // 2 + 1, -(-V // 32)
            keep = torch.rand(n, words, 32, generator=g, device="cuda") >= case["masked"]
            bits = torch.arange(32, device="cuda", dtype=torch.int64)
            masks = (keep.long() << bits).sum(-1)
            masks = torch.where(masks >= 2 ** 31, masks - 2 ** 32, masks).to(torch.int32)
            rows = torch.where(torch.arange(T, device="cuda") % 2 == 0, torch.arange(T, device="cuda") // 2, -1).to(torch.int32)
        return dict(logits=normal(T, V, std=3.0, dtype=types[case["dtype"]]), history=hist,
                    prompt=(total * 0.7).to(torch.int32), total=total,
                    repetition=1 + 0.3 * torch.rand(T, generator=g, device="cuda"),
                    presence=torch.rand(T, generator=g, device="cuda"), frequency=0.5 * torch.rand(T, generator=g, device="cuda"),
                    bias_start=start, bias_ids=bias_ids, bias=normal(T * nb, std=5.0, dtype=torch.float32),
                    masks=masks, mask_rows=rows, out=torch.empty(T, V, device="cuda", dtype=types[case["dtype"]]))
    if op == "append4":
        T, D, page, pages = case["T"], case["dim"], case["page"], case["pages"]
        Hq, Hkv, rot = case["heads"], case["kv_heads"], case["rot"]
        if T > 256:  # a prompt: consecutive tokens on pages of its own, from the middle of one
            order = torch.randperm(pages, generator=g, device="cuda")
            at = page // 2 - 1 + torch.arange(T, device="cuda")
            slots = order[at // page] * page + at % page
            positions = at.to(torch.int32)
        else:  # the new token of T requests
            slots = torch.randperm(pages, generator=g, device="cuda")[:T] * page
            slots = slots + torch.randint(0, page, (T,), generator=g, device="cuda")
            positions = ints(0, 16384, T)
        cos = sin = None
        if rot:
            f = 500000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") * 2 / rot)
            a = torch.arange(16384, dtype=torch.float64, device="cuda")[:, None] * f
            cos, sin = a.cos().float(), a.sin().float()
        qn = normal(D, std=0.1) + 1 if case["norm"] else None
        kn = normal(D, std=0.1) + 1 if case["norm"] else None
        e = lambda h: torch.empty(T, h * D, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        return dict(data=_fill4(case, pages, g), qkv=normal(T, (Hq + 2 * Hkv) * D), slots=slots.to(torch.int64),
                    positions=positions, cos=cos, sin=sin, q_norm=qn, k_norm=kn, q=e(Hq), k=e(Hkv), v=e(Hkv))
    if op == "attn4":
        B, D, page, Hq = case["B"], case["dim"], case["page"], case["heads"]
        lens = _lengths(case, seed)
        shared = case["prefix"] // page
        per = -(-(lens - case["prefix"]) // page)
        pages = shared + int(per.sum())
        order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
        table = torch.zeros(B, shared + int(per.max()), device="cuda", dtype=torch.int32)
        table[:, :shared] = order[:shared]
        at = shared
        for b, n in enumerate(per.tolist()):
            table[b, shared:shared + n] = order[at:at + n]
            at += n
        return dict(data=_fill4(case, pages, g), table=table, lens=lens.to(torch.int32).cuda(), q=normal(B, Hq * D),
                    sinks=normal(Hq, dtype=torch.float32) if case["sinks"] else None,
                    out=torch.empty(B, Hq * D, device="cuda", dtype=torch.bfloat16))
    # a pool in use: groups of sequences that share the whole pages of a common first half
    R, page, pages, G = case["rows"], case["page"], case["pages"], case["group"]
    lens = torch.randint(1, case["tokens"] + 1, (R,), generator=host)
    lens[0] = case["tokens"]
    head = torch.arange(R) // G * G  # a group's first sequence
    same = torch.minimum(lens // 2 // page, lens[head] // 2 // page)  # whole pages of it that are shared
    same[head == torch.arange(R)] = 0
    used = -(-lens // page)
    width = -(-(case["tokens"] + case["grow"]) // page) + 1
    order = torch.randperm(pages, generator=host)
    j = torch.arange(width)
    mine = (j >= same[:, None]) & (j < used[:, None])
    table = torch.full((R, width), -1, dtype=torch.int64)
    table[mine] = order[:int(mine.sum())]
    table = torch.where(j < same[:, None], table[head], table)
    refs = torch.bincount(table[table >= 0], minlength=pages)
    free = torch.full((pages,), -1, dtype=torch.int64)
    n_free = int((refs == 0).sum())
    free[:n_free] = order[pages - n_free:]
    # a group's new rows continue some of its old ones; one request in eight has ended
    parent = head + torch.randint(0, G, (R,), generator=host)
    parent = torch.where((parent >= R) | (torch.rand(R, generator=host) < 0.125), -1, parent)
    if G == 1:
        parent = torch.where(parent >= 0, torch.arange(R), -1)
    i32 = lambda t: t.to(torch.int32).cuda()  # noqa: E731
    if case["bits"] == 4:
        arrays = [_fill4(case, pages, g) for _ in range(case["layers"])]
    else:
        shape = (pages, case["kv_heads"], page, case["dim"])
        arrays = [torch.randint(-2 ** 15, 2 ** 15, shape if i % 2 == 0 else (shape[0], shape[1], shape[3], shape[2]), generator=g,
                                device="cuda", dtype=torch.int16) for i in range(2 * case["layers"])]
    old = dict(refs=i32(refs), free=i32(free), n_free=i32(torch.tensor([n_free])), table=i32(table), lens=i32(lens))
    return dict(arrays=arrays, old=old, new={k: torch.empty_like(v) for k, v in old.items()}, parent=i32(parent),
                grow=torch.full((R,), case["grow"], device="cuda", dtype=torch.int32),
                slots=torch.empty(R, case["grow"], device="cuda", dtype=torch.int64),
                moved=torch.empty(pages, device="cuda", dtype=torch.int32))


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own:  # the descriptors and the workspace that a program makes once
        import sparse_moe_transformer_wave_amd as fm

        op = case["op"]
        if op == "lora":
            state["plan"] = fm.LoraAdapters(state["a"], state["b"], scales=state["scales"])
            state["ws"] = fm.lora_workspace(state["plan"], case["T"])
        elif op == "logits":
            state["plan"] = fm.LogitRules(
                history=state["history"], prompt_len=state["prompt"], total_len=state["total"], repetition=state["repetition"],
                presence=state["presence"], frequency=state["frequency"], bias_start=state["bias_start"],
                bias_ids=state["bias_ids"], bias=state["bias"], masks=state["masks"], mask_rows=state["mask_rows"])
        elif op in ("append4", "attn4"):
            cache = fm.KV4Cache(state["data"], case["heads"], case["kv_heads"], case["dim"], case["page"])
            if op == "append4":
                state["plan"] = (cache, fm.QKTransform(state["q_norm"], state["k_norm"], 1e-6, state["cos"], state["sin"],
                                                       case["style"] == "pairs"))
            else:
                state["plan"] = (cache, fm.AttnDecode(case["dim"] ** -0.5, case["window"], state["sinks"]))
                state["ws"] = fm.kv4_attn_decode_workspace(cache, case["B"])
        else:
            a = state["arrays"]
            if case["bits"] == 4:
                caches = [fm.KV4Cache(d, case["kv_heads"], case["kv_heads"], case["dim"], case["page"]) for d in a]
            else:
                caches = [fm.KVCache(a[i], a[i + 1], case["kv_heads"]) for i in range(0, len(a), 2)]
            pages = fm.KVPages(caches)
            o, n = (fm.KVState(s["refs"], s["free"], s["n_free"], s["table"], s["lens"]) for s in (state["old"], state["new"]))
            state["plan"], state["ws"] = (pages, o, n), fm.kv_pages_workspace(pages, case["rows"])
    return state


# ---- plain forms -----------------------------------------------------------------------
def _lora(s):
    case = s["case"]
    T, n, r = case["T"], case["adapters"], case["rank"]
    h = (s["x"].float() @ s["a"].float().view(n * r, -1).t()).view(T, n, r)
    mine = s["ids"].long()[:, None] == torch.arange(n, device="cuda")
    h = torch.where(mine[:, :, None], h * s["scales"][:, None], 0.0)
    y = h.view(T, n * r) @ s["b"].float().permute(0, 2, 1).reshape(n * r, -1)
    if s["base"] is not None:
        y = y + s["base"].float()
    return y.to(s["y"].dtype)


def _logits(s):
    T, V = s["logits"].shape
    at = torch.arange(s["history"].shape[1], device="cuda")
    seen_at = at < s["total"][:, None]
    out_at = seen_at & (at >= s["prompt"][:, None])
    ids = s["history"].long()
    seen = torch.zeros(T, V, device="cuda").scatter_add_(1, ids, seen_at.float()) > 0
    count = torch.zeros(T, V, device="cuda").scatter_add_(1, ids, out_at.float())
    x = s["logits"].float()
    rep = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias"].numel():
        x = x.scatter_add(1, s["bias_ids"].long().view(T, -1), s["bias"].view(T, -1))
    if s["masks"] is not None:
        v = torch.arange(V, device="cuda")
        rows = s["mask_rows"].long()
        keep = (s["masks"][rows.clamp(min=0)][:, v // 32] >> (v % 32)) & 1 == 1
        x = torch.where(keep | (rows < 0)[:, None], x, -math.inf)
    return x.to(s["out"].dtype)


def _norm(x, w, eps=1e-6):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(x.dtype)


def _rotate(x, cos, sin, style):
    rot = 2 * cos.shape[-1]
    a, rest = x[..., :rot], x[..., rot:]
    c, s = cos[:, None].to(x.dtype), sin[:, None].to(x.dtype)
    if style == "half":
        u, v = a[..., :rot // 2], a[..., rot // 2:]
        a = torch.cat([u * c - v * s, v * c + u * s], -1)
    else:
        u, v = a[..., 0::2], a[..., 1::2]
        a = torch.stack([u * c - v * s, v * c + u * s], -1).flatten(-2)
    return torch.cat([a, rest], -1)


def _quantise(x):
    """Codes, scale bytes and the values they stand for, of blocks of 32 channels (x in 64 bits, as
    codes next to a border depend on it): the least power of two with max |x| <= 7 of it, and the
    nearest of the eight magnitudes, the even code at a tie."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    f, e = torch.frexp(top / 7)
    e = torch.where(f == 0.5, e - 1, e).clamp(-125, 125)
    y = b.abs() * torch.exp2(-e.double())
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda", dtype=torch.float64)
    up = torch.tensor([False, True] * 3 + [False], device="cuda")  # a tie goes up to the even code
    code = ((y[..., None] > borders) | ((y[..., None] == borders) & up)).sum(-1)
    value = torch.tensor(E2M1, device="cuda", dtype=torch.float64)[code] * torch.exp2(e.double()) * torch.where(b < 0, -1.0, 1.0)
    code = (code + 8 * torch.signbit(b)).to(torch.uint8)
    return code.flatten(-2), (e.squeeze(-1) + 127).to(torch.uint8), value.flatten(-2)


def _parts(data, case):
    """The cache's key and value codes [page][head][token][dim / 2] and scales [page][head][dim / 32][token]."""
    n, h, page, d = data.shape[0], case["kv_heads"], case["page"], case["dim"]
    c, z = h * page * d // 2, h * page * d // 32
    return (data[:, :c].view(n, h, page, d // 2), data[:, c:2 * c].view(n, h, page, d // 2),
            data[:, 2 * c:2 * c + z].view(n, h, d // 32, page), data[:, 2 * c + z:].view(n, h, d // 32, page))


def _append4(s):
    case = s["case"]
    T, Hq, Hkv, D, page = case["T"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    x = s["qkv"].view(T, Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq].float(), x[:, Hq:Hq + Hkv].double(), x[:, Hq + Hkv:].double()
    if case["norm"]:
        q, k = _norm(q, s["q_norm"]), _norm(k, s["k_norm"])
    if case["rot"]:
        c, n = s["cos"][s["positions"].long()], s["sin"][s["positions"].long()]
        q, k = _rotate(q, c, n, case["style"]), _rotate(k, c, n, case["style"])
    (kc, ks, k), (vc, vs, v) = _quantise(k), _quantise(v)
    pg, off = s["slots"] // page, s["slots"] % page
    k_codes, v_codes, k_scales, v_scales = _parts(s["data"], case)
    k_codes[pg, :, off] = kc[..., 0::2] | kc[..., 1::2] << 4  # the even channel in the low nibble
    v_codes[pg, :, off] = vc[..., 0::2] | vc[..., 1::2] << 4
    k_scales[pg, :, :, off] = ks
    v_scales[pg, :, :, off] = vs
    return dict(q=q.flatten(1).to(torch.bfloat16), k=k.flatten(1).to(torch.bfloat16), v=v.flatten(1).to(torch.bfloat16),
                data=s["data"])


def _values(codes, scales, table, dtype):
    """What the pages of a table [B][n] hold: [B][heads][n * page][dim]."""
    c = codes[table]  # [B][n][heads][page][dim / 2]
    m = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda", dtype=dtype)
    x = torch.stack([m[(c & 15).long()], m[(c >> 4).long()]], -1).flatten(-2)
    z = torch.exp2(scales[table].to(dtype) - 127).transpose(-1, -2)  # [B][n][heads][page][dim / 32]
    x = (x.unflatten(-1, (-1, 32)) * z[..., None]).flatten(-2)
    return x.transpose(1, 2).flatten(2, 3)


def _attn4(s):
    case = s["case"]
    B, Hq, Hkv, D = case["B"], case["heads"], case["kv_heads"], case["dim"]
    kc, vc, ks, vs = _parts(s["data"], case)
    table = s["table"].long()
    L = table.shape[1] * case["page"]
    q = s["q"].view(B, Hkv, Hq // Hkv, D).float()
    x = torch.matmul(q, _values(kc, ks, table, torch.float32).transpose(-1, -2).contiguous()) * D ** -0.5
    at = torch.arange(L, device="cuda")
    n = s["lens"].long()[:, None]
    seen = at < n
    if case["window"]:
        seen = seen & (at >= n - case["window"])
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    if case["sinks"]:
        sink = s["sinks"].view(1, Hkv, Hq // Hkv, 1)
        m = torch.maximum(m, sink)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    if case["sinks"]:
        l = l + torch.exp(sink - m)
    return (torch.matmul(p, _values(vc, vs, table, torch.float32)) / l).reshape(B, Hq * D).to(torch.bfloat16)


def _advance(s):
    case, old = s["case"], s["old"]
    R, page, grow = case["rows"], case["page"], s["grow"].long()
    pages, width = old["refs"].numel(), old["table"].shape[1]
    table, lens, j = old["table"].long(), old["lens"].long(), torch.arange(width, device="cuda")
    # a page is held once more for each further row that continues its row, once less where none does
    parent, alive = s["parent"].long().clamp(min=0), s["parent"] >= 0
    children = torch.zeros(R, device="cuda", dtype=torch.int64).index_add_(0, parent, alive.long())
    held = j < -(-lens // page)[:, None]
    refs = old["refs"].long().index_add(0, table.clamp(min=0).flatten(), (held * (children - 1)[:, None]).flatten())
    freed = ((refs == 0) & (old["refs"] > 0)).nonzero()[:, 0]
    stack = torch.cat([old["free"][:old["n_free"].item()].long(), freed])
    # copy on write: of the rows that grow into a page, all but the last that holds it alone
    L = torch.where(alive, lens[parent], 0)
    used, rows = -(-L // page), torch.arange(R, device="cuda")
    last = table[parent, (used - 1).clamp(min=0)]
    fits = L + grow <= width * page
    into = (L % page > 0) & (grow > 0) & fits
    before = ((last[:, None] == last) & into & (rows < rows[:, None])).sum(1)
    copy = into & (refs[last.clamp(min=0)] - before > 1)
    # pages from the top of the stack, row after row; a row that finds too few does not grow, nor
    # does one that keeps a page which a row ahead would have had to copy
    want = torch.where(fits, -(-(L + grow) // page) - used + copy, 0)
    end = want.cumsum(0)
    served = fits & (((want == 0) & (before == 0)) | (end <= stack.numel()))
    copy = copy & served
    want = torch.where(served, want, 0)
    grow = torch.where(served, grow, 0)
    taken = want.sum()
    first = used - copy.long()  # a row's first new entry
    k = (end - want)[:, None] + j - first[:, None]
    new = (j >= first[:, None]) & (j < (first + want)[:, None])
    fresh = stack.flip(0)[torch.where(new, k, 0).clamp(0, max(stack.numel() - 1, 0))] if stack.numel() else torch.full_like(k, -1)
    out = torch.where(new, fresh, torch.where(j < used[:, None], table[parent], -1))
    refs = refs.index_add(0, last.clamp(min=0), -copy.long())
    refs[fresh[new]] = 1
    at = L[:, None] + torch.arange(s["slots"].shape[1], device="cuda")
    ok = at < (L + grow)[:, None]
    slots = torch.where(ok, out.gather(1, (at // page).clamp(max=width - 1)) * page + at % page, -1)
    src, dst = last[copy], out[rows, first][copy]
    for a in s["arrays"]:
        a[dst] = a[src]
    n_free = stack.numel() - taken
    place = torch.arange(pages, device="cuda")
    free = torch.where(place < n_free, torch.cat([stack, place.new_zeros(pages)])[:pages], -1)
    return dict(refs=refs.int(), free=free.int(), n_free=n_free.int().view(1), table=out.int(), lens=(L + grow).int(), slots=slots,
                arrays=s["arrays"])


def _compact(s):
    case, old = s["case"], s["old"]
    pages, place = old["refs"].numel(), torch.arange(old["refs"].numel(), device="cuda")
    live = old["refs"] > 0
    n = live.sum()
    src, dst = (live & (place >= n)).nonzero()[:, 0], (~live & (place < n)).nonzero()[:, 0]
    moved = torch.where(live, place, -1)
    moved[src] = dst
    refs = torch.where(place < n, old["refs"], 0)
    refs[dst] = old["refs"][src]
    for a in s["arrays"]:
        a[dst] = a[src]
    used = -(-old["lens"].long() // case["page"])
    held = torch.arange(old["table"].shape[1], device="cuda") < used[:, None]
    table = torch.where(held, moved[old["table"].long().clamp(min=0)], -1)
    free = torch.where(place < pages - n, pages - 1 - place, -1)
    return dict(refs=refs, free=free.int(), n_free=(pages - n).int().view(1), table=table.int(), lens=old["lens"], moved=moved.int(),
                arrays=s["arrays"])


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"lora": _lora, "logits": _logits, "append4": _append4, "attn4": _attn4, "advance": _advance, "compact": _compact}[op](s)
    import sparse_moe_transformer_wave_amd as fm

    if op == "lora":
        fm.lora(s["plan"], s["x"], s["ids"], s["base"], s["y"], s["ws"])
        return s["y"]
    if op == "logits":
        fm.logits_adjust(s["plan"], s["logits"], s["out"])
        return s["out"]
    if op == "append4":
        cache, transform = s["plan"]
        fm.kv4_append(cache, transform, s["qkv"], s["positions"], s["slots"], s["q"], s["k"], s["v"])
        return dict(q=s["q"], k=s["k"], v=s["v"], data=s["data"])
    if op == "attn4":
        cache, attn = s["plan"]
        fm.kv4_attn_decode(cache, attn, s["q"], s["table"], s["lens"], s["case"]["prefix"], s["out"], s["ws"])
        return s["out"]
    pages, old, new = s["plan"]
    if op == "advance":
        fm.kv_advance(pages, old, new, s["parent"], s["grow"], s["slots"], s["ws"])
        return dict(s["new"], slots=s["slots"], arrays=s["arrays"])
    fm.kv_compact(pages, old, new, s["moved"], s["ws"])
    return dict(s["new"], moved=s["moved"], arrays=s["arrays"])


# ---- what a pass cannot do without -------------------------------------------------------
def work(case):
    op = case["op"]
    size = dict(bf16=2, fp32=4, none=0)
    if op == "lora":
        T, K, N, r = case["T"], case["K"], case["N"], case["rank"]
        n = min(case["adapters"], T)
        return dict(bytes=2 * T * K + 2 * n * r * (K + N) + T * N * (size[case["base"]] + size[case["out"]]) + 4 * T,
                    flops=2 * T * r * (K + N))
    if op == "logits":
        T, V = case["T"], case["V"]
        mask = (T // 2 + 1) * V // 8 if case["masked"] else 0
        return dict(bytes=2 * T * V * size[case["dtype"]] + 2 * T * case["history"] + 8 * T * case["bias"] + mask, flops=2 * T * V)
    if op == "append4":
        T, D, Hq, Hkv = case["T"], case["dim"], case["heads"], case["kv_heads"]
        width = (Hq + 2 * Hkv) * D
        new = 2 * Hkv * (D // 2 + D // 32)
        return dict(bytes=T * (4 * width + new + 4 * case["rot"] + 12), flops=8 * T * width)
    if op == "attn4":
        B, kv, D = case["B"], case["kv_heads"], case["dim"]
        tail = case["suffix"] + (B - 1) * (case["suffix"] + 1) / 2  # the mean of the ragged suffixes
        unique, seen = case["prefix"] + tail, B * case["prefix"] + tail
        if case["window"]:
            unique = seen = min(seen, B * case["window"])
        return dict(bytes=2 * unique * kv * (D // 2 + D // 32) + 4 * B * case["heads"] * D, flops=4 * seen * case["heads"] * D)
    page = 2 * case["kv_heads"] * case["page"] * (case["dim"] // 2 + case["dim"] // 32 if case["bits"] == 4 else 2 * case["dim"])
    used = case["rows"] * (case["tokens"] / case["page"] / 2 + 1)  # entries of the tables
    state = 8 * used + 8 * case["pages"] + 4 * min(case["pages"], used)
    if op == "advance":  # about half of the rows of a group that forks copy a page
        copies = 0 if case["group"] == 1 else case["rows"] / 2
        return dict(bytes=state + 2 * copies * page * case["layers"], flops=used)
    live = min(0.9, 0.8 * used / case["pages"])  # live pages beyond the last live one's new place
    return dict(bytes=state + 2 * case["pages"] * live * (1 - live) * page * case["layers"], flops=used)


# ---- 64 bits -----------------------------------------------------------------------------
def _codes(x):
    """Values of x in 4 bits: the nearest of the sixteen times a block's power of two."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    b = x.reshape(-1, 32)
    top = b.abs().max(1).values
    e = torch.full_like(top, -125)
    for i in range(-124, 126):  # as long as the largest is over 7 of the power before
        e = torch.where(top > 7 * 2.0 ** (i - 1), float(i), e)
        if bool((top <= 7 * 2.0 ** i).all()):
            break
    z = 2.0 ** e[:, None]
    out = torch.empty_like(b)
    for a in range(0, b.shape[0], 65536):
        part, zz = b[a:a + 65536], z[a:a + 65536]
        far = (part.abs() / zz)[..., None] - grid
        far = far.abs() + (torch.arange(8, device="cuda") % 2) * 1e-300  # the even code at a tie
        near = far.min(-1, keepdim=True).values
        even = ((far == near) & (torch.arange(8, device="cuda") % 2 == 0)).any(-1)
        odd_first = (far == near).float().argmax(-1)
        even_first = ((far == near) & (torch.arange(8, device="cuda") % 2 == 0)).float().argmax(-1)
        out[a:a + 65536] = grid[torch.where(even, even_first, odd_first)] * zz * torch.sign(part)
    return out.view(x.shape)


def exact(case, seed):
    op, f64 = case["op"], torch.float64
    if op in ("advance", "compact"):
        return None  # whole numbers and copies
    s = _inputs(case, seed)
    if op == "lora":
        y = torch.zeros(case["T"], case["N"], dtype=f64, device="cuda")
        for i in range(case["adapters"]):
            t = (s["ids"] == i).nonzero()[:, 0]
            y[t] = (s["x"][t].to(f64) @ s["a"][i].to(f64).t()) @ s["b"][i].to(f64).t() * s["scales"][i].to(f64)
        return y if s["base"] is None else y + s["base"].to(f64)
    if op == "logits":
        out = s["logits"].to(f64)
        for t in range(case["T"]):
            n, p = int(s["total"][t]), int(s["prompt"][t])
            x = out[t]
            seen = torch.unique(s["history"][t, :n].long())
            r = s["repetition"][t].to(f64)
            x[seen] = torch.where(x[seen] > 0, x[seen] / r, x[seen] * r)
            said, times = torch.unique(s["history"][t, p:n].long(), return_counts=True)
            x[said] -= times.to(f64) * s["frequency"][t].to(f64) + s["presence"][t].to(f64)
            lo, hi = int(s["bias_start"][t]), int(s["bias_start"][t + 1])
            x[s["bias_ids"][lo:hi].long()] += s["bias"][lo:hi].to(f64)
            if s["masks"] is not None and int(s["mask_rows"][t]) >= 0:
                words = s["masks"][int(s["mask_rows"][t])].long() & 0xffffffff
                keep = (words[:, None] // 2 ** torch.arange(32, device="cuda") % 2).flatten()[:case["V"]]
                x[keep == 0] = -math.inf
        return out
    if op == "append4":
        T, Hq, Hkv, D, rot = case["T"], case["heads"], case["kv_heads"], case["dim"], case["rot"]
        x = s["qkv"].to(f64).view(T, -1, D).clone()
        for lo, hi, w in ((0, Hq, s["q_norm"]), (Hq, Hq + Hkv, s["k_norm"])):
            if w is not None:
                part = x[:, lo:hi]
                x[:, lo:hi] = part / (part.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.to(f64)
        if rot:
            p = s["positions"].long()
            z = torch.complex(s["cos"].to(f64), s["sin"].to(f64))[p][:, None]
            i = torch.arange(rot // 2, device="cuda")
            u, v = (i, i + rot // 2) if case["style"] == "half" else (2 * i, 2 * i + 1)
            r = torch.complex(x[:, :Hq + Hkv][..., u], x[:, :Hq + Hkv][..., v]) * z
            x[:, :Hq + Hkv, u], x[:, :Hq + Hkv, v] = r.real, r.imag
        return dict(q=x[:, :Hq].reshape(T, -1), k=_codes(x[:, Hq:Hq + Hkv]).reshape(T, -1),
                    v=_codes(x[:, Hq + Hkv:]).reshape(T, -1), data=None)
    B, Hq, Hkv, D, page = case["B"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    out = torch.empty(B, Hq, D, dtype=f64, device="cuda")
    c, z = Hkv * page * D // 2, Hkv * page * D // 32
    grid = torch.tensor([m for x in E2M1 for m in (x,)] + [-x for x in E2M1], dtype=f64, device="cuda")

    def read(pg, base, scale, h):
        """Head h of the pages pg: [tokens][D] from bytes `base` on, with scales from `scale` on."""
        d = s["data"][pg]
        b = d[:, base + h * page * D // 2:base + (h + 1) * page * D // 2].reshape(-1, D // 2).long()
        x = torch.empty(b.shape[0], D, dtype=f64, device="cuda")
        x[:, 0::2], x[:, 1::2] = grid[b % 16], grid[b // 16]
        e = d[:, scale + h * page * D // 32:scale + (h + 1) * page * D // 32].reshape(len(pg), D // 32, page)
        return x * (2.0 ** (e.to(f64) - 127)).transpose(1, 2).reshape(-1, D // 32).repeat_interleave(32, 1)

    for b, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        pg = s["table"][b, :-(-n // page)].long()
        for h in range(Hkv):
            k, v = read(pg, 0, 2 * c, h)[lo:n], read(pg, c, 2 * c + z, h)[lo:n]
            rows = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = s["q"][b].view(Hq, D)[rows].to(f64) @ k.t() / math.sqrt(D)
            if case["sinks"]:  # one more score, whose value is zero
                x = torch.cat([x, s["sinks"][rows].to(f64)[:, None]], 1)
            p = torch.softmax(x, -1)
            out[b, rows] = p[:, :n - lo] @ v
    return out.view(B, Hq * D)
