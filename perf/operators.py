"""Timed and compared cases of the decode-step operators around the MoE layer.

  linear     flint_linear_int4      a decode batch through a linear layer with 4-bit weights
  append     flint_kv_append        norm, rotation and the paged cache's new keys and values
  attn       flint_attn_decode      one query per sequence over the paged cache, shared prefix read once
  logprobs   flint_token_logprobs   log probabilities of given tokens, entropy, top alternatives

`own` selects the side: False runs the plain form (elementary torch operations in 32 bits,
rounded once), True the library's entry points.  Both sides get the same inputs.
"""
import math

import torch

own = False

HEADS, KV_HEADS, HEAD_DIM = 32, 4, 128  # the Flint model's attention heads
# (query heads, key heads) of the drawn cases: one head, shared by odd and even numbers of queries, wide
GROUPS = ((1, 1), (8, 1), (6, 2), (10, 2), (4, 4), (20, 4), (32, 4), (40, 8), (64, 8))


# ---- cases ---------------------------------------------------------------------------
def listed():
    lin = dict(op="linear", group=128, out="bf16", residual=False)
    app = dict(op="append", heads=HEADS, kv_heads=KV_HEADS, dim=HEAD_DIM, page=64, rot=128, style="half", norm=True)
    att = dict(op="attn", heads=HEADS, kv_heads=KV_HEADS, dim=HEAD_DIM, page=64, window=0, sinks=True)
    lp = dict(op="logprobs", masked=0.0)
    return [
        # one token through the attention output projection of the 2048-wide layer, residual added
        dict(lin, name="linear_t1_out_proj", T=1, K=4096, N=2048, residual=True),
        # eight requests through the fused query, key and value projection
        dict(lin, name="linear_t8_qkv", T=8, K=2048, N=5120),
        # one token through the output layer: fp32 logits of an odd vocabulary, groups of 64
        dict(lin, name="linear_t1_vocab", T=1, K=2048, N=130953, group=64, out="fp32"),
        # the new token of eight requests
        dict(app, name="append_t8", T=8, pages=1024),
        # a batch without rotation (the full-attention layers), 16-token pages
        dict(app, name="append_t97_norope", T=97, pages=4096, page=16, rot=0),
        # an 8192-token prompt
        dict(app, name="append_t8192", T=8192, pages=1024),
        # one request on a sliding-window layer: the smallest call, latency
        dict(att, name="attn_b1_window", B=1, prefix=0, suffix=700, window=513),
        # thirty-two requests that share a 32768-token prefix
        dict(att, name="attn_b32_shared_32k", B=32, prefix=32768, suffix=1000),
        # eight requests at 100K tokens, a 96K prefix shared
        dict(att, name="attn_b8_shared_96k", B=8, prefix=98304, suffix=4000),
        # the sampled token of one request and its alternatives
        dict(lp, name="logprobs_t1", T=1, V=130953, dtype="fp32", top=20),
        # a decode batch under a grammar that masks most of the vocabulary
        dict(lp, name="logprobs_t32_masked", T=32, V=32001, dtype="bf16", top=5, masked=0.9),
        # the tokens of a scored prompt
        dict(lp, name="logprobs_t1024", T=1024, V=131072, dtype="bf16", top=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "append", "attn", "logprobs"])
    if op == "linear":
        K = 128 * (2 * _log(rng, 1, 32) + 1)  # blocks that split unevenly over waves
        N = _log(rng, 16, min(131072, 268000000 // K))
        out = rng.choice(["bf16", "fp32"])
        return dict(op=op, T=_log(rng, 1, 64), K=K, N=N, group=rng.choice([32, 64, 128]), out=out,
                    residual=rng.random() < 0.4)
    if op == "append":
        (heads, kv), dim = rng.choice(GROUPS), rng.choice([64, 128])
        page = rng.choice([16, 32, 64, 128])
        T = _log(rng, 1, min(8192, 8192 * 40 * 128 // ((heads + 2 * kv) * dim)))
        return dict(op=op, T=T, heads=heads, kv_heads=kv, dim=dim, page=page,
                    pages=(2 * T + 4096) // page + 8, rot=rng.choice([0, dim // 2, dim]),
                    style=rng.choice(["half", "pairs"]), norm=rng.random() < 0.6)
    if op == "attn":
        (heads, kv), dim = rng.choice(GROUPS), rng.choice([64, 128])
        page = rng.choice([16, 32, 64, 128])
        B = _log(rng, 1, 128)
        most = 3200000 // (B * kv)  # keys of one sequence: the plain form gathers them all
        prefix = rng.choice([0, 1]) * _log(rng, 256, 98304)
        prefix = min(prefix, most // 2) // page * page
        return dict(op=op, B=B, heads=heads, kv_heads=kv, dim=dim, page=page, prefix=prefix,
                    suffix=min(_log(rng, 1, 8192), most // 2), window=rng.choice([0, 0, 513]),
                    sinks=rng.random() < 0.5)
    T = _log(rng, 1, 1024)
    V = _log(rng, 1000, min(200000, 134000000 // T))
    return dict(op=op, T=T, V=V, dtype=rng.choice(["bf16", "fp32"]), top=rng.choice([0, 1, 5, 20, 32]),
                masked=rng.choice([0.0, 0.0, 0.5, 0.9]))


# ---- inputs --------------------------------------------------------------------------
def _lengths(case, seed):
    """Tokens of each sequence: the shared prefix and a suffix of 1 ... suffix, ragged; the
    first has the longest."""
    g = torch.Generator().manual_seed(seed)
    own_part = torch.randint(1, case["suffix"] + 1, (case["B"],), generator=g)
    own_part[0] = case["suffix"]
    return case["prefix"] + own_part


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    op = case["op"]
    if op == "linear":
        T, K, N, G = case["T"], case["K"], case["N"], case["group"]
        return dict(x=normal(T, K),
                    codes=torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
                    scales=((torch.rand(N, K // G, generator=g, device="cuda") + 0.5) * (0.02 / 4)).to(torch.bfloat16),
                    residual=normal(T, N) if case["residual"] else None,
                    y=torch.empty(T, N, device="cuda", dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32))
    if op == "append":
        T, D, page, pages = case["T"], case["dim"], case["page"], case["pages"]
        Hq, Hkv, rot = case["heads"], case["kv_heads"], case["rot"]
        k = normal(pages, Hkv, page, D)
        v = normal(pages, Hkv, D, page)
        if T > 256:  # a prompt: consecutive tokens on pages of its own, from the middle of one
            order = torch.randperm(pages, generator=g, device="cuda")
            at = page // 2 - 1 + torch.arange(T, device="cuda")
            slots = order[at // page] * page + at % page
            positions = at.to(torch.int32)
        else:  # the new token of T requests
            slots = torch.randperm(pages, generator=g, device="cuda")[:T] * page
            slots = slots + torch.randint(0, page, (T,), generator=g, device="cuda")
            positions = torch.randint(0, 16384, (T,), generator=g, device="cuda", dtype=torch.int32)
        cos = sin = None
        if rot:
            f = 500000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") * 2 / rot)
            a = torch.arange(16384, dtype=torch.float64, device="cuda")[:, None] * f
            cos, sin = a.cos().float(), a.sin().float()
        qn = normal(D, std=0.1) + 1 if case["norm"] else None
        kn = normal(D, std=0.1) + 1 if case["norm"] else None
        return dict(k=k, v=v, qkv=normal(T, (Hq + 2 * Hkv) * D), slots=slots.to(torch.int64), positions=positions,
                    cos=cos, sin=sin, q_norm=qn, k_norm=kn,
                    q=torch.empty(T, Hq * D, device="cuda", dtype=torch.bfloat16))
    if op == "attn":
        B, D, page = case["B"], case["dim"], case["page"]
        Hq, Hkv = case["heads"], case["kv_heads"]
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
        return dict(k=normal(pages, Hkv, page, D), v=normal(pages, Hkv, D, page), table=table,
                    lens=lens.to(torch.int32).cuda(), q=normal(B, Hq * D, std=2.0),
                    sinks=normal(Hq, dtype=torch.float32) if case["sinks"] else None,
                    out=torch.empty(B, Hq * D, device="cuda", dtype=torch.bfloat16))
    T, V, n = case["T"], case["V"], case["top"]
    x = normal(T, V, std=3.0, dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    if case["masked"]:
        off = torch.rand(T, V, generator=g, device="cuda") < case["masked"]
        off.scatter_(1, tokens.long()[:, None], False)
        x.masked_fill_(off, -math.inf)
    f32 = dict(device="cuda", dtype=torch.float32)
    return dict(logits=x, tokens=tokens, logprob=torch.empty(T, **f32), entropy=torch.empty(T, **f32),
                top_ids=torch.empty(T, n, device="cuda", dtype=torch.int32), top_logprobs=torch.empty(T, n, **f32))


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own:  # the descriptors and the workspace that a program makes once
        import sparse_moe_transformer_wave_amd as fm

        op = case["op"]
        if op == "linear":
            state["plan"] = fm.Int4Linear(state["codes"], state["scales"])
        elif op == "append":
            state["plan"] = (fm.KVCache(state["k"], state["v"], case["heads"]),
                             fm.QKTransform(state["q_norm"], state["k_norm"], 1e-6, state["cos"], state["sin"],
                                            case["style"] == "pairs"))
        elif op == "attn":
            cache = fm.KVCache(state["k"], state["v"], case["heads"])
            state["plan"] = (cache, fm.AttnDecode(case["dim"] ** -0.5, case["window"], state["sinks"]))
            state["ws"] = fm.attn_decode_workspace(cache, case["B"])
        else:
            state["ws"] = fm.token_logprobs_workspace(case["T"], case["V"], case["top"])
    return state


# ---- plain forms -----------------------------------------------------------------------
def _linear(s):
    K, G = s["case"]["K"], s["case"]["group"]
    N = s["codes"].shape[0]
    lo = (s["codes"] & 15).to(torch.int8)
    hi = (s["codes"] >> 4).to(torch.int8)
    q = torch.stack([lo, hi], -1).view(N, K)  # the even column in the low nibble
    q = torch.where(q > 7, q - 16, q).float()
    w = (q.view(N, K // G, G) * s["scales"].float()[:, :, None]).view(N, K)
    y = s["x"].float() @ w.t()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["y"].dtype)


def _norm(x, w, eps=1e-6):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(x.dtype)


def _rotate(x, cos, sin, style):
    rot = 2 * cos.shape[-1]
    a, rest = x[..., :rot], x[..., rot:]
    c, s = cos[:, None], sin[:, None]
    if style == "half":
        u, v = a[..., :rot // 2], a[..., rot // 2:]
        a = torch.cat([u * c - v * s, v * c + u * s], -1)
    else:
        u, v = a[..., 0::2], a[..., 1::2]
        a = torch.stack([u * c - v * s, v * c + u * s], -1).flatten(-2)
    return torch.cat([a, rest], -1)


def _split(s, dtype):
    case = s["case"]
    T, Hq, Hkv, D = case["T"], case["heads"], case["kv_heads"], case["dim"]
    x = s["qkv"].view(T, Hq + 2 * Hkv, D)
    q, k = x[:, :Hq].to(dtype), x[:, Hq:Hq + Hkv].to(dtype)
    if case["norm"]:
        q, k = _norm(q, s["q_norm"]), _norm(k, s["k_norm"])
    return q, k, x[:, Hq + Hkv:]


def _append(s):
    case = s["case"]
    q, k, v = _split(s, torch.float32)
    if case["rot"]:
        c, n = s["cos"][s["positions"].long()], s["sin"][s["positions"].long()]
        q, k = _rotate(q, c, n, case["style"]), _rotate(k, c, n, case["style"])
    page, off = s["slots"] // case["page"], s["slots"] % case["page"]
    s["k"][page, :, off] = k.to(torch.bfloat16)
    s["v"][page, :, :, off] = v
    return dict(q=q.flatten(1).to(torch.bfloat16), k=s["k"], v=s["v"])


def _attn(s):
    case = s["case"]
    B, Hq, Hkv, D = case["B"], case["heads"], case["kv_heads"], case["dim"]
    table = s["table"].long()
    L = table.shape[1] * case["page"]
    k = s["k"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D).float()
    v = s["v"][table].permute(0, 2, 1, 4, 3).reshape(B, Hkv, L, D).float()
    q = s["q"].view(B, Hkv, Hq // Hkv, D).float()
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()) * D ** -0.5
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
    return (torch.matmul(p, v) / l).reshape(B, Hq * D).to(torch.bfloat16)


def _logprobs(s):
    x, V, n = s["logits"].float(), s["case"]["V"], s["case"]["top"]
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    lse = m + torch.log(z)
    logprob = (x.gather(1, s["tokens"].long()[:, None]) - lse)[:, 0]
    entropy = torch.log(z)[:, 0] - (torch.where(e > 0, e * (x - m), 0.0).sum(-1) / z[:, 0])
    # a key that falls with the value and, among equal values, with the index
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits + 2 ** 31), bits) * 2 ** 20 - torch.arange(V, device="cuda")
    ids = key.topk(n, -1).indices if n else torch.empty(x.shape[0], 0, device="cuda", dtype=torch.int64)
    return dict(logprob=logprob, entropy=entropy, top_ids=ids.int(), top_logprobs=x.gather(1, ids) - lse)


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"linear": _linear, "append": _append, "attn": _attn, "logprobs": _logprobs}[op](s)
    import sparse_moe_transformer_wave_amd as fm

    if op == "linear":
        fm.linear_int4(s["plan"], s["x"], s["y"], s["residual"])
        return s["y"]
    if op == "append":
        cache, transform = s["plan"]
        fm.kv_append(cache, transform, s["qkv"], s["positions"], s["slots"], s["q"])
        return dict(q=s["q"], k=s["k"], v=s["v"])
    if op == "attn":
        cache, attn = s["plan"]
        fm.attn_decode(cache, attn, s["q"], s["table"], s["lens"], s["case"]["prefix"], s["out"], s["ws"])
        return s["out"]
    fm.token_logprobs(s["logits"], s["tokens"], s["logprob"], s["entropy"], s["top_ids"], s["top_logprobs"], s["ws"])
    return dict(logprob=s["logprob"], entropy=s["entropy"], top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])


# ---- what a pass cannot do without -------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        out = T * N * ((2 if case["out"] == "bf16" else 4) + (2 if case["residual"] else 0))
        return dict(bytes=N * K // 2 + 2 * N * (K // case["group"]) + 2 * T * K + out, flops=2 * T * N * K)
    if op == "append":
        T, width = case["T"], (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        rows = 4 * T * case["rot"]  # the positions' cosines and sines, fp32
        return dict(bytes=4 * T * width + rows + 12 * T, flops=6 * T * width)
    if op == "attn":
        B, kv, D = case["B"], case["kv_heads"], case["dim"]
        tail = case["suffix"] + (B - 1) * (case["suffix"] + 1) / 2  # the mean of the ragged suffixes
        unique, seen = case["prefix"] + tail, B * case["prefix"] + tail
        if case["window"]:
            unique = seen = min(seen, B * case["window"])
        return dict(bytes=4 * unique * kv * D + 4 * B * case["heads"] * D, flops=4 * seen * case["heads"] * D)
    T, V, n = case["T"], case["V"], case["top"]
    return dict(bytes=T * V * (2 if case["dtype"] == "bf16" else 4) + T * (12 + 8 * n), flops=5 * T * V)


# ---- 64 bits -----------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "linear":
        c = s["codes"].to(torch.int32)
        N, K, G = case["N"], case["K"], case["group"]
        out = torch.empty(case["T"], N, dtype=f64, device="cuda")
        x = s["x"].to(f64)
        for a in range(0, N, 16384):  # rows at a time: 64-bit weights are large
            part, sc = c[a:a + 16384], s["scales"][a:a + 16384].to(f64)
            w = torch.empty(part.shape[0], K, dtype=f64, device="cuda")
            w[:, 0::2] = (((part & 15) ^ 8) - 8).to(f64)
            w[:, 1::2] = (((part >> 4) ^ 8) - 8).to(f64)
            w *= sc.repeat_interleave(G, 1)
            out[:, a:a + 16384] = x @ w.t()
        return out if s["residual"] is None else out + s["residual"].to(f64)
    if op == "append":
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
        k, v = s["k"].to(f64), s["v"].to(f64)
        at = s["slots"].tolist()
        if T > 256:
            pg, off = s["slots"] // case["page"], s["slots"] % case["page"]
            k.transpose(1, 2)[pg, off] = x[:, Hq:Hq + Hkv]
            v.permute(0, 3, 1, 2)[pg, off] = x[:, Hq + Hkv:]
        else:
            for t, slot in enumerate(at):
                pg, off = divmod(slot, case["page"])
                k[pg, :, off], v[pg, :, :, off] = x[t, Hq:Hq + Hkv], x[t, Hq + Hkv:]
        return dict(q=x[:, :Hq].reshape(T, -1), k=k, v=v)
    if op == "attn":
        B, Hq, Hkv, D = case["B"], case["heads"], case["kv_heads"], case["dim"]
        out = torch.empty(B, Hq, D, dtype=f64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            lo = max(0, n - case["window"]) if case["window"] else 0
            pg = s["table"][b, :-(-n // case["page"])].long()
            for h in range(Hkv):
                k = s["k"][pg, h].reshape(-1, D)[lo:n].to(f64)
                v = s["v"][pg, h].transpose(1, 2).reshape(-1, D)[lo:n].to(f64)
                rows = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                x = s["q"][b].view(Hq, D)[rows].to(f64) @ k.t() / math.sqrt(D)
                if case["sinks"]:  # one more score, whose value is zero
                    x = torch.cat([x, s["sinks"][rows].to(f64)[:, None]], 1)
                p = torch.softmax(x, -1)
                out[b, rows] = p[:, :n - lo] @ v
        return out.view(B, Hq * D)
    T, n = case["T"], case["top"]
    res = dict(logprob=[], entropy=[], top_logprobs=[])
    for t in range(T):
        x = s["logits"][t].to(f64)
        lp = torch.log_softmax(x, 0)
        fin = lp[lp > -math.inf]
        res["logprob"].append(lp[s["tokens"][t].long()])
        res["entropy"].append(-(fin.exp() * fin).sum())
        res["top_logprobs"].append(lp.sort(descending=True).values[:n])
    res = {name: torch.stack(v) for name, v in res.items()}
    return dict(res, top_ids=None)
