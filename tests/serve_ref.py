"""Plain 64-bit forms of the operators of include/flint_serve.h on the CPU, with the a-priori error
bounds that the GPU tests hold the kernels to (u = 2^-24, see ops_ref.py), and the page tables' next
step as a loop over rows."""
import math

import torch

from ops_ref import F64, U

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---- 4-bit cache -----------------------------------------------------------------------
def quantise(x):
    """(codes, scale bytes, values) of blocks of 32 of the last dimension, value by value."""
    x = x.to(F64)
    shape = x.shape
    codes, scales, values = [], [], []
    for block in x.reshape(-1, 32).tolist():
        if not all(math.isfinite(v) for v in block):
            codes += [0] * 32
            scales.append(255)
            values += [math.nan] * 32
            continue
        top, e = max(abs(v) for v in block), -125
        while e < 125 and top > 7 * 2.0 ** e:
            e += 1
        if top == 0:
            e = 0
        scales.append(e + 127)
        for v in block:
            y = abs(v) / 2.0 ** e
            near = min(range(8), key=lambda c: (abs(GRID[c] - y), c % 2))
            codes.append(near + (8 if math.copysign(1, v) < 0 else 0))
            values.append(math.copysign(GRID[near] * 2.0 ** e, v))
    return (torch.tensor(codes, dtype=torch.uint8).view(shape),
            torch.tensor(scales, dtype=torch.uint8).view(*shape[:-1], shape[-1] // 32), torch.tensor(values, dtype=F64).view(shape))


def values(codes, scales):
    """[page][head][token][D] from codes [page][head][token][D / 2] and scales [page][head][D / 32][token]."""
    grid = torch.tensor(GRID + [-v for v in GRID], dtype=F64)
    c = codes.long()
    x = torch.stack([grid[c & 15], grid[c >> 4]], -1).flatten(-2)
    z = torch.pow(torch.tensor(2.0, dtype=F64), scales.to(F64) - 127)
    z = torch.where(scales == 255, torch.full_like(z, math.nan), z)
    return x * z.transpose(-1, -2).repeat_interleave(32, -1)


# ---- pages -----------------------------------------------------------------------------
def _pages_of(n, page):
    return -(-n // page)


def advance(page, old, parent, grow, lds):
    """The next state as lists: old = dict(refs, free (n_free entries), table, lens).  Returns the new
    one with slots and the copied pages (src, dst)."""
    width, n_pages = len(old["table"][0]) if old["table"] else old["width"], len(old["refs"])
    lens = [min(max(n, 0), width * page) for n in old["lens"]]
    page_ok = lambda p: 0 <= p < n_pages  # noqa: E731
    parent = [p if 0 <= p < len(lens) else -1 for p in parent]
    grow = [max(g, 0) for g in grow]
    refs = list(old["refs"])
    for r, n in enumerate(lens):
        more = sum(p == r for p in parent) - 1
        for p in old["table"][r][:_pages_of(n, page)]:
            if page_ok(p):
                refs[p] += more
    stack = list(old["free"]) + [p for p in range(n_pages) if old["refs"][p] > 0 and refs[p] == 0]
    rows, needed, holders, sharers = [], 0, list(refs), {}
    for r, p in enumerate(parent):
        n = lens[p] if p >= 0 else 0
        fits = n + grow[r] <= width * page
        entries = list(old["table"][p][:_pages_of(n, page)]) if p >= 0 else []
        last = entries[-1] if n % page and grow[r] and fits and page_ok(entries[-1]) else None
        copies = keeps = False
        if last is not None:
            copies = holders[last] > 1
            keeps = not copies and sharers.get(last, 0) > 0
            sharers[last] = sharers.get(last, 0) + 1
            if copies:
                holders[last] -= 1
        want = _pages_of(n + grow[r], page) - _pages_of(n, page) + copies if fits else 0
        needed += want
        rows.append((n, entries, fits, copies, keeps, want, needed))
    have, copied, table, new_lens, slots = len(stack), [], [], [], []
    for r, (n, entries, fits, copies, keeps, want, end) in enumerate(rows):
        ok = fits and ((want == 0 and not keeps) or end <= have)
        if ok:
            fresh = [stack.pop() for _ in range(want)]
            for p in fresh:
                refs[p] = 1
            if copies:
                refs[entries[-1]] -= 1
                copied.append((entries[-1], fresh[0]))
                entries = entries[:-1]
            entries = entries + fresh
        add = grow[r] if ok else 0
        at = [(entries[j // page], j % page) for j in range(n, n + add)]
        slots.append(([p * page + o if page_ok(p) else -1 for p, o in at] + [-1] * lds)[:lds])
        table.append(entries + [-1] * (width - len(entries)))
        new_lens.append(n + add)
    return dict(refs=refs, free=stack, table=table, lens=new_lens, slots=slots, copied=copied)


def compact(page, old):
    """The state after the live pages have moved to the front, and moved."""
    refs, n_pages = old["refs"], len(old["refs"])
    live = [p for p in range(n_pages) if refs[p] > 0]
    n = len(live)
    holes = [p for p in range(n) if refs[p] <= 0]
    moved = [-1] * n_pages
    for p in live:
        moved[p] = p if p < n else holes.pop(0)
    new = [0] * n_pages
    for p in live:
        new[moved[p]] = refs[p]
    table, lens = [], []
    for row, length in zip(old["table"], old["lens"]):
        length = min(max(length, 0), len(row) * page)
        used = _pages_of(length, page)
        table.append([(moved[p] if 0 <= p < n_pages else p) if j < used else -1 for j, p in enumerate(row)])
        lens.append(length)
    return dict(refs=new, free=list(range(n_pages - 1, n - 1, -1)), table=table, lens=lens, moved=moved)


# ---- adapters --------------------------------------------------------------------------
def lora(x, ids, a, b, ranks=None, scales=None, base=None, bf16=True):
    """(y, bound): a token's K products are exact and summed in fp32 in any order, so are its rank's."""
    T, n, K, R = x.shape[0], a.shape[0], x.shape[1], a.shape[1]
    y = torch.zeros(T, b.shape[1], dtype=F64) if base is None else base.to(F64).clone()
    mag, low = y.abs(), torch.zeros_like(y)
    for i in range(n):
        t = (ids == i).nonzero()[:, 0]
        r = R if ranks is None else min(max(int(ranks[i]), 0), R)
        if len(t) == 0 or r == 0:
            continue
        s = 1.0 if scales is None else float(scales[i])
        ai, bi, xt = a[i, :r].to(F64), b[i, :, :r].to(F64), x[t].to(F64)
        y[t] += xt @ ai.t() @ bi.t() * s
        low[t] = xt.abs() @ ai.abs().t() @ bi.abs().t() * abs(s)
    # A x: K sums; its scale and three parts: 3 u; R products and sums; the base
    return y, (K + R + 16) * U * low + 2 * U * (mag + low) + (2.0 ** -8 * y.abs() if bf16 else 0)


# ---- logits ----------------------------------------------------------------------------
def logits(x, history=None, prompt_len=None, total_len=None, repetition=None, frequency=None, presence=None, bias_start=None,
           bias_ids=None, bias=None, masks=None, mask_rows=None, bf16=True):
    """(x', bound): at most six roundings to fp32 of numbers no larger than the magnitudes that are added up."""
    T, V = x.shape
    out, mag = x.to(F64).clone(), x.to(F64).abs()
    for t in range(T):
        if history is not None:
            L = history.shape[1]
            n = L if total_len is None else min(max(int(total_len[t]), 0), L)
            m = 0 if prompt_len is None else min(max(int(prompt_len[t]), 0), n)
            h = [v for v in history[t, :n].tolist()]
            own = {}
            for v in h[m:]:
                if 0 <= v < V:
                    own[v] = own.get(v, 0) + 1
            rep = 1.0 if repetition is None else float(repetition[t])
            f = 0.0 if frequency is None else float(frequency[t])
            p = 0.0 if presence is None else float(presence[t])
            for v in {v for v in h if 0 <= v < V}:
                y = float(out[t, v])
                y = y / rep if y > 0 else y * rep
                y = math.copysign(math.inf, y) if abs(y) >= 2.0 ** 128 - 2.0 ** 103 else y  # in fp32
                mag[t, v] = max(float(mag[t, v]), abs(y)) + (f * own[v] + abs(p) if v in own else 0)
                out[t, v] = y - f * own[v] - p if v in own else y
        if bias_start is not None:
            last = {}
            for i in range(max(int(bias_start[t]), 0), min(int(bias_start[t + 1]), len(bias_ids))):
                if 0 <= int(bias_ids[i]) < V:
                    last[int(bias_ids[i])] = float(bias[i])
            for v, add in last.items():
                out[t, v] += add
                mag[t, v] += abs(add)
        if masks is not None:
            m = t if mask_rows is None else int(mask_rows[t])
            if 0 <= m < masks.shape[0]:
                v = torch.arange(V)
                keep = (masks[m].long()[v // 32] >> (v % 32)) & 1 == 1
                out[t, ~keep] = -math.inf
    over = out.abs() >= 2.0 ** 128 - 2.0 ** (119 if bf16 else 103)  # rounds to an infinity
    out = torch.where(over, torch.copysign(torch.full_like(out, math.inf), out), out)
    mag = torch.where(torch.isfinite(out), mag, torch.zeros_like(mag))
    return out, 6 * U * mag + (2.0 ** -8 * out.abs().nan_to_num(0, 0, 0) if bf16 else 0)
