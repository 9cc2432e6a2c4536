"""The example's serving step (examples/serve_step.py): every operator's output against its plain
64-bit form on the inputs it had, over several steps with forks and sequences that end, and the
captured steps against the eager ones."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(__file__))
sys.path.insert(0, os.path.join(os.path.dirname(__file__), "..", "examples"))

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import ops_ref  # noqa: E402
import serve_ref as ref  # noqa: E402

BF, I32 = torch.bfloat16, torch.int32
SMALL = dict(rows=6, prompt=37, room=40, hidden=256, heads=8, kv_heads=2, dim=64, vocab=1000, page=16, adapters=3, rank=8, top=4, spare=3)


def c(t):
    return t.detach().cpu()


def _close(got, want, bound, what):
    over = (c(got).double() - want).abs() - bound
    assert (over <= 0).all(), "%s: over its bound by %g" % (what, over.max())


def _begin(**kw):
    from serve_step import ServeStep
    s = ServeStep(**{**SMALL, **kw})
    g = torch.Generator().manual_seed(5)
    tokens = torch.randint(0, 1000, (3, 37), generator=g).to(I32).cuda()
    s.prompts(tokens, torch.tensor([1, -1, 2], dtype=I32).cuda(), 2, torch.tensor([0, -1, 1], dtype=I32).cuda())
    return s


def _lists(st):
    n = st.n_free.item()
    return dict(refs=st.refs.tolist(), free=st.free_list.tolist()[:n], table=st.table.tolist(), lens=st.kv_len.tolist())


def _parents(s, i):
    """What the steps continue: all rows; a fork of one whose sibling ends; beams in another order."""
    s.parent.copy_(torch.tensor([[0, 1, 2, 3, 4, 5], [0, 0, 2, 3, 4, 5], [1, 0, 5, 5, 5, 2], [0, 1, 2, 3, 4, 5]][i % 4], dtype=I32))


@pytest.mark.parametrize("window", [0, 30])
def test_serve_step_operator_by_operator(window):
    s = _begin(window=window)
    from serve_step import rms_norm
    st = _lists(s.states[0])
    assert st["lens"] == [37] * 6 and [r for r in st["refs"] if r] == [2] * 9
    for i in range(6):
        _parents(s, i)
        turn = i % 2
        new = s.states[1 - turn]
        before, total = _lists(s.states[turn]), c(s.total)[c(s.parent).long()]
        of = c(s.parent).long()
        data, history = c(s.cache.data).clone(), c(s.history)[of]
        hidden = s.step(turn)
        # the tables, and the copied pages
        want = ref.advance(16, before, s.parent.tolist(), [1] * 6, 1)
        assert {k: want[k] for k in before} == _lists(new)
        assert s.slots.tolist() == want["slots"]
        for src, dst in want["copied"]:
            data[dst] = data[src]
        at = torch.tensor(want["lens"]) - 1
        # the projection with the adapters
        x = rms_norm(hidden)
        w, b = ops_ref.linear(c(s.qkv_w.codes), c(s.qkv_w.scales), c(x), bf16=False)
        _close(s.shared, w, b, "shared projection")
        w, b = ref.lora(c(x), c(s.adapter), c(s.qkv_a.a), c(s.qkv_a.b), None, c(s.qkv_a.scales), c(s.shared))
        _close(s.qkv, w, b, "qkv")
        # queries; the new tokens in the cache: half of a code's step from the key, and nothing else
        heads, t = c(s.qkv).view(6, 12, 64), s.transform
        cos, sin = c(t.cos)[at][:, None], c(t.sin)[at][:, None]
        w, b = ops_ref.transform(heads[:, :8], c(t.q_norm), 1e-6, cos, sin, False)
        _close(s.q.view(6, 8, 64), w, b, "q")
        page, off = torch.tensor([t[n // 16] for t, n in zip(want["table"], at.tolist())]), at % 16
        for name, codes, scales, x64 in (("k", s.cache.k_codes, s.cache.k_scales, ops_ref.transform(heads[:, 8:10], c(t.k_norm), 1e-6, cos, sin, False)[0]),
                                         ("v", s.cache.v_codes, s.cache.v_scales, heads[:, 10:].double())):
            got = ref.values(c(codes)[page], c(scales)[page])[torch.arange(6), :, off]
            top = torch.pow(2.0, c(scales)[page][torch.arange(6), :, :, off].double() - 127).repeat_interleave(32, -1)
            # a code's step is at most 2 (of 4 to 6) and 7 is the furthest from 6; the key's own error is far less
            assert ((got - x64).abs() <= 1.0001 * top).all(), name
        now = c(s.cache.data)
        rest = torch.ones(s.pool.n_pages, dtype=torch.bool)
        rest[page] = False
        assert torch.equal(now[rest], data[rest]), "other pages"
        # attention over the new tables
        k = ref.values(c(s.cache.k_codes), c(s.cache.k_scales))
        v = ref.values(c(s.cache.v_codes), c(s.cache.v_scales)).transpose(-1, -2).contiguous()
        w, b = ops_ref.attn(c(s.q).view(6, 8, 64), k, v, c(new.table), c(new.kv_len), 64 ** -0.5, window, c(s.attn.sinks))
        _close(s.mixed.view(6, 8, 64), w, b, "attention")
        # the output projection, rounded to bf16, with its adapters on top of that
        w, b = ops_ref.linear(c(s.o_w.codes), c(s.o_w.scales), c(s.mixed), c(hidden))
        wl, bl = ref.lora(c(s.mixed), c(s.adapter), c(s.o_a.a), c(s.o_a.b), None, c(s.o_a.scales), w)
        _close(s.after, wl, b * (1 + 2.0 ** -8) + bl, "output projection")
        w, b = ops_ref.linear(c(s.head_w.codes), c(s.head_w.scales), c(rms_norm(s.after)), bf16=False)
        _close(s.raw, w, b, "output layer")
        # rules and log probabilities
        h = s.rules.held
        w, b = ref.logits(c(s.raw), history, c(s.prompt_len), total, *(c(x) for x in h[3:]), bf16=False)
        inf = torch.isinf(w)
        assert torch.equal(torch.isinf(c(s.logits)), inf)
        _close(s.logits.nan_to_num(0, 0, 0), w.nan_to_num(0, 0, 0), b.nan_to_num(0, 0, 0), "rules")
        assert torch.equal(c(s.ids)[:, 0].long(), c(s.logits).argmax(-1))
        assert torch.equal(c(s.tokens), c(s.ids)[:, 0]) and torch.equal(c(s.history)[torch.arange(6), total.long()], c(s.tokens))


def test_serve_step_captured():
    """Two captured steps (one for each direction between the states) replayed by turns are the eager
    steps, bit for bit."""
    eager, graphed = _begin(), _begin()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm up away from the state that counts
        warm = _begin()
        warm.step(0)
        warm.step(1)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for turn in (0, 1):
        with torch.cuda.graph(graphs[turn]):
            graphed.step(turn)
    for i in range(8):
        for s in (eager, graphed):
            _parents(s, i)
        eager.step(i % 2)
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        a, b = eager.states[1 - i % 2], graphed.states[1 - i % 2]
        for name in ("refs", "free_list", "n_free", "table", "kv_len"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name
        for name in ("qkv", "mixed", "after", "logits", "logprob", "entropy", "ids", "tokens", "history", "total"):
            assert torch.equal(getattr(eager, name), getattr(graphed, name)), name
        assert torch.equal(eager.cache.data, graphed.cache.data)


def test_serve_step_compacts_between_steps():
    """Pages moved to the front between two steps change nothing that is said."""
    import sparse_moe_transformer_wave_amd as fm
    plain, moved = _begin(), _begin()
    for i in range(4):
        for s in (plain, moved):
            _parents(s, i)
            s.step(i % 2)
        state, other = moved.states[1 - i % 2], moved.states[i % 2]
        where = torch.empty(moved.pool.n_pages, dtype=I32, device="cuda")
        fm.kv_compact(moved.pool, state, other, where, moved.pages_ws)
        live = int((c(state.refs) > 0).sum())
        assert (c(other.refs)[:live] > 0).all() and int(c(other.refs)[live:].abs().sum()) == 0
        moved.states[0], moved.states[1] = (other, state) if (i + 1) % 2 == 0 else (state, other)
        for name in ("qkv", "mixed", "after", "logits", "ids"):
            assert torch.equal(getattr(plain, name), getattr(moved, name)), (i, name)


def test_serve_step_of_more_rows_than_a_linear_call_takes():
    """70 sequences: every projection goes through in pieces, and the last rows are as the others."""
    from serve_step import ServeStep, rms_norm
    s = ServeStep(**{**SMALL, "rows": 70, "spare": 70})
    g = torch.Generator().manual_seed(6)
    tokens = torch.randint(0, 1000, (35, 37), generator=g).to(I32).cuda()
    s.prompts(tokens, torch.arange(35, device="cuda", dtype=I32) % 4 - 1, 2)
    hidden = s.step(0)
    assert s.states[1].kv_len.tolist() == [38] * 70
    x = rms_norm(hidden)
    w, b = ops_ref.linear(c(s.qkv_w.codes), c(s.qkv_w.scales), c(x), bf16=False)
    _close(s.shared, w, b, "shared projection")
    w, b = ops_ref.linear(c(s.o_w.codes), c(s.o_w.scales), c(s.mixed), c(hidden))
    wl, bl = ref.lora(c(s.mixed), c(s.adapter), c(s.o_a.a), c(s.o_a.b), None, c(s.o_a.scales), w)
    _close(s.after, wl, b * (1 + 2.0 ** -8) + bl, "output projection")
    w, b = ops_ref.linear(c(s.head_w.codes), c(s.head_w.scales), c(rms_norm(s.after)), bf16=False)
    _close(s.raw, w, b, "output layer")


def test_serve_step_of_prompts_of_one_token():
    """The output projection's adapters are twice as wide as the first one's and need more workspace, which
    no long prompt covers here."""
    from serve_step import ServeStep
    s = ServeStep(rows=40, prompt=1, room=4, vocab=1000)
    tokens = torch.arange(40, device="cuda", dtype=I32)[:, None] * 20
    s.prompts(tokens, torch.arange(40, device="cuda", dtype=I32) % 4 - 1)
    s.step(0)
    s.step(1)
    assert s.states[0].kv_len.tolist() == [3] * 40 and torch.isfinite(s.entropy).all()


def test_serve_step_of_prompts_of_more_tokens_than_an_adapter_call_takes():
    """33 prompts of 2000 tokens: their adapters go through in pieces."""
    from serve_step import rms_norm, ServeStep
    s = ServeStep(**{**SMALL, "rows": 33, "prompt": 2000, "room": 2})
    g = torch.Generator().manual_seed(7)
    tokens = torch.randint(0, 1000, (33, 2000), generator=g).to(I32).cuda()
    adapter = torch.arange(33, device="cuda", dtype=I32) % 4 - 1
    s.prompts(tokens, adapter)
    x = rms_norm(s.embed[tokens.long().flatten()])
    qkv, ids = s.project(x, adapter.repeat_interleave(2000)), adapter.repeat_interleave(2000)
    at = torch.tensor([0, 1999, 65535, 65536, 65999])  # either side of a piece's end, and the ends
    shared, _ = ops_ref.linear(c(s.qkv_w.codes), c(s.qkv_w.scales), c(x)[at], bf16=False)
    w, b = ref.lora(c(x)[at], c(ids)[at], c(s.qkv_a.a), c(s.qkv_a.b), None, c(s.qkv_a.scales), shared)
    _, more = ops_ref.linear(c(s.qkv_w.codes), c(s.qkv_w.scales), c(x)[at], bf16=False)
    _close(qkv[at.cuda()], w, b + more * (1 + 2.0 ** -8), "qkv")
    s.step(0)
    assert s.states[1].kv_len.tolist() == [2001] * 33 and torch.isfinite(s.entropy).all()
