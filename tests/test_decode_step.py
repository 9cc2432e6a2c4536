"""The example's decode step (examples/decode_step.py): every operator's output against its
plain 64-bit form on the inputs it had, over several steps, and the captured step against the
eager one."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(__file__))
sys.path.insert(0, os.path.join(os.path.dirname(__file__), "..", "examples"))

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import ops_ref as ref  # noqa: E402

SMALL = dict(batch=3, prefix=256, room=128, hidden=256, heads=8, kv_heads=2, dim=64, inter=128, experts=8, vocab=1000, page=32, top=4)


def _close(got, want, bound, what):
    over = (got.detach().cpu().double() - want).abs() - bound
    assert (over <= 0).all(), "%s: over its bound by %g" % (what, over.max())


@pytest.mark.parametrize("window", [0, 300])
def test_decode_step_operator_by_operator(window):
    from decode_step import DecodeStep, rms_norm
    s = DecodeStep(window=window, **SMALL)
    c = lambda t: t.detach().cpu()
    hidden = torch.randn(3, 256, generator=s.g, device="cuda").to(torch.bfloat16)
    tokens = torch.tensor([5, 0, 999], dtype=torch.int32, device="cuda")
    for _ in range(3):
        x, at = rms_norm(hidden), c(s.lens).clone()
        before_k = c(s.cache.k).clone()
        new = s.step(hidden, tokens)
        w, b = ref.linear(c(s.qkv_w.codes), c(s.qkv_w.scales), c(x))
        _close(s.qkv, w, b, "qkv")
        heads = c(s.qkv).view(3, 12, 64)
        t = s.transform
        cos, sin = c(t.cos)[at.long()][:, None], c(t.sin)[at.long()][:, None]
        w, b = ref.transform(heads[:, :8], c(t.q_norm), 1e-6, cos, sin, False)
        _close(s.q.view(3, 8, 64), w, b, "q")
        w, b = ref.transform(heads[:, 8:10], c(t.k_norm), 1e-6, cos, sin, False)
        page = c(s.table)[torch.arange(3), at.long() // 32].long()
        _close(s.cache.k[page.cuda(), :, at.cuda().long() % 32], w, b, "k")
        assert torch.equal(c(s.cache.v)[page, :, :, at.long() % 32], heads[:, 10:])
        before_k[page, :, at.long() % 32] = c(s.cache.k)[page, :, at.long() % 32]
        assert torch.equal(before_k, c(s.cache.k)), "other tokens' keys"
        w, b = ref.attn(c(s.q).view(3, 8, 64), c(s.cache.k), c(s.cache.v), c(s.table), at + 1, 64 ** -0.5, window, c(s.attn.sinks))
        _close(s.mixed.view(3, 8, 64), w, b, "attention")
        w, b = ref.linear(c(s.o_w.codes), c(s.o_w.scales), c(s.mixed), c(hidden))
        _close(s.after, w, b, "output projection")
        w, b = ref.linear(c(s.head_w.codes), c(s.head_w.scales), c(rms_norm(new)), bf16=False)
        _close(s.logits, w, b, "logits")
        wl, wh, wi, wt, bl, bh = ref.logprobs(c(s.logits), c(tokens), 4)
        _close(s.logprob, wl, bl, "logprob")
        _close(s.entropy, wh, bh, "entropy")
        _close(s.top_logprobs, wt, bl[:, None], "top")
        assert torch.equal(c(s.ids).long(), wi)
        hidden, tokens = new, s.ids[:, 0].contiguous()


def test_decode_step_captured():
    """A captured step replayed is the eager step: the same tokens, bit for bit, step after step."""
    from decode_step import DecodeStep
    eager, graphed = DecodeStep(**SMALL), DecodeStep(**SMALL)
    hidden = torch.randn(3, 256, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").to(torch.bfloat16)
    tokens = torch.zeros(3, dtype=torch.int32, device="cuda")
    h, t = hidden.clone(), tokens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm up away from the state that counts
        DecodeStep(**SMALL).step(h, t)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = graphed.step(h, t)
    for _ in range(4):
        want = eager.step(hidden, tokens)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((out, want), (graphed.ids, eager.ids), (graphed.logprob, eager.logprob), (graphed.cache.k, eager.cache.k),
                     (graphed.cache.v, eager.cache.v), (graphed.lens, eager.lens)):
            assert torch.equal(a, b)
        hidden, tokens = want, eager.ids[:, 0].contiguous()
        h.copy_(hidden)
        t.copy_(tokens)
