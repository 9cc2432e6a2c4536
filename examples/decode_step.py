"""A decode step of one transformer layer and the output layer, from this library's operators.

    hidden -> norm -> 4-bit qkv projection -> append (norm, rotation, paged cache)
           -> attention over the cache, the batch's shared prefix read once
           -> 4-bit output projection + residual -> norm -> sparse MoE layer + residual
           -> 4-bit output layer -> log probabilities of the chosen tokens, entropy, alternatives

Random weights of the Flint model's attention shape (32 query and 4 key/value heads of 128, a
2048-wide hidden state); only the norms and residual sums between the operators are torch's.
Run:  python examples/decode_step.py [--batch 8] [--prefix 4096] [--steps 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import sparse_moe_transformer_wave_amd as fm  # noqa: E402

BF = torch.bfloat16


def rms_norm(x, eps=1e-6):
    x = x.float()
    return (x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + eps)).to(BF)


class DecodeStep:
    """Weights, cache and buffers of a batch that shares a prefix; step() makes one token each."""

    def __init__(self, batch=8, prefix=4096, room=256, hidden=2048, heads=32, kv_heads=4, dim=128, inter=768,
                 experts=32, vocab=32000, page=64, top=5, window=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.batch, self.prefix, self.top = g, batch, prefix // page * page, top

        def int4(out, inp):
            codes = torch.randint(0, 256, (out, inp // 2), generator=g, device="cuda", dtype=torch.uint8)
            scales = torch.full((out, inp // 128), 0.2 / inp ** 0.5, device="cuda", dtype=BF)
            return fm.Int4Linear(codes, scales)

        def normal(*shape, std=1.0, dtype=BF):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

        # projections and the output layer
        self.qkv_w, self.o_w, self.head_w = int4((heads + 2 * kv_heads) * dim, hidden), int4(hidden, heads * dim), int4(vocab, hidden)
        # the prefix's pages, shared, and each sequence's own
        shared, own = self.prefix // page, -(-room // page)
        pages = shared + batch * own
        self.cache = fm.KVCache(normal(pages, kv_heads, page, dim), normal(pages, kv_heads, dim, page), heads)
        order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
        self.table = torch.cat([order[:shared].expand(batch, shared), order[shared:].view(batch, own)], 1).contiguous()
        self.page, self.room = page, own * page
        # rotary angles, norms, sinks
        top_pos = self.prefix + self.room
        f = 500000.0 ** (-torch.arange(dim // 2, dtype=torch.float64, device="cuda") * 2 / dim)
        a = torch.arange(top_pos, dtype=torch.float64, device="cuda")[:, None] * f
        self.transform = fm.QKTransform(normal(dim, std=0.1) + 1, normal(dim, std=0.1) + 1, 1e-6, a.cos().float(), a.sin().float())
        self.attn = fm.AttnDecode(dim ** -0.5, window, normal(heads, dtype=torch.float32))
        self.attn_ws = fm.attn_decode_workspace(self.cache, batch)
        # the MoE layer
        self.desc = fm.desc(hidden, inter, n_experts=experts, top_k=min(6, experts))
        bits = lambda *s: normal(*s, std=0.02).view(torch.int16)
        self.moe = fm.Weights(fm.WFMT_BF16, bits(experts, inter, hidden), bits(experts, inter, hidden), bits(experts, hidden, inter),
                              bits(1, inter, hidden), bits(1, inter, hidden), bits(1, hidden, inter))
        self.router, self.moe_ws = normal(experts, hidden, std=0.02, dtype=torch.float32), fm.workspace(self.desc, batch)
        # state and buffers
        e = lambda *s, dtype=BF: torch.empty(*s, device="cuda", dtype=dtype)
        self.lens = torch.full((batch,), self.prefix, device="cuda", dtype=torch.int32)  # tokens already in the cache
        self.qkv, self.q, self.mixed, self.after = e(batch, (heads + 2 * kv_heads) * dim), e(batch, heads * dim), e(batch, heads * dim), e(batch, hidden)
        self.moe_out = e(batch, hidden, dtype=torch.int16)
        self.logits = e(batch, vocab, dtype=torch.float32)
        self.logprob, self.entropy = e(batch, dtype=torch.float32), e(batch, dtype=torch.float32)
        self.ids, self.top_logprobs = e(batch, top, dtype=torch.int32), e(batch, top, dtype=torch.float32)
        self.lp_ws = fm.token_logprobs_workspace(batch, vocab, top)
        self.rows = torch.arange(batch, device="cuda")

    def step(self, hidden, tokens):
        """hidden: bf16 [batch][hidden] of the new token; tokens: int32 [batch], whose log
        probabilities are wanted.  Advances the cache by one token; returns the new hidden state."""
        positions = self.lens
        page = self.table[self.rows, torch.div(positions, self.page, rounding_mode="floor").long()].long()
        slots = page * self.page + positions % self.page
        fm.linear_int4(self.qkv_w, rms_norm(hidden), self.qkv)
        fm.kv_append(self.cache, self.transform, self.qkv, positions, slots, self.q)
        self.lens += 1
        fm.attn_decode(self.cache, self.attn, self.q, self.table, self.lens, self.prefix, self.mixed, self.attn_ws)
        fm.linear_int4(self.o_w, self.mixed, self.after, hidden)
        x = rms_norm(self.after)
        fm.layer(self.desc, self.moe, self.batch, x.view(torch.int16), self.router, None, self.moe_out, self.moe_ws)
        out = (self.after.float() + self.moe_out.view(BF).float()).to(BF)
        fm.linear_int4(self.head_w, rms_norm(out), self.logits)
        fm.token_logprobs(self.logits, tokens, self.logprob, self.entropy, self.ids, self.top_logprobs, self.lp_ws)
        return out


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--prefix", type=int, default=4096)
    p.add_argument("--steps", type=int, default=4)
    a = p.parse_args()
    s = DecodeStep(a.batch, a.prefix)
    hidden = torch.randn(a.batch, 2048, generator=s.g, device="cuda").to(BF)
    tokens = torch.zeros(a.batch, device="cuda", dtype=torch.int32)
    for i in range(min(a.steps, s.room)):
        hidden = s.step(hidden, tokens)
        print("step %d: first sequence: token %d has log probability %.3f, entropy %.3f, best %s" % (
            i, tokens[0].item(), s.logprob[0].item(), s.entropy[0].item(), s.ids[0].tolist()))
        tokens = s.ids[:, 0].contiguous()
    assert fm.workspace_status(s.moe_ws) == 0


if __name__ == "__main__":
    main()
