"""A decode step of a server with many requests: one attention layer and the output layer, each
request with an adapter of its own, a cache in 4 bits, and rules on what may be said next.

    page tables: continue, fork or end sequences, room for a token, copy on write
           -> norm -> 4-bit qkv projection + the requests' adapters
           -> append to the 4-bit paged cache -> attention over it
           -> 4-bit output projection + residual + the requests' adapters
           -> 4-bit output layer -> penalties, biases, grammar masks
           -> log probabilities, entropy, the best tokens

Random weights of the Flint model's attention shape (32 query and 4 key/value heads of 128, a
2048-wide hidden state); the norms, the history of tokens and the next tokens' embeddings are
torch's.
Run:  python examples/serve_step.py [--requests 4] [--samples 2] [--prompt 300] [--steps 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import sparse_moe_transformer_wave_amd as fm  # noqa: E402

BF, I32 = torch.bfloat16, torch.int32
LORA_TOKENS = 65536  # of a call at most


def linear(w, x, y, residual=None):
    """fm.linear_int4 for any number of rows: a call takes up to 64."""
    for t in range(0, x.shape[0], 64):
        fm.linear_int4(w, x[t:t + 64], y[t:t + 64], None if residual is None else residual[t:t + 64])


def rms_norm(x, eps=1e-6):
    x = x.float()
    return (x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + eps)).to(BF)


class ServeStep:
    """Weights, cache and buffers of up to `rows` sequences; prompts() begins them, step() makes one
    token each."""

    def __init__(self, rows=8, prompt=300, room=64, hidden=2048, heads=32, kv_heads=4, dim=128, vocab=32000, page=64, adapters=3,
                 rank=16, top=5, window=0, spare=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.rows, self.heads, self.kv_heads, self.dim, self.vocab = g, rows, heads, kv_heads, dim, vocab

        def int4(out, inp):
            codes = torch.randint(0, 256, (out, inp // 2), generator=g, device="cuda", dtype=torch.uint8)
            return fm.Int4Linear(codes, torch.full((out, inp // 128), 0.2 / inp ** 0.5, device="cuda", dtype=BF))

        def normal(*shape, std=1.0, dtype=BF):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

        def adapter(out, inp):
            scales = torch.linspace(0.5, 1, adapters, device="cuda")
            return fm.LoraAdapters(normal(adapters, rank, inp, std=inp ** -0.5), normal(adapters, out, rank, std=rank ** -0.5), scales=scales)

        width = (heads + 2 * kv_heads) * dim
        self.qkv_w, self.o_w, self.head_w = int4(width, hidden), int4(hidden, heads * dim), int4(vocab, hidden)
        self.qkv_a, self.o_a = adapter(width, hidden), adapter(hidden, heads * dim)
        self.embed = normal(vocab, hidden)
        # a pool with room for every sequence's own pages, and who holds them, now and next
        per_row = -(-(prompt + room) // page)
        pages = rows * per_row + spare
        self.cache = fm.KV4Cache(torch.zeros(pages, fm.KV4Cache.page_bytes(kv_heads, dim, page), device="cuda", dtype=torch.uint8),
                                 heads, kv_heads, dim, page)
        self.pool = fm.KVPages([self.cache])
        self.states = [fm.kv_state(pages, rows, per_row), fm.kv_state(pages, rows, per_row)]
        self.pages_ws = fm.kv_pages_workspace(self.pool, rows)
        # rotary angles and norms
        f = 500000.0 ** (-torch.arange(dim // 2, dtype=torch.float64, device="cuda") * 2 / dim)
        a = torch.arange(prompt + room, dtype=torch.float64, device="cuda")[:, None] * f
        self.transform = fm.QKTransform(normal(dim, std=0.1) + 1, normal(dim, std=0.1) + 1, 1e-6, a.cos().float(), a.sin().float())
        self.attn = fm.AttnDecode(dim ** -0.5, window, normal(heads, dtype=torch.float32))
        self.attn_ws = fm.kv4_attn_decode_workspace(self.cache, rows)
        # for the prompts' tokens at one projection, for a step's rows at both: the wider one's needs may be the larger
        self.lora_ws = max(fm.lora_workspace(self.qkv_a, min(rows * prompt, LORA_TOKENS)), fm.lora_workspace(self.o_a, rows), key=lambda w: w.nbytes)
        # what may be said next: each sequence's history, two biased tokens, and a grammar's masks
        e = lambda *s, dtype=BF: torch.zeros(*s, device="cuda", dtype=dtype)  # noqa: E731
        self.history, self.total, self.prompt_len = e(rows, prompt + room, dtype=I32), e(rows, dtype=I32), e(rows, dtype=I32)
        self.mask_rows = e(rows, dtype=I32) - 1
        self.masks = torch.randint(-2 ** 31, 2 ** 31, (2, -(-vocab // 32)), generator=g, device="cuda").to(I32)
        one = torch.ones(rows, device="cuda")
        self.rules = fm.LogitRules(
            history=self.history, prompt_len=self.prompt_len, total_len=self.total, repetition=one * 1.2, frequency=one * 0.1,
            presence=one * 0.2, bias_start=torch.arange(rows + 1, device="cuda", dtype=I32) * 2,
            bias_ids=torch.tensor([0, 1], device="cuda", dtype=I32).repeat(rows), bias=torch.tensor([-4.0, 1.0], device="cuda").repeat(rows),
            masks=self.masks, mask_rows=self.mask_rows)
        # buffers of a step
        self.adapter = e(rows, dtype=I32) - 1
        self.parent, self.grow, self.slots = torch.arange(rows, device="cuda", dtype=I32), e(rows, dtype=I32) + 1, e(rows, 1, dtype=torch.int64)
        self.shared, self.qkv = e(rows, width, dtype=torch.float32), e(rows, width)
        self.q, self.mixed, self.after = e(rows, heads * dim), e(rows, heads * dim), e(rows, hidden)
        self.raw, self.logits = e(rows, vocab, dtype=torch.float32), e(rows, vocab, dtype=torch.float32)
        self.tokens, self.logprob, self.entropy = e(rows, dtype=I32), e(rows, dtype=torch.float32), e(rows, dtype=torch.float32)
        self.ids, self.top_logprobs = e(rows, top, dtype=I32), e(rows, top, dtype=torch.float32)
        self.lp_ws = fm.token_logprobs_workspace(rows, vocab, top)

    def project(self, x, ids):
        """The qkv projection of a prompt's or a step's tokens, with their adapters."""
        T = x.shape[0]
        shared = self.shared if T == self.rows else torch.empty(T, self.shared.shape[1], device="cuda")
        linear(self.qkv_w, x, shared)
        qkv = self.qkv if T == self.rows else torch.empty(T, self.qkv.shape[1], device="cuda", dtype=BF)
        for t in range(0, T, LORA_TOKENS):
            part = slice(t, t + LORA_TOKENS)
            fm.lora(self.qkv_a, x[part], ids[part], shared[part], qkv[part], self.lora_ws)
        return qkv

    def prompts(self, tokens, adapter, samples=1, masks=None):
        """Begins sequences: tokens int32 [requests][n], adapter int32 [requests]; then each request's
        `samples` rows share its pages."""
        R, n = tokens.shape
        grow = torch.zeros(self.rows, device="cuda", dtype=I32)
        grow[:R] = n
        slots = torch.empty(self.rows, n, device="cuda", dtype=torch.int64)
        fm.kv_advance(self.pool, self.states[0], self.states[1], torch.full_like(grow, -1), grow, slots, self.pages_ws)
        x = rms_norm(self.embed[tokens.long().flatten()])
        qkv = self.project(x, adapter.repeat_interleave(n))
        positions = torch.arange(n, device="cuda", dtype=I32).repeat(R)
        fm.kv4_append(self.cache, self.transform, qkv, positions, slots[:R].flatten(), torch.empty(R * n, self.heads * self.dim, device="cuda", dtype=BF))
        # the fork: no page is copied until a row writes to one that others hold
        of = torch.arange(self.rows, device="cuda") // samples
        parent = torch.where(of < R, of, -1).to(I32)
        fm.kv_advance(self.pool, self.states[1], self.states[0], parent, torch.zeros_like(grow), None, self.pages_ws)
        live, of = of < R, of.clamp(max=R - 1)
        self.history[:, :n] = torch.where(live[:, None], tokens[of], 0)
        self.total.copy_(live * n)
        self.prompt_len.copy_(self.total)
        self.adapter.copy_(torch.where(live, adapter[of], -1))
        if masks is not None:
            self.mask_rows.copy_(masks[of])
        self.tokens.copy_(tokens[of, -1])

    def step(self, turn):
        """A token for every row: row r goes on from row parent[r] (itself unless that is changed) with
        tokens[r].  turn: 0, 1, 0, ... by turns, the state that is read."""
        old, new = self.states[turn], self.states[1 - turn]
        of = self.parent.long().clamp(min=0)
        for t in (self.history, self.total, self.prompt_len, self.adapter, self.mask_rows):
            t.copy_(t[of])
        fm.kv_advance(self.pool, old, new, self.parent, self.grow, self.slots, self.pages_ws)
        hidden = self.embed[self.tokens.long()]
        positions = new.kv_len - 1
        qkv = self.project(rms_norm(hidden), self.adapter)
        fm.kv4_append(self.cache, self.transform, qkv, positions, self.slots.view(-1), self.q)
        fm.kv4_attn_decode(self.cache, self.attn, self.q, new.table, new.kv_len, 0, self.mixed, self.attn_ws)
        linear(self.o_w, self.mixed, self.after, hidden)
        fm.lora(self.o_a, self.mixed, self.adapter, self.after, self.after, self.lora_ws)
        linear(self.head_w, rms_norm(self.after), self.raw)
        fm.logits_adjust(self.rules, self.raw, self.logits)
        fm.token_logprobs(self.logits, self.tokens, self.logprob, self.entropy, self.ids, self.top_logprobs, self.lp_ws)
        best = self.ids[:, 0]
        self.history.scatter_(1, self.total.long()[:, None], best[:, None])
        self.total += 1
        self.tokens.copy_(best)
        return hidden


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--requests", type=int, default=4)
    p.add_argument("--samples", type=int, default=2)
    p.add_argument("--prompt", type=int, default=300)
    p.add_argument("--steps", type=int, default=4)
    a = p.parse_args()
    s = ServeStep(a.requests * a.samples, a.prompt, max(a.steps, 1))
    tokens = torch.randint(0, s.vocab, (a.requests, a.prompt), generator=s.g, device="cuda").to(I32)
    s.prompts(tokens, torch.arange(a.requests, device="cuda", dtype=I32) % 4 - 1, a.samples)
    for i in range(a.steps):
        s.step(i % 2)
        state = s.states[1 - i % 2]
        print("step %d: %d of %d pages in use; first sequence: entropy %.3f, best %s" % (
            i, s.pool.n_pages - state.n_free.item(), s.pool.n_pages, s.entropy[0].item(), s.ids[0].tolist()))


if __name__ == "__main__":
    main()
