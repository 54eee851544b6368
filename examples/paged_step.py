"""Serving steps over a 4-bit paged KV cache, with drafted tokens.

A small decoder with random weights (8-bit weights and activations in every
projection) serves a batch of requests.  A step runs, without a look at the
GPU's results from the host:

    build_block_tables   blocks, slots and positions of the step's tokens
    kv4_cache_write      their keys and values, per layer
    kv4_attention        over the cache: prompts first, then a few drafted
                         tokens of each request at once
    verify_drafts        which drafted tokens stand, and the token after them

The draft is a fixed table of next-token probabilities, which is bad enough to
show rejections: the blocks that only rejected tokens needed go back to the
free list.

    python examples/paged_step.py [--steps 8] [--drafts 3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import int8_w8a8_scaled_gb300 as w8  # noqa: E402

LAYERS, HIDDEN, Q_HEADS, KV_HEADS, HEAD_DIM, VOCAB = 2, 512, 8, 2, 64, 1000
BLOCK_SIZE, MAX_BLOCKS = 16, 16


class Projection:
    """A linear layer with e4m3 weights, one scale for each output channel."""

    def __init__(self, gen, n, k):
        w = (torch.randn(n, k, generator=gen, device="cuda") / k ** 0.5).bfloat16()
        self.q = torch.empty(n, k, dtype=torch.float8_e4m3fn, device="cuda")
        self.scale = torch.empty(n, dtype=torch.float32, device="cuda")
        w8.scaled_quant(w, self.q, self.scale, per_token=True, dynamic=True)

    def __call__(self, x):
        out = torch.empty(x.shape[0], self.q.shape[0], dtype=torch.bfloat16, device="cuda")
        return w8.quant_scaled_mm(x, self.q, self.scale, out)


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.pow(2).mean(1, keepdim=True) + 1e-6)).bfloat16()


def rotate(x, positions):
    """Rotary position embedding of [tokens, heads, head_dim]."""
    half = x.shape[2] // 2
    angle = positions[:, None].double() * 10000.0 ** (-torch.arange(half, device=x.device).double() / half)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x.float().split(half, 2)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], 2).to(x.dtype)


class Server:
    def __init__(self, batch, num_blocks, seed=0, kind="e2m1"):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.gen, self.kind, self.batch = gen, kind, batch
        self.embed = torch.randn(VOCAB, HIDDEN, generator=gen, device="cuda").bfloat16()
        qkv = (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM
        self.layers = [(Projection(gen, qkv, HIDDEN), Projection(gen, HIDDEN, Q_HEADS * HEAD_DIM)) for _ in range(LAYERS)]
        self.head = Projection(gen, VOCAB, HIDDEN)
        self.bigram = torch.softmax(2.0 * torch.randn(VOCAB, VOCAB, generator=gen, device="cuda"), 1)
        self.caches = [torch.zeros(w8.kv4_cache_shape(num_blocks, KV_HEADS, BLOCK_SIZE, HEAD_DIM), dtype=torch.uint8, device="cuda")
                       for _ in range(LAYERS)]
        # scales of an earlier calibration: keys and values stay below 8
        largest = {"e2m1": 6.0, "int4": 7.0}[kind] * 448.0
        self.scale = torch.full((1,), 8.0 / largest, device="cuda")
        ints = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table = torch.full((batch, MAX_BLOCKS), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(num_blocks, generator=gen, device="cuda").int()
        self.free_count, self.held = ints(1) + num_blocks, ints(batch)

    def forward(self, tokens, new, most):
        """Logits of the packed new tokens, `new` of each request (most the largest)."""
        ints = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        start, lens, positions = ints(self.batch + 1), ints(self.batch), ints(tokens.numel())
        slots = torch.zeros(tokens.numel(), dtype=torch.int64, device="cuda")
        balance, count = ints(1), ints(1)
        w8.build_block_tables(self.held, new, self.free, self.free_count, self.table, BLOCK_SIZE, start, lens, slots,
                              positions, balance, free_count_out=count)
        self.free_count, self.allocated = count, lens
        x = self.embed[tokens.long()]
        for (qkv, proj), cache in zip(self.layers, self.caches):
            rows = qkv(norm(x)).view(tokens.numel(), -1, HEAD_DIM)
            q, k, v = rows.split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
            q, k = rotate(q, positions), rotate(k, positions)
            w8.kv4_cache_write(k, v, cache, slots, self.scale, self.scale, kind=self.kind)
            out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
            w8.kv4_attention(q, cache, lens, self.table, self.scale, self.scale, out, query_start=start,
                             max_query_len=most, kind=self.kind)
            x = x + proj(out.flatten(1))
        return self.head(norm(x)).float(), start

    def keep(self, lengths):
        """Requests hold `lengths` tokens from now on: the blocks past them are free again."""
        blocks = lambda n: (n + BLOCK_SIZE - 1) // BLOCK_SIZE  # noqa: E731
        col = torch.arange(MAX_BLOCKS, device="cuda")[None, :]
        gone = (col >= blocks(lengths)[:, None]) & (col < blocks(self.allocated)[:, None])
        place = self.free_count + gone.flatten().int().cumsum(0, dtype=torch.int32) - 1
        place = torch.where(gone.flatten(), place, self.free.numel())          # the rest past the end
        wide = torch.cat([self.free, self.free[:1]])
        self.free = wide.scatter_(0, place.long(), self.table.flatten())[:-1].contiguous()
        self.free_count = self.free_count + gone.sum(dtype=torch.int32)
        self.table = torch.where(gone, -1, self.table)
        self.held = lengths

    def prompt(self, prompts):
        """Takes the prompts in and returns each request's next token."""
        new = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        tokens = torch.cat([torch.as_tensor(p, dtype=torch.int32) for p in prompts]).cuda()
        logits, start = self.forward(tokens, new, max(len(p) for p in prompts))
        self.keep(self.allocated)
        return self.sample(torch.softmax(logits[start[1:].long() - 1], 1))

    def sample(self, probs):
        """One token of each row's distribution: no drafts, only the extra token."""
        out = torch.empty(self.batch, 1, dtype=torch.int32, device="cuda")
        none, count = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (0, self.batch))
        w8.verify_drafts(probs, None, none, torch.zeros(self.batch + 1, dtype=torch.int32, device="cuda"),
                         torch.empty(0, device="cuda"), torch.rand(self.batch, generator=self.gen, device="cuda"), out, count)
        return out[:, 0]

    def step(self, last, drafts):
        """Tokens of one step after each request's `last`: [batch, drafts + 1], -1 behind the ones that stand."""
        b = self.batch
        tokens, probs = [last], []
        for _ in range(drafts):
            probs.append(self.bigram[tokens[-1].long()])
            tokens.append(self.sample(probs[-1]))
        new = torch.full((b,), drafts + 1, dtype=torch.int32, device="cuda")
        logits, _ = self.forward(torch.stack(tokens, 1).flatten(), new, drafts + 1)
        out = torch.empty(b, drafts + 1, dtype=torch.int32, device="cuda")
        accepted = torch.empty(b, dtype=torch.int32, device="cuda")
        start = torch.arange(b + 1, dtype=torch.int32, device="cuda") * drafts
        drafted = torch.stack(tokens[1:], 1).flatten() if drafts else torch.empty(0, dtype=torch.int32, device="cuda")
        draft_probs = torch.stack(probs, 1).flatten(0, 1) if drafts else None
        w8.verify_drafts(torch.softmax(logits, 1), draft_probs, drafted, start,
                         torch.rand(b * drafts, generator=self.gen, device="cuda"),
                         torch.rand(b, generator=self.gen, device="cuda"), out, accepted)
        # the last token and the accepted ones are in the cache to stay; the new one comes with the next step
        self.keep(self.held + 1 + accepted)
        return out, accepted


def main(argv=None):
    args = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    args.add_argument("--steps", type=int, default=8)
    args.add_argument("--drafts", type=int, default=3)
    args.add_argument("--kind", default="e2m1", choices=("e2m1", "int4"))
    args = args.parse_args(argv)
    server = Server(batch=4, num_blocks=64, kind=args.kind)
    last = server.prompt([list(range(1, n + 1)) for n in (40, 7, 1, 23)])
    texts = [[t] for t in last.tolist()]
    for _ in range(args.steps):
        out, accepted = server.step(last, args.drafts)
        last = out.gather(1, accepted[:, None].long())[:, 0]
        for text, row, n in zip(texts, out.tolist(), accepted.tolist()):
            text += row[:n + 1]
    for text, held in zip(texts, server.held.tolist()):
        print(f"{len(text)} tokens after the prompt, {held} cached:", *text)
    return server, texts


if __name__ == "__main__":
    main()
