"""A prompt, then greedy decoding with one pruned decoder layer, every step
between its products on the library's serving operators:

    q, k, v     spmm of the row-stacked projections; kv_append puts the new keys
                and values into the paged cache
    attention   prompt_attention over the prompt, then paged_attention, adding
                a step's attention weights up per cached row; a prompt adds
                none, so its rows are ranked by the steps behind it alone
    o_proj      spmm_epilogue with the residual stream
    FFN         gate_up_silu, then spmm_epilogue with the residual stream
    cache       kv_evict once a sequence is `slack` tokens over its budget
    lm_head     spmm, then token_logprobs: the next token, its log probability
                and the entropy of the step

Random weights (seeded), magnitude-pruned; norms have no gain and there is no
position encoding.  The state on the host is the step number and the length of
each sequence.

    python examples/pruned_decode.py [--hidden 4096 --ffn 11008 --heads 32
        --kv-heads 32 --vocab 32000 --batch 4 --prompt 16 --steps 64 --budget 32 ...]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_weight_matmul_amd as swm  # noqa: E402


def norm(x):
    """Root-mean-square norm without a gain, in fp32."""
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-5)).to(x.dtype)


class Layer:
    """Pruned weights, compressed once, and the dense copies they came from (for checks)."""

    def __init__(self, hidden, ffn, heads, kv_heads, vocab, sparsity=0.5, seed=0):
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, hidden // heads
        kv = self.dim * kv_heads
        shapes = {"qkv": (hidden + 2 * kv, hidden), "o": (hidden, hidden), "gate": (ffn, hidden),
                  "up": (ffn, hidden), "down": (hidden, ffn), "head": (vocab, hidden)}
        r = np.random.default_rng(seed)
        self.dense, self.fmt = {}, {}
        for name, (m, k) in shapes.items():
            w = (r.standard_normal((m, k), dtype=np.float32) * 0.7 / np.sqrt(k)).astype(np.float16)
            cut = np.quantile(np.abs(w[: max(1, 200000 // k)].astype(np.float32)), sparsity)
            w[np.abs(w) < cut] = 0
            self.dense[name], self.fmt[name] = w, swm.sparse_compress(w)
        self.embed = torch.from_numpy(r.standard_normal((vocab, hidden), dtype=np.float32).astype(np.float16)).cuda()


class Session:
    """A batch of sequences: their cache, the accumulated weights and the positions."""

    def __init__(self, layer, batch, budget, slack, recent, page_size):
        self.layer, self.batch, self.budget, self.slack, self.recent = layer, batch, budget, slack, recent
        per = -(-(budget + slack) // page_size)
        shape = (batch * per, page_size, layer.kv_heads, layer.dim)
        self.k, self.v = (torch.zeros(shape, dtype=torch.float16, device="cuda") for _ in range(2))
        self.table = torch.randperm(batch * per, device="cuda").to(torch.int32).view(batch, per)
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.cache = swm.PagedCache(self.k, self.v, self.table, self.lengths)
        slots = (shape[0], layer.kv_heads, page_size)
        self.weights = torch.zeros(slots, device="cuda")
        self.positions = torch.zeros(slots, dtype=torch.int32, device="cuda")
        self.used, self.seen, self.page_size = 0, 0, page_size  # tokens in the cache, tokens so far

    def append(self, k, v, n):
        """The next n tokens of every sequence into their slots, with no attention weight yet."""
        at = torch.arange(n, device="cuda")
        page = self.table[:, (self.used + at) // self.page_size].long()
        slots = page * self.page_size + (self.used + at) % self.page_size
        positions = (self.seen + at).to(torch.int32).repeat(self.batch)
        swm.kv_append(self.cache, k, v, slots.view(-1), weights=self.weights, positions=self.positions, at=positions)
        self.used += n
        self.seen += n
        self.lengths.fill_(self.used)

    def prompt(self, tokens):
        """Next tokens, their log probabilities and the entropies after prompts, (batch, n) tokens, n below
        budget + slack; the cache is empty."""
        n = tokens.shape[1]
        if self.used or not 0 < n < self.budget + self.slack:
            raise ValueError(f"a prompt begins a session and has 1 to {self.budget + self.slack - 1} tokens")
        starts = torch.arange(0, self.batch * n + 1, n, dtype=torch.int32, device="cuda")
        return self.forward(tokens.reshape(-1), n, lambda q, k, v: swm.prompt_attention(q, k, v, starts))

    def step(self, tokens):
        """Next tokens, their log probabilities and the entropies for a batch of tokens."""
        return self.forward(tokens, 1, lambda q, k, v: swm.paged_attention(self.cache, q, weights=self.weights))

    def forward(self, tokens, n, attend):
        y, f = self.layer, self.layer.fmt
        rows = self.batch * n
        x = y.embed[tokens]
        qkv = swm.spmm(f["qkv"], norm(x))
        kv = y.kv_heads * y.dim
        q = qkv[:, :y.hidden].view(rows, y.heads, y.dim)  # strided: the stacked product as it is
        k, v = (qkv[:, i:i + kv].view(rows, y.kv_heads, y.dim) for i in (y.hidden, y.hidden + kv))
        self.append(k, v, n)
        a = attend(q, k, v)
        x = swm.spmm_epilogue(f["o"], a.view(rows, y.hidden), residual=x)
        need = swm.gate_up_silu_workspace_bytes(f["gate"], f["up"], rows)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        h = swm.gate_up_silu_ws(f["gate"], f["up"], norm(x), ws)
        swm.spmm_epilogue(f["down"], h, residual=x, Y=x)
        x = x[n - 1::n].contiguous()  # the last token of every sequence
        if self.used == self.budget + self.slack:
            swm.kv_evict(self.cache, self.weights, self.positions, self.budget, self.recent)
            self.used = self.budget
        logits = swm.spmm(f["head"], norm(x))
        _, entropy, ids, logp = swm.token_logprobs(logits, top=1)
        return ids[:, 0], logp[:, 0], entropy


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("hidden", 4096), ("ffn", 11008), ("heads", 32), ("kv-heads", 32), ("vocab", 32000),
                        ("batch", 4), ("prompt", 16), ("steps", 64), ("budget", 32), ("slack", 8), ("recent", 8),
                        ("page-size", 16)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args(argv)
    s = Session(Layer(a.hidden, a.ffn, a.heads, a.kv_heads, a.vocab), a.batch, a.budget, a.slack, a.recent,
                a.page_size)
    tokens = torch.arange(a.batch * max(a.prompt, 1), device="cuda").view(a.batch, -1) % a.vocab
    tokens, _, _ = s.prompt(tokens)
    s.step(tokens)  # the first call loads the kernels
    torch.cuda.synchronize()
    t, total = time.perf_counter(), torch.zeros(a.batch, device="cuda")
    for _ in range(a.steps):
        tokens, logp, entropy = s.step(tokens)
        total += logp
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.steps} steps of {a.batch} sequences: {t / a.steps * 1e6:.0f} us a step; mean log probability "
          f"{(total / a.steps).mean().item():.3f}, last entropy {entropy.mean().item():.3f}, "
          f"{s.used} of {s.seen} tokens cached")


if __name__ == "__main__":
    main()
