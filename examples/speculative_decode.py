"""Speculative decoding with a small random decoder, run end to end on the library:
quantised products (qkv, o, gate/up with SwiGLU, down, vocabulary head), the paged
key-value cache, attention over it and the verification of drafted tokens.

    python -m examples.speculative_decode [--steps 24] [--drafts 4]

The weights are random, so the text means nothing; the calls and their order are
those of a serving loop:

  prompts    every prompt token goes through the layers once; kv_append stores its keys
             and values, kv_attention lets it see the tokens before it
  each step  1. draft: copy the tokens that followed the last occurrence of the newest
                token in the sequence so far (no draft probabilities)
             2. run the newest token and the drafts through the layers as one step of
                a ragged batch (kv_append, kv_attention)
             3. draft_verify against the head's probabilities: the drafts that stand,
                and one more token
             4. the cache keeps the tokens that stand; the entries of fallen drafts are
                past the sequence's length and are overwritten by the next step

Embedding, the layers' RMS norms and the residual additions are torch operations; the
per-head norms of queries and keys and the rotation are part of kv_append.
"""
from __future__ import annotations

import argparse

import torch

import qmoe_mnb_matmul_gb300 as mnb


class Weight:
    """A random packed INT4 weight [N, K] with scales of about K ** -0.5."""

    def __init__(self, g, N, K, bs=32):
        self.N, self.bs = N, bs
        self.packed = torch.randint(0, 256, (N, K // bs, bs // 2), generator=g, dtype=torch.uint8, device="cuda")
        self.scales = (torch.rand((N, K // bs), generator=g, device="cuda") + 0.5) * (0.22 * K ** -0.5)

    def __call__(self, x, dtype=None):
        y = torch.empty((x.shape[0], self.N), dtype=dtype or x.dtype, device=x.device)
        mnb.mnb_matmul(x, self.packed, self.scales, None, self.N, 4, self.bs, y)
        return y


class Decoder:
    """A decoder of `layers` layers over `batch` sequences of at most max_len tokens."""

    def __init__(self, seed=0, layers=2, hidden=256, heads=8, kv_heads=2, dim=64, ffn=512, vocab=997, batch=3, max_len=512,
                 page=16, dtype=torch.float16):
        g = torch.Generator("cuda").manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.dim, self.ffn, self.vocab = hidden, heads, kv_heads, dim, ffn, vocab
        self.dtype, self.max_len = dtype, max_len
        self.embedding = torch.randn((vocab, hidden), generator=g, device="cuda").to(dtype)
        self.layers = []
        pages = -(-max_len // page)
        for _ in range(layers):
            shape = (batch * pages, kv_heads, page, dim)
            k, v = (torch.empty(shape, dtype=dtype, device="cuda") for _ in range(2))
            self.layers.append({
                "qkv": Weight(g, (heads + 2 * kv_heads) * dim, hidden), "o": Weight(g, hidden, heads * dim),
                "gate_up": Weight(g, 2 * ffn, hidden), "down": Weight(g, hidden, ffn), "cache": mnb.kv_cache(k, v)})
        self.head = Weight(g, vocab, hidden)
        # every sequence's pages, in no order
        self.table = torch.randperm(batch * pages, generator=g, device="cuda").to(torch.int32).view(batch, pages)
        angle = torch.arange(max_len, device="cuda")[:, None] * 1e4 ** (-torch.arange(0, dim, 2, device="cuda") / dim)
        norm = torch.ones(dim, device="cuda")
        self.rope = mnb.kv_rope(torch.cat([angle.cos(), angle.sin()], 1), q_norm=norm, k_norm=norm)

    def _norm(self, x):
        x = x.float()
        return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).to(self.dtype)

    def forward(self, tokens, lens):
        """Runs one ragged step: tokens[b] are sequence b's new tokens, lens[b] its length before them.  Returns the
        logits (fp32) of every new token, sequence after sequence."""
        counts = [len(t) for t in tokens]
        start = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
        after = torch.tensor([n + c for n, c in zip(lens, counts)], dtype=torch.int32).cuda()
        total = sum(counts)
        step = mnb.kv_step(after, self.table, new_start=start, tokens=total, max_new=max(counts))
        workspace = torch.empty(mnb.kv_attention_workspace_size(self.heads, self.kv_heads, self.dim, max(counts)),
                                dtype=torch.uint8, device="cuda")
        return self.run_layers([t for seq in tokens for t in seq], step, workspace)

    def run_layers(self, ids, step, workspace):
        """The logits (fp32) of a step's tokens."""
        total = len(ids)
        x = self.embedding[torch.tensor(ids).cuda()]
        q_end, k_end = self.heads * self.dim, (self.heads + self.kv_heads) * self.dim
        for layer in self.layers:
            qkv = layer["qkv"](self._norm(x))
            q, k, v = (part.unflatten(1, (-1, self.dim)) for part in (qkv[:, :q_end], qkv[:, q_end:k_end], qkv[:, k_end:]))
            seen = torch.empty((total, self.heads, self.dim), dtype=self.dtype, device="cuda")
            mnb.kv_append(layer["cache"], step, q, k, v, q, self.rope)       # the queries turn in place
            mnb.kv_attention(layer["cache"], step, q, seen, workspace)
            x = x + layer["o"](seen.flatten(1))
            hidden = torch.empty((total, self.ffn), dtype=self.dtype, device="cuda")
            w = layer["gate_up"]
            mnb.mnb_gate_up_swiglu(self._norm(x), w.packed, w.scales, None, self.ffn, 4, w.bs, hidden)
            x = x + layer["down"](hidden)
        return self.head(self._norm(x), torch.float32)


def lookup_drafts(history, most):
    """The tokens that followed the last earlier occurrence of the newest token."""
    for i in range(len(history) - 2, -1, -1):
        if history[i] == history[-1]:
            return history[i + 1:i + 1 + most]
    return []


def generate(model, prompts, steps, drafts, seed=1, temperature=0.7):
    """Extends every prompt by `steps` verified steps; returns the sequences and how many drafts stood and fell."""
    g = torch.Generator("cuda").manual_seed(seed)
    seqs = [list(p) for p in prompts]
    batch, V = len(seqs), model.vocab
    if any(len(p) > 1 for p in prompts):
        model.forward([p[:-1] for p in prompts], [0] * batch)  # the newest token waits for its step
    stood = fell = 0
    out = torch.empty((batch, drafts + 1), dtype=torch.int32, device="cuda")
    accepted = torch.empty(batch, dtype=torch.int32, device="cuda")
    for _ in range(steps):
        proposed = [lookup_drafts(s, drafts) for s in seqs]
        logits = model.forward([[s[-1]] + d for s, d in zip(seqs, proposed)], [len(s) - 1 for s in seqs])
        probs = torch.softmax(logits / temperature, -1)
        # one row of drafts + 1 distributions per sequence; rows past a sequence's drafts are not read
        target = torch.zeros((batch, drafts + 1, V), device="cuda")
        tokens = torch.zeros((batch, drafts), dtype=torch.int32, device="cuda")
        at = 0
        for b, d in enumerate(proposed):
            target[b, :len(d) + 1] = probs[at:at + len(d) + 1]
            tokens[b, :len(d)] = torch.tensor(d, dtype=torch.int32)
            at += len(d) + 1
        n_drafts = torch.tensor([len(d) for d in proposed], dtype=torch.int32).cuda()
        uniforms = torch.rand((batch, drafts + 1), generator=g, device="cuda")
        mnb.draft_verify(target, None, tokens, uniforms, out, accepted, n_drafts=n_drafts)
        for b, (row, n) in enumerate(zip(out.tolist(), accepted.tolist())):
            seqs[b] += row[:n + 1]
            stood += n
            fell += len(proposed[b]) - n
    return seqs, stood, fell


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=24)
    p.add_argument("--drafts", type=int, default=4)
    a = p.parse_args()
    model = Decoder()
    prompts = [[5, 17, 99, 5, 17, 99, 5], [3], list(range(40, 90))]
    seqs, stood, fell = generate(model, prompts, a.steps, a.drafts)
    if mnb.mnb_get_last_device_error() != 0:
        raise SystemExit("a device error was recorded")
    for s, q in zip(seqs, prompts):
        print(f"{len(q)} -> {len(s)} tokens: {s[len(q):len(q) + 16]} ...")
    print(f"drafts that stood: {stood}, that fell: {fell}")


if __name__ == "__main__":
    main()
