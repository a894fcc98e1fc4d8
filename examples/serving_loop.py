"""A serving loop on the device-side operators: the small random decoder of
examples/speculative_decode.py over a paged cache of 8-bit codes, with fewer pages than all
sequences together would need.

    python -m examples.serving_loop [--steps 24] [--drafts 3] [--pages 24]

Each step
  1. kv_plan: sequences drop the tokens of fallen drafts, finished ones give their pages back, and
     the step's tokens get pages and places; who is refused for want of pages waits, and where all
     wait the shortest one gives its pages back until another has ended
  2. the layers: kv_append stores e4m3 codes (a scale for each block of tokens and head),
     kv_attention reads them
  3. token_probs: the ragged step's logits become one row of probabilities per draft, with
     penalties for what a sequence has said, biases, a grammar mask and its temperature
  4. draft_verify: the drafts that stand and one more token
"""
from __future__ import annotations

import argparse

import torch

import qmoe_mnb_matmul_gb300 as mnb
from examples.speculative_decode import Decoder, lookup_drafts


class Server(Decoder):
    """`batch` sequences over a pool of `pages` pages of 8-bit codes."""

    def __init__(self, pages=24, page=16, block=16, batch=3, max_len=512, **kw):
        super().__init__(batch=batch, max_len=max_len, page=page, **kw)
        shape = (pages, self.kv_heads, page, self.dim)
        for layer in self.layers:
            k, v = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
            scales = (torch.zeros((pages, self.kv_heads, page // block), device="cuda") for _ in range(2))
            layer["cache"] = mnb.kv_cache(k, v, *scales)

        def i32(*n):
            return torch.zeros(n, dtype=torch.int32, device="cuda")

        self.batch, self.pages = batch, pages
        self.table, self.held, self.free_count = i32(batch, -(-max_len // page)), i32(batch), i32(1)
        self.free_pages = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.free_count.fill_(pages)
        self.pool = mnb.kv_pool(self.held, self.table, self.free_pages, self.free_count, page)
        self.seq_lens, self.new_start, self.refused = i32(batch), i32(batch + 1), i32(batch)

    def step(self, tokens, keep):
        """Runs tokens[b] after the first keep[b] of sequence b.  Returns the logits of the tokens that found room, sequence
        after sequence, and which sequences were refused."""
        def ints(values):
            return torch.tensor(values, dtype=torch.int32, device="cuda")

        counts = [len(t) for t in tokens]
        mnb.kv_plan(self.pool, ints(keep), ints(counts), self.seq_lens, self.new_start, max_tokens=sum(counts),
                    refused=self.refused)
        refused = self.refused.tolist()
        ids = [t for seq, no in zip(tokens, refused) if not no for t in seq]
        if not ids:
            return None, refused
        most = max(counts)
        step = mnb.kv_step(self.seq_lens, self.table, new_start=self.new_start, tokens=len(ids), max_new=most)
        workspace = torch.empty(mnb.kv_attention_workspace_size(self.heads, self.kv_heads, self.dim, most),
                                dtype=torch.uint8, device="cuda")
        return self.run_layers(ids, step, workspace), refused


def serve(model, prompts, steps, drafts, seed=1, temperature=0.7, presence=0.0, frequency=0.0, repetition=1.0, mask=None,
          limit=None):
    """Extends every prompt by up to `steps` steps (a sequence of `limit` tokens is finished, its pages go back).  mask: int32
    words of the tokens that may be drawn.  Returns the sequences and how often one was refused."""
    g = torch.Generator("cuda").manual_seed(seed)
    batch, V = len(prompts), model.vocab
    seqs, done, waits = [list(p) for p in prompts], [0] * batch, 0
    cached = [0] * batch                                   # tokens of each sequence in the cache
    most = max(max(len(p) for p in prompts), 1) + steps * (drafts + 1)
    history = torch.zeros((batch, most), dtype=torch.int32, device="cuda")
    lens, prompt_lens = (torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda") for _ in range(2))
    for b, p in enumerate(prompts):
        history[b, :len(p)] = torch.tensor(p, dtype=torch.int32)

    def each(value):
        return torch.full((batch,), float(value), device="cuda")

    rules = mnb.token_rules(temperature=each(temperature), history=history, history_lens=lens, prompt_lens=prompt_lens,
                            repetition=each(repetition), frequency=each(frequency), presence=each(presence))
    target = torch.zeros((batch, drafts + 1, V), device="cuda")
    if mask is not None:
        mask = mask.expand(batch, drafts + 1, mask.shape[-1])
    draft_tokens = torch.zeros((batch, drafts), dtype=torch.int32, device="cuda")
    out = torch.empty((batch, drafts + 1), dtype=torch.int32, device="cuda")
    accepted = torch.empty(batch, dtype=torch.int32, device="cuda")
    paused, left = set(), batch
    for _ in range(10 * steps):
        active = [n < steps and (limit is None or len(s) < limit) for n, s in zip(done, seqs)]
        if not any(active):
            break
        if sum(active) < left:                             # one has ended: room for those that gave way
            paused, left = set(), sum(active)
        active = [a and b not in paused for b, a in enumerate(active)]
        if not any(active):                                # one alone needs more pages than there are
            break
        proposed = [lookup_drafts(s, drafts) if a else [] for s, a in zip(seqs, active)]
        tokens = [s[n:] + d if a else [] for s, n, d, a in zip(seqs, cached, proposed, active)]
        logits, refused = model.step(tokens, [n if a else 0 for n, a in zip(cached, active)])
        waits += sum(refused)
        cached = [n if a else 0 for n, a in zip(cached, active)]
        if logits is None:
            paused.add(min((b for b in range(batch) if active[b]), key=lambda b: cached[b]))
            continue
        # the rows that predict: the newest token's and the drafts'
        at, row_start, rows = 0, [0], []
        for b, t in enumerate(tokens):
            n = 0 if refused[b] else len(t)
            if n:
                rows += range(at + n - len(proposed[b]) - 1, at + n)
            row_start.append(len(rows))
            at += n
            draft_tokens[b, :len(proposed[b])] = torch.tensor(proposed[b], dtype=torch.int32)
        logits = logits[torch.tensor(rows, device="cuda")]
        starts = torch.tensor(row_start, dtype=torch.int32, device="cuda")
        mnb.token_probs(logits, rules, target, row_start=starts, draft_tokens=draft_tokens, mask=mask)
        n_drafts = torch.tensor([len(d) for d in proposed], dtype=torch.int32, device="cuda")
        uniforms = torch.rand((batch, drafts + 1), generator=g, device="cuda")
        mnb.draft_verify(target, None, draft_tokens, uniforms, out, accepted, n_drafts=n_drafts)
        for b, (row, n) in enumerate(zip(out.tolist(), accepted.tolist())):
            if not tokens[b] or refused[b]:
                continue
            cached[b] = len(seqs[b]) + n                   # the newest token waits for its step
            history[b, len(seqs[b]):len(seqs[b]) + n + 1] = out[b, :n + 1]
            seqs[b] += row[:n + 1]
            lens[b] += n + 1
            done[b] += 1
    return seqs, waits


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=24)
    p.add_argument("--drafts", type=int, default=3)
    p.add_argument("--pages", type=int, default=24)
    a = p.parse_args()
    prompts = [[5, 17, 99, 5, 17, 99, 5], [3], list(range(40, 90))]
    seqs, waits = serve(Server(pages=a.pages), prompts, a.steps, a.drafts, presence=0.3, frequency=0.2, repetition=1.1)
    if mnb.mnb_get_last_device_error() != 0:
        raise SystemExit("a device error was recorded")
    for s, q in zip(seqs, prompts):
        print(f"{len(q)} -> {len(s)} tokens: {s[len(q):len(q) + 16]} ...")
    print(f"steps that waited for pages: {waits}")


if __name__ == "__main__":
    main()
