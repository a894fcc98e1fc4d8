"""Workloads of a serving step around an 8-bit paged cache: planning the step's pages and slots on the GPU
(``kv_plan``), appending to a cache of e4m3 codes with a scale for each block of tokens and head (``kv_append``),
attention over it (``kv_attention``), and the step's logits with penalties, biases and grammar masks on their way to
the probabilities that a sampler or ``draft_verify`` draws from (``token_probs``).

``run`` makes the library's calls where ``own`` is true and computes the same in elementary torch operations, in
32 bits, where it is false.  Lengths follow from a case alone (so ``work`` needs no seed); everything else is drawn
from the seed.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODES = torch.float8_e4m3fn
GOLDEN = 0.6180339887498949  # spreads lengths evenly over their range, in no order
EPS = 1e-6                   # of the per-head norms


def _append(name, batch, new_lo, new_hi, ctx, heads, kv_heads, dim, rot, page, block, dtype, norm, interleaved):
    return {"name": name, "op": "append", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "ctx": ctx,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "page": page, "block": block,
            "dtype": dtype, "norm": norm, "interleaved": interleaved}


def _attention(name, batch, new_lo, new_hi, ctx_lo, ctx_hi, heads, kv_heads, dim, page, block, dtype, window):
    return {"name": name, "op": "attention", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "block": block,
            "dtype": dtype, "window": window}


def _probs(name, batch, rows, vocab, dtype, history, ragged, penalties, biases, mask):
    return {"name": name, "op": "probs", "batch": batch, "rows": rows, "vocab": vocab, "dtype": dtype,
            "history": history, "ragged": ragged, "penalties": penalties, "biases": biases, "mask": mask}


def _plan(name, batch, new_lo, new_hi, ctx, drop, page, short, budget):
    return {"name": name, "op": "plan", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "ctx": ctx, "drop": drop,
            "page": page, "short": short, "budget": budget}


def listed():
    return [
        # one user's decode step of the 1.7B decoder (16 query heads over 8 key-value heads, fp32 activations)
        _append("append8 one token", 1, 1, 1, 4095, 16, 8, 128, 128, 16, 16, "f32", True, False),
        # a serving batch that drafts: one to five new tokens per sequence, blocks that earlier steps began
        _append("append8 drafts b64", 64, 1, 5, 3000, 32, 4, 128, 128, 32, 32, "bf16", True, False),
        # prompts of many lengths entering an empty cache together
        _append("append8 prompts", 12, 17, 2700, 0, 16, 8, 128, 128, 64, 16, "bf16", True, False),
        # one user, a short conversation: latency
        _attention("attend8 short", 1, 1, 1, 777, 777, 16, 8, 128, 16, 16, "f32", 0),
        # one user, a whole book in the cache
        _attention("attend8 long", 1, 1, 1, 131072, 131072, 32, 4, 128, 64, 64, "bf16", 0),
        # a serving batch whose conversations are of every length
        _attention("attend8 batch b64", 64, 1, 1, 1, 8192, 16, 8, 128, 16, 16, "bf16", 0),
        # a batch that drafts, narrow heads, a sliding window, pages that end inside a tile
        _attention("attend8 drafts odd", 16, 1, 5, 5, 16000, 20, 5, 80, 24, 8, "f16", 5000),
        # one user's drafts over the 151936-token vocabulary, penalties on a conversation of 2000 tokens
        _probs("probs one", 1, 5, 151936, "f32", 2000, False, True, 0, False),
        # a serving batch's step, fewer rows where the drafter gave up early, grammars and a few biases
        _probs("probs b64", 64, 6, 151936, "bf16", 3000, True, True, 16, True),
        # a vocabulary that is no multiple of anything, many biases, no penalties
        _probs("probs odd", 13, 4, 50257, "f16", 1, True, False, 300, True),
        # a batch's decode step that drafts: a few tokens fell in the step before, a page for a few sequences
        _plan("plan decode b64", 64, 1, 5, 3000, 4, 16, False, 512),
        # prompts among decoding sequences, more than the pool and the step have room for
        _plan("plan prompts b1000", 1000, 1, 1500, 2000, 30, 16, True, 500000),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "probs", "plan"])
    if op == "probs":
        batch, rows = _spread(rng, 1, 64), rng.randint(1, 6)
        case = _probs("", batch, rows, _spread(rng, 30000, 152000), rng.choice(["f32", "f16", "bf16"]),
                      _spread(rng, 1, 8000), rng.random() < 0.5, rng.random() < 0.7,
                      rng.choice([0, 1, _spread(rng, 2, 300)]), rng.random() < 0.5)
    elif op == "plan":
        hi = _spread(rng, 1, 1500)
        batch = _spread(rng, 1, 1000)
        case = _plan("", batch, max(1, hi // rng.randint(1, 20)), hi, _spread(rng, 1, 2000), rng.randint(0, 30),
                     rng.choice([8, 16, 24, 32, 64, 128]), rng.random() < 0.5, _spread(rng, 1, min(batch * hi, 500000)))
    else:
        kv_heads = rng.choice([1, 2, 4, 5, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
        dim = rng.choice([64, 80, 96, 112, 128, 128, 128, 256])
        page = rng.choice([8, 16, 24, 32, 64, 128])
        block = rng.choice([b for b in (8, 16, 32, 64, 128) if page % b == 0])
        dtype = rng.choice(["bf16", "f16", "f32"])
        if op == "append":
            rot = rng.choice([dim, dim, dim // 2 // 8 * 8])
            batch = _spread(rng, 1, 64)
            hi = max(1, min(_spread(rng, 1, 4000), 16000 // batch))
            case = _append("", batch, max(1, hi // rng.randint(1, 20)), hi, _spread(rng, 1, 3000), heads, kv_heads, dim,
                           rot, page, block, dtype, rng.random() < 0.5, rng.random() < 0.3)
        else:
            batch = _spread(rng, 1, 64)
            most = int(64 * 4096 * 8 * 128 / (batch * kv_heads * dim))  # the largest listed case reads as much
            hi = _spread(rng, 40, max(41, min(131072, most)))
            new = rng.choice([1, 1, 1, rng.randint(2, 6)])
            window = rng.choice([0, 0, 0, _spread(rng, 30, 4000)])
            case = _attention("", batch, 1, new, max(new, hi // rng.choice([1, 2, 10, 100])), hi, heads, kv_heads, dim,
                              page, block, dtype, window)
    return {k: v for k, v in case.items() if k != "name"}


# ------------------------------------------------------------------ lengths and work

def _lengths(lo, hi, count, phase):
    return [lo + int((hi - lo + 1) * ((i * GOLDEN + phase) % 1.0)) for i in range(count)]


def _new_tokens(case):
    if case["op"] == "probs":  # rows of a sequence
        return _lengths(1, case["rows"], case["batch"], 0.37) if case["ragged"] else [case["rows"]] * case["batch"]
    return _lengths(case["new_lo"], case["new_hi"], case["batch"], 0.37)


def _seq_lens(case):
    """Cache lengths after the step, the new tokens among them."""
    new = _new_tokens(case)
    if case["op"] == "append":
        return [case["ctx"] + n for n in new]
    return [max(c, n) for c, n in zip(_lengths(case["ctx_lo"], case["ctx_hi"], case["batch"], 0.71), new)]


def _history_lens(case):
    return _lengths((case["history"] + 1) // 2, case["history"], case["batch"], 0.11)


def _plan_lens(case):
    """Tokens in the cache before the step, of which the last `dropped` fell; every seventh sequence ends."""
    had = _lengths(1, case["ctx"], case["batch"], 0.53)
    kept = [max(0, h - d) for h, d in zip(had, _lengths(0, case["drop"], case["batch"], 0.29))]
    new = _new_tokens(case)
    for i in range(3, case["batch"], 7):
        kept[i], new[i] = 0, 0
    return had, kept, new


def _ceil(a, b):
    return -(-a // b)


def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    if case["op"] == "probs":
        b, v = case["batch"], case["vocab"]
        rows = sum(_new_tokens(case))
        read = rows * v * _size(case["dtype"]) + (rows * _ceil(v, 32) * 4 if case["mask"] else 0)
        read += sum(_history_lens(case)) * 4 if case["penalties"] else 0
        return {"bytes": float(read + b * case["biases"] * 8 + rows * v * 4), "flops": 6.0 * rows * v}
    if case["op"] == "plan":
        had, kept, new = _plan_lens(case)
        page, b = case["page"], case["batch"]
        grown = sum(max(0, _ceil(k + n, page) - _ceil(h, page)) for h, k, n in zip(had, kept, new))
        tokens = min(sum(new), case["budget"])
        return {"bytes": float(4 * 6 * b + 8 * grown + 8 * tokens), "flops": 10.0 * b + 4.0 * tokens}
    hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    tokens = sum(_new_tokens(case))
    if case["op"] == "append":
        es = _size(case["dtype"])
        moved = tokens * d * ((hq + 2 * hkv) * es + hq * es + 2 * hkv) + tokens * case["rot"] * 4
        return {"bytes": float(moved), "flops": 12.0 * tokens * d * (hq + hkv)}
    flops, read = 0, 0
    for length, n in zip(_seq_lens(case), _new_tokens(case)):
        first = length - n
        lo = max(0, first + 1 - case["window"]) if case["window"] else 0
        read += length - lo
        for i in range(n):
            seen = first + i + 1
            flops += 4 * hq * d * (min(seen, case["window"]) if case["window"] else seen)
    return {"bytes": float(read * 2 * hkv * (d + 4 / case["block"]) + 2 * tokens * hq * d * _size(case["dtype"])),
            "flops": float(flops)}


# ------------------------------------------------------------------ inputs

def _cache_inputs(case, g, dev):
    """The paged cache of codes with its scales, the page table (pages in no order) and the step's lengths."""
    page, hkv, d = case["page"], case["kv_heads"], case["dim"]
    lens = torch.tensor(_seq_lens(case), dtype=torch.int32, device=dev)
    new = torch.tensor(_new_tokens(case), dtype=torch.int32, device=dev)
    pages = (lens + page - 1) // page
    pool = int(pages.sum()) + 3
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((len(lens), int(pages.max())), dtype=torch.int32, device=dev)
    table[torch.arange(table.shape[1], device=dev) < pages[:, None]] = order[:pool - 3]
    s = {"page_table": table, "seq_lens": lens, "max_new": max(_new_tokens(case))}
    for name in ("k", "v"):
        codes = torch.empty((pool, hkv, page, d), dtype=torch.float16, device=dev).normal_(0.0, 90.0, generator=g)
        s[name + "_cache"] = codes.clamp_(-448.0, 448.0).to(CODES)
        # scales as appending leaves them: powers of two around a largest value of 448 codes
        power = torch.randint(-8, -5, (pool, hkv, page // case["block"]), generator=g, device=dev)
        s[name + "_scale"] = torch.ldexp(torch.ones(power.shape, device=dev), power)
    s["new_start"] = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0, dtype=torch.int32)])
    s["tokens"] = int(s["new_start"][-1])
    return s


def _append_inputs(case, g, dev):
    s = _cache_inputs(case, g, dev)
    hq, hkv, d, rot = case["heads"], case["kv_heads"], case["dim"], case["rot"]
    # one row per token of the fused projection's output, as the product before it leaves it
    qkv = torch.randn((s["tokens"], (hq + 2 * hkv) * d), generator=g, device=dev).to(DTYPES[case["dtype"]])
    s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    inv = 1e6 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
    angle = torch.arange(max(_seq_lens(case)), device=dev, dtype=torch.float64)[:, None] * inv
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["q_norm"] = s["k_norm"] = None
    if case["norm"]:
        s["q_norm"] = torch.rand(d, generator=g, device=dev) * 2 + 0.2
        s["k_norm"] = torch.rand(d, generator=g, device=dev) * 2 + 0.2
    s["q_out"] = torch.empty((s["tokens"], hq, d), dtype=qkv.dtype, device=dev)
    return s


def _attention_inputs(case, g, dev):
    s = _cache_inputs(case, g, dev)
    shape = (s["tokens"], case["heads"], case["dim"])
    s["q"] = (torch.randn(shape, generator=g, device=dev) * 2).to(DTYPES[case["dtype"]])
    s["out"] = torch.empty(shape, dtype=s["q"].dtype, device=dev)
    return s


def _probs_inputs(case, g, dev):
    b, n, v = case["batch"], case["rows"], case["vocab"]
    rows = torch.tensor(_new_tokens(case), dtype=torch.int32, device=dev)
    start = torch.cat([torch.zeros_like(rows[:1]), rows.cumsum(0, dtype=torch.int32)])
    logits = (torch.randn((sum(_new_tokens(case)), v), generator=g, device=dev) * 3).to(DTYPES[case["dtype"]])
    s = {"logits": logits if case["ragged"] else logits.view(b, n, v), "row_start": start if case["ragged"] else None,
         "history": None, "history_lens": None, "prompt_lens": None, "repetition": None, "frequency": None,
         "presence": None, "bias_tokens": None, "bias_values": None, "mask": None, "draft_tokens": None,
         "out": torch.zeros((b, n, v), device=dev)}

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=dev)

    def tokens(*shape):  # few tokens often, most hardly ever
        return (uniform(*shape).pow(4) * v).to(torch.int32).clamp_(0, v - 1)

    s["temperature"] = uniform(b) * 0.9 + 0.3
    if b > 2:
        s["temperature"][b // 2] = 0.0  # one sequence decodes greedily
    if case["penalties"]:
        s["history"] = tokens(b, case["history"])
        s["history_lens"] = torch.tensor(_history_lens(case), dtype=torch.int32, device=dev)
        s["prompt_lens"] = s["history_lens"] // 3
        s["repetition"], s["frequency"], s["presence"] = uniform(b) * 0.5 + 0.9, uniform(b) * 0.4, uniform(b) - 0.3
        s["draft_tokens"] = tokens(b, n - 1)
    if case["biases"]:
        s["bias_tokens"], s["bias_values"] = tokens(b, case["biases"]), uniform(b, case["biases"]) * 20 - 10
    if case["mask"]:  # most sequences may go anywhere, some along a grammar that allows few tokens
        words = torch.randint(-2 ** 31, 2 ** 31, (b, n, -(-v // 32)), generator=g, device=dev).to(torch.int32)
        narrow = torch.randint(-2 ** 31, 2 ** 31, words.shape, generator=g, device=dev).to(torch.int32)
        narrow &= words & torch.randint(-2 ** 31, 2 ** 31, words.shape, generator=g, device=dev).to(torch.int32)
        free = (torch.arange(b, device=dev) % 3 != 1)[:, None, None]
        s["mask"] = torch.where(free, torch.full_like(words, -1), narrow)
    return s


def _plan_inputs(case, g, dev):
    had, kept, new = _plan_lens(case)
    page, b = case["page"], case["batch"]
    held = torch.tensor([_ceil(h, page) for h in had], dtype=torch.int32, device=dev)
    grown = sum(max(0, _ceil(k + n, page) - _ceil(h, page)) for h, k, n in zip(had, kept, new))
    spare = grown * 2 // 3 + 1 if case["short"] else grown + 17
    used = int(held.sum())
    pool = used + spare
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    columns = max(max(_ceil(k + n, page), _ceil(h, page)) for h, k, n in zip(had, kept, new))
    table = torch.full((b, columns), -1, dtype=torch.int32, device=dev)
    table[torch.arange(columns, device=dev) < held[:, None]] = order[:used]
    free = torch.full((pool,), -1, dtype=torch.int32, device=dev)
    free[:spare] = order[used:]

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    budget = case["budget"]
    return {"held": held, "page_table": table, "free_pages": free, "free_count": ints([spare]), "keep": ints(kept),
            "new": ints(new), "held_out": torch.zeros_like(held), "free_count_out": ints([0]),
            "seq_lens": torch.zeros_like(held), "new_start": torch.zeros(b + 1, dtype=torch.int32, device=dev),
            "refused": torch.zeros_like(held), "slots": torch.full((budget,), -1, dtype=torch.int64, device=dev)}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(int(seed))
    make = {"append": _append_inputs, "attention": _attention_inputs, "probs": _probs_inputs, "plan": _plan_inputs}
    s = make[case["op"]](case, g, dev)
    s["case"] = case
    if own:  # the descriptors and the workspace that a serving loop keeps
        import qmoe_mnb_matmul_gb300 as mnb
        if case["op"] == "plan":
            s["pool"] = mnb.kv_pool(s["held"], s["page_table"], s["free_pages"], s["free_count"], case["page"],
                                    held_out=s["held_out"], free_count_out=s["free_count_out"])
        elif case["op"] == "probs":
            s["rules"] = mnb.token_rules(
                temperature=s["temperature"], history=s["history"], history_lens=s["history_lens"],
                prompt_lens=s["prompt_lens"], repetition=s["repetition"], frequency=s["frequency"],
                presence=s["presence"], bias_tokens=s["bias_tokens"], bias_values=s["bias_values"])
        else:
            s["cache"] = mnb.kv_cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
            s["step"] = mnb.kv_step(s["seq_lens"], s["page_table"], new_start=s["new_start"], tokens=s["tokens"],
                                    max_new=s["max_new"])
        if case["op"] == "append":
            s["rope"] = mnb.kv_rope(s["cos_sin"], interleaved=case["interleaved"], q_norm=s["q_norm"],
                                    k_norm=s["k_norm"], eps=EPS)
        elif case["op"] == "attention":
            need = mnb.kv_attention_workspace_size(case["heads"], case["kv_heads"], case["dim"], s["max_new"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ one pass

def _token_places(s):
    """Sequence, position, page and row in the page of every new token."""
    t = torch.arange(s["tokens"], device=s["seq_lens"].device)
    seq = (t[:, None] >= s["new_start"][None, 1:]).sum(1)
    pos = s["seq_lens"].long()[seq] - s["new_start"].long()[seq + 1] + t
    size = s["k_cache"].shape[2]
    return seq, pos, s["page_table"].long()[seq, pos // size], pos % size


def _rotated(x, weight, table, case):
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    half = case["rot"] // 2
    cos, sin = table[:, None, :half], table[:, None, half:]
    y = x.clone()
    if case["interleaved"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
    return y


def _smallest_scale(largest):
    """The smallest power of two s, at least 2^-126, with largest <= 448 s; 0 for 0."""
    part, power = torch.frexp(largest)  # largest = part 2^power, part in [0.5, 1); 448 = 0.875 * 2^9
    power = (power + torch.where(part > 0.875, -8, -9)).clamp_min(-126)
    return torch.where(largest > 0, torch.ldexp(torch.ones_like(largest), power), torch.zeros_like(largest))


def _quantised(x, scale):
    return torch.where(scale > 0, x / scale, torch.zeros_like(x)).to(CODES)


def _plain_store(s, codes, scales, x, seq, page, row):
    """Stores x [tokens, kv_heads, dim] in codes and scales."""
    block = s["case"]["block"]
    pages, heads, size, dim = codes.shape
    per = size // block
    at = page * per + row // block                                        # the token's block in the pool
    flat = scales.transpose(1, 2).reshape(pages * per, heads)
    largest = torch.zeros_like(flat).scatter_reduce_(0, at[:, None].expand(-1, heads), x.abs().amax(-1), "amax")
    # a sequence's first new token may find older ones in its block, whose scale then stands or grows
    head = s["new_start"][:-1].long()
    older = row[head] % block
    first = at[head]
    fresh = torch.ones(pages * per, dtype=torch.bool, device=at.device)
    fresh[first] = older == 0
    touched = torch.zeros_like(fresh)
    touched[at] = True
    old = torch.where(fresh[:, None], torch.zeros_like(flat), flat)
    need = _smallest_scale(largest)
    now = torch.where(touched[:, None], torch.where(need > old, need, old), flat)
    # the older tokens of a block whose scale grew
    j = torch.arange(block, device=at.device)
    rows = (first % per * block)[:, None] + j
    mine = codes[page[head][:, None], :, rows]                                     # [batch, block, heads, dim]
    again = _quantised(mine.float() * flat[first][:, None, :, None], now[first][:, None, :, None])
    grew = (now[first] > flat[first])[:, None, :, None] & (j[None] < older[:, None])[:, :, None, None]
    # (bytes are what torch scatters)
    kept = torch.where(grew, again.view(torch.uint8), mine.view(torch.uint8))
    raw = codes.view(torch.uint8)
    raw[page[head][:, None], :, rows] = kept
    raw[page, :, row] = _quantised(x, now[at][..., None]).view(torch.uint8)
    scales.copy_(now.view(pages, per, heads).transpose(1, 2))


def _plain_append(s):
    case = s["case"]
    seq, pos, page, row = _token_places(s)
    table = s["cos_sin"][pos]
    s["q_out"].copy_(_rotated(s["q"].float(), s["q_norm"], table, case))
    _plain_store(s, s["k_cache"], s["k_scale"], _rotated(s["k"].float(), s["k_norm"], table, case), seq, page, row)
    _plain_store(s, s["v_cache"], s["v_scale"], s["v"].float(), seq, page, row)
    return s["q_out"], s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    seq, pos, _, _ = _token_places(s)
    batch, most = s["seq_lens"].shape[0], s["max_new"]
    slot = torch.arange(s["tokens"], device=seq.device) - s["new_start"].long()[seq]
    table = s["page_table"].long()

    def read(name):  # [b, length, kv head, d]
        values = s[name + "_cache"].view(torch.uint8)[table].view(CODES).float()
        scale = s[name + "_scale"][table].repeat_interleave(case["block"], 3)
        return (values * scale[..., None]).transpose(2, 3).reshape(batch, -1, hkv, d)

    keys, values = read("k"), read("v")
    q = torch.zeros((batch, most, hkv, hq // hkv, d), device=seq.device)
    q[seq, slot] = s["q"].float().view(-1, hkv, hq // hkv, d)
    at = torch.full((batch, most), -1, device=seq.device, dtype=torch.long)
    at[seq, slot] = pos
    j = torch.arange(keys.shape[1], device=seq.device)
    seen = j <= at[..., None]
    if case["window"]:
        seen = seen & (j > at[..., None] - case["window"])
    scores = torch.einsum("bihgd,bjhd->bhgij", q, keys) / math.sqrt(d)
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    e = torch.exp(scores - scores.amax(-1, keepdim=True).clamp_min(-3e38))
    o = torch.einsum("bhgij,bjhd->bihgd", e, values) / e.sum(-1).permute(0, 3, 1, 2)[..., None]
    s["out"].copy_(o[seq, slot].reshape(-1, hq, d))
    return s["out"]


def _plain_probs(s):
    logits, out = s["logits"], s["out"]
    batch, rows, vocab = out.shape
    dev = out.device
    i = torch.arange(rows, device=dev)
    if s["row_start"] is None:
        valid, x = torch.ones((batch, rows), dtype=torch.bool, device=dev), logits.float()
    else:
        start = s["row_start"].long()
        valid = i < (start[1:] - start[:-1])[:, None]
        x = logits[torch.where(valid, start[:-1, None] + i, torch.zeros_like(i))].float()

    def each(name):
        return s[name][:, None, None]

    if s["history"] is not None:
        j = torch.arange(s["history"].shape[1], device=dev)
        past, lens = s["history"].long(), s["history_lens"][:, None]
        seen = torch.zeros((batch, vocab), device=dev).scatter_add_(1, past, (j < lens).float())
        said = ((j < lens) & (j >= s["prompt_lens"][:, None])).float()
        count = torch.zeros((batch, vocab), device=dev).scatter_add_(1, past, said)
        # row i comes after the drafts before it
        before = (i[:rows - 1] < i[:, None]).float().expand(batch, rows, rows - 1)
        drafts = s["draft_tokens"].long()[:, None].expand(batch, rows, rows - 1)
        extra = torch.zeros((batch, rows, vocab), device=dev).scatter_add_(2, drafts, before)
        seen, count = seen[:, None] + extra, count[:, None] + extra
        factor = each("repetition")
        x = torch.where(seen > 0, torch.where(x > 0, x / factor, x * factor), x)
        x = x - each("frequency") * count
        x = torch.where(count > 0, x - each("presence"), x)
    if s["bias_tokens"] is not None:  # of several biases of one token the last one counts
        tokens = s["bias_tokens"].long()
        e = torch.arange(tokens.shape[1], device=dev)
        later = (tokens[:, :, None] == tokens[:, None]) & (e[None, :] > e[:, None])
        values = torch.where(later.any(-1), torch.zeros_like(s["bias_values"]), s["bias_values"])
        x = x + torch.zeros((batch, vocab), device=dev).scatter_add_(1, tokens, values)[:, None]
    if s["mask"] is not None:
        at = torch.arange(vocab, device=dev)
        x = torch.where((s["mask"][..., at // 32] >> (at % 32)) & 1 == 1, x, torch.full_like(x, -math.inf))
    temperature = each("temperature")
    top = x.amax(-1, keepdim=True)
    y = x / torch.where(temperature > 0, temperature, torch.ones_like(temperature))
    y = torch.exp(y - y.amax(-1, keepdim=True).clamp_min(-3e38))
    total = y.sum(-1, keepdim=True)
    y = torch.where(total > 0, y / total, torch.zeros_like(y))
    at = torch.arange(vocab, device=dev)
    winner = torch.where((x == top) & (top > -math.inf), at, vocab).amin(-1, keepdim=True)
    y = torch.where(temperature > 0, y, (at == winner).float())
    out[valid] = y[valid]
    return out


def _plain_plan(s):
    case = s["case"]
    page, table, free = case["page"], s["page_table"], s["free_pages"]
    held, n, total_free = s["held"].long(), s["new"].long(), s["free_count"].long()
    batch, columns = table.shape
    budget, dev = s["slots"].shape[0], table.device
    keep = torch.minimum(s["keep"].long(), held * page)
    want = (keep + n + page - 1) // page
    long = want > columns
    target = torch.where(long, held, want)
    grow, back = (target - held).clamp_min(0), (held - target).clamp_min(0)
    grows, backs = grow.cumsum(0), back.cumsum(0)
    room = total_free + backs[-1]
    step = torch.where(long, torch.zeros_like(n), n)
    refused = (n > 0) & (long | ((grow > 0) & (grows > room)) | (step.cumsum(0) > budget))
    n, grow = torch.where(refused, torch.zeros_like(n), n), torch.where(refused, torch.zeros_like(grow), grow)
    start = torch.cat([torch.zeros_like(n[:1]), n.cumsum(0)])
    taken = grow.sum()
    # one stack: the free pages, then the released ones, the first released on top
    i = torch.arange(free.shape[0], device=dev)
    seq = torch.searchsorted(backs, i, right=True).clamp_max(batch - 1)
    column = (target[seq] + i - (backs - back)[seq]).clamp(0, columns - 1)
    released = table[seq, column]                                    # of number i, where i < backs[-1]
    number = room - 1 - i
    stack = torch.where(i < total_free, free, released[number.clamp(0, free.shape[0] - 1)])
    left = room - taken
    # pages of the growing sequences: the stack's top goes to the first
    c = torch.arange(columns, device=dev)
    order = (grow.cumsum(0) - grow)[:, None] + c - held[:, None]
    takes = (c >= held[:, None]) & (c < (held + grow)[:, None])
    table.copy_(torch.where(takes, stack[(room - 1 - order).clamp(0, free.shape[0] - 1)], table))
    free.copy_(torch.where((i >= total_free) & (i < left), stack, free))
    s["held_out"].copy_(held + grow - back)
    s["free_count_out"].copy_(left)
    s["seq_lens"].copy_(keep + n)
    s["new_start"].copy_(start)
    s["refused"].copy_(refused)
    t = torch.arange(budget, device=dev)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp_max(batch - 1)
    pos = keep[b] + t - start[b]
    slot = table[b, (pos // page).clamp(0, columns - 1)].long() * page + pos % page
    s["slots"].copy_(torch.where(t < start[-1], slot, s["slots"]))
    return tuple(s[k] for k in PLAN_OUTPUTS)


PLAN_OUTPUTS = ("held_out", "page_table", "free_pages", "free_count_out", "seq_lens", "new_start", "slots", "refused")


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "probs": _plain_probs, "plan": _plain_plan}[op](s)
    import qmoe_mnb_matmul_gb300 as mnb
    if op == "append":
        mnb.kv_append(s["cache"], s["step"], s["q"], s["k"], s["v"], s["q_out"], s["rope"])
        return s["q_out"], s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]
    if op == "attention":
        mnb.kv_attention(s["cache"], s["step"], s["q"], s["out"], s["workspace"], window=s["case"]["window"])
        return s["out"]
    if op == "probs":
        mnb.token_probs(s["logits"], s["rules"], s["out"], row_start=s["row_start"], draft_tokens=s["draft_tokens"],
                        mask=s["mask"])
        return s["out"]
    mnb.kv_plan(s["pool"], s["keep"], s["new"], s["seq_lens"], s["new_start"], slots=s["slots"], refused=s["refused"])
    return tuple(s[k] for k in PLAN_OUTPUTS)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_append(s):
    """The codes before their rounding."""
    case = s["case"]
    rot, half, block, size = case["rot"], case["rot"] // 2, case["block"], case["page"]
    first = list(range(0, rot, 2)) if case["interleaved"] else list(range(half))
    second = list(range(1, rot, 2)) if case["interleaved"] else list(range(half, rot))
    starts, lens = s["new_start"].tolist(), s["seq_lens"].tolist()
    table = s["page_table"].long()
    q_out = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=table.device)

    def turned(x, weight, angle_cos, angle_sin):
        if weight is not None:
            x = x * weight.double() * (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).rsqrt()
        y = x.clone()
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(angle_cos, angle_sin)[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    new = {"k": torch.zeros(s["k"].shape, dtype=torch.float64, device=table.device), "v": s["v"].double()}
    for b, length in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        pos = torch.arange(length - (hi - lo), length, device=table.device)
        cos, sin = s["cos_sin"][pos, :half].double(), s["cos_sin"][pos, half:].double()
        q_out[lo:hi] = turned(s["q"][lo:hi].double(), s["q_norm"], cos, sin)
        new["k"][lo:hi] = turned(s["k"][lo:hi].double(), s["k_norm"], cos, sin)
    found = [q_out]
    for name in ("k", "v"):
        codes, scales = s[name + "_cache"].double(), s[name + "_scale"].double()
        for b, length in enumerate(lens):
            lo, hi = starts[b], starts[b + 1]
            begin = length - (hi - lo)
            x = new[name][lo:hi]
            # whole blocks of the sequence, the older tokens of the first one in front and nothing behind the last
            front, back = begin % block, -length % block
            places = torch.arange(begin - front, length + back, block, device=table.device)
            page, part = table[b, places // size], places % size // block
            x = torch.cat([x.new_zeros((front,) + x.shape[1:]), x, x.new_zeros((back,) + x.shape[1:])])
            x = x.view(-1, block, *x.shape[1:])                                     # [blocks, token, head, dim]
            largest = x.abs().amax((1, 3))
            scale = torch.exp2(torch.ceil(torch.log2(largest / 448.0)).clamp_min(-126.0))
            scale[largest == 0] = 0.0
            old = scales[page[0], :, part[0]].clone()
            if front:
                scale[0] = torch.maximum(scale[0], old)
            scales[page, :, part] = scale
            rows = part[:, None] * block + torch.arange(block, device=table.device)
            there = codes[page[:, None], :, rows]                                   # [blocks, token, head, dim]
            moved = torch.where(scale[:, None, :, None] > 0, x / scale[:, None, :, None], torch.zeros_like(x))
            older = there[0, :front] * torch.where(scale[0] > 0, old / scale[0], torch.zeros_like(old))[:, None]
            at = places[:, None] + torch.arange(block, device=table.device)
            written = ((at >= begin) & (at < length))[:, :, None, None]
            there = torch.where(written, moved, there)
            there[0, :front] = older
            codes[page[:, None], :, rows] = there
        found += [codes, scales]
    return tuple(found)


def _exact_attention(s):
    case = s["case"]
    hkv, group, d = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    starts, lens = s["new_start"].tolist(), s["seq_lens"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    size, block = case["page"], case["block"]
    for b, length in enumerate(lens):
        pages = s["page_table"][b, :-(-length // size)].long()
        for h in range(hkv):
            def read(name):
                codes = s[name + "_cache"][:, h].view(torch.uint8)[pages].view(CODES).double().view(-1, block, d)
                return (codes * s[name + "_scale"][pages, h].double().view(-1, 1, 1)).view(-1, d)[:length]

            keys, values = read("k"), read("v")
            for t in range(starts[b], starts[b + 1]):
                end = length - (starts[b + 1] - 1 - t)
                begin = max(0, end - case["window"]) if case["window"] else 0
                q = s["q"][t, h * group:(h + 1) * group].double()
                p = torch.softmax(q @ keys[begin:end].T * d ** -0.5, -1)
                out[t, h * group:(h + 1) * group] = p @ values[begin:end]
    return out


def _exact_probs(s):
    out = s["out"].double()
    batch, rows, vocab = out.shape
    for b in range(batch):
        if s["row_start"] is None:
            x = s["logits"][b].double()
        else:
            x = s["logits"][int(s["row_start"][b]):int(s["row_start"][b + 1])].double()
        for i in range(x.shape[0]):
            y = x[i]
            if s["history"] is not None:
                past = s["history"][b, :int(s["history_lens"][b])].long()
                drafts = s["draft_tokens"][b, :i].long()
                seen = torch.bincount(torch.cat([past, drafts]), minlength=vocab) > 0
                count = torch.bincount(torch.cat([past[int(s["prompt_lens"][b]):], drafts]), minlength=vocab)
                factor = s["repetition"][b].double()
                y = torch.where(seen, y * torch.where(y > 0, 1.0 / factor, factor), y)
                y = y - s["frequency"][b].double() * count - s["presence"][b].double() * (count > 0)
            if s["bias_tokens"] is not None:
                last = dict(zip(s["bias_tokens"][b].tolist(), s["bias_values"][b].tolist()))
                at = torch.tensor(list(last), device=y.device)
                y = y.index_add(0, at, torch.tensor(list(last.values()), dtype=torch.float64, device=y.device))
            if s["mask"] is not None:
                bits = s["mask"][b, i].view(-1, 1) >> torch.arange(32, dtype=torch.int32, device=y.device) & 1
                y = y.masked_fill(bits.flatten()[:vocab] == 0, -math.inf)
            if bool((y == -math.inf).all()):
                out[b, i] = 0.0
            elif float(s["temperature"][b]) > 0:
                out[b, i] = torch.softmax(y / s["temperature"][b].double(), 0)
            else:
                out[b, i] = 0.0
                out[b, i, int((y == y.max()).nonzero()[0])] = 1.0
    return out


def _exact_plan(s):
    page = s["case"]["page"]
    table, free = s["page_table"].cpu().clone(), s["free_pages"].cpu().clone()
    held, keep, new = s["held"].tolist(), s["keep"].tolist(), s["new"].tolist()
    count, columns, budget = int(s["free_count"][0]), table.shape[1], s["slots"].shape[0]
    stack, released = free[:count].tolist(), []
    held_out, seq_lens, refused, start, slots = [], [], [], [0], s["slots"].cpu().clone()
    keep = [min(k, h * page) for k, h in zip(keep, held)]
    want = [_ceil(k + n, page) for k, n in zip(keep, new)]
    for b, w in enumerate(want):
        if w < held[b]:
            released += table[b, w:held[b]].tolist()
    stack += released[::-1]
    room, pages, tokens = len(stack), 0, 0
    for b, w in enumerate(want):
        grow = w - held[b] if held[b] < w <= columns else 0
        pages += grow
        tokens += new[b] if w <= columns else 0
        bad = new[b] > 0 and (w > columns or (grow > 0 and pages > room) or tokens > budget)
        n = 0 if bad else new[b]
        refused.append(int(bad))
        seq_lens.append(keep[b] + n)
        if grow and not bad:
            table[b, held[b]:w] = torch.tensor([stack.pop() for _ in range(grow)], dtype=torch.int32)
        held_out.append(held[b] if w > columns or (grow and bad) else w)
        at = torch.arange(keep[b], keep[b] + n)
        slots[start[-1]:start[-1] + n] = table[b, at // page].long() * page + at % page
        start.append(start[-1] + n)
    if len(stack) > count:
        free[count:len(stack)] = torch.tensor(stack[count:], dtype=torch.int32)
    as_int = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return (as_int(held_out), table, free, as_int([len(stack)]), as_int(seq_lens), as_int(start), slots, as_int(refused))


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "probs": _exact_probs, "plan": _exact_plan}[case["op"]](s)
