"""Workloads of the serving operators around the quantised products: appending to a paged key-value cache with the
position rotation on the way (``kv_append``), attention of a step's new tokens over that cache (``kv_attention``) and
the verification of drafted tokens (``draft_verify``).

``run`` makes the library's calls where ``own`` is true and computes the same in elementary torch operations, in
32 bits, where it is false.  Lengths follow from a case alone (so ``work`` needs no seed); everything else is drawn
from the seed.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
GOLDEN = 0.6180339887498949  # spreads lengths evenly over their range, in no order
EPS = 1e-6                   # of the per-head norms
FIXED = 2.0 ** 40            # unit of the sampling weights: whole numbers, so that every order of summation agrees


def _append(name, batch, new_lo, new_hi, ctx, heads, kv_heads, dim, rot, page, dtype, cache, norm, interleaved):
    return {"name": name, "op": "append", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "ctx": ctx,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "page": page, "dtype": dtype,
            "cache": cache, "norm": norm, "interleaved": interleaved}


def _attention(name, batch, new_lo, new_hi, ctx_lo, ctx_hi, heads, kv_heads, dim, page, dtype, cache, window):
    return {"name": name, "op": "attention", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype,
            "cache": cache, "window": window}


def _verify(name, batch, drafts, vocab, ragged, probs):
    return {"name": name, "op": "verify", "batch": batch, "drafts": drafts, "vocab": vocab, "ragged": ragged,
            "probs": probs}


def listed():
    return [
        # one user's decode step of the 1.7B decoder (16 query heads over 8 key-value heads, fp32 activations)
        _append("append one token", 1, 1, 1, 4095, 16, 8, 128, 128, 16, "f32", "bf16", True, False),
        # a serving batch that drafts: one to five new tokens per sequence, 32 query heads over 4
        _append("append drafts b64", 64, 1, 5, 3000, 32, 4, 128, 128, 32, "bf16", "bf16", True, False),
        # prompts of many lengths entering an empty cache together
        _append("append prompts", 12, 17, 2700, 0, 16, 8, 128, 128, 64, "bf16", "bf16", True, False),
        # narrow heads, a quarter of them rotated in interleaved pairs, pages of 24 tokens
        _append("append odd f16", 7, 1, 299, 1000, 10, 5, 80, 32, 24, "f16", "f16", False, True),
        # one user, a short conversation: latency
        _attention("attend short", 1, 1, 1, 777, 777, 16, 8, 128, 16, "f32", "bf16", 0),
        # one user, a whole book in the cache
        _attention("attend long", 1, 1, 1, 131072, 131072, 32, 4, 128, 64, "bf16", "bf16", 0),
        # a serving batch whose conversations are of every length
        _attention("attend batch b64", 64, 1, 1, 1, 8192, 16, 8, 128, 16, "bf16", "bf16", 0),
        # a batch that drafts: up to five new tokens of each sequence share one pass over its cache
        _attention("attend drafts b16", 16, 1, 5, 900, 16000, 32, 4, 128, 32, "f16", "f16", 0),
        # a sliding window, narrow heads, pages that end inside a tile
        _attention("attend window odd", 9, 1, 3, 5, 5000, 10, 5, 80, 24, "f16", "f16", 1000),
        # one user's drafts over the 151936-token vocabulary
        _verify("verify one", 1, 4, 151936, False, True),
        # a serving batch's drafts, fewer of them where the drafter gave up early
        _verify("verify b64", 64, 5, 151936, True, True),
        # drafts copied from the prompt (no draft probabilities), a vocabulary that is no multiple of anything
        _verify("verify lookup odd", 13, 3, 50257, True, False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "verify"])
    if op == "verify":
        return {k: v for k, v in _verify("", _spread(rng, 1, 64), rng.randint(1, 6), _spread(rng, 30000, 152000),
                                         rng.random() < 0.5, rng.random() < 0.7).items() if k != "name"}
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    dim = rng.choice([64, 80, 96, 112, 128, 128, 128, 256])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    cache = rng.choice(["f16", "bf16"])
    dtype = rng.choice([cache, cache, "f32"])
    if op == "append":
        rot = rng.choice([dim, dim, dim // 2 // 8 * 8])
        batch = _spread(rng, 1, 64)
        hi = max(1, min(_spread(rng, 1, 4000), 16000 // batch))
        case = _append("", batch, max(1, hi // rng.randint(1, 20)), hi, _spread(rng, 1, 3000), heads, kv_heads, dim, rot,
                       page, dtype, cache, rng.random() < 0.5, rng.random() < 0.3)
    else:
        batch = _spread(rng, 1, 64)
        most = int(64 * 4096 * 8 * 128 / (batch * kv_heads * dim))  # the largest listed case reads as much
        hi = _spread(rng, 40, max(41, min(131072, most)))
        new = rng.choice([1, 1, 1, rng.randint(2, 6)])
        window = rng.choice([0, 0, 0, _spread(rng, 30, 4000)])
        case = _attention("", batch, 1, new, max(new, hi // rng.choice([1, 2, 10, 100])), hi, heads, kv_heads, dim, page,
                          dtype, cache, window)
    return {k: v for k, v in case.items() if k != "name"}


# ------------------------------------------------------------------ lengths and work

def _lengths(lo, hi, count, phase):
    return [lo + int((hi - lo + 1) * ((i * GOLDEN + phase) % 1.0)) for i in range(count)]


def _new_tokens(case):
    return _lengths(case["new_lo"], case["new_hi"], case["batch"], 0.37)


def _seq_lens(case):
    """Cache lengths after the step, the new tokens among them."""
    new = _new_tokens(case)
    if case["op"] == "append":
        return [case["ctx"] + n for n in new]
    return [max(c, n) for c, n in zip(_lengths(case["ctx_lo"], case["ctx_hi"], case["batch"], 0.71), new)]


def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    if case["op"] == "verify":
        b, n, v = case["batch"], case["drafts"], case["vocab"]
        rows = 2 if case["probs"] else 1
        return {"bytes": 4.0 * b * (rows * v + 4 * n + 3), "flops": 4.0 * b * v}
    hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    tokens = sum(_new_tokens(case))
    if case["op"] == "append":
        es, cs = _size(case["dtype"]), _size(case["cache"])
        moved = tokens * d * ((hq + 2 * hkv) * es + hq * es + 2 * hkv * cs) + tokens * case["rot"] * 4
        return {"bytes": float(moved), "flops": 10.0 * tokens * d * (hq + hkv)}
    flops, read = 0, 0
    for length, n in zip(_seq_lens(case), _new_tokens(case)):
        first = length - n
        lo = max(0, first + 1 - case["window"]) if case["window"] else 0
        read += length - lo
        for i in range(n):
            seen = first + i + 1
            flops += 4 * hq * d * (min(seen, case["window"]) if case["window"] else seen)
    return {"bytes": float(read * 2 * hkv * d * _size(case["cache"]) + 2 * tokens * hq * d * _size(case["dtype"])),
            "flops": float(flops)}


# ------------------------------------------------------------------ inputs

def _cache_inputs(case, g, dev):
    """The paged cache, its page table (pages in no order) and the step's lengths."""
    page, hkv, d = case["page"], case["kv_heads"], case["dim"]
    lens = torch.tensor(_seq_lens(case), dtype=torch.int32, device=dev)
    new = torch.tensor(_new_tokens(case), dtype=torch.int32, device=dev)
    pages = (lens + page - 1) // page
    pool = int(pages.sum()) + 3
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((len(lens), int(pages.max())), dtype=torch.int32, device=dev)
    table[torch.arange(table.shape[1], device=dev) < pages[:, None]] = order[:pool - 3]
    dt = DTYPES[case["cache"]]
    k = torch.empty((pool, hkv, page, d), dtype=dt, device=dev).normal_(generator=g)
    v = torch.empty((pool, hkv, page, d), dtype=dt, device=dev).normal_(0.1, 0.6, generator=g)
    start = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0, dtype=torch.int32)])
    return {"k_cache": k, "v_cache": v, "page_table": table, "seq_lens": lens, "new_start": start,
            "tokens": int(start[-1]), "max_new": max(_new_tokens(case))}


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


def _verify_inputs(case, g, dev):
    b, n, v = case["batch"], case["drafts"], case["vocab"]
    logits = torch.randn((b, n + 1, v), generator=g, device=dev) * 3
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits[:, :n] + torch.randn((b, n, v), generator=g, device=dev) * 0.5, -1)
    tokens = torch.multinomial(draft.flatten(0, 1), 1, generator=g).view(b, n).to(torch.int32)
    s = {"target": target, "draft": draft if case["probs"] else None, "draft_tokens": tokens,
         "uniforms": torch.rand((b, n + 1), generator=g, device=dev), "n_drafts": None,
         "tokens": torch.empty((b, n + 1), dtype=torch.int32, device=dev),
         "accepted": torch.empty(b, dtype=torch.int32, device=dev)}
    if case["ragged"]:
        s["n_drafts"] = torch.randint(0, n + 1, (b,), generator=g, device=dev, dtype=torch.int32)
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(int(seed))
    s = {"append": _append_inputs, "attention": _attention_inputs, "verify": _verify_inputs}[case["op"]](case, g, dev)
    s["case"] = case
    if own and case["op"] != "verify":  # the descriptors and the workspace that a serving loop keeps
        import qmoe_mnb_matmul_gb300 as mnb
        s["cache"] = mnb.kv_cache(s["k_cache"], s["v_cache"])
        s["step"] = mnb.kv_step(s["seq_lens"], s["page_table"], new_start=s["new_start"], tokens=s["tokens"],
                                max_new=s["max_new"])
        if case["op"] == "append":
            s["rope"] = mnb.kv_rope(s["cos_sin"], interleaved=case["interleaved"], q_norm=s["q_norm"],
                                    k_norm=s["k_norm"], eps=EPS)
        else:
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


def _plain_append(s):
    case = s["case"]
    _, pos, page, row = _token_places(s)
    table = s["cos_sin"][pos]
    s["q_out"].copy_(_rotated(s["q"].float(), s["q_norm"], table, case))
    dt = s["k_cache"].dtype
    s["k_cache"][page, :, row] = _rotated(s["k"].float(), s["k_norm"], table, case).to(dt)
    s["v_cache"][page, :, row] = s["v"].to(dt)
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    seq, pos, _, _ = _token_places(s)
    batch, most = s["seq_lens"].shape[0], s["max_new"]
    slot = torch.arange(s["tokens"], device=seq.device) - s["new_start"].long()[seq]
    table = s["page_table"].long()
    keys = s["k_cache"][table].float().transpose(2, 3).reshape(batch, -1, hkv, d)    # [b, length, kv head, d]
    values = s["v_cache"][table].float().transpose(2, 3).reshape(batch, -1, hkv, d)
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


def _plain_verify(s):
    target, draft, x = s["target"], s["draft"], s["draft_tokens"].long()
    b, n = x.shape
    i = torch.arange(n + 1, device=x.device)
    given = torch.full((b,), n, device=x.device) if s["n_drafts"] is None else s["n_drafts"].long()
    p = target[:, :n].gather(2, x[..., None])[..., 0]
    q = torch.ones_like(p) if draft is None else draft.gather(2, x[..., None])[..., 0]
    ok = (s["uniforms"][:, :n] * q < p) & (i[:n] < given[:, None])
    count = ok.long().cumprod(1).sum(1)
    row = torch.arange(b, device=x.device)
    weight = target[row, count]
    rejected = count < given
    r = count.clamp_max(n - 1)
    if draft is None:
        drafted = torch.zeros_like(weight).scatter_(1, x[row, r][:, None], weight.gather(1, x[row, r][:, None]))
    else:
        drafted = draft[row, r]
    weight = torch.where(rejected[:, None], weight - drafted, weight)
    whole = (weight.clamp(0.0, 1.0) * FIXED).long()
    sums = whole.cumsum(1)
    u = (s["uniforms"][:, n] * 2.0 ** 24).long()
    total = sums[:, -1]
    goal = (total >> 24) * u + (((total & 0xFFFFFF) * u) >> 24)
    last = (sums <= goal[:, None]).sum(1)
    tokens = torch.where(i[:n] < count[:, None], x, torch.full_like(x, -1))
    tokens = torch.cat([tokens, torch.full_like(x[:, :1], -1)], 1)
    tokens[row, count] = last
    s["tokens"].copy_(tokens)
    s["accepted"].copy_(count)
    return s["tokens"], s["accepted"]


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "verify": _plain_verify}[op](s)
    import qmoe_mnb_matmul_gb300 as mnb
    if op == "append":
        mnb.kv_append(s["cache"], s["step"], s["q"], s["k"], s["v"], s["q_out"], s["rope"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "attention":
        mnb.kv_attention(s["cache"], s["step"], s["q"], s["out"], s["workspace"], window=s["case"]["window"])
        return s["out"]
    mnb.draft_verify(s["target"], s["draft"], s["draft_tokens"], s["uniforms"], s["tokens"], s["accepted"],
                     n_drafts=s["n_drafts"])
    return s["tokens"], s["accepted"]


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_append(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    first = list(range(0, rot, 2)) if case["interleaved"] else list(range(half))
    second = list(range(1, rot, 2)) if case["interleaved"] else list(range(half, rot))
    starts, lens = s["new_start"].tolist(), s["seq_lens"].tolist()
    table, size = s["page_table"].long(), s["k_cache"].shape[2]
    q_out = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=table.device)
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()

    def turned(x, weight, angle_cos, angle_sin):
        if weight is not None:
            x = x * weight.double() * (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).rsqrt()
        y = x.clone()
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(angle_cos, angle_sin)[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    for b, length in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        pos = torch.arange(length - (hi - lo), length, device=table.device)
        cos, sin = s["cos_sin"][pos, :half].double(), s["cos_sin"][pos, half:].double()
        page, row = table[b, torch.div(pos, size, rounding_mode="floor")], pos.remainder(size)
        q_out[lo:hi] = turned(s["q"][lo:hi].double(), s["q_norm"], cos, sin)
        k_cache[page, :, row] = turned(s["k"][lo:hi].double(), s["k_norm"], cos, sin)
        v_cache[page, :, row] = s["v"][lo:hi].double()
    return q_out, k_cache, v_cache


def _exact_attention(s):
    case = s["case"]
    hkv, group, d = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    starts, lens = s["new_start"].tolist(), s["seq_lens"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    size = case["page"]
    for b, length in enumerate(lens):
        pages = s["page_table"][b, :-(-length // size)].long()
        for h in range(hkv):
            keys = s["k_cache"][pages, h].reshape(-1, d)[:length].double()
            values = s["v_cache"][pages, h].reshape(-1, d)[:length].double()
            for t in range(starts[b], starts[b + 1]):
                end = length - (starts[b + 1] - 1 - t)
                begin = max(0, end - case["window"]) if case["window"] else 0
                q = s["q"][t, h * group:(h + 1) * group].double()
                p = torch.softmax(q @ keys[begin:end].T * d ** -0.5, -1)
                out[t, h * group:(h + 1) * group] = p @ values[begin:end]
    return out


def _exact_verify(s):
    b, n = s["draft_tokens"].shape
    xs, us = s["draft_tokens"].tolist(), s["uniforms"].double().tolist()
    tokens, accepted = torch.full((b, n + 1), -1, dtype=torch.int32), torch.zeros(b, dtype=torch.int32)
    for k in range(b):
        given = n if s["n_drafts"] is None else int(s["n_drafts"][k])
        r = 0
        while r < given:
            q = 1.0 if s["draft"] is None else float(s["draft"][k, r, xs[k][r]])
            if not us[k][r] * q < float(s["target"][k, r, xs[k][r]]):
                break
            tokens[k, r] = xs[k][r]
            r += 1
        weight = s["target"][k, r].double()
        if r < given:
            if s["draft"] is None:
                weight[xs[k][r]] = 0.0
            else:
                # the weight is the single-precision difference: its rounding is part of the definition
                weight = (s["target"][k, r] - s["draft"][k, r]).double()
        whole = torch.floor(weight.clamp(0.0, 1.0) * FIXED).long().cpu()
        ends = whole.cumsum(0)
        goal = int(ends[-1]) * int(us[k][n] * 2 ** 24) >> 24
        tokens[k, r] = int(torch.searchsorted(ends, torch.tensor(goal), right=True))
        accepted[k] = r
    dev = s["tokens"].device
    return tokens.to(dev), accepted.to(dev)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "verify": _exact_verify}[case["op"]](s)
