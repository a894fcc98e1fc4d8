"""token_probs against its definition in 64 bits.

Tolerances.  A changed logit of magnitude up to X takes at most five fp32 operations (2^-24 each of a value up to X) and
a difference from the row's largest; with u = 2^-24 the exponent's argument errs by less than 6 u X / T + 2 u |argument|,
the exponential by 2^-22 and the sum and its division by a few u.  Rows here have X <= 64 after the changes and
T >= 0.3, so a probability is off by at most 2^-24 (6 * 64 / 0.3 + 2 * 128) + 2^-20 < 2^-13 relative."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402

REL = 2.0 ** -13
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def changed(row, b, i, r):
    """Row i of sequence b in 64 bits: the logits after penalties, biases and mask."""
    x, V = row.double(), row.shape[0]
    seen, count = torch.zeros(V, device="cuda").bool(), torch.zeros(V, device="cuda").double()
    tokens = []
    if r.get("history") is not None:
        n = min(max(int(r["history_lens"][b]), 0), r["history"].shape[1])
        p = int(r["prompt_lens"][b]) if r.get("prompt_lens") is not None else 0
        tokens = [(t, j >= p) for j, t in enumerate(r["history"][b, :n].tolist())]
    if r.get("draft_tokens") is not None:
        tokens += [(t, True) for t in r["draft_tokens"][b, :i].tolist()]
    for t, said in tokens:
        if 0 <= t < V:
            seen[t] = True
            count[t] += said
    get = lambda name, default: default if r.get(name) is None else r[name][b].double()  # noqa: E731
    rep = get("repetition", 1.0)
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = torch.where(seen, x - get("frequency", 0.0) * count, x)
    x = torch.where(count > 0, x - get("presence", 0.0), x)
    if r.get("bias_tokens") is not None:
        last = {t: v for t, v in zip(r["bias_tokens"][b].tolist(), r["bias_values"][b].tolist()) if 0 <= t < V}
        for t, v in last.items():
            x[t] += v
    if r.get("mask") is not None:
        bits = (r["mask"][b, i].view(-1, 1) >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        x = torch.where(bits.flatten()[:V] == 1, x, -math.inf)
    return x


def wanted(row, b, i, r, softmax=True):
    x = changed(row, b, i, r)
    T = 1.0 if r.get("temperature") is None else float(r["temperature"][b])
    if not softmax:
        return x / T if T > 0 else x
    if bool((x == -math.inf).all()):
        return torch.zeros_like(x)
    if T > 0:
        return torch.softmax(x / T, 0)
    y = torch.zeros_like(x)
    y[int((x == x.max()).nonzero()[0])] = 1.0
    return y


def rules(r, batch):
    keys = ("temperature", "history", "history_lens", "prompt_lens", "repetition", "frequency", "presence", "bias_tokens",
            "bias_values")
    return mnb.token_rules(batch=batch, **{k: r.get(k) for k in keys})


def inputs(seed, B, R, V, dtype, history=0, biases=0, mask=False, penalties=True):
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    ints = lambda hi, *s: torch.randint(0, hi, s, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    r = {"logits": (torch.randn((B, R, V), generator=g, device="cuda") * 4).to(DT[dtype]), "temperature": rand(B) + 0.3}
    few = max(1, V // 3)
    if history:
        r["history"] = ints(few, B, history)
        r["history"][:, ::7] = -1                     # padding
        r["history"][:, 3::11] = V + 5
        r["history_lens"] = torch.tensor([(history * (b + 1)) // B for b in range(B)], dtype=torch.int32, device="cuda")
        r["prompt_lens"] = r["history_lens"] // 2
        if R > 1:
            r["draft_tokens"] = ints(few, B, R - 1)
    if penalties:
        r["repetition"], r["frequency"], r["presence"] = rand(B) + 0.6, rand(B) * 0.2, rand(B) - 0.5
    if biases:
        r["bias_tokens"], r["bias_values"] = ints(few, B, biases) - 1, rand(B, biases) * 20 - 10
    if mask:
        r["mask"] = torch.randint(-2 ** 31, 2 ** 31, (B, R, -(-V // 32)), generator=g, device="cuda").to(torch.int32)
    return r


def check(out, r, softmax=True, rel=REL, rows=None):
    B, R, V = out.shape
    for b in range(B):
        for i in range(R if rows is None else rows[b]):
            src = r["logits"][b, i] if rows is None else r["logits"][sum(rows[:b]) + i]
            want = wanted(src, b, i, r, softmax)
            got = out[b, i].double()
            fine = torch.isfinite(want)
            assert torch.equal(got[~fine], want[~fine]), (b, i)
            # (an exponential below 2^-126 may be zero)
            scale = want.abs() if softmax else want.abs().clamp_min(1.0)
            assert ((got - want).abs()[fine] <= rel * scale[fine] + 2.0 ** -120).all(), (b, i)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,R,V,history,biases,mask", [
    (1, 1, 1, 0, 0, False), (2, 1, 3, 5, 2, True), (1, 5, 151936, 2000, 0, False), (3, 2, 50257, 100, 300, True),
    (5, 3, 997, 50, 16, True), (2, 2, 2048, 0, 7, False), (2, 2, 2049, 9, 0, True), (1, 2, 163841, 30, 3, False),
    (1, 1, 400000, 3000, 1, True), (1, 1, 400000, 30000, 2047, False), (3, 1, 262144, 20000, 9, True), (2, 4, 32768, 1, 0, False), (1, 1, 163968, 0, 0, True)])
def test_probabilities(dtype, B, R, V, history, biases, mask):
    r = inputs(B * 1000 + R, B, R, V, dtype, history, biases, mask)
    out = torch.full((B, R, V), 7.0, device="cuda")
    mnb.token_probs(r["logits"], rules(r, B), out, draft_tokens=r.get("draft_tokens"), mask=r.get("mask"))
    assert mnb.mnb_get_last_device_error() == 0
    check(out, r)
    again = torch.empty_like(out)
    mnb.token_probs(r["logits"], rules(r, B), again, draft_tokens=r.get("draft_tokens"), mask=r.get("mask"))
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype,V", [("f32", 50257), ("bf16", 4096), ("f16", 300001)])
def test_changed_logits(dtype, V):
    """The changed logits themselves: six roundings of values up to 64 / 0.3."""
    r = inputs(3, 3, 2, V, dtype, 200, 40, True)
    out = torch.empty((3, 2, V), device="cuda")
    mnb.token_probs(r["logits"], rules(r, 3), out, draft_tokens=r["draft_tokens"], mask=r["mask"], softmax=False)
    check(out, r, softmax=False, rel=6 * 64 / 0.3 * 2.0 ** -24)


def test_greedy_takes_the_first_of_equals():
    V = 40000
    logits = torch.zeros((4, 1, V), dtype=torch.bfloat16, device="cuda")
    logits[0, 0, [39999, 20001, 31000]] = 5.0
    logits[2, 0] = -math.inf
    logits[2, 0, [17, 30000]] = -9.0
    mask = torch.full((4, 1, V // 32), -1, dtype=torch.int32, device="cuda")
    mask[3] = 0
    mask[3, 0, 900] = 0b1100
    out = torch.empty((4, 1, V), device="cuda")
    mnb.token_probs(logits, mnb.token_rules(temperature=torch.tensor([0.0, -1.0, 0.0, 0.0], device="cuda")), out, mask=mask)
    assert out.sum(-1).flatten().tolist() == [1.0] * 4
    assert out.argmax(-1).flatten().tolist() == [20001, 0, 17, 900 * 32 + 2]


@pytest.mark.parametrize("V", [100, 50257, 200000])
def test_masked_places_and_rows_with_nothing_left(V):
    g = torch.Generator("cuda").manual_seed(1)
    logits = torch.randn((6, 1, V), generator=g, device="cuda")
    allowed = torch.rand((6, 1, V), generator=g, device="cuda") < 0.4
    allowed[1] = False
    allowed[4] = False
    logits[:, 0, ::5] = math.inf                      # in masked places alone
    logits[:, 0, 1::5] = math.nan
    allowed[:, 0, ::5] = False
    allowed[:, 0, 1::5] = False
    logits[3, 0, 2] = torch.finfo(torch.float32).min  # a mask of the lowest value, as far as that goes
    allowed[3, 0, 2] = True
    allowed[5, 0] = False
    allowed[5, 0, 2] = True
    logits[5, 0, 2] = -math.inf                       # allowed, and nothing
    padded = torch.zeros((6, 1, -(-V // 32) * 32), dtype=torch.int64, device="cuda")
    padded[..., :V] = allowed
    padded[..., V:] = 1                               # bits past the vocabulary mean nothing
    words = (padded.view(6, 1, -1, 32) << torch.arange(32, device="cuda")).sum(-1).to(torch.int32)
    T = torch.tensor([1.0, 1.0, 0.5, 2.0, 0.0, 1.0], device="cuda")
    out = torch.empty((6, 1, V), device="cuda")
    mnb.token_probs(logits, mnb.token_rules(temperature=T), out, mask=words)
    assert (out[[1, 4, 5]] == 0).all()
    check(out, {"logits": logits, "temperature": T, "mask": words})


def test_infinities_and_nan_that_are_allowed():
    V = 60000
    logits = torch.randn((4, 1, V), device="cuda")
    logits[0, 0, 5] = math.inf
    logits[1, 0, 59999] = math.nan
    logits[2, 0, 31000] = math.nan
    logits[3, 0, 123] = math.inf
    out = torch.empty((4, 1, V), device="cuda")
    mnb.token_probs(logits, mnb.token_rules(temperature=torch.tensor([1.0, 1.0, 0.0, 0.0], device="cuda")), out)
    assert out[:3].isnan().all()
    assert out[3].sum() == 1 and out[3, 0, 123] == 1


def test_extreme_temperatures():
    logits = torch.tensor([[[1.0, 3.0, 2.0, 3.0]]] * 3, device="cuda")
    out = torch.empty((3, 1, 4), device="cuda")
    T = torch.tensor([1e-42, 1e-30, math.inf], device="cuda")
    mask = torch.full((3, 1, 1), 0b1110, dtype=torch.int32, device="cuda")
    mnb.token_probs(logits, mnb.token_rules(temperature=T), out, mask=mask)
    assert out[:2].flatten().tolist() == [0.0, 0.5, 0.0, 0.5] * 2
    assert (out[2, 0] - torch.tensor([0.0, 1 / 3, 1 / 3, 1 / 3], device="cuda")).abs().max() < 1e-6


@pytest.mark.parametrize("dtype,V", [("f32", 1000), ("f16", 2001)])
def test_ragged_rows_strides_and_rows_left_alone(dtype, V):
    rows, B, R = [2, 0, 3, 1], 4, 3
    r = inputs(8, B, R, V, dtype, 40, 5, True)
    wide = torch.randn((sum(rows) + 2, V + 4), device="cuda").to(DT[dtype])
    r["logits"] = wide[:, :V]
    start = torch.tensor([0, 2, 2, 5, 6], dtype=torch.int32, device="cuda")
    big = torch.full((B, R + 1, V + 4), 7.0, device="cuda")
    out = big[:, :R, :V]
    mnb.token_probs(r["logits"], rules(r, B), out, row_start=start, draft_tokens=r["draft_tokens"], mask=r["mask"])
    check(out, r, rows=rows)
    for b, n in enumerate(rows):
        assert (big[b, n:] == 7.0).all() and (big[b, :, V:] == 7.0).all()
    assert mnb.mnb_get_last_device_error() == 0


def test_shared_rows_strided_history_and_in_place():
    V, B, R = 5000, 3, 2
    r = inputs(4, B, R, V, "f32", 30, 4, True)
    wide = torch.zeros((B, 64), dtype=torch.int32, device="cuda")
    wide[:, :30] = r["history"]
    r["history"] = wide[:, :30]
    r["mask"] = r["mask"][:1, :1].expand(B, R, -1)
    one = r["logits"][:1].expand(B, R, V)
    out = torch.empty((B, R, V), device="cuda")
    mnb.token_probs(one, rules(r, B), out, draft_tokens=r["draft_tokens"], mask=r["mask"])
    check(out, {**r, "logits": one})
    same = r["logits"].clone()
    mnb.token_probs(same, rules(r, B), same, draft_tokens=r["draft_tokens"], mask=r["mask"])
    check(same, r)


def test_no_rules_no_history_and_no_rows():
    logits = torch.randn((2, 1, 777), device="cuda")
    out = torch.empty_like(logits)
    mnb.token_probs(logits, mnb.token_rules(batch=2), out)
    check(out, {"logits": logits})
    empty = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    mnb.token_probs(logits, mnb.token_rules(history=empty, history_lens=lens, bias_tokens=empty,
                                            bias_values=empty.float()), out)
    check(out, {"logits": logits})
    none = torch.empty((2, 0, 777), device="cuda")
    mnb.token_probs(none, mnb.token_rules(batch=2), none)
    out.fill_(3.0)
    mnb.token_probs(torch.empty((0, 777), device="cuda"), mnb.token_rules(batch=2), out,
                    row_start=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert (out == 3.0).all()


def test_heavily_repeated_and_neighbouring_tokens():
    """Histories of one token and of a run of neighbours, the same token in the biases again and again, all of it in one
    CTA's words; counts stay whole numbers."""
    V, n = 151936, 6000
    g = torch.Generator("cuda").manual_seed(3)
    history = torch.stack([torch.full((n,), 7, device="cuda"), torch.arange(n, device="cuda") % 128,
                           torch.arange(n, device="cuda"), torch.full((n,), V - 1, device="cuda")]).to(torch.int32)
    r = {"logits": torch.randn((4, 2, V), generator=g, device="cuda"), "history": history,
         "history_lens": torch.full((4,), n, dtype=torch.int32, device="cuda"),
         "frequency": torch.full((4,), 2.0 ** -8, device="cuda"), "presence": torch.full((4,), 0.25, device="cuda"),
         "repetition": torch.full((4,), 1.25, device="cuda"),
         "bias_tokens": torch.full((4, 900), 7, dtype=torch.int32, device="cuda"),
         "bias_values": torch.linspace(-3, 3, 900, device="cuda").repeat(4, 1).contiguous(),
         "draft_tokens": torch.full((4, 1), 7, dtype=torch.int32, device="cuda")}
    out = torch.empty((4, 2, V), device="cuda")
    mnb.token_probs(r["logits"], rules(r, 4), out, draft_tokens=r["draft_tokens"])
    check(out, r)
    mnb.token_probs(r["logits"], rules(r, 4), out, draft_tokens=r["draft_tokens"], softmax=False)
    check(out, r, softmax=False, rel=6 * 64 * 2.0 ** -24)


def test_captured_beside_an_eager_call_and_on_another_stream():
    r = inputs(6, 2, 3, 33000, "bf16", 64, 3, True)
    out, eager = torch.empty((2, 3, 33000), device="cuda"), torch.empty((2, 3, 33000), device="cuda")
    d = rules(r, 2)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        mnb.token_probs(r["logits"], d, out, draft_tokens=r["draft_tokens"], mask=r["mask"])
    for k in range(2):
        r["history_lens"].fill_(10 + 20 * k)
        r["logits"].copy_(torch.randn_like(r["logits"]) * 3)
        torch.cuda.synchronize()
        graph.replay()
        mnb.token_probs(r["logits"], d, eager, draft_tokens=r["draft_tokens"], mask=r["mask"], stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        check(out, r)


def test_drafts_are_verified_against_these_probabilities():
    """Row i of a sequence counts the drafts ahead of it, and draft_verify takes the rows as they are: with the greedy
    temperature every draft that is the penalised row's largest token stands."""
    B, n, V = 3, 3, 5000
    g = torch.Generator("cuda").manual_seed(2)
    logits = torch.randn((B, n + 1, V), generator=g, device="cuda")
    drafts = torch.zeros((B, n), dtype=torch.int32, device="cuda")
    presence = torch.full((B,), 100.0, device="cuda")  # no token twice
    logits[:, :, 42] = 50.0                            # every row's largest, and allowed once
    drafts[:, 0] = 42
    for b in range(B):
        for i in range(1, n):
            drafts[b, i] = int(torch.cat([logits[b, i, :42], torch.tensor([-99.0], device="cuda"), logits[b, i, 43:]])
                               .index_fill(0, drafts[b, :i].long(), -99.0).argmax())
    drafts[2, 2] = 42                                  # said already: falls
    probs = torch.empty((B, n + 1, V), device="cuda")
    mnb.token_probs(logits, mnb.token_rules(temperature=torch.zeros(B, device="cuda"), presence=presence), probs,
                    draft_tokens=drafts)
    tokens, accepted = torch.empty((B, n + 1), dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    mnb.draft_verify(probs, None, drafts, torch.full((B, n + 1), 0.5, device="cuda"), tokens, accepted)
    assert accepted.tolist() == [3, 3, 2]
    assert mnb.mnb_get_last_device_error() == 0
