"""draft_verify against a plain implementation of its definition: 64-bit numbers
and whole-number sums, one token after the other.  Every output is a whole
number and has to be equal."""
import zlib

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402

CONTENT = 7


def rng(*key):
    return np.random.default_rng(zlib.crc32(repr(key).encode()))


def draw(weight, uniform):
    """The smallest entry whose inclusive whole-number sum passes floor(U sum / 2^24); None without weight."""
    w = np.nan_to_num(weight.astype(np.float64), nan=0.0, posinf=1.0, neginf=0.0).clip(0.0, 1.0)
    ends = np.cumsum(np.floor(w * 2.0 ** 40).astype(np.int64))
    if ends[-1] == 0:
        return None
    U = int(np.floor(np.float64(uniform) * 2 ** 24)) if uniform > 0 else 0
    goal = (int(ends[-1]) * min(U, 2 ** 24 - 1)) >> 24
    return int(np.searchsorted(ends, goal, side="right"))


def reference(target, draft, tokens, uniforms, given):
    B, n1, V = target.shape
    n = n1 - 1
    out, acc = np.full((B, n1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        m = n if given is None else min(max(int(given[b]), 0), n)
        r = 0
        while r < m:
            x = int(tokens[b, r])
            if not 0 <= x < V:
                break
            q = np.float32(1) if draft is None else draft[b, r, x]
            if not np.float32(uniforms[b, r] * q) < target[b, r, x]:
                break
            out[b, r] = x
            r += 1
        weight = target[b, r].copy()
        if r < m:
            if draft is not None:
                with np.errstate(invalid="ignore"):
                    weight = target[b, r] - draft[b, r]
            elif 0 <= tokens[b, r] < V:
                weight[tokens[b, r]] = 0
        x = draw(weight, uniforms[b, n])
        if x is None:
            x = draw(target[b, r], uniforms[b, n])
        out[b, r] = -1 if x is None else x
        acc[b] = r
    return out, acc


def run(target, draft, tokens, uniforms, given=None, stream=None):
    cu = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    B, n1, _ = target.shape
    out = torch.full((B, n1), -9, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    mnb.draft_verify(cu(target), cu(draft), cu(tokens), cu(uniforms), out, acc, n_drafts=cu(given), stream=stream)
    torch.cuda.synchronize()
    return out.cpu().numpy(), acc.cpu().numpy()


def inputs(g, B, n, V, spread=3.0, apart=0.5):
    def softmax(x):
        e = np.exp(x - x.max(-1, keepdims=True))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)
    logits = g.standard_normal((B, n + 1, V)) * spread
    draft = softmax(logits[:, :n] + g.standard_normal((B, n, V)) * apart)
    target = softmax(logits)
    tokens = np.zeros((B, n), np.int32)
    for b in range(B):
        for i in range(n):
            tokens[b, i] = min(np.searchsorted(np.cumsum(draft[b, i].astype(np.float64)), g.random()), V - 1)
    return target, draft, tokens, g.random((B, n + 1)).astype(np.float32)


@pytest.mark.parametrize("B,n,V", [(1, 4, 151936), (1, 1, 1), (3, 2, 2), (5, 3, 31), (7, 5, 128), (40, 4, 129),
                                   (2, 3, 50257), (33, 6, 1000), (300, 2, 4099), (1, 0, 777), (6, 40, 257)])
@pytest.mark.parametrize("probs,ragged", [(True, False), (True, True), (False, True)])
def test_matches_the_definition(B, n, V, probs, ragged):
    g = rng("match", B, n, V, probs, ragged)
    target, draft, tokens, uniforms = inputs(g, B, n, V)
    given = g.integers(-1, n + 2, B).astype(np.int32) if ragged else None
    draft = draft if probs else None
    out, acc = run(target, draft, tokens, uniforms, given)
    rout, racc = reference(target, draft, tokens, uniforms, given)
    assert np.array_equal(acc, racc) and np.array_equal(out, rout)
    assert mnb.mnb_get_last_device_error() == 0


def test_uniforms_at_both_ends_and_on_boundaries():
    """Flat rows of 2^k entries put the drawn point on a boundary between entries for every multiple of 2^-k."""
    V, B = 1024, 64
    target = np.full((B, 1, V), 1.0 / V, np.float32)
    u = (np.arange(B, dtype=np.float32) / B).reshape(B, 1)
    u[-1] = np.float32(1) - np.float32(2.0 ** -24)
    out, _ = run(target, None, np.zeros((B, 0), np.int32), u)
    want = np.floor(u[:, 0].astype(np.float64) * V).astype(np.int32)
    assert np.array_equal(out[:, 0], want) and out[0, 0] == 0 and out[-1, 0] == V - 1
    # outside [0, 1), and NaN: the nearest end
    u = np.array([[-0.5], [1.0], [7.0], [np.nan], [np.inf]], np.float32)
    out, _ = run(target[:5], None, np.zeros((5, 0), np.int32), u)
    assert out[:, 0].tolist() == [0, V - 1, V - 1, 0, V - 1]


def test_only_one_entry_has_weight():
    for V in (1, 5, 4096, 151936):
        for at in {0, V // 2, V - 1}:
            target = np.zeros((2, 1, V), np.float32)
            target[:, 0, at] = [1.0, 1e-9]
            out, _ = run(target, None, np.zeros((2, 0), np.int32), np.array([[0.0], [0.9999999]], np.float32))
            assert out[:, 0].tolist() == [at, at]


def test_equal_distributions_and_zero_probabilities():
    g = rng("equal")
    target, _, tokens, uniforms = inputs(g, 8, 3, 500)
    draft = target[:, :3].copy()
    out, acc = run(target, draft, tokens, uniforms)       # p = q: every draft stands
    assert np.array_equal(acc, np.full(8, 3)) and np.array_equal(out[:, :3], tokens)
    target2 = target.copy()
    target2[np.arange(8)[:, None], np.arange(3), tokens] = 0  # the target never says the drafted token
    out, acc = run(target2, draft, tokens, uniforms)
    rout, racc = reference(target2, draft, tokens, uniforms, None)
    assert np.array_equal(acc, np.zeros(8)) and np.array_equal(out, rout) and np.array_equal(racc, acc)


def test_nothing_left_of_the_weights():
    """p <= q everywhere and the draft falls: drawn from p; a row of zeros gives -1 and is reported."""
    V = 300
    target = np.full((2, 2, V), 0.001, np.float32)
    draft = np.full((2, 1, V), 0.002, np.float32)
    tokens = np.zeros((2, 1), np.int32)
    uniforms = np.array([[0.9, 0.5], [0.9, 0.1]], np.float32)
    out, acc = run(target, draft, tokens, uniforms)
    rout, _ = reference(target, draft, tokens, uniforms, None)
    assert acc.tolist() == [0, 0] and np.array_equal(out, rout)
    assert mnb.mnb_get_last_device_error() == 0
    target[1] = 0
    out, acc = run(target, draft, tokens, uniforms)
    assert out[1].tolist() == [-1, -1] and acc[1] == 0
    assert mnb.mnb_get_last_device_error() == CONTENT


def test_nan_infinity_and_tokens_outside_the_vocabulary():
    g = rng("odd")
    target, draft, tokens, uniforms = inputs(g, 6, 2, 700)
    target[0, 0, 5] = np.nan
    draft[1, 0, 7] = np.nan
    target[2, 1, 9] = np.inf
    target[3, 0, 11] = -np.inf
    out, acc = run(target, draft, tokens, uniforms)
    rout, racc = reference(target, draft, tokens, uniforms, None)
    assert np.array_equal(out, rout) and np.array_equal(acc, racc)
    assert mnb.mnb_get_last_device_error() == 0
    for bad in (-1, 700, 2 ** 31 - 1):
        tokens[4, 0] = bad
        for probs in (draft, None):
            out, acc = run(target, probs, tokens, uniforms)
            rout, racc = reference(target, probs, tokens, uniforms, None)
            assert np.array_equal(out, rout) and np.array_equal(acc, racc) and acc[4] == 0
            assert mnb.mnb_get_last_device_error() == CONTENT


def test_strided_probabilities():
    """Rows padded to a wider vocabulary, sequences apart, rows that are not 16-byte aligned."""
    g = rng("strided")
    B, n, V = 5, 3, 1000
    target, draft, tokens, uniforms = inputs(g, B, n, V)
    rout, racc = reference(target, draft, tokens, uniforms, None)
    for pad, lead in ((24, 0), (24, 4), (1, 0), (24, 1)):
        T = torch.full((B, n + 3, V + pad), 9.0, device="cuda")
        D = torch.full((B, n + 2, V + pad), -9.0, device="cuda")
        t, d = T[:, 1:n + 2, lead:V + lead] if lead + V <= V + pad else T[:, 1:n + 2, :V], D[:, :n, :V]
        t.copy_(torch.from_numpy(target))
        d.copy_(torch.from_numpy(draft))
        out = torch.empty((B, n + 1), dtype=torch.int32, device="cuda")
        acc = torch.empty(B, dtype=torch.int32, device="cuda")
        mnb.draft_verify(t, d, torch.from_numpy(tokens).cuda(), torch.from_numpy(uniforms).cuda(), out, acc)
        assert np.array_equal(out.cpu().numpy(), rout) and np.array_equal(acc.cpu().numpy(), racc)


def test_draws_follow_the_target_distribution():
    """Drafting and verifying gives the target's distribution, whatever the drafts: 2e5 first tokens over 8
    entries against their probabilities, within five standard deviations."""
    g = rng("distribution")
    N, V = 200_000, 8
    p = np.array([0.3, 0.05, 0.2, 0.01, 0.14, 0.1, 0.15, 0.05], np.float32)
    q = np.array([0.1, 0.2, 0.1, 0.2, 0.1, 0.1, 0.1, 0.1], np.float32)
    target = torch.from_numpy(p).cuda().expand(N, 2, V)
    for probs in (True, False):
        draft = torch.from_numpy(q).cuda().expand(N, 1, V) if probs else None
        tokens = torch.from_numpy(g.choice(V, size=(N, 1), p=q / q.sum()).astype(np.int32)).cuda()
        uniforms = torch.from_numpy(g.random((N, 2)).astype(np.float32)).cuda()
        out = torch.empty((N, 2), dtype=torch.int32, device="cuda")
        acc = torch.empty(N, dtype=torch.int32, device="cuda")
        mnb.draft_verify(target, draft, tokens, uniforms, out, acc)
        share = np.bincount(out[:, 0].cpu().numpy(), minlength=V) / N
        if probs:
            assert np.all(np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / N))
        # a fixed draft that stands with its own probability, else another token by what is left of p
        else:
            assert np.all(np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / N))


def test_another_stream_and_refusals():
    g = rng("refuse")
    target, draft, tokens, uniforms = inputs(g, 3, 2, 400)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, acc = run(target, draft, tokens, uniforms, stream=s)
    rout, racc = reference(target, draft, tokens, uniforms, None)
    assert np.array_equal(out, rout) and np.array_equal(acc, racc)
    t = torch.from_numpy(target).cuda()
    x, u = torch.from_numpy(tokens).cuda(), torch.from_numpy(uniforms).cuda()
    o, a = torch.empty((3, 3), dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        mnb.draft_verify(t.half(), None, x, u, o, a)
    with pytest.raises(ValueError):
        mnb.draft_verify(t, t, x, u, o, a)
    with pytest.raises(ValueError):
        mnb.draft_verify(t, None, x[:, :1], u, o, a)
    with pytest.raises(TypeError):
        mnb.draft_verify(t, None, x.long(), u, o, a)
    with pytest.raises(ValueError):
        mnb.draft_verify(t.cpu(), None, x, u, o, a)
    with pytest.raises(ValueError):
        mnb.draft_verify(t.transpose(1, 2), None, x, u, o, a)
