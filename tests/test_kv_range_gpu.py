"""kv_attention at the ends of its numbers' ranges: weights far below a row's largest,
queries with outliers or of extreme magnitude, infinite values, lengths past the
page table.  References and tolerances are those of tests/test_kv_gpu.py unless a test
derives a closer one."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402
from tests.test_kv_gpu import CONTENT, DT, HALF_ULP, TINY, Batch, check, reference, rng  # noqa: E402

# (query heads per key-value head, new tokens): row tiles of 8, 32 and 64 rows
ROWS = [(2, 1), (8, 3), (8, 6)]


def run(bt, q, scale=None, window=0, error=0):
    out = torch.full_like(q, 77.0)
    lse = torch.full(q.shape[:2], 77.0, device="cuda")
    mnb.kv_attention(bt.cache, bt.step, q, out, scale=scale, window=window, lse=lse)
    assert mnb.mnb_get_last_device_error() == error
    return out, lse


def set_token(bt, b, pos, k=None, v=None):
    page, row = bt.place(b, pos)
    if k is not None:
        bt.k[page, :, row] = k
    if v is not None:
        bt.v[page, :, row] = v


@pytest.mark.parametrize("cache,dtype", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("length", [60, 2048, 40001])  # one tile, one CTA's range, split over the GPU
@pytest.mark.parametrize("nats", [10, 14, 18, 22])
def test_weights_far_below_the_largest(cache, dtype, group, new, length, nats):
    """The first token leads all others by `nats` and its value is zero, so that the output is made of small weights
    alone (an attention sink).  One product of a score is not zero, so scores are exact; to log2 units they err by
    2^-22 of `nats` at most, the weights' parts and the sums as everywhere."""
    g = rng("sink", cache, dtype, group, new, length, nats)
    bt = Batch(g, [length], [new], 1, 128, 16, cache)
    bt.fill(g)
    pages = bt.table[0, :-(-length // 16)].long()
    bt.k[pages] = 0
    v = torch.rand((len(pages), 1, 16, 128), generator=g, device="cuda") * 2000 + 1000
    bt.v[pages] = v.to(bt.v.dtype)
    lead = torch.zeros(128, device="cuda")
    lead[3] = nats
    set_token(bt, 0, 0, lead.to(bt.k.dtype), 0.0)
    q = torch.zeros((new, group, 128), dtype=DT[dtype], device="cuda")
    q[..., 3] = 1.0
    out, lse = run(bt, q, scale=1.0)
    ref, rlse, (_, V) = reference(bt, q, group, 1.0, 0)
    parts = 2.0 ** -21 if dtype == "f32" else 2.0 ** -16
    tol = HALF_ULP[dtype] * ref.abs() + (V * (2 * nats * 2.0 ** -22 + parts + 2.0 ** -20))[..., None] + TINY[dtype]
    worst = ((out.double() - ref).abs() / tol).max().item()
    assert worst <= 1.0, f"output off by {worst:.3g} of its tolerance"
    assert bool(((lse.double() - rlse).abs() <= 2.0 ** -19 * (1 + rlse.abs())).all())


@pytest.mark.parametrize("cache,dtype", [("f16", "f16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("group,new", ROWS)
def test_spread_weights_below_a_sink(cache, dtype, group, new):
    """As above with other tokens of every weight from e^-16 to e^-8 of the first one's."""
    g = rng("spread", cache, dtype, group, new)
    bt = Batch(g, [1000, 130], [new, new], 2, 64, 24, cache)
    bt.fill(g)
    for b in range(2):
        for pos in range(bt.lens[b]):
            page, row = bt.place(b, pos)
            bt.k[page, :, row, 0] = 0.0 if pos else 12.0
            bt.v[page, :, row] = bt.v[page, :, row].abs() * 1000 if pos else 0.0
    q = torch.randn((bt.tokens, 2 * group, 64), generator=g, device="cuda") * 0.15
    q[..., 0] = 1.0
    q = q.to(DT[dtype])
    out, lse = run(bt, q, scale=1.0)
    check(bt, q, out, lse, group, 1.0, 0, dtype)


@pytest.mark.parametrize("cache", ["f16", "bf16"])
@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("scale,spread", [(1e-30, 1e-16), (1e-38, 1e-30), (2.0 ** -149, 1.0), (1e-31, 1e31), (1e-37, 1e37),
                                          (1e31, 1e-31), (1e36, 1e-37), (1e3, 1e-41)])
def test_queries_and_scales_of_any_magnitude(cache, group, new, scale, spread):
    """fp32 queries far from 1 with a scale that brings the scores back, or that leaves nothing of them (all weights
    equal)."""
    g = rng("magnitude", cache, group, new, scale, spread)
    bt = Batch(g, [300, 65, 1], [new, new, 1], 2, 128, 16, cache)
    bt.fill(g)
    q = torch.randn((bt.tokens, 2 * group, 128), generator=g, device="cuda") * spread
    q[0, 0] = 0.0
    out, lse = run(bt, q, scale=scale)
    check(bt, q, out, lse, group, float(torch.tensor(scale)), 0, "f32")


@pytest.mark.parametrize("cache", ["f16", "bf16"])
@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("ratio", [2.0 ** 8, 2.0 ** 12, 2.0 ** 16])
def test_a_query_element_that_dwarfs_the_others(cache, group, new, ratio):
    """The keys are zero where the query is large: the scores are made of its small elements."""
    g = rng("outlier", cache, group, new, ratio)
    bt = Batch(g, [300, 65], [new, new], 2, 128, 16, cache)
    bt.fill(g)
    for b in range(2):
        pages = bt.table[b, :-(-bt.lens[b] // 16)].long()
        bt.k[pages, :, :, 7] = 0
    q = torch.randn((bt.tokens, 2 * group, 128), generator=g, device="cuda") * 2
    q[..., 7] = 2.0 * ratio
    out, lse = run(bt, q)
    check(bt, q, out, lse, group, 128 ** -0.5, 0, "f32")


def past_the_table(g, cache, group, new, window, dtype):
    """Two sequences, the first longer than its page table of 7 pages of 16 tokens."""
    bt = Batch(g, [112, 70], [new, new], 2, 64, 16, cache)
    bt.fill(g)
    bt.seq_lens[0] = 112 + new - 1 if new > 1 else 112 + 5
    q = torch.randn((bt.tokens, 2 * group, 64), generator=g, device="cuda").to(DT[dtype])
    out, lse = run(bt, q, window=window, error=CONTENT)
    length, out64 = int(bt.seq_lens[0]), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    V = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    for i in range(new):
        pos = length - new + i
        lo, hi = (max(0, pos + 1 - window) if window else 0), min(pos + 1, 112)
        for h in range(2 * group):
            k, v = bt.rows_of(0, h // group)
            if lo < hi:
                p = torch.softmax(q[i, h].double() @ k[lo:hi].T / 8, -1)
                out64[i, h], V[i, h] = p @ v[lo:hi], (p @ v[lo:hi].abs()).max()
            assert bool(torch.isfinite(lse[i, h])) == (lo < hi)
    tol = HALF_ULP[dtype] * out64[:new].abs() + (V[:new] * 2.0 ** -12)[..., None] + TINY[dtype]
    assert bool(((out[:new].double() - out64[:new]).abs() <= tol).all())
    # the other sequence is as always
    bt.seq_lens[0] = 112
    again, _ = run(bt, q, window=window)
    check(bt, q, again, None, group, 0.125, window, dtype)
    assert torch.equal(again[new:], out[new:])


@pytest.mark.parametrize("cache,dtype", [("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("group,new", [(2, 1), (2, 4), (8, 3), (8, 6), (3, 40)])
@pytest.mark.parametrize("window", [0, 3, 50, 112, 120])
def test_a_length_past_the_page_table(cache, dtype, group, new, window):
    """New tokens keep their positions, and with them what they see of the tokens that have a page; the length is
    reported."""
    past_the_table(rng("past", cache, dtype, group, new, window), cache, group, new, window, dtype)


@pytest.mark.parametrize("cache,dtype", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("length,at", [(300, 10), (300, 100), (300, 290), (40001, 20000), (40001, 39990)])
def test_an_infinite_value_gives_that_infinity(cache, dtype, group, new, length, at):
    """Wherever the token lies in its tile and whatever its weight: a positive share of an infinity."""
    g = rng("infinite", cache, dtype, group, new, length, at)
    bt = Batch(g, [length, 70], [new, new], 2, 80, 16, cache)
    bt.fill(g)
    page, row = bt.place(0, at)
    bt.v[page, 0, row, 5] = math.inf
    bt.v[page, 1, row, 6] = -math.inf
    bt.v[page, 1, row, 79] = math.nan
    page, row = bt.place(0, 40)
    bt.v[page, 0, row, 9] = math.inf
    page, row = bt.place(0, 41)
    bt.v[page, 0, row, 9] = -math.inf
    q = (torch.randn((bt.tokens, 2 * group, 80), generator=g, device="cuda") * 2).to(DT[dtype])
    out, lse = run(bt, q)
    inf = torch.full((new, group), math.inf, dtype=out.dtype, device="cuda")
    assert torch.equal(out[:new, :group, 5], inf) and torch.equal(out[:new, group:, 6], -inf)
    assert bool(torch.isnan(out[:new, group:, 79]).all()) and bool(torch.isnan(out[:new, :group, 9]).all())
    odd = torch.zeros_like(out, dtype=torch.bool)
    odd[:new, :group, 5] = odd[:new, :group, 9] = odd[:new, group:, 6] = odd[:new, group:, 79] = True
    torch.nan_to_num_(bt.v, 0.0, 0.0, 0.0)  # what is not odd is as if those values were zero
    ref, rlse, (A, V) = reference(bt, q, group, 80 ** -0.5, 0)
    tol = HALF_ULP[dtype] * ref.abs() + (V * 2.0 ** -12)[..., None] + TINY[dtype]
    assert bool(((out.double() - ref).abs() <= tol)[~odd].all())
    assert bool(((lse.double() - rlse).abs() <= 1e-3).all())


@pytest.mark.parametrize("cache,dtype", [("f16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("lead", [0, 17000, 39000])  # before, among and after the infinite value's own part
def test_an_infinite_value_of_a_weight_below_fp32(cache, dtype, group, new, lead):
    """Another token leads by 200 nats: e^-200 is no fp32 number, and no zero."""
    g = rng("faint", cache, dtype, group, new, lead)
    bt = Batch(g, [40000], [new], 1, 64, 16, cache)
    bt.fill(g)
    pages = bt.table[0, :2500].long()
    bt.k[pages, :, :, 0] = 0
    set_token(bt, 0, lead, k=torch.nn.functional.one_hot(torch.tensor(0), 64).cuda() * 200.0)
    page, row = bt.place(0, 20000)
    bt.v[page, 0, row, 11] = math.inf
    q = torch.randn((new, group, 64), generator=g, device="cuda") * 0.1
    q[..., 0] = 1.0
    q = q.to(DT[dtype])
    out, _ = run(bt, q, scale=1.0)
    assert bool((out[..., 11] == math.inf).all())
    assert bool(torch.isfinite(out[..., :11]).all()) and bool(torch.isfinite(out[..., 12:]).all())


def test_a_value_that_overflows_the_cache_and_a_window_past_it():
    """fp32 values above 65504 become infinities of an fp16 cache; a window that has left them sees none."""
    g = rng("overflow")
    bt = Batch(g, [200], [1], 1, 64, 16, "f16", new_start=False)
    bt.fill(g)
    q = torch.randn((1, 2, 64), generator=g, device="cuda")
    k, v = torch.randn((1, 1, 64), generator=g, device="cuda"), torch.ones((1, 1, 64), device="cuda")
    v[0, 0, 3] = 1e6
    mnb.kv_append(bt.cache, bt.step, None, k, v, None)
    out, _ = run(bt, q)
    assert bool((out[..., 3] == math.inf).all()) and bool(torch.isfinite(out[..., 4:]).all())
    set_token(bt, 0, 199, v=0.0)
    page, row = bt.place(0, 150)
    bt.v[page, 0, row, 20] = -math.inf
    assert bool((run(bt, q)[0][..., 20] == -math.inf).all())
    assert bool((run(bt, q, window=50)[0][..., 20] == -math.inf).all())
    assert bool(torch.isfinite(run(bt, q, window=49)[0][..., 20]).all())
