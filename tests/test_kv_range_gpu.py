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
