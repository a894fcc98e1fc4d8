"""kv_attention over 8-bit codes at the ends of its numbers' ranges: values, keys, queries and scales of any
magnitude.  References and tolerances are those of tests/test_kv_gpu.py unless a test derives another."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402
from tests.test_kv8_gpu import Codes, codes_of  # noqa: E402
from tests.test_kv_gpu import DT, HALF_ULP, TINY, check, reference, rng  # noqa: E402

# (query heads per key-value head, new tokens): row tiles of 8, 32 and 64 rows
ROWS = [(2, 1), (8, 3), (8, 6)]
LENGTHS = [1, 60, 2048, 40001]  # one token, one tile, one CTA's range, split over the GPU


def run(bt, q, scale=None):
    out = torch.full_like(q, 77.0)
    lse = torch.full(q.shape[:2], 77.0, device="cuda")
    mnb.kv_attention(bt.cache, bt.step, q, out, scale=scale, lse=lse)
    assert mnb.mnb_get_last_device_error() == 0
    return out, lse


def codes(g, like, largest):
    x = torch.randn(like.shape, generator=g, device="cuda").clamp(-4, 4) * (largest / 4)
    return codes_of(x.cpu()).to("cuda")


@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("power,largest", [(119, 448), (108, 448), (60, 448), (127, 1.5), (126, 3), (-110, 448)])
def test_values_of_any_magnitude(group, new, length, dtype, power, largest):
    """Up to 3.3e38, as appending leaves them and as scales alone allow; every weight about the same, so that sums of
    products with whole weights would pass the type's end."""
    length = max(length, new)
    g = rng("values", group, new, length, dtype, power)
    bt = Codes(g, [length], [new], 1, 128, 16, 16)
    bt.fill(g)
    bt.v.copy_(codes(g, bt.v, largest).abs() if length % 2 else codes(g, bt.v, largest))
    bt.vs.fill_(2.0 ** power)
    q = (torch.randn((new, group, 128), generator=g, device="cuda") * 0.05).to(DT[dtype])
    out, lse = run(bt, q)
    check(bt, q, out, lse, group, 128 ** -0.5, 0, dtype)


@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("length", [300, 3000, 40001])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("power", [40, 70, 100, 119])
def test_ordinary_values_beside_huge_ones_of_no_weight(group, new, length, first, power):
    """Half of the tokens have huge values and scores 200 below the others' (weights of 2^-288): the output is the other
    half's, with all of its bits; what is left of the huge ones is 2^-169 of an ordinary value."""
    g = rng("beside", group, new, length, first, power)
    bt = Codes(g, [length], [new], 1, 64, 16, 16)
    bt.fill(g)
    half = length // 2 // 64 * 64
    for pos in range(0, length, 16):
        page, _ = bt.place(0, pos)
        huge = (pos < half) == first
        bt.ks[page] = 2.0 ** -7
        bt.k[page] = 0xC6 if huge else 0x46  # -3.5 or 3.5: scores of +-100 at 2^-7 * 3.5 * 64 * q / 8
        bt.vs[page] = 2.0 ** (power if huge else -7)
    q = torch.full((new, group, 64), 100.0 / (2.0 ** -7 * 3.5 * 64 / 8), device="cuda")
    out, lse = run(bt, q)
    ref, rlse, (A, V) = reference(bt, q, group, 64 ** -0.5, 0)
    check(bt, q, out, lse, group, 64 ** -0.5, 0, "f32")


@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("length", [60, 2048, 40001])
@pytest.mark.parametrize("power,spread", [(100, 2.0 ** -107), (119, 2.0 ** -126), (60, 2.0 ** -67), (-60, 2.0 ** 53),
                                          (-126, 2.0 ** 119), (-100, 2.0 ** 93)])
def test_keys_of_any_magnitude_with_queries_that_bring_the_scores_back(group, new, length, power, spread):
    g = rng("keys", group, new, length, power)
    bt = Codes(g, [length], [new], 1, 128, 16, 16)
    bt.fill(g)
    bt.k.copy_(codes(g, bt.k, 400))
    bt.ks.fill_(2.0 ** power)
    q = torch.randn((new, group, 128), generator=g, device="cuda") * spread
    out, lse = run(bt, q)
    check(bt, q, out, lse, group, 128 ** -0.5, 0, "f32")


@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("power", [97, 110, 117])
def test_keys_that_leave_one_token(group, new, power):
    """Scores of up to 2^126: the largest takes all."""
    g = rng("one token", group, new, power)
    bt = Codes(g, [200], [new], 1, 64, 16, 16)
    bt.fill(g)
    bt.k.fill_(0x38)                                        # 1
    bt.ks.fill_(2.0 ** power)
    page, row = bt.place(0, 77)
    bt.k[page, :, row] = 0x40                               # 2
    q = torch.ones((new, group, 64), device="cuda")
    out, lse = run(bt, q)
    _, v = bt.rows_of(0, 0)
    assert bool(((out.double() - v[77]).abs() <= 2.0 ** -20 * v[77].abs()).all())
    assert bool((lse == 2.0 ** (power + 4)).all())          # 64^-0.5 * 64 * 2 * 2^power


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("scale,spread", [(1e-30, 1e-16), (1e-38, 1e-30), (2.0 ** -149, 1.0), (1e-31, 1e31), (1e-37, 1e37),
                                          (1e31, 1e-31), (1e36, 1e-37)])
def test_queries_and_scales_of_any_magnitude(dtype, group, new, scale, spread):
    """Queries far from 1 with a scale that brings the scores back, or that leaves nothing of them."""
    g = rng("magnitude", dtype, group, new, scale)
    bt = Codes(g, [300, 65, 1], [new, new, 1], 2, 128, 16, 16)
    bt.fill(g)
    q = (torch.randn((bt.tokens, 2 * group, 128), generator=g, device="cuda") * spread).to(DT[dtype])
    q[0, 0] = 0.0
    out, lse = run(bt, q, scale=scale)
    check(bt, q, out, lse, group, float(torch.tensor(scale)), 0, dtype)
