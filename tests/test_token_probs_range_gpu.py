"""token_probs at the ends of its ranges: row starts that no step has, equal logits in many places, temperatures
of any size.  The definition is tests/test_token_probs_gpu.py's."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402
from tests.test_token_probs_gpu import DT, check, inputs, rules  # noqa: E402

CONTENT = 7


@pytest.mark.parametrize("V", [1000, 2001])
def test_row_starts_at_the_end_of_32_bits(V):
    """The first row of sequence 1 would be the last that 32 bits count: it and the rows behind it are not there."""
    B, R = 3, 4
    r = inputs(5, B, R, V, "f32")
    r["logits"] = r["logits"][0, :2].contiguous()
    start = torch.tensor([0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    r["logits"] = torch.cat([r["logits"], r["logits"] + 1])
    out = torch.full((B, R, V), 7.0, device="cuda")
    mnb.token_probs(r["logits"], rules(r, B), out, row_start=start)
    check(out, r, rows=[4, 0, 0])
    assert bool((out[1:] == 7.0).all())
    assert mnb.mnb_get_last_device_error() == 0


@pytest.mark.parametrize("B,V", [(1, 151936), (3, 50257), (8, 32000), (64, 30001)])
@pytest.mark.parametrize("seed", range(4))
def test_equal_logits_get_equal_probabilities(B, V, seed):
    """Tokens of one logit in every lane, warp and CTA, whose own sums and largest values differ; some come to that
    logit by a bias (both numbers and their sum are whole), so that they are joined apart."""
    r = inputs(seed, B, 2, V, "f32", penalties=False)
    r["logits"][..., 5::37] = 3.0
    listed = torch.arange(17, V, 331, dtype=torch.int32, device="cuda")[:90]
    r["logits"][..., listed.long()] = -2.0
    r["bias_tokens"] = listed.expand(B, -1).contiguous()
    r["bias_values"] = torch.full((B, len(listed)), 5.0, device="cuda")
    out = torch.empty((B, 2, V), device="cuda")
    mnb.token_probs(r["logits"], rules(r, B), out)
    equal = torch.zeros(V, dtype=torch.bool, device="cuda")
    equal[5::37] = True
    equal[listed.long()] = True
    p = out[..., equal]
    assert bool((p > 0).all()) and bool((p == p[..., :1]).all())
    for b in range(0, B, 16):
        check(out[b:b + 1], {k: v[b:b + 1] for k, v in r.items() if v is not None})


def test_rows_that_the_logits_do_not_have_are_reported():
    """A sequence's rows that lie outside the step's logits: their probabilities are left alone, and the error word says
    so.  Rows that a sequence does not ask for are no error."""
    V, B, R = 1500, 3, 3
    r = inputs(9, B, R, V, "bf16")
    r["logits"] = r["logits"].flatten(0, 1)[:5].contiguous()
    d = rules(r, B)

    def run(*start):
        out = torch.full((B, R, V), 7.0, device="cuda")
        mnb.token_probs(r["logits"], d, out, row_start=torch.tensor(start, dtype=torch.int32, device="cuda"))
        return out, mnb.mnb_get_last_device_error()

    whole, error = run(0, 2, 2, 5)
    assert error == 0
    check(whole, r, rows=[2, 0, 3])
    out, error = run(0, 2, 2, 6)             # sequence 2 has four rows, three places in out: no row past the logits
    assert error == 0 and torch.equal(out, whole)
    out, error = run(0, 2, 3, 6)             # the last row of sequence 2 is row 5 of 5
    assert error == CONTENT
    assert bool((out[2, 2] == 7.0).all()) and bool((out[1, 1:] == 7.0).all()) and torch.equal(out[0], whole[0])
    out, error = run(-2, 2, 2, 5)            # sequence 0 begins before the logits
    assert error == CONTENT
    assert bool((out[0] == 7.0).all()) and torch.equal(out[1:], whole[1:])
    out, error = run(7, 7, 7, 7)             # no rows at all
    assert error == 0 and bool((out == 7.0).all())
    out, error = run(0, 2, 2, 5)
    assert error == 0 and torch.equal(out, whole)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("temperature", [1e30, 1e37, 1.2e38, 2e38, 3.4e38])
def test_temperatures_as_large_as_the_logits(dtype, temperature):
    """(x - m) / T is of the order of one: its two roundings are 2^-24 of at most 4 each and the logarithm's base a
    third, the exponential and the sum err by a few 2^-22."""
    r = inputs(11, 2, 2, 3001, "f32", penalties=False)
    r["logits"] = (r["logits"].clamp(-7, 7) / 7 * min(1.6e38, 2 * temperature)).to(DT[dtype])
    r["temperature"] = torch.tensor([temperature, 1.0], device="cuda")
    out = torch.empty((2, 2, 3001), device="cuda")
    mnb.token_probs(r["logits"], rules(r, 2), out)
    check(out, r, rel=2.0 ** -18)


def test_an_infinite_temperature_leaves_the_row_even():
    x = torch.tensor([[[1.0, -3e38, 2e37, 0.0]]], device="cuda")
    out = torch.empty_like(x)
    mnb.token_probs(x, mnb.token_rules(temperature=torch.full((1,), float("inf"), device="cuda")), out)
    # 1 / T is held as fp32's smallest number, 2^-149, so that -infinity times it stays that: differences of less than
    # 2^129 come out as exponents below 2^-20
    assert bool(((out - 0.25).abs() <= 0.25 * 2.0 ** -19).all())
