"""token_probs at the ends of its ranges: row starts that no step has, equal logits in many places, temperatures
of any size.  The definition is tests/test_token_probs_gpu.py's."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402
from tests.test_token_probs_gpu import check, inputs, rules  # noqa: E402


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
