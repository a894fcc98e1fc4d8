"""The example that runs the plan, the 8-bit cache, the token probabilities and the draft verification together
(examples/serving_loop.py)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402
from examples.serving_loop import Server, serve  # noqa: E402
from examples.speculative_decode import Decoder  # noqa: E402

PROMPTS = [[5, 17, 99, 5, 17, 99, 5], [3], list(range(40, 90))]


def test_the_loop_runs_twice_alike_and_gives_its_pages_back():
    model = Server()
    seqs, waits = serve(model, PROMPTS, steps=10, drafts=3)
    assert mnb.mnb_get_last_device_error() == 0
    for s, p in zip(seqs, PROMPTS):
        assert s[:len(p)] == p and len(s) >= len(p) + 10
        assert all(0 <= t < model.vocab for t in s)
    assert int(model.held.sum() + model.free_count) == model.pages
    owned = [int(p) for row, n in zip(model.table.tolist(), model.held.tolist()) for p in row[:n]]
    assert sorted(owned + model.free_pages[:int(model.free_count)].tolist()) == list(range(model.pages))
    again, _ = serve(Server(), PROMPTS, steps=10, drafts=3)
    assert again == seqs and waits == 0


def test_a_pool_too_small_makes_sequences_wait_for_those_that_end():
    model = Server(pages=6)  # 96 tokens; the three want 7, 1 and 50 and grow to 70 each
    seqs, waits = serve(model, PROMPTS, steps=60, drafts=2, limit=70)
    assert mnb.mnb_get_last_device_error() == 0
    assert waits > 0
    assert int(model.held.sum() + model.free_count) == 6
    assert len(seqs[2]) >= 70


def test_penalties_and_masks_reach_the_draw():
    model = Server(vocab=61, batch=2, pages=40)
    prompts = [[1, 2, 3], [7, 8]]
    once, _ = serve(model, prompts, steps=20, drafts=2, presence=1000.0)
    for s, p in zip(once, prompts):
        said = s[len(p):]
        assert len(said) == len(set(said))              # no token twice
    words = torch.zeros(2, dtype=torch.int32, device="cuda")
    words[0] = 0b111 << 20
    few, _ = serve(Server(vocab=61, batch=2, pages=40), prompts, steps=20, drafts=2, mask=words)
    for s, p in zip(few, prompts):
        assert set(s[len(p):]) <= {20, 21, 22}


def test_logits_over_codes_are_near_those_over_a_16_bit_cache():
    """Codes carry values to 2^-4 at most, 2^-5 in the mean, of which an average over a few tokens leaves less, against
    random residual streams of the same size: a quarter of the logits' norm is far above, a wrong page or scale far below."""
    tokens = [[7, 8, 9, 10, 11, 12, 13], [400, 401, 402], list(range(100, 140))]
    plain = Decoder().forward(tokens, [0, 0, 0])
    model = Server()
    model.step([t[:-2] for t in tokens], [0, 0, 0])
    codes, refused = model.step([t[-2:] for t in tokens], [len(t) - 2 for t in tokens])
    assert refused == [0, 0, 0] and mnb.mnb_get_last_device_error() == 0
    at = 0
    for b, t in enumerate(tokens):
        a, c = plain[at + len(t) - 2:at + len(t)], codes[2 * b:2 * b + 2]
        assert float((a - c).norm() / a.norm()) < 0.25
        at += len(t)
