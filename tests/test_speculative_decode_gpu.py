"""The example that runs the products, the paged cache, the attention and the draft
verification together (examples/speculative_decode.py)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402
from examples.speculative_decode import Decoder, generate  # noqa: E402

PROMPTS = [[5, 17, 99, 5, 17, 99, 5], [3], list(range(40, 90))]


def test_a_ragged_step_of_drafts_gives_the_logits_of_one_token_at_a_time():
    """The same tokens in one ragged step and one by one.  The two ways round every layer's activations to fp16 at the
    same places but add in other orders (other product kernels, other row tiles), so logits of magnitude about 1 may
    differ by a few fp16 roundings (2^-11) per layer: 2^-6 covers two layers of five roundings each."""
    model = Decoder(batch=2)
    first = [[7, 8, 9, 10, 11], [400]]
    drafts = [[12, 13, 14], [401, 402, 403, 404]]
    model.forward(first, [0, 0])
    together = model.forward(drafts, [5, 1])
    other = Decoder(batch=2)
    other.forward(first, [0, 0])
    alone = [[], []]
    for b in range(2):
        for i, t in enumerate(drafts[b]):
            logits = other.forward([[t] if s == b else [] for s in range(2)], [5 + (len(drafts[0]) if b else i), 1 + i if b else 1])
            alone[b].append(logits[0])
    alone = torch.stack(alone[0] + alone[1])
    assert torch.isfinite(together).all()
    assert (together - alone).abs().max() <= 2.0 ** -6 * alone.abs().max().clamp_min(1.0)
    assert mnb.mnb_get_last_device_error() == 0


def test_the_loop_runs_and_keeps_what_stands():
    model = Decoder()
    seqs, stood, fell = generate(model, PROMPTS, steps=12, drafts=4)
    assert mnb.mnb_get_last_device_error() == 0
    assert stood + fell > 0
    for s, p in zip(seqs, PROMPTS):
        assert s[:len(p)] == p and len(s) >= len(p) + 12
        assert all(0 <= t < model.vocab for t in s)
    # every step adds one token and the drafts that stood
    assert sum(len(s) - len(p) for s, p in zip(seqs, PROMPTS)) == 12 * len(PROMPTS) + stood
    # the same seeds, the same sequences
    again, _, _ = generate(Decoder(), PROMPTS, steps=12, drafts=4)
    assert again == seqs


def test_a_confident_model_accepts_its_own_repetitions():
    """Near zero temperature the model repeats itself, lookup finds the repetition and drafts stand."""
    model = Decoder(seed=3, vocab=61, batch=1)
    seqs, stood, fell = generate(model, [[1, 2, 3]], steps=60, drafts=4, temperature=1e-3)
    assert stood > 0
