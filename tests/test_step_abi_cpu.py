"""CPU-side checks of kv_plan and token_probs: metadata errors come before any GPU work, and the binding refuses tensors
of the wrong shape, type, layout or device."""
import ctypes

import pytest

import qmoe_mnb_matmul_gb300 as mnb
from qmoe_mnb_matmul_gb300 import _binding, _build

torch = pytest.importorskip("torch")

from tests.test_kv_binding_cpu import Tensor, f32, i32  # noqa: E402
from tests.test_kv_binding_cpu import lib as fake  # noqa: E402,F401

OK, INVALID, UNSUPPORTED, OVERFLOW = 0, 1, 2, 3
FAKE = 0x10000  # 64 KiB-aligned fake device address: never dereferenced by these calls


@pytest.fixture(scope="module")
def real():
    _build.build()
    return mnb.load_library()


def plan(lib, keep=FAKE, add=FAKE, lens=FAKE, start=FAKE, most=100, slots=FAKE, refused=FAKE, **kw):
    d = dict(held=FAKE, page_table=FAKE, table_stride=10, free_pages=FAKE, free_count=FAKE, held_out=FAKE, free_count_out=FAKE,
             batch=4, max_pages=10, num_pages=50, page_size=16)
    d.update(kw)
    return lib.kv_plan(ctypes.byref(mnb.KvPoolDesc(**d)), keep, add, lens, start, most, slots, refused, None)


def test_plan_errors(real):
    assert real.kv_plan(None, FAKE, FAKE, FAKE, FAKE, 1, None, None, None) == INVALID
    for bad in (dict(held=None), dict(page_table=None), dict(free_pages=None), dict(free_count=None), dict(held_out=None),
                dict(free_count_out=None), dict(batch=-1), dict(num_pages=-1), dict(page_size=0), dict(max_pages=0),
                dict(table_stride=9), dict(keep=None), dict(add=None), dict(lens=None), dict(start=None), dict(most=-1)):
        assert plan(real, **bad) == INVALID, bad
    for bad in (dict(batch=8193), dict(held=FAKE + 2), dict(page_table=FAKE + 1), dict(free_pages=FAKE + 2),
                dict(free_count=FAKE + 2), dict(held_out=FAKE + 2), dict(free_count_out=FAKE + 1), dict(keep=FAKE + 2),
                dict(add=FAKE + 2), dict(lens=FAKE + 2), dict(start=FAKE + 2), dict(slots=FAKE + 4), dict(refused=FAKE + 2)):
        assert plan(real, **bad) == UNSUPPORTED, bad
    for bad in (dict(most=(1 << 30) + 1), dict(table_stride=1 << 61)):
        assert plan(real, **bad) == OVERFLOW, bad


def probs(lib, logits=FAKE, dt=0, ls=5000, lr=1000, start=None, tokens=0, drafts=None, mask=None, ms=320, mr=32, rows=5,
          vocab=1000, out=FAKE, os=5000, orow=1000, softmax=1, **kw):
    rules = mnb.TokenRules(**{**dict(batch=2), **kw})
    return lib.token_probs(logits, dt, ls, lr, start, tokens, ctypes.byref(rules), drafts, mask, ms, mr, rows, vocab, out, os,
                           orow, softmax, None)


def test_probs_errors(real):
    assert real.token_probs(FAKE, 0, 1, 1, None, 0, None, None, None, 0, 0, 1, 1, FAKE, 1, 1, 1, None) == INVALID
    for bad in (dict(logits=None), dict(out=None), dict(dt=3), dict(dt=-1), dict(batch=-1), dict(rows=-1), dict(vocab=0),
                dict(ls=-1), dict(lr=-1), dict(ms=-1), dict(mr=-1), dict(orow=999), dict(os=10), dict(tokens=-1),
                dict(history=FAKE, history_columns=5, history_stride=5), dict(history_columns=-1), dict(biases=-1),
                dict(history=FAKE, history_lens=FAKE, history_columns=5, history_stride=4),
                dict(biases=3, bias_tokens=FAKE, bias_stride=3), dict(biases=3, bias_values=FAKE, bias_stride=3),
                dict(biases=3, bias_tokens=FAKE, bias_values=FAKE, bias_stride=2)):
        assert probs(real, **bad) == INVALID, bad
    long = dict(os=1 << 24, orow=1 << 23, ls=1 << 24, lr=1 << 23)
    lots = dict(history=FAKE, history_lens=FAKE, history_columns=500000, history_stride=500000)
    extra = dict(biases=1, bias_tokens=FAKE, bias_values=FAKE, bias_stride=1)
    for bad in (dict(vocab=1 << 22, **long), dict(rows=1026, os=1 << 21), dict(logits=FAKE + 2), dict(logits=FAKE + 1, dt=1),
                dict(out=FAKE + 2), dict(start=FAKE + 2, tokens=9), dict(drafts=FAKE + 2), dict(mask=FAKE + 1),
                dict(temperature=FAKE + 2), dict(presence=FAKE + 2), dict(vocab=1 << 21, **lots, **long),
                dict(vocab=460801, **lots, **extra, **long),
                dict(history=FAKE, history_lens=FAKE, history_columns=1 << 20, history_stride=1 << 20),
                dict(biases=2048, bias_tokens=FAKE, bias_values=FAKE, bias_stride=2048)):
        assert probs(real, **bad) == UNSUPPORTED, bad
    for bad in (dict(lr=1 << 61), dict(os=1 << 61), dict(mask=FAKE, ms=1 << 61), dict(batch=1 << 26),
                dict(start=FAKE, tokens=1 << 40, lr=1 << 40)):
        assert probs(real, **bad) == OVERFLOW, bad
    assert probs(real, batch=0, logits=None, out=None) == OK
    assert probs(real, rows=0, logits=None, out=None) == OK


# ------------------------------------------------------------------ the binding

def pool(device=0, **kw):
    d = dict(held=i32(3, device=device), page_table=i32(3, 4, device=device), free_pages=i32(9, device=device),
             free_count=i32(1, device=device))
    d.update(kw)
    return mnb.kv_pool(d.pop("held"), d.pop("page_table"), d.pop("free_pages"), d.pop("free_count"), 16, **d)


def test_pool_and_plan_refusals(fake):  # noqa: F811
    go = lambda p=None, keep=None, new=None, lens=None, start=None, **kw: mnb.kv_plan(  # noqa: E731
        p or pool(), keep or i32(3), new or i32(3), lens or i32(3), start or i32(4), **kw)
    go(slots=Tensor((20,), torch.int64), refused=i32(3))
    name, args = fake.calls.pop()
    assert name == "kv_plan" and args[5] == 20
    go()
    assert fake.calls.pop()[1][5] == 1 << 30
    go(slots=Tensor((20,), torch.int64), max_tokens=7)
    assert fake.calls.pop()[1][5] == 7
    for bad in (dict(page_table=i32(2, 4)), dict(page_table=i32(12)), dict(free_count=i32(2)), dict(free_pages=i32(3, 3)),
                dict(held_out=i32(4)), dict(free_count_out=i32(2)), dict(held=i32(3, device=-1))):
        with pytest.raises(ValueError):
            pool(**bad)
    with pytest.raises(TypeError):
        pool(held=f32(3))
    for bad in (dict(keep=i32(2)), dict(new=i32(4)), dict(lens=i32(4)), dict(start=i32(3)), dict(refused=i32(2)),
                dict(slots=Tensor((20,), torch.int64), max_tokens=21), dict(p=pool(1)), dict(new=i32(3, device=1)),
                dict(keep=i32(3, device=1))):
        with pytest.raises(ValueError):
            go(**bad)
    for bad in (dict(slots=i32(20)), dict(keep=Tensor((3,), torch.int64))):
        with pytest.raises(TypeError):
            go(**bad)
    assert fake.calls == []


def test_rules_and_probs_refusals(fake):  # noqa: F811
    for bad in (dict(), dict(temperature=f32(3), presence=f32(4)), dict(history=i32(3, 5)), dict(history_lens=i32(3)),
                dict(prompt_lens=i32(3)), dict(bias_tokens=i32(3, 5)), dict(bias_tokens=i32(3, 5), bias_values=f32(3, 4)),
                dict(history=i32(3, 5), history_lens=i32(4)), dict(history=i32(15), history_lens=i32(3)),
                dict(temperature=f32(3), presence=f32(3, device=1)), dict(temperature=f32(3, device=-1))):
        with pytest.raises(ValueError):
            mnb.token_rules(**bad)
    with pytest.raises(TypeError):
        mnb.token_rules(temperature=i32(3))
    rules = mnb.token_rules(temperature=f32(3), history=i32(3, 5), history_lens=i32(3))
    assert (rules.batch, rules.history_columns, rules.history_stride) == (3, 5, 5)
    go = lambda logits=None, r=rules, out=None, **kw: mnb.token_probs(  # noqa: E731
        logits or Tensor((3, 2, 100)), r, out or f32(3, 2, 100), **kw)
    go(draft_tokens=i32(3, 1), mask=i32(3, 2, 4))
    assert fake.calls.pop()[0] == "token_probs"
    go(logits=Tensor((5, 100)), row_start=i32(4))
    assert fake.calls.pop()[1][5] == 5
    for bad in (dict(logits=Tensor((3, 2, 99))), dict(logits=Tensor((5, 100))), dict(logits=Tensor((5, 99)), row_start=i32(4)),
                dict(logits=Tensor((5, 100)), row_start=i32(3)), dict(out=f32(4, 2, 100)), dict(draft_tokens=i32(3, 2)),
                dict(mask=i32(3, 2, 3)), dict(logits=Tensor((3, 2, 100), device=1)), dict(mask=i32(3, 2, 4, device=1)),
                dict(out=f32(3, 2, 100, device=1))):
        with pytest.raises(ValueError):
            go(**bad)
    for bad in (dict(out=Tensor((3, 2, 100))), dict(logits=i32(3, 2, 100)), dict(mask=f32(3, 2, 4))):
        with pytest.raises(TypeError):
            go(**bad)
    with pytest.raises(ValueError):
        go(r=mnb.token_rules(temperature=f32(3, device=1)))
    assert fake.calls == []
    assert _binding.TokenRules.device is None
