"""CPU-side checks of the paged-cache and draft-verification entry points: every
metadata error is reported before any GPU work, and an empty step is a success
that enqueues nothing."""
import ctypes

import pytest

import qmoe_mnb_matmul_gb300 as mnb
from qmoe_mnb_matmul_gb300 import _build

OK, INVALID, UNSUPPORTED, OVERFLOW, WORKSPACE = 0, 1, 2, 3, 4
FAKE = 0x10000  # 64 KiB-aligned fake device address: never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mnb.load_library()


def cache(**kw):
    d = dict(k=FAKE, v=FAKE, num_pages=100, page_stride=8 * 16 * 128, head_stride=16 * 128, token_stride=128,
             page_size=16, kv_heads=8, head_dim=128, dtype=2)
    d.update(kw)
    return mnb.KvCacheDesc(**d)


def step(**kw):
    d = dict(seq_lens=FAKE, new_start=FAKE, page_table=FAKE, table_stride=10, batch=4, tokens=9, max_new=3, max_pages=10)
    d.update(kw)
    return mnb.KvStepDesc(**d)


def append(lib, c=None, s=None, rope=None, q=FAKE, qs=2048, qh=16, k=FAKE, ks=1024, v=FAKE, vs=1024, dt=2, o=FAKE, os=2048):
    c, s = c or cache(), s or step()
    return lib.kv_append(ctypes.byref(c), ctypes.byref(s), None if rope is None else ctypes.byref(rope), q, qs, qh, k,
                         ks, v, vs, dt, o, os, None)


def attention(lib, c=None, s=None, q=FAKE, qs=2048, qh=16, dt=2, o=FAKE, os=2048, lse=None, scale=0.1, window=0,
              ws=FAKE, size=1 << 40):
    c, s = c or cache(), s or step()
    return lib.kv_attention(ctypes.byref(c), ctypes.byref(s), q, qs, qh, dt, o, os, lse, scale, window, ws, size, None)


BAD_CACHE = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
             (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID), (dict(dtype=5), INVALID),
             (dict(dtype=0), UNSUPPORTED), (dict(head_dim=100), UNSUPPORTED), (dict(head_dim=8), UNSUPPORTED),
             (dict(head_dim=264), UNSUPPORTED), (dict(page_size=12), UNSUPPORTED), (dict(k=FAKE + 8), UNSUPPORTED),
             (dict(v=FAKE + 2), UNSUPPORTED), (dict(token_stride=64), INVALID), (dict(token_stride=132), UNSUPPORTED),
             (dict(head_stride=-128), INVALID), (dict(page_stride=1 << 38), UNSUPPORTED),
             (dict(num_pages=1 << 40, page_stride=1 << 30), OVERFLOW), (dict(num_pages=1 << 32, page_stride=128), OVERFLOW)]
BAD_STEP = [(dict(seq_lens=None), INVALID), (dict(page_table=None), INVALID), (dict(batch=-1), INVALID),
            (dict(tokens=-1), INVALID), (dict(max_new=0), INVALID), (dict(max_pages=0), INVALID),
            (dict(table_stride=9), INVALID), (dict(new_start=None), INVALID),  # 9 tokens of 4 sequences
            (dict(tokens=(1 << 30) + 1), OVERFLOW), (dict(seq_lens=FAKE + 2), UNSUPPORTED), (dict(table_stride=1 << 61), OVERFLOW)]


@pytest.mark.parametrize("bad,code", BAD_CACHE)
def test_cache_errors(lib, bad, code):
    assert append(lib, c=cache(**bad)) == code
    assert attention(lib, c=cache(**bad)) == code


@pytest.mark.parametrize("bad,code", BAD_STEP)
def test_step_errors(lib, bad, code):
    assert append(lib, s=step(**bad)) == code
    assert attention(lib, s=step(**bad)) == code


def test_null_descriptors(lib):
    c, s = cache(), step()
    assert lib.kv_append(None, ctypes.byref(s), None, FAKE, 2048, 16, FAKE, 1024, FAKE, 1024, 2, FAKE, 2048, None) == INVALID
    assert lib.kv_append(ctypes.byref(c), None, None, FAKE, 2048, 16, FAKE, 1024, FAKE, 1024, 2, FAKE, 2048, None) == INVALID
    assert lib.kv_attention(None, ctypes.byref(s), FAKE, 2048, 16, 2, FAKE, 2048, None, 0.1, 0, FAKE, 1 << 40, None) == INVALID


def test_append_errors(lib):
    assert append(lib, k=None) == INVALID
    assert append(lib, v=None) == INVALID
    assert append(lib, o=None) == INVALID          # queries without an output
    assert append(lib, q=None) == INVALID          # an output without queries
    assert append(lib, qh=0) == INVALID
    assert append(lib, dt=9) == INVALID
    assert append(lib, dt=1) == UNSUPPORTED        # fp16 rows into a bf16 cache
    assert append(lib, qs=2040) == INVALID         # rows that overlap
    assert append(lib, ks=1000) == INVALID
    assert append(lib, vs=1028) == UNSUPPORTED     # rows off a 16-byte boundary
    assert append(lib, q=FAKE + 4) == UNSUPPORTED
    assert append(lib, os=1 << 61) == OVERFLOW
    rope = lambda **kw: mnb.KvRopeDesc(**{**dict(cos_sin=FAKE, max_pos=10, rot_dim=128, interleaved=0, eps=1e-6), **kw})  # noqa: E731
    assert append(lib, rope=rope(max_pos=0)) == INVALID
    assert append(lib, rope=rope(rot_dim=136)) == INVALID
    assert append(lib, rope=rope(rot_dim=0)) == INVALID
    assert append(lib, rope=rope(rot_dim=60)) == UNSUPPORTED
    assert append(lib, rope=rope(cos_sin=FAKE + 4)) == UNSUPPORTED
    assert append(lib, rope=rope(q_norm=FAKE, eps=-1.0)) == INVALID
    assert append(lib, rope=rope(k_norm=FAKE, eps=float("nan"))) == INVALID
    assert append(lib, rope=rope(k_norm=FAKE + 8)) == UNSUPPORTED


def test_attention_errors(lib):
    assert attention(lib, q=None) == INVALID
    assert attention(lib, o=None) == INVALID
    assert attention(lib, qh=12) == INVALID        # not a multiple of the key-value heads
    assert attention(lib, qh=0) == INVALID
    assert attention(lib, dt=4) == INVALID
    assert attention(lib, dt=1) == UNSUPPORTED
    assert attention(lib, window=-1) == INVALID
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert attention(lib, scale=scale) == INVALID
    assert attention(lib, qs=2000) == INVALID
    assert attention(lib, os=2052) == UNSUPPORTED
    assert attention(lib, o=FAKE + 8) == UNSUPPORTED
    assert attention(lib, lse=FAKE + 2) == UNSUPPORTED
    assert attention(lib, ws=None) == WORKSPACE
    assert attention(lib, size=1000) == WORKSPACE
    assert attention(lib, ws=FAKE + 128) == UNSUPPORTED
    assert attention(lib, qh=1 << 40, qs=1 << 50) == OVERFLOW
    assert attention(lib, s=step(tokens=(1 << 26) + 1)) == OVERFLOW   # 16 heads: 2^30 rows


def test_attention_workspace(lib):
    n = ctypes.c_size_t(7)
    size = lambda *a: lib.kv_attention_workspace_size(*a, ctypes.byref(n))  # noqa: E731
    assert lib.kv_attention_workspace_size(16, 8, 128, 1, None) == INVALID
    assert size(16, 8, 128, 1) == OK and n.value > 0
    one = n.value
    assert size(16, 8, 128, 4) == OK and n.value == one       # 8 rows
    assert size(16, 8, 128, 5) == OK and n.value > one        # 10 rows
    assert size(16, 8, 128, 10 ** 6) == OK and n.value < 64 << 20
    assert size(15, 8, 128, 1) == INVALID
    assert size(16, 8, 128, 0) == INVALID
    assert size(16, 8, 100, 1) == UNSUPPORTED
    assert size(1 << 40, 1, 128, 1) == OVERFLOW


def test_empty_steps_succeed(lib):
    assert append(lib, s=step(batch=0, tokens=0, seq_lens=None, page_table=None), q=None, o=None, k=None, v=None) == OK
    assert append(lib, s=step(tokens=0)) == OK
    assert attention(lib, s=step(tokens=0), q=None, o=None) == OK
    assert attention(lib, s=step(batch=0, tokens=0), ws=None) == OK


def verify(lib, t=FAKE, ts=5000, tr=1000, d=FAKE, ds=4000, dr=1000, x=FAKE, g=None, u=FAKE, B=2, n=4, V=1000, o=FAKE, a=FAKE):
    return lib.draft_verify(t, ts, tr, d, ds, dr, x, g, u, B, n, V, o, a, None)


def test_draft_verify_errors(lib):
    for bad in (dict(t=None), dict(x=None), dict(u=None), dict(o=None), dict(a=None), dict(B=-1), dict(n=-1), dict(V=0),
                dict(tr=-1), dict(ts=-5), dict(dr=-1), dict(ds=-1)):
        assert verify(lib, **bad) == INVALID, bad
    for bad in (dict(V=1 << 22), dict(n=1025), dict(B=1 << 31), dict(t=FAKE + 1), dict(d=FAKE + 2), dict(u=FAKE + 2),
                dict(g=FAKE + 1), dict(o=FAKE + 2), dict(a=FAKE + 3)):
        assert verify(lib, **bad) == UNSUPPORTED, bad
    assert verify(lib, ts=1 << 61) == OVERFLOW
    assert verify(lib, dr=1 << 61) == OVERFLOW
    assert verify(lib, B=0) == OK
