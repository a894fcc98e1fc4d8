"""A decoder's steps over the cache of 8-bit codes with rotated keys: a prompt, single tokens, drafts of which some
fall and are written again, a second prompt.  After each step every kept token's cached key and value and each output
are held against 64 bits.

Tolerances.  A code is off by half its step, 2^-4 of the value, or by 2^-10 of its scale where it is subnormal.  A
block whose scale grows (by powers of two) rounds its subnormal codes again: the scales at least double, so that all
these roundings are below 2^-9 of the last scale.  A key's own error is 2^-19 of the magnitudes that enter it.  The
attention over what the cache holds has the tolerances of tests/test_kv_gpu.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402
from tests.test_kv8_gpu import Codes  # noqa: E402
from tests.test_kv_gpu import DT, check, cos_sin_table, near, prepared, rng  # noqa: E402

STEPS = [([30, 7], [30, 7]), ([1, 1], [1, 1]), ([4, 5], [2, 5]), ([5, 1], [5, 1]), ([1, 6], [1, 0]), ([3, 6], [0, 6]),
         ([25, 40], [25, 40])]  # new tokens, and those that stay


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,rot,hq,hkv,page,block,norm,interleaved", [(64, 64, 8, 2, 16, 16, False, False),
                                                                        (128, 128, 4, 4, 32, 32, True, False),
                                                                        (80, 40, 10, 2, 24, 8, True, True)])
def test_steps_with_rotated_keys(dtype, dim, rot, hq, hkv, page, block, norm, interleaved):
    g = rng("rotated steps", dtype, dim)
    bt = Codes(g, [sum(n[b] for n, _ in STEPS) for b in range(2)], [0, 0], hkv, dim, page, block)
    table = cos_sin_table(150, rot)
    qn, kn = (torch.rand(dim, generator=g, device="cuda") + 0.5 for _ in range(2)) if norm else (None, None)
    rope = mnb.kv_rope(table, interleaved=interleaved, q_norm=qn, k_norm=kn, eps=1e-5)
    had, kept = [0, 0], [[], []]  # per sequence: (key, magnitudes, value) of each kept token
    for counts, keep in STEPS:
        bt.new, bt.starts, bt.tokens = counts, [0, counts[0], sum(counts)], sum(counts)
        bt.lens = [a + n for a, n in zip(had, counts)]
        after = torch.tensor(bt.lens, dtype=torch.int32, device="cuda")
        start = torch.tensor(bt.starts, dtype=torch.int32, device="cuda")
        step = mnb.kv_step(after, bt.table, new_start=start, tokens=bt.tokens, max_new=max(counts))
        size = float(torch.rand((), generator=g, device="cuda")) * 4 + 0.1  # blocks whose scales grow
        q, k, v = (torch.randn((bt.tokens, h, dim), generator=g, device="cuda") for h in (hq, hkv, hkv))
        q, k, v = q.to(DT[dtype]), (k * size).to(DT[dtype]), (v * size).to(DT[dtype])
        turned, out = torch.empty_like(q), torch.empty_like(q)
        lse = torch.empty(q.shape[:2], device="cuda")
        mnb.kv_append(bt.cache, step, q, k, v, turned, rope)
        mnb.kv_attention(bt.cache, step, turned, out, lse=lse)
        assert mnb.mnb_get_last_device_error() == 0
        for b in range(2):
            now = []
            for i in range(counts[b]):
                t, pos = bt.starts[b] + i, had[b] + i
                ref, magnitudes = prepared(q[t], table[pos], qn, rot, interleaved, 1e-5)
                assert near(turned[t], ref, magnitudes, dtype)
                now.append((*prepared(k[t], table[pos], kn, rot, interleaved, 1e-5), v[t].double()))
            here = kept[b] + now
            for pos, (key, magnitudes, value) in enumerate(here):
                at, row = bt.place(b, pos)
                for raw, scale, want, slack in ((bt.k, bt.ks, key, magnitudes * 2.0 ** -19), (bt.v, bt.vs, value, 0.0)):
                    s = scale[at, :, row // block].double()[:, None]
                    got = raw[at, :, row].contiguous().view(torch.float8_e4m3fn).double() * s
                    assert bool(((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -9 * s + slack * 1.0625).all()), (b, pos)
            kept[b] = here[:had[b] + keep[b]]
        check(bt, turned, out, lse, hq // hkv, dim ** -0.5, 0, dtype)
        had = [a + n for a, n in zip(had, keep)]
