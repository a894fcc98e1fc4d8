"""The paged cache of 8-bit codes: kv_append and kv_attention against plain 64-bit implementations of include/mnb.h.

Tolerances.  kv_attention: those of the 16-bit cache (test_kv_gpu.py), whose derivation holds for the values that
the codes stand for: the codes are exact operands, a score is multiplied by its scale once more and a weight by the ratio of
two scales (2^-24 each, within the 2^-20 of the sums).  kv_append: a key errs by 2^-19 of the magnitudes that enter it
before it is divided by the scale (as over 16 bits) and rounded to the nearest code: half a step of the code, which is 2^-4
of its binade's start and never less than 2^-10, of the value with that error."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402
from tests._util import guarded_workspace, guards_intact  # noqa: E402
from tests.test_kv_gpu import CONTENT, DT, HALF_ULP, attend, check, cos_sin_table, near, prepared, reference, rng  # noqa: E402

NAN = 0x7F  # a code
E4M3 = torch.float8_e4m3fn
STEPS = torch.tensor([2.0 ** (max(e, 1) - 10) for e in range(16)], dtype=torch.float64)  # between codes, by their exponent


def values(codes):
    """uint8 codes as the numbers they stand for, in 64 bits."""
    return codes.contiguous().view(E4M3).double()


def codes_of(x):
    """The nearest codes of |x| <= 448, ties to even."""
    return x.float().to(E4M3).view(torch.uint8)


def smallest_scale(a):
    if a == 0:
        return 0.0
    e = max(math.ceil(math.log2(a / 448)), -126)
    while e > -126 and a <= 448 * 2.0 ** (e - 1):
        e -= 1
    while a > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Codes:
    """A paged cache of codes and a step over it: every slot that no sequence holds is NaN, its scale too, every
    page-table entry that no sequence needs is an impossible page."""

    def __init__(self, g, lens, new, kv_heads, dim, page, block, layout="heads", new_start=True, spare=3):
        self.lens, self.new, self.page, self.hkv, self.dim, self.block = lens, new, page, kv_heads, dim, block
        pages = [-(-n // page) for n in lens]
        pool = sum(pages) + spare
        if layout == "heads":
            raw = [torch.empty((pool, kv_heads, page, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
            scale = [torch.empty((pool, kv_heads, page // block), device="cuda") for _ in range(2)]
        elif layout == "rows":     # [pages, rows, heads, dim], scales of a head apart
            raw = [torch.empty((pool, page, kv_heads, dim), dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in range(2)]
            scale = [torch.empty((kv_heads, pool, page // block), device="cuda").transpose(0, 1) for _ in range(2)]
        else:                      # keys and values side by side, rows padded
            both = torch.empty((pool, 2, kv_heads, page + 8, dim + 16), dtype=torch.uint8, device="cuda")
            raw = [both[:, i, :, :page, :dim] for i in range(2)]
            wide = torch.empty((pool, 2, kv_heads, page // block + 1), device="cuda")
            scale = [wide[:, i, :, :page // block] for i in range(2)]
        (self.k, self.v), (self.ks, self.vs) = raw, scale
        for t in raw:
            t.fill_(NAN)
        for t in scale:
            t.fill_(math.nan)
        order = torch.randperm(pool, generator=g, device="cuda").tolist()
        self.table = torch.full((len(lens), max(pages + [1]) + 2), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.table = self.table.cuda()
        self.starts = [0]
        for n in new:
            self.starts.append(self.starts[-1] + n)
        self.tokens = self.starts[-1]
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.new_start = torch.tensor(self.starts, dtype=torch.int32, device="cuda") if new_start else None
        self.cache = mnb.kv_cache(self.k.view(E4M3), self.v.view(E4M3), self.ks, self.vs)
        self.step = mnb.kv_step(self.seq_lens, self.table[:, :max(pages + [1])], new_start=self.new_start,
                                tokens=self.tokens, max_new=max(new + [1]))

    def place(self, b, pos):
        return int(self.table[b, pos // self.page]), pos % self.page

    def fill(self, g, lens=None, spread=4, power=True):
        """Random codes for every token (of the first lens[b] of each sequence), a scale for each of their blocks."""
        for b, n in enumerate(self.lens if lens is None else lens):
            if n == 0:
                continue
            pos = torch.arange(n, device="cuda")
            pages, rows = self.table[b].long()[pos // self.page], pos % self.page
            for raw, scale, shift in ((self.k, self.ks, 0.0), (self.v, self.vs, 20.0)):
                x = torch.randn((n, self.hkv, self.dim), generator=g, device="cuda") * 100 + shift
                raw[pages, :, rows] = codes_of(x.clamp(-448, 448))
                e = torch.randint(-spread, spread + 1, (n, self.hkv), generator=g, device="cuda") - 7
                s = torch.exp2(e.float())
                if not power:
                    s = s * (1 + torch.rand(s.shape, generator=g, device="cuda"))
                # (of a block's tokens one gives the scale)
                first = torch.arange(0, n, self.block, device="cuda")
                scale[pages[first], :, rows[first] // self.block] = s[first]

    def rows_of(self, b, h):
        pos = torch.arange(self.lens[b], device="cuda")
        pages, rows = self.table[b].long()[pos // self.page], pos % self.page
        blocks = rows // self.block
        return (values(self.k[pages, h, rows]) * self.ks[pages, h, blocks].double()[:, None],
                values(self.v[pages, h, rows]) * self.vs[pages, h, blocks].double()[:, None])


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,hkv,group,page,block", [(128, 8, 2, 16, 16), (128, 4, 8, 64, 64), (64, 2, 7, 32, 8),
                                                      (80, 5, 2, 24, 8), (256, 2, 4, 8, 8), (16, 1, 1, 40, 8),
                                                      (96, 1, 20, 128, 128), (144, 2, 3, 16, 8), (32, 3, 8, 256, 32)])
def test_one_token_of_ragged_sequences(dtype, dim, hkv, group, page, block):
    g = rng("one", dtype, dim, hkv, group, page)
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 1, 0, 777]
    bt = Codes(g, lens, [1] * len(lens), hkv, dim, page, block, new_start=False)
    bt.fill(g, power=dim != 128)
    attend(bt, g, group, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,hkv,group", [(128, 2, 8), (64, 1, 5), (80, 3, 2), (256, 1, 3)])
@pytest.mark.parametrize("new", [[1, 5, 2, 0, 3, 1, 4], [9, 1, 0, 12, 2, 2, 7], [70, 3, 33, 1, 129, 0, 64]])
def test_several_new_tokens(dtype, dim, hkv, group, new):
    """Row tiles of 16, 32 and 64 rows, more rows than a tile, tokens cut between row tiles, prompts from zero."""
    g = rng("several", dtype, dim, hkv, group, tuple(new))
    lens = [new[0], 300, 65, 40, new[4] + 1, 64, 200]
    bt = Codes(g, lens, new, hkv, dim, 16, 16 if dim == 128 else 8)
    bt.fill(g, power=dim == 64)
    attend(bt, g, group, dtype)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 127, 128, 129, 5000])
@pytest.mark.parametrize("dtype,group", [("f16", 3), ("f32", 1)])
def test_sliding_window(window, dtype, group):
    g = rng("window", window, dtype)
    lens, new = [1, 64, 65, 300, 129, 1000], [1, 3, 1, 2, 5, 4]
    bt = Codes(g, lens, new, 2, 80, 24, 8)
    bt.fill(g)
    attend(bt, g, group, dtype, window=window)


@pytest.mark.parametrize("layout", ["rows", "side by side"])
@pytest.mark.parametrize("dim,page,block", [(128, 16, 16), (80, 24, 8), (256, 32, 16)])
def test_other_cache_layouts_and_strided_rows(layout, dim, page, block):
    g = rng("layout", layout, dim, page)
    bt = Codes(g, [100, 33, 257], [2, 1, 3], 4, dim, page, block, layout=layout)
    bt.fill(g)
    q, out, _ = attend(bt, g, 2, "bf16")
    wide = torch.full((bt.tokens, 12 * dim), math.nan, dtype=q.dtype, device="cuda")
    wide[:, dim:9 * dim] = q.flatten(1)
    buf = torch.full((bt.tokens, 10 * dim), 3.0, dtype=q.dtype, device="cuda")
    mnb.kv_attention(bt.cache, bt.step, wide[:, dim:9 * dim].unflatten(1, (8, dim)), buf[:, dim:9 * dim].unflatten(1, (8, dim)))
    assert torch.equal(buf[:, dim:9 * dim].reshape(out.shape), out)
    assert bool((buf[:, :dim] == 3).all()) and bool((buf[:, 9 * dim:] == 3).all())


@pytest.mark.parametrize("dtype,dim,hkv,group,n", [("bf16", 128, 1, 8, 1), ("f32", 128, 2, 4, 3), ("f32", 256, 1, 4, 1),
                                                   ("f16", 64, 1, 16, 4), ("f32", 128, 1, 8, 1)])
def test_one_long_sequence_is_split_over_the_gpu(dtype, dim, hkv, group, n):
    g = rng("long", dtype, dim)
    bt = Codes(g, [70001], [n], hkv, dim, 32, 32)
    bt.fill(g)
    q, out, stat = attend(bt, g, group, dtype)
    again, again_stat = torch.empty_like(out), torch.empty_like(stat)
    mnb.kv_attention(bt.cache, bt.step, q, again, lse=again_stat)
    assert torch.equal(out, again) and torch.equal(stat, again_stat)


def test_many_short_sequences_and_some_without_new_tokens():
    g = rng("many")
    lens = [(i * 37) % 90 for i in range(700)]
    new = [0 if i % 3 == 0 else 1 + i % 2 for i in range(700)]
    lens = [max(a, b) for a, b in zip(lens, new)]
    bt = Codes(g, lens, new, 1, 64, 8, 8)
    bt.fill(g)
    attend(bt, g, 4, "bf16")


def test_peaked_and_flat_scores_and_queries_of_any_size():
    g = rng("peaked")
    bt = Codes(g, [300, 64, 1], [1, 2, 1], 2, 128, 16, 16)
    bt.fill(g, spread=1)
    attend(bt, g, 2, "f16", spread=16.0)
    attend(bt, g, 2, "bf16", spread=40.0)
    attend(bt, g, 2, "f32", spread=1e-6)
    attend(bt, g, 2, "f32", scale=3.0, spread=30.0)
    attend(bt, g, 2, "f32", scale=1e-30, spread=1e25)
    attend(bt, g, 2, "bf16", scale=1e-30, spread=1e25)
    attend(bt, g, 2, "bf16", scale=1e20, spread=1e-24)


@pytest.mark.parametrize("dtype,n", [("f32", 1), ("f32", 9), ("bf16", 5)])
def test_weights_far_below_the_largest_keep_their_bits(dtype, n):
    """A first token draws the attention (its score 20 above the others', weights 2^-29) and has a value of zero: the output
    is made of the others, of scales that differ by 2^8."""
    g = rng("far", dtype, n)
    bt = Codes(g, [200], [n], 1, 64, 16, 8)
    bt.fill(g)
    page, row = bt.place(0, 0)
    bt.k[:] = codes_of(torch.randn(bt.k.shape, generator=g, device="cuda").cpu() * 8).cuda()
    bt.ks.fill_(2.0 ** -7)
    bt.k[page, 0, row] = codes_of(torch.full((64,), 256.0)).cuda()  # 2 per element
    bt.vs.copy_(torch.exp2(torch.randint(-8, 1, bt.vs.shape, generator=g, device="cuda").float()))
    first = bt.v[page, 0, row]
    first.zero_()
    q = torch.full((n, 1, 64), 1.25, device="cuda").to(DT[dtype])  # 1.25 * 2 * 64 / 8 = 20
    out = torch.empty_like(q)
    mnb.kv_attention(bt.cache, bt.step, q, out)
    ref, _, (A, V) = reference(bt, q, 1, 64 ** -0.5, 0)
    ds = (64 / 16 + 2) * 2.0 ** -22 * A
    # weights are at least 2^-31 (scores above -21.5 in all), over the ratio of 2^8 of the scales 2^-39 of the largest: an
    # error of 2^-51 of the largest weight times the block of the largest scale is 2^-12 of the smallest contribution alone
    tol = HALF_ULP[dtype] * ref.abs() + (V * (2 * ds + 2.0 ** -14))[..., None]
    assert bool(((out.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("new", [[5, 3, 6], [1, 1, 1], [40, 20, 30]])
@pytest.mark.parametrize("window", [0, 40])
def test_unseen_tokens_never_reach_a_row(new, window):
    """A NaN that a later token's row sees leaves the rows before it alone."""
    g = rng("unseen", tuple(new), window)
    bt = Codes(g, [100, 64, 67], new, 2, 64, 16, 8)
    bt.fill(g)
    spots = ((0, 2), (1, 1), (2, 6))  # how many tokens from the end
    for b, back in spots:
        page, row = bt.place(b, bt.lens[b] - back)
        bt.v[page, :, row, ::3] = NAN
        bt.k[page, 1, row, 0] = 0xFF
    q = torch.randn((bt.tokens, 4, 64), generator=g, device="cuda").bfloat16()
    out = torch.empty_like(q)
    mnb.kv_attention(bt.cache, bt.step, q, out, window=window)
    for b, back in spots:
        page, row = bt.place(b, bt.lens[b] - back)
        bt.v[page, :, row, ::3] = 0
        bt.k[page, 1, row, 0] = 0
    ref, _, (A, V) = reference(bt, q, 2, 64 ** -0.5, window)
    for b, back in spots:
        before = max(0, bt.new[b] - back)
        t = slice(bt.starts[b], bt.starts[b] + before)
        tol = HALF_ULP["bf16"] * ref[t].abs() + (V[t] * 2.0 ** -14)[..., None]
        assert bool(((out[t].double() - ref[t]).abs() <= tol).all())
        seen = out[bt.starts[b] + before, :2]
        if not window or back <= window:
            assert bool(torch.isnan(seen[:, ::3]).all())
            assert bool(torch.isfinite(seen[:, 1::3]).all())
            assert bool(torch.isnan(out[bt.starts[b] + before, 2:]).all())


def test_a_bad_query_spoils_its_own_row_only():
    g = rng("badquery")
    for new in ([3, 1], [1, 1], [20, 1]):
        bt = Codes(g, [130, 64], new, 2, 128, 16, 16)
        bt.fill(g)
        for dtype in ("bf16", "f32"):
            q = torch.randn((sum(new), 8, 128), generator=g, device="cuda").to(DT[dtype])
            clean = torch.empty_like(q)
            mnb.kv_attention(bt.cache, bt.step, q, clean)
            out = torch.empty_like(q)
            for bad in (math.nan, math.inf):
                spoiled = q.clone()
                spoiled[1, 2, 5] = bad
                mnb.kv_attention(bt.cache, bt.step, spoiled, out)
                rows = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
                rows[1, 2] = False
                assert torch.equal(out[rows], clean[rows])
                assert not bool(torch.isfinite(out[1, 2]).any())


@pytest.mark.parametrize("lens", [[40], [9000, 70]])
def test_output_in_place_of_the_queries(lens):
    g = rng("alias", tuple(lens))
    bt = Codes(g, lens, [2] * len(lens), 2, 128, 16, 16)
    bt.fill(g)
    q, out, _ = attend(bt, g, 3, "bf16")
    same = q.clone()
    mnb.kv_attention(bt.cache, bt.step, same, same)
    assert torch.equal(same, out)


def test_rows_of_no_sequence_padding_rows_and_more_rows_than_announced():
    g = rng("padding")
    bt = Codes(g, [10, 0, 5], [1, 1, 2], 2, 64, 8, 8)
    bt.fill(g)
    bt.new_start += 3
    tokens = bt.tokens + 5
    step = mnb.kv_step(bt.seq_lens, bt.table, new_start=bt.new_start, tokens=tokens, max_new=2)
    q = torch.randn((tokens, 4, 64), generator=g, device="cuda").bfloat16()
    out = torch.full_like(q, 7.0)
    lse = torch.full((tokens, 4), 7.0, device="cuda")
    mnb.kv_attention(bt.cache, step, q, out, lse=lse)
    assert bool((out[:3] == 7).all()) and bool((out[-2:] == 7).all()) and bool((lse[:3] == 7).all())
    assert bool((out[4] == 0).all()) and bool((lse[4] == -math.inf).all())
    check(bt, q[3:-2], out[3:-2], lse[3:-2], 2, 0.125, 0, "bf16")
    bt = Codes(g, [300, 90], [30, 6], 2, 128, 16, 16)
    bt.fill(g)
    bt.step.max_new = 1
    attend(bt, g, 2, "bf16")
    bt = Codes(g, [3], [8], 1, 64, 16, 8)  # positions -5 .. 2
    bt.fill(g)
    attend(bt, g, 2, "bf16")


def test_bad_pages_are_reported_and_read_as_zeros():
    g = rng("badpages")
    bt = Codes(g, [100], [1], 1, 64, 16, 16)
    bt.fill(g)
    q = torch.randn((1, 2, 64), generator=g, device="cuda").bfloat16()
    for page in (-5, bt.k.shape[0], 2 ** 31 - 1):
        table = bt.table.clone()
        table[0, 1] = page
        out = torch.empty_like(q)
        mnb.kv_attention(bt.cache, mnb.kv_step(bt.seq_lens, table), q, out)
        assert mnb.mnb_get_last_device_error() == CONTENT
        k, v = bt.rows_of(0, 0)
        k[16:32] = v[16:32] = 0
        p = torch.softmax(q[0].double() @ k.T / 8, -1)
        assert torch.allclose(out[0].double(), p @ v, rtol=2 ** -7, atol=1e-3)
    long = mnb.kv_step(torch.tensor([1000], dtype=torch.int32, device="cuda"), bt.table[:, :7])
    out = torch.empty_like(q)
    mnb.kv_attention(bt.cache, long, q, out)  # cut at 7 pages: 112 positions, of which the last 12 hold NaN
    assert mnb.mnb_get_last_device_error() == CONTENT
    assert bool(torch.isnan(out).all())


def test_cache_larger_than_32_bit_offsets():
    """Pages whose offsets pass 2^32, and the step that appends there."""
    g = rng("huge")
    pages, hkv, page, dim = 33000, 8, 128, 128  # 4.3e9 codes
    k = torch.empty((pages, hkv, page, dim), dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    ks, vs = (torch.full((pages, hkv, 4), 2.0 ** -7, device="cuda") for _ in range(2))
    use = [pages - 1, 3, pages - 2]
    for p in use:
        for t in (k, v):
            t[p] = codes_of(torch.randn((hkv, page, dim), generator=g, device="cuda") * 100)
    table = torch.tensor([use], dtype=torch.int32, device="cuda")
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    cache, step = mnb.kv_cache(k.view(E4M3), v.view(E4M3), ks, vs), mnb.kv_step(lens, table)
    q = torch.randn((1, 16, dim), generator=g, device="cuda").bfloat16()
    nk, nv = (torch.randn((1, hkv, dim), generator=g, device="cuda").bfloat16() for _ in range(2))
    mnb.kv_append(cache, step, q, nk, nv, q)
    assert torch.equal(k[pages - 2, :, 43], codes_of(nk[0].double() / ks[pages - 2, :, 1, None].double()))
    out = torch.empty_like(q)
    mnb.kv_attention(cache, step, q, out)

    def rows(t, s):
        return torch.cat([values(t[p]) * s[p].double().repeat_interleave(32, 1)[..., None] for p in use], 1)[:, :300]

    s = torch.einsum("hgd,hjd->hgj", q[0].double().view(hkv, 2, dim), rows(k, ks)) * dim ** -0.5
    ref = torch.einsum("hgj,hjd->hgd", torch.softmax(s, -1), rows(v, vs)).view(16, dim)
    fine = torch.isfinite(ref)  # (a draw past 448 is a NaN among the codes: its head is NaN)
    assert bool(fine.any()) and torch.equal(fine, torch.isfinite(out[0]))
    assert bool(((out[0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4)[fine].all())
    assert mnb.mnb_get_last_device_error() == 0


def test_another_stream_a_captured_graph_and_a_shared_workspace():
    g = rng("stream")
    bt = Codes(g, [700, 3], [1, 1], 2, 128, 16, 16)
    bt.fill(g)
    q, out, _ = attend(bt, g, 2, "bf16", lse=False)
    ws = torch.empty(mnb.kv_attention_workspace_size(4, 2, 128, 1), dtype=torch.uint8, device="cuda")
    other = torch.empty_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mnb.kv_attention(bt.cache, bt.step, q, other, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, other)
    graphs, outs = [], [torch.empty_like(out) for _ in range(2)]
    for o in outs:  # two graphs that take the same workspace, one after the other
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            mnb.kv_attention(bt.cache, bt.step, q, o, ws)
    bt.seq_lens[0] = 650
    graphs[0].replay()
    bt.seq_lens[0] = 640
    graphs[1].replay()
    torch.cuda.synchronize()
    for n, o in zip((650, 640), outs):
        bt.lens = [n, 3]
        check(bt, q, o, None, 2, 128 ** -0.5, 0, "bf16")


# --------------------------------------------------------------------- append

def expected(bt, x, size, raw, scale, before_raw, before_scale, limit=None):
    """Checks one of keys or values: x [tokens, heads, dim] in 64 bits with the magnitudes `size` that enter it, what the
    cache holds now and what it held.  limit: positions from there on are left out."""
    touched = torch.zeros(raw.shape[:3], dtype=torch.bool, device="cuda")
    scales_touched = torch.zeros(scale.shape, dtype=torch.bool, device="cuda")
    for b, length in enumerate(bt.lens):
        n = bt.new[b]
        p0 = max(0, length - n)
        end = length if limit is None else min(length, limit)
        for start in range(p0 // bt.block * bt.block, end, bt.block):
            lo, hi = max(start, p0), min(start + bt.block, end)
            if lo >= hi:
                continue
            page, row = bt.place(b, start)
            t = slice(bt.starts[b] + n - (length - lo), bt.starts[b] + n - (length - hi))
            for h in range(bt.hkv):
                y, sz = x[t, h], size[t, h]
                fine = torch.isfinite(y)
                largest = float(y[fine].abs().max()) if bool(fine.any()) else 0.0
                old = float(before_scale[page, h, row // bt.block]) if lo > start else 0.0
                got = float(scale[page, h, row // bt.block])
                # (a largest value within its error of a border may fall on either side)
                err = float(sz[fine].max()) * 2.0 ** -19 if bool(fine.any()) else 0.0
                either = {max(old, smallest_scale(a)) for a in (largest, max(0.0, largest - err), largest + err)} \
                    if largest else {old}
                assert got in either, (b, start, h, got, either)
                q = y / got if got else torch.zeros_like(y)
                c = values(raw[page, h, row + lo - start:row + hi - start])
                assert torch.equal(torch.isnan(c), ~fine)
                step = STEPS.cuda()[(raw[page, h, row + lo - start:row + hi - start].long() >> 3) & 15][fine]
                slack = sz[fine] * 2.0 ** -19 / got if got else 0.0
                over = (c[fine] - q[fine]).abs() - (step / 2 + slack)
                worst = over.max().item() if over.numel() else 0.0
                assert worst <= 0, (b, start, h, worst)
                if lo > start:
                    was = before_raw[page, h, row:row + lo - start]
                    now = raw[page, h, row:row + lo - start]
                    if got > old:
                        was = codes_of((values(was).float() * (torch.tensor(old) / got).item()).double())
                    assert torch.equal(now, was), (b, start, h, old, got)
                scales_touched[page, h, row // bt.block] = True
                touched[page, h, row:row + hi - start] = True
    assert torch.equal(raw[~touched], before_raw[~touched])                            # what no sequence holds is left alone
    now, was = scale[~scales_touched], before_scale[~scales_touched]
    assert torch.equal(now.isnan(), was.isnan()) and torch.equal(now[~now.isnan()], was[~was.isnan()])


def append(bt, g, hq, dtype, rot, norm, interleaved, spread=1.0, edit=None, max_pos=None):
    dim, hkv = bt.dim, bt.hkv
    qkv = (torch.randn((bt.tokens, (hq + 2 * hkv) * dim), generator=g, device="cuda") * spread).to(DT[dtype])
    q, k, v = (t.unflatten(1, (-1, dim)) for t in qkv.split([hq * dim, hkv * dim, hkv * dim], 1))
    if edit:
        edit(q, k, v)
    table = cos_sin_table(max_pos or max(bt.lens + [1]), rot) if rot else None
    qn, kn = (torch.rand(dim, generator=g, device="cuda") + 0.5 for _ in range(2)) if norm else (None, None)
    rope = mnb.kv_rope(table, interleaved=interleaved, q_norm=qn, k_norm=kn, eps=1e-5)
    before = [t.clone() for t in (bt.k, bt.ks, bt.v, bt.vs)]
    out = torch.full((bt.tokens, hq, dim), 9.0, dtype=DT[dtype], device="cuda")
    mnb.kv_append(bt.cache, bt.step, q, k, v, out, rope)
    torch.cuda.synchronize()
    y, size = k.double(), k.double().abs()
    for b, length in enumerate(bt.lens):
        for i in range(bt.new[b]):
            t, pos = bt.starts[b] + i, length - bt.new[b] + i
            if pos < 0 or (max_pos and rot and pos >= max_pos):
                assert bool((out[t] == 9).all())
                continue
            row = table[pos] if rot else None
            ref, sz = prepared(q[t], row, qn, rot, interleaved, 1e-5)
            assert near(out[t], ref, sz, dtype)
            y[t], size[t] = prepared(k[t], row, kn, rot, interleaved, 1e-5)
    limit = max_pos if rot else None
    expected(bt, y, size, bt.k, bt.ks, before[0], before[1], limit)
    expected(bt, v.double(), torch.zeros_like(v.double()), bt.v, bt.vs, before[2], before[3], limit)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,rot,hq,hkv,page,block", [(128, 128, 16, 8, 16, 16), (64, 64, 7, 1, 8, 8), (80, 40, 10, 5, 24, 8),
                                                       (256, 64, 3, 1, 64, 64), (16, 8, 1, 1, 8, 8), (96, 96, 5, 5, 32, 16),
                                                       (144, 128, 4, 2, 16, 16), (128, 0, 8, 2, 128, 128), (256, 256, 2, 3, 128, 128),
                                                       (64, 32, 4, 3, 64, 32)])
@pytest.mark.parametrize("norm,interleaved", [(True, False), (False, True)])
def test_append_to_blocks_that_hold_older_tokens(dtype, dim, rot, hq, hkv, page, block, norm, interleaved):
    g = rng("append", dtype, dim, rot, page, norm)
    lens = [1, 5, 40, 17, 130, 64, 3, 200, 0, 33]
    new = [1, 5, 3, 1, 66, 64, 8, 1, 1, 0]   # sequence 6: positions -5 .. 2, 8: a padding row
    bt = Codes(g, lens, new, hkv, dim, page, block)
    bt.fill(g, lens=[max(0, n - m) for n, m in zip(lens, new)])
    append(bt, g, hq, dtype, rot, norm, interleaved)
    assert mnb.mnb_get_last_device_error() == 0
    # what other calls see: the same bits for a second call, which finds its own scales
    now = [t.clone() for t in (bt.k, bt.v)]
    g2 = rng("append", dtype, dim, rot, page, norm)
    Codes(g2, lens, new, hkv, dim, page, block).fill(g2, lens=[max(0, n - m) for n, m in zip(lens, new)])
    append(bt, g2, hq, dtype, rot, norm, interleaved)
    assert torch.equal(now[0], bt.k) and torch.equal(now[1], bt.v)


def test_append_one_token_each_without_new_start():
    g = rng("append one")
    lens = [1, 2, 16, 17, 100, 0, 33]
    bt = Codes(g, lens, [1] * 7, 3, 128, 16, 16, new_start=False)
    bt.fill(g, lens=[max(0, n - 1) for n in lens])
    append(bt, g, 6, "bf16", 128, True, False)


@pytest.mark.parametrize("layout", ["rows", "side by side"])
def test_append_to_other_layouts(layout):
    g = rng("append layout", layout)
    bt = Codes(g, [30, 100, 7], [2, 50, 7], 4, 80, 24, 8, layout=layout)
    bt.fill(g, lens=[28, 50, 0])
    append(bt, g, 8, "bf16", 80, False, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_values_of_every_size(dtype):
    """Scales that grow by many powers of two, zeros, tiny and huge values, borders, infinities and NaN."""
    g = rng("append sizes", dtype)
    lens, new = [40, 24, 16, 16, 50, 33, 9], [30, 3, 16, 16, 20, 3, 2]
    bt = Codes(g, lens, new, 2, 64, 16, 16)
    bt.fill(g, lens=[a - b for a, b in zip(lens, new)], power=False)

    def edit(q, k, v):
        s = bt.starts
        v[s[0]:s[1]] *= torch.logspace(-12, 12, 30, device="cuda")[:, None, None].to(v.dtype)
        v[s[1]:s[2]] = 0
        k[s[1]:s[2]] = 0
        v[s[2]:s[3]] = 0                       # a fresh block of zeros, and of the smallest numbers
        k[s[2]:s[3]] = 1e-38
        v[s[3]:s[4]] = 448.0 * 2.0 ** -3       # a border
        k[s[3]:s[4]] = 450.0 * 2.0 ** -3
        v[s[4], 0, 5] = math.inf
        v[s[4] + 1, 1, 6] = -math.inf
        v[s[4] + 2, 0, :] = math.nan
        k[s[4] + 3, 1, 7] = math.nan
        v[s[5]:s[6], 0] = math.nan             # nothing finite beside older tokens
        v[s[6]:] = 3e38
        k[s[6]:] = -3e38

    append(bt, g, 2, dtype, 0, False, False, edit=edit)
    assert mnb.mnb_get_last_device_error() == 0


def test_append_grows_scales_that_are_no_powers_of_two():
    g = rng("append odd scales")
    lens, new = [9 + i for i in range(20)], [1 + i % 3 for i in range(20)]
    bt = Codes(g, lens, new, 2, 128, 32, 32)
    bt.fill(g, lens=[a - b for a, b in zip(lens, new)], power=False, spread=2)
    append(bt, g, 2, "f32", 128, False, False, spread=3.0)


def test_append_skips_tokens_without_a_page_or_angles():
    g = rng("append skips")
    bt = Codes(g, [40, 20], [30, 2], 2, 64, 16, 16)
    bt.fill(g, lens=[10, 18])
    append(bt, g, 2, "bf16", 64, True, False, max_pos=35)
    assert mnb.mnb_get_last_device_error() == CONTENT
    for bad in (-1, bt.k.shape[0], 2 ** 31 - 1):
        table = bt.table.clone()
        table[0, 1] = bad
        before = [t.clone() for t in (bt.k, bt.ks)]
        step = mnb.kv_step(bt.seq_lens, table, new_start=bt.new_start, tokens=32)
        k = torch.full((32, 2, 64), 1000.0, device="cuda").bfloat16()
        q = torch.full((32, 2, 64), 9.0, device="cuda").bfloat16()
        out = torch.full_like(q, 5.0)
        mnb.kv_append(bt.cache, step, q, k, k, out)
        assert mnb.mnb_get_last_device_error() == CONTENT
        assert bool((out[6:22] == 5).all()) and bool((out[:6] == 9).all()) and bool((out[22:] == 9).all())
        page = int(bt.table[0, 1])
        assert torch.equal(bt.k[page], before[0][page]) and torch.equal(bt.ks[page], before[1][page])
    short = mnb.kv_step(bt.seq_lens, bt.table[:, :2], new_start=bt.new_start, tokens=32)  # 32 positions
    out = torch.full_like(q, 5.0)
    mnb.kv_append(bt.cache, short, q, k, k, out)
    assert mnb.mnb_get_last_device_error() == CONTENT
    assert bool((out[22:30] == 5).all()) and bool((out[:22] == 9).all()) and bool((out[30:] == 9).all())


def test_append_without_queries_in_place_and_captured():
    g = rng("append graph")
    bt = Codes(g, [17, 40], [1, 3], 2, 128, 16, 16)
    bt.fill(g, lens=[16, 37])
    twin = Codes(rng("append graph"), [17, 40], [1, 3], 2, 128, 16, 16)
    for t, s in ((twin.k, bt.k), (twin.v, bt.v), (twin.ks, bt.ks), (twin.vs, bt.vs)):
        t.copy_(s)
    k, v, q = (torch.randn((4, h, 128), generator=g, device="cuda").bfloat16() for h in (2, 2, 6))
    rope = mnb.kv_rope(cos_sin_table(64, 128))
    want = torch.empty_like(q)
    mnb.kv_append(bt.cache, bt.step, q, k, v, want, rope)
    mnb.kv_append(twin.cache, twin.step, None, k, v, None, rope)
    assert torch.equal(bt.k, twin.k) and torch.equal(bt.v, twin.v)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    same = q.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        mnb.kv_append(twin.cache, twin.step, same, k, v, same, rope)
    twin.k.fill_(NAN)
    twin.ks.fill_(2.0 ** -20)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(same, want)
    page, row = bt.place(0, 16)
    assert torch.equal(twin.k[page, :, row], bt.k[page, :, row])   # the block's first token: the old scale means nothing
    assert mnb.mnb_get_last_device_error() == 0


def test_append_and_attention_over_steps():
    """A prompt, then single tokens and drafts of which some fall: the attention over the codes is that over the keys and
    values themselves but for their rounding: 2^-4 of each, half that in the mean."""
    g = rng("steps")
    hq, hkv, dim, page, block = 8, 2, 64, 16, 16
    bt = Codes(g, [90, 71], [0, 0], hkv, dim, page, block)
    rope = mnb.kv_rope(cos_sin_table(100, dim))
    lens, kept = [0, 0], [[[], []], [[], []]]
    for counts, keep in (([30, 7], [30, 7]), ([1, 1], [1, 1]), ([4, 5], [2, 5]), ([1, 3], [1, 1]), ([25, 40], [25, 40])):
        start = torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32, device="cuda")
        after = torch.tensor([a + n for a, n in zip(lens, counts)], dtype=torch.int32, device="cuda")
        step = mnb.kv_step(after, bt.table, new_start=start, tokens=sum(counts), max_new=max(counts))
        k, v, q = (torch.randn((sum(counts), h, dim), generator=g, device="cuda").bfloat16() for h in (hkv, hkv, hq))
        out = torch.empty_like(q)
        plain = mnb.kv_rope()
        mnb.kv_append(bt.cache, step, q, k, v, q, plain)
        mnb.kv_attention(bt.cache, step, q, out)
        for b in range(2):
            t = slice(int(start[b]), int(start[b + 1]))
            ks = torch.cat(kept[b][0] + [k[t]]).double()
            vs = torch.cat(kept[b][1] + [v[t]]).double()
            for i in range(counts[b]):
                n = lens[b] + i + 1
                s = torch.einsum("hgd,jhd->hgj", q[t][i].double().view(hkv, hq // hkv, dim), ks[:n]) * dim ** -0.5
                ref = torch.einsum("hgj,jhd->hgd", torch.softmax(s, -1), vs[:n]).reshape(hq, dim)
                assert float((out[t][i].double() - ref).norm() / ref.norm()) < 2.0 ** -4
            kept[b][0].append(k[t][:keep[b]])
            kept[b][1].append(v[t][:keep[b]])
            lens[b] += keep[b]
    assert rope is not None and mnb.mnb_get_last_device_error() == 0
