"""GPU parity of the paged key-value cache (kv_append) and of the attention over
it (kv_attention) against plain 64-bit implementations of the definitions in
include/mnb.h.

Tolerances.  kv_append: the one rounding to the stored dtype (half a unit in
the last place) plus 2^-19 of the magnitudes that enter an element: its few
fp32 operations and the fp32 mean under the norm's root each err by 2^-23 or
less.  kv_attention: with A the largest sum_d |scale q_d k_d| of a row and V
the row's mean of |v| under its probabilities, a score errs by at most (D / 16
+ 2) 2^-22 A (one truncation per matrix instruction), which moves the output by
at most twice that times V; the probabilities' 16-bit parts leave 2^-16 of
them (22 significant bits, 2^-21, for fp32 outputs), the fp32 sums 2^-20; then
the one rounding of the output."""
import math
import zlib

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402
from tests._util import guarded_workspace, guards_intact  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # of a value's magnitude, with the last binade's slack
TINY = {"f32": 2.0 ** -140, "f16": 2.0 ** -24, "bf16": 2.0 ** -130}
CONTENT = 7


def rng(*key):
    return torch.Generator("cuda").manual_seed(zlib.crc32(repr(key).encode()))


class Batch:
    """A paged cache and a step over it.  Every slot that no sequence holds is NaN, every page-table entry that
    no sequence needs is an impossible page."""

    def __init__(self, g, lens, new, kv_heads, dim, page, cache, layout="heads", new_start=True, spare=3):
        self.lens, self.new, self.page, self.hkv, self.dim, self.cache_dt = lens, new, page, kv_heads, dim, cache
        pages = [-(-n // page) for n in lens]
        pool = sum(pages) + spare
        dt = DT[cache]
        if layout == "heads":      # [pages, heads, rows, dim]
            self.k, self.v = (torch.empty((pool, kv_heads, page, dim), dtype=dt, device="cuda") for _ in range(2))
        elif layout == "rows":     # [pages, rows, heads, dim]
            self.k, self.v = (torch.empty((pool, page, kv_heads, dim), dtype=dt, device="cuda").transpose(1, 2)
                              for _ in range(2))
        else:                      # keys and values side by side, rows padded
            both = torch.empty((pool, 2, kv_heads, page + 8, dim + 8), dtype=dt, device="cuda")
            self.k, self.v = both[:, 0, :, :page, :dim], both[:, 1, :, :page, :dim]
        self.k.fill_(math.nan)
        self.v.fill_(math.nan)
        order = torch.randperm(pool, generator=g, device="cuda").tolist()
        self.table = torch.full((len(lens), max(pages + [1]) + 2), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.unused = order[at:]
        self.table = self.table.cuda()
        self.starts = [0]
        for n in new:
            self.starts.append(self.starts[-1] + n)
        self.tokens = self.starts[-1]
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.new_start = torch.tensor(self.starts, dtype=torch.int32, device="cuda") if new_start else None
        self.cache = mnb.kv_cache(self.k, self.v)
        self.step = mnb.kv_step(self.seq_lens, self.table[:, :max(pages + [1])], new_start=self.new_start,
                                tokens=self.tokens, max_new=max(new + [1]))
        # the table's rows are wider than what the step describes
        assert self.step.table_stride == self.table.shape[1] or len(lens) <= 1

    def place(self, b, pos):
        return int(self.table[b, pos // self.page]), pos % self.page

    def fill(self, g, spread=1.0):
        """Random keys and values for every token of every sequence."""
        for b, n in enumerate(self.lens):
            if n == 0:
                continue
            pos = torch.arange(n, device="cuda")
            pages, rows = self.table[b].long()[pos // self.page], pos % self.page
            shape = (n, self.hkv, self.dim)
            self.k[pages, :, rows] = (torch.randn(shape, generator=g, device="cuda") * spread).to(self.k.dtype)
            self.v[pages, :, rows] = (torch.randn(shape, generator=g, device="cuda") + 0.2).to(self.v.dtype)

    def rows_of(self, b, h):
        n = self.lens[b]
        pos = torch.arange(n, device="cuda")
        pages, rows = self.table[b].long()[pos // self.page], pos % self.page
        return self.k[pages, h, rows].double(), self.v[pages, h, rows].double()


def reference(bt, q, group, scale, window):
    """out, lse, and per row the A and V of the tolerance, in 64 bits."""
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    size = torch.zeros((2,) + q.shape[:2], dtype=torch.float64, device="cuda")
    for b, length in enumerate(bt.lens):
        n = bt.new[b]
        for h in range(bt.hkv):
            k, v = bt.rows_of(b, h)
            for i in range(n):
                pos = length - n + i
                lo = max(0, pos + 1 - window) if window else 0
                if pos < 0:
                    continue
                t, hs = bt.starts[b] + i, slice(h * group, (h + 1) * group)
                x = q[t, hs].double()
                s = x @ k[lo:pos + 1].T * scale
                m = s.amax(-1, keepdim=True)
                e = torch.exp(s - m)
                out[t, hs] = e @ v[lo:pos + 1] / e.sum(-1, keepdim=True)
                lse[t, hs] = (m + torch.log(e.sum(-1, keepdim=True)))[:, 0]
                size[0, t, hs] = (x.abs() @ k[lo:pos + 1].abs().T * scale).amax(-1)
                size[1, t, hs] = (e @ v[lo:pos + 1].abs() / e.sum(-1, keepdim=True)).amax(-1)
    return out, lse, size


def check(bt, q, out, lse, group, scale, window, dtype):
    ref, rlse, (A, V) = reference(bt, q, group, scale, window)
    ds = (bt.dim / 16 + 2) * 2.0 ** -22 * A
    parts = 2.0 ** -21 if dtype == "f32" else 2.0 ** -16
    tol = HALF_ULP[dtype] * ref.abs() + (V * (2 * ds + parts + 2.0 ** -20))[..., None] + TINY[dtype]
    err = (out.double() - ref).abs()
    assert not torch.isnan(out).any()
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"output off by {worst:.3g} of its tolerance"
    if lse is not None:
        seen = torch.isfinite(rlse)
        assert torch.equal(seen, torch.isfinite(lse))
        assert torch.equal(lse[~seen].double(), rlse[~seen])
        d = (lse.double() - rlse).abs()[seen]
        lim = (2 * ds + 2.0 ** -19 * (1 + rlse.abs()))[seen]
        assert bool((d <= lim).all()), f"lse off by {(d / lim).max().item():.3g} of its tolerance"


def attend(bt, g, group, dtype, scale=None, window=0, spread=2.0, lse=True):
    q = (torch.randn((bt.tokens, bt.hkv * group, bt.dim), generator=g, device="cuda") * spread).to(DT[dtype])
    out = torch.full_like(q, math.nan)
    stat = torch.full(q.shape[:2], math.nan, device="cuda") if lse else None
    need = mnb.kv_attention_workspace_size(bt.hkv * group, bt.hkv, bt.dim, bt.step.max_new)
    ws, full = guarded_workspace(need)
    mnb.kv_attention(bt.cache, bt.step, q, out, ws, scale=scale, window=window, lse=stat)
    torch.cuda.synchronize()
    assert guards_intact(full, 256)
    assert mnb.mnb_get_last_device_error() == 0
    check(bt, q, out, stat, group, bt.dim ** -0.5 if scale is None else scale, window, dtype)
    return q, out, stat


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("dim,hkv,group,page", [(128, 8, 2, 16), (128, 4, 8, 64), (64, 2, 7, 32), (80, 5, 2, 24),
                                                (256, 2, 4, 8), (16, 1, 1, 40), (96, 1, 20, 128), (136, 2, 3, 16)])
def test_one_token_of_ragged_sequences(cache, dtype, dim, hkv, group, page):
    g = rng("one", cache, dtype, dim, hkv, group, page)
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 1, 0, 777]
    bt = Batch(g, lens, [1] * len(lens), hkv, dim, page, cache, new_start=False)
    bt.fill(g)
    attend(bt, g, group, dtype)


@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("dim,hkv,group", [(128, 2, 8), (64, 1, 5), (80, 3, 2), (256, 1, 3)])
@pytest.mark.parametrize("new", [[1, 5, 2, 0, 3, 1, 4], [9, 1, 0, 12, 2, 2, 7], [70, 3, 33, 1, 129, 0, 64]])
def test_several_new_tokens(cache, dtype, dim, hkv, group, new):
    """Row tiles of 16, 32 and 64 rows, more rows than a tile, tokens cut between row tiles, prompts from zero."""
    g = rng("several", cache, dtype, dim, hkv, group, tuple(new))
    lens = [new[0], 300, 65, 40, new[4] + 1, 64, 200]
    bt = Batch(g, lens, new, hkv, dim, 16, cache)
    bt.fill(g)
    attend(bt, g, group, dtype)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 5000])
@pytest.mark.parametrize("cache,dtype", [("f16", "f16"), ("bf16", "f32")])
def test_sliding_window(window, cache, dtype):
    g = rng("window", window, cache, dtype)
    lens, new = [1, 64, 65, 300, 129, 1000], [1, 3, 1, 2, 5, 4]
    bt = Batch(g, lens, new, 2, 80, 24, cache)
    bt.fill(g)
    attend(bt, g, 3, dtype, window=window)


@pytest.mark.parametrize("layout", ["rows", "side by side"])
@pytest.mark.parametrize("dim,page", [(128, 16), (80, 24)])
def test_other_cache_layouts_and_strided_rows(layout, dim, page):
    g = rng("layout", layout, dim, page)
    bt = Batch(g, [100, 33, 257], [2, 1, 3], 4, dim, page, "bf16", layout=layout)
    bt.fill(g)
    q, out, _ = attend(bt, g, 2, "bf16")
    # the queries as part of a wider projection output, the output as part of a wider buffer
    wide = torch.full((bt.tokens, 12 * dim), math.nan, dtype=q.dtype, device="cuda")
    wide[:, dim:9 * dim] = q.flatten(1)
    buf = torch.full((bt.tokens, 10 * dim), 3.0, dtype=q.dtype, device="cuda")
    mnb.kv_attention(bt.cache, bt.step, wide[:, dim:9 * dim].unflatten(1, (8, dim)), buf[:, dim:9 * dim].unflatten(1, (8, dim)))
    assert torch.equal(buf[:, dim:9 * dim].reshape(out.shape), out)
    assert bool((buf[:, :dim] == 3).all()) and bool((buf[:, 9 * dim:] == 3).all())


@pytest.mark.parametrize("cache,dtype,dim,hkv,group,n", [("bf16", "bf16", 128, 1, 8, 1), ("f16", "f32", 128, 2, 4, 3),
                                                         ("bf16", "f32", 256, 1, 4, 1), ("f16", "f16", 64, 1, 16, 4)])
def test_one_long_sequence_is_split_over_the_gpu(cache, dtype, dim, hkv, group, n):
    g = rng("long", cache, dtype, dim)
    bt = Batch(g, [40001], [n], hkv, dim, 32, cache)
    bt.fill(g)
    q, out, stat = attend(bt, g, group, dtype)
    again, again_stat = torch.empty_like(out), torch.empty_like(stat)
    mnb.kv_attention(bt.cache, bt.step, q, again, lse=again_stat)
    assert torch.equal(out, again) and torch.equal(stat, again_stat)  # the same bits on every run


def test_many_short_sequences_and_some_without_new_tokens():
    g = rng("many")
    lens = [(i * 37) % 90 for i in range(700)]
    new = [0 if i % 3 == 0 else 1 + i % 2 for i in range(700)]
    lens = [max(a, b) for a, b in zip(lens, new)]
    bt = Batch(g, lens, new, 1, 64, 8, "bf16")
    bt.fill(g)
    attend(bt, g, 4, "bf16")


def test_peaked_and_flat_scores():
    g = rng("peaked")
    bt = Batch(g, [300, 64, 1], [1, 2, 1], 2, 128, 16, "f16")
    bt.fill(g, spread=4.0)
    attend(bt, g, 2, "f16", spread=16.0)       # scores in the hundreds: a softmax of one token
    attend(bt, g, 2, "f32", spread=1e-6)       # all weights equal
    attend(bt, g, 2, "f32", scale=3.0, spread=30.0)
    attend(bt, g, 2, "f32", scale=1e-30, spread=1e25)  # large fp32 queries keep their range in a fp16 cache


def test_unseen_tokens_never_reach_a_row():
    """A NaN or an infinity that a later token's row sees leaves the rows before it alone."""
    g = rng("unseen")
    for bad in (math.nan, math.inf, -math.inf):
        for window in (0, 40):
            bt = Batch(g, [100, 64, 67], [5, 3, 6], 2, 64, 16, "bf16")
            bt.fill(g)
            for b, back in ((0, 2), (1, 1), (2, 6)):  # how many tokens from the end
                page, row = bt.place(b, bt.lens[b] - back)
                bt.v[page, :, row, ::3] = bad
                bt.k[page, 1, row, 0] = bad
            q = torch.randn((bt.tokens, 4, 64), generator=g, device="cuda").bfloat16()
            out = torch.empty_like(q)
            mnb.kv_attention(bt.cache, bt.step, q, out, window=window)
            clean = Batch(rng("unseen2"), bt.lens, bt.new, 2, 64, 16, "bf16")
            clean.k, clean.v, clean.table, clean.lens, clean.new = bt.k.clone(), bt.v.clone(), bt.table, bt.lens, bt.new
            for b, back in ((0, 2), (1, 1), (2, 6)):
                page, row = bt.place(b, bt.lens[b] - back)
                clean.v[page, :, row, ::3] = 0
                clean.k[page, 1, row, 0] = 0
            ref, _, (A, V) = reference(clean, q, 2, 64 ** -0.5, window)
            for b, back in ((0, 2), (1, 1), (2, 6)):
                before = bt.new[b] - back  # rows ahead of the bad token
                t = slice(bt.starts[b], bt.starts[b] + before)
                tol = HALF_ULP["bf16"] * ref[t].abs() + (V[t] * 2.0 ** -14)[..., None]
                assert bool(((out[t].double() - ref[t]).abs() <= tol).all())
                seen = out[bt.starts[b] + before, :2]  # key-value head 0: only the values are bad
                assert not bool(torch.isfinite(seen[:, ::3]).any())
                assert bool(torch.isfinite(seen[:, 1::3]).all())


def test_a_bad_query_spoils_its_own_row_only():
    g = rng("badquery")
    bt = Batch(g, [130, 64], [3, 1], 2, 128, 16, "bf16")
    bt.fill(g)
    for dtype in ("bf16", "f32"):
        q = torch.randn((4, 8, 128), generator=g, device="cuda").to(DT[dtype])
        clean = torch.empty_like(q)
        mnb.kv_attention(bt.cache, bt.step, q, clean)
        out = torch.empty_like(q)
        for bad in (math.nan, math.inf):
            spoiled = q.clone()
            spoiled[1, 2, 5] = bad
            mnb.kv_attention(bt.cache, bt.step, spoiled, out)
            rows = torch.ones((4, 8), dtype=torch.bool, device="cuda")
            rows[1, 2] = False
            assert torch.equal(out[rows], clean[rows])
            assert not bool(torch.isfinite(out[1, 2]).any())


@pytest.mark.parametrize("lens", [[40], [9000, 70]])  # within one CTA's range, split over many
def test_output_in_place_of_the_queries(lens):
    g = rng("alias", tuple(lens))
    bt = Batch(g, lens, [2] * len(lens), 2, 128, 16, "bf16")
    bt.fill(g)
    q, out, _ = attend(bt, g, 3, "bf16")
    same = q.clone()
    mnb.kv_attention(bt.cache, bt.step, same, same)
    assert torch.equal(same, out)


def test_window_leaves_bad_old_tokens_behind():
    g = rng("old")
    bt = Batch(g, [200], [4], 1, 64, 16, "f16")
    bt.fill(g)
    q = torch.randn((4, 2, 64), generator=g, device="cuda").half()
    page0, row0 = bt.place(0, 200 - 4 - 19)  # the oldest token that the first new token's window of 20 holds
    bt.v[page0, :, row0] = math.inf
    out = torch.empty_like(q)
    mnb.kv_attention(bt.cache, bt.step, q, out, window=20)
    assert not bool(torch.isfinite(out[0]).any())
    assert bool(torch.isfinite(out[1:]).all())


def test_rows_of_no_sequence_and_padding_rows():
    g = rng("padding")
    bt = Batch(g, [10, 0, 5], [1, 1, 2], 2, 64, 8, "bf16")  # sequence 1 is a padding row of length 0
    bt.fill(g)
    bt.new_start += 3  # rows 0..2 and the last two belong to no sequence
    tokens = bt.tokens + 5
    step = mnb.kv_step(bt.seq_lens, bt.table, new_start=bt.new_start, tokens=tokens, max_new=2)
    q = torch.randn((tokens, 4, 64), generator=g, device="cuda").bfloat16()
    out = torch.full_like(q, 7.0)
    lse = torch.full((tokens, 4), 7.0, device="cuda")
    mnb.kv_attention(bt.cache, step, q, out, lse=lse)
    assert bool((out[:3] == 7).all()) and bool((out[-2:] == 7).all()) and bool((lse[:3] == 7).all())
    assert bool((out[4] == 0).all()) and bool((lse[4] == -math.inf).all())
    check(bt, q[3:-2], out[3:-2], lse[3:-2], 2, 0.125, 0, "bf16")
    assert mnb.mnb_get_last_device_error() == 0


def test_more_new_tokens_than_max_new_and_a_sequence_of_more_new_tokens_than_length():
    g = rng("maxnew")
    bt = Batch(g, [300, 90], [30, 6], 2, 128, 16, "bf16")
    bt.fill(g)
    bt.step.max_new = 1
    attend(bt, g, 2, "bf16")
    bt = Batch(g, [3], [8], 1, 64, 16, "bf16")  # positions -5 .. 2
    bt.fill(g)
    attend(bt, g, 2, "bf16")


def test_bad_pages_and_lengths_are_reported_and_read_as_zeros():
    g = rng("badpages")
    bt = Batch(g, [100], [1], 1, 64, 16, "bf16")
    bt.fill(g)
    q = torch.randn((1, 2, 64), generator=g, device="cuda").bfloat16()
    for page in (-5, bt.k.shape[0], 2 ** 31 - 1):
        table = bt.table.clone()
        table[0, 1] = page
        out = torch.empty_like(q)
        mnb.kv_attention(bt.cache, mnb.kv_step(bt.seq_lens, table), q, out)
        assert mnb.mnb_get_last_device_error() == CONTENT
        assert bool(torch.isfinite(out).all())
        k, v = bt.rows_of(0, 0)
        k[16:32] = v[16:32] = 0
        p = torch.softmax(q[0].double() @ k.T / 8, -1)
        assert torch.allclose(out[0].double(), p @ v, rtol=2 ** -7, atol=1e-3)
    long = mnb.kv_step(torch.tensor([1000], dtype=torch.int32, device="cuda"), bt.table[:, :7])
    out = torch.empty_like(q)
    mnb.kv_attention(bt.cache, long, q, out)  # cut at 7 pages: 112 positions, of which the last 12 hold NaN
    mnb.mnb_get_last_device_error()
    assert bool(torch.isnan(out).all())


def test_cache_larger_than_32_bit_offsets():
    """Pages whose element offsets pass 2^32."""
    g = rng("huge")
    pages, hkv, page, dim = 33000, 8, 128, 128  # 4.3e9 elements
    k = torch.empty((pages, hkv, page, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    use = [pages - 1, 3, pages - 2]
    for p in use:
        k[p] = torch.randn((hkv, page, dim), generator=g, device="cuda").bfloat16()
        v[p] = torch.randn((hkv, page, dim), generator=g, device="cuda").bfloat16()
    table = torch.tensor([use], dtype=torch.int32, device="cuda")
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    cache, step = mnb.kv_cache(k, v), mnb.kv_step(lens, table)
    q = torch.randn((1, 16, dim), generator=g, device="cuda").bfloat16()
    nk, nv = (torch.randn((1, hkv, dim), generator=g, device="cuda").bfloat16() for _ in range(2))
    mnb.kv_append(cache, step, q, nk, nv, q)
    assert torch.equal(k[pages - 2, :, 43], nk[0]) and torch.equal(v[pages - 2, :, 43], nv[0])
    out = torch.empty_like(q)
    mnb.kv_attention(cache, step, q, out)
    keys = torch.cat([k[p] for p in use], 1)[:, :300].double()
    vals = torch.cat([v[p] for p in use], 1)[:, :300].double()
    s = torch.einsum("hgd,hjd->hgj", q[0].double().view(hkv, 2, dim), keys) * dim ** -0.5
    ref = torch.einsum("hgj,hjd->hgd", torch.softmax(s, -1), vals).view(16, dim)
    assert bool(((out[0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4).all())
    assert mnb.mnb_get_last_device_error() == 0


def test_another_stream_and_a_captured_graph():
    g = rng("stream")
    bt = Batch(g, [700, 3], [1, 1], 2, 128, 16, "bf16")
    bt.fill(g)
    q, out, _ = attend(bt, g, 2, "bf16", lse=False)
    ws = torch.empty(mnb.kv_attention_workspace_size(4, 2, 128, 1), dtype=torch.uint8, device="cuda")
    other = torch.empty_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mnb.kv_attention(bt.cache, bt.step, q, other, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, other)
    for handle in (s, s.cuda_stream):  # without a workspace the call makes one for that stream
        other.zero_()
        s.wait_stream(torch.cuda.current_stream())
        mnb.kv_attention(bt.cache, bt.step, q, other, stream=handle)
        s.synchronize()
        assert torch.equal(out, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mnb.kv_attention(bt.cache, bt.step, q, other, ws)
    other.zero_()
    bt.seq_lens[0] = 650  # lengths are read when the graph runs
    graph.replay()
    bt.lens = [650, 3]
    torch.cuda.synchronize()
    check(bt, q, other, None, 2, 128 ** -0.5, 0, "bf16")


def test_empty_steps_do_nothing():
    g = rng("empty")
    bt = Batch(g, [10], [1], 1, 64, 8, "bf16")
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    step = mnb.kv_step(none, torch.empty((0, 4), dtype=torch.int32, device="cuda"))
    q = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    mnb.kv_attention(bt.cache, step, q, q.clone())
    mnb.kv_append(bt.cache, step, q, k, k, q.clone())
    torch.cuda.synchronize()
    assert mnb.mnb_get_last_device_error() == 0
    # sequences, but none with a new token: the first row belongs to none
    step = mnb.kv_step(bt.seq_lens, bt.table, new_start=torch.zeros(2, dtype=torch.int32, device="cuda"), tokens=1)
    out = torch.full((1, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    mnb.kv_attention(bt.cache, step, torch.zeros_like(out), out)
    assert bool((out == 5).all())


# --------------------------------------------------------------------- append

def cos_sin_table(rows, rot):
    inv = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepared(x, table_row, weight, rot, interleaved, eps):
    """A head vector normed and rotated in 64 bits, and the magnitudes that enter each element."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    y, size = x.clone(), x.abs()
    if rot:
        c, s = table_row[:rot // 2].double(), table_row[rot // 2:].double()
        i = torch.arange(rot // 2, device="cuda")
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size


def near(got, ref, size, dtype):
    tol = HALF_ULP[dtype] * ref.abs() + 2.0 ** -19 * size + TINY[dtype]
    return bool(((got.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("dim,rot,hq,hkv,page", [(128, 128, 16, 8, 16), (64, 64, 7, 1, 8), (80, 40, 10, 5, 24),
                                                 (256, 64, 3, 1, 64), (16, 8, 1, 1, 8), (96, 96, 5, 5, 32),
                                                 (136, 128, 4, 2, 16), (128, 0, 8, 2, 16)])
@pytest.mark.parametrize("interleaved,norm", [(False, True), (True, False)])
def test_append(cache, dtype, dim, rot, hq, hkv, page, interleaved, norm):
    g = rng("append", cache, dtype, dim, rot, hq, hkv, page, interleaved, norm)
    lens, new = [1, 40, 64, 0, 33, 257, 9], [1, 3, 64, 0, 1, 5, 2]
    bt = Batch(g, lens, new, hkv, dim, page, cache, layout=["heads", "rows", "side by side"][(dim + hq) % 3])
    before = bt.k.clone(), bt.v.clone()
    # parts of one projection's output rows
    qkv = torch.randn((bt.tokens, (hq + 2 * hkv) * dim), generator=g, device="cuda").to(DT[dtype])
    q, k, v = (x.unflatten(1, (-1, dim)) for x in qkv.split([hq * dim, hkv * dim, hkv * dim], 1))
    table = cos_sin_table(300, rot) if rot else None
    wq, wk = ((torch.rand(dim, generator=g, device="cuda") + 0.5) for _ in range(2)) if norm else (None, None)
    rope = mnb.kv_rope(table, interleaved=interleaved, q_norm=wq, k_norm=wk, eps=1e-5)
    q_out = torch.full((bt.tokens, hq, dim), math.nan, dtype=q.dtype, device="cuda")
    mnb.kv_append(bt.cache, bt.step, q, k, v, q_out, rope)
    assert mnb.mnb_get_last_device_error() == 0
    for b, n in enumerate(new):
        for i in range(n):
            t, pos = bt.starts[b] + i, lens[b] - n + i
            row = table[pos] if rot else None
            pg, r = bt.place(b, pos)
            assert near(q_out[t], *prepared(q[t], row, wq, rot, interleaved, 1e-5), dtype)
            assert near(bt.k[pg, :, r], *prepared(k[t], row, wk, rot, interleaved, 1e-5), cache)
            assert torch.equal(bt.v[pg, :, r], v[t].to(bt.v.dtype))
            before[0][pg, :, r], before[1][pg, :, r] = bt.k[pg, :, r], bt.v[pg, :, r]
    # nothing else in the cache has changed
    assert torch.equal(torch.nan_to_num(bt.k, 77.0), torch.nan_to_num(before[0], 77.0))
    assert torch.equal(torch.nan_to_num(bt.v, 77.0), torch.nan_to_num(before[1], 77.0))


def test_append_one_token_per_sequence_in_place_and_without_queries():
    g = rng("inplace")
    lens = [5, 1, 0, 200]
    bt = Batch(g, lens, [1] * 4, 2, 64, 16, "bf16", new_start=False)
    q = torch.randn((4, 6, 64), generator=g, device="cuda").bfloat16()
    k, v = (torch.randn((4, 2, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    rope = mnb.kv_rope(cos_sin_table(200, 64))
    out, same = torch.full_like(q, 9.0), q.clone()
    mnb.kv_append(bt.cache, bt.step, q, k, v, out, rope)
    mnb.kv_append(bt.cache, bt.step, same, k, v, same, rope)
    assert torch.equal(out[[0, 1, 3]], same[[0, 1, 3]])
    assert bool((out[2] == 9).all()) and torch.equal(same[2], q[2])  # a padding row is left alone
    keys = bt.k.clone()
    bt.k.fill_(0)
    mnb.kv_append(bt.cache, bt.step, None, k, v, None, rope)
    for b in (0, 1, 3):
        pg, r = bt.place(b, lens[b] - 1)
        assert torch.equal(bt.k[pg, :, r], keys[pg, :, r])
    assert mnb.mnb_get_last_device_error() == 0


def test_append_many_tokens():
    """More tokens than CTAs, sequences found among more than 32."""
    g = rng("appendmany")
    new = [(i * 131) % 700 for i in range(90)]
    bt = Batch(g, [n + 7 for n in new], new, 1, 64, 16, "f16")
    k, v = (torch.randn((bt.tokens, 1, 64), generator=g, device="cuda").half() for _ in range(2))
    mnb.kv_append(bt.cache, bt.step, None, k, v, None)
    for b, n in enumerate(new):
        pos = torch.arange(7, 7 + n, device="cuda")
        pages, rows = bt.table[b].long()[pos // 16], pos % 16
        s = slice(bt.starts[b], bt.starts[b] + n)
        assert torch.equal(bt.k[pages, :, rows], k[s]) and torch.equal(bt.v[pages, :, rows], v[s])


def test_append_skips_and_reports_tokens_without_a_place():
    g = rng("noplace")
    bt = Batch(g, [20, 20, 20], [1, 1, 1], 1, 64, 16, "bf16", new_start=False)
    bt.k.fill_(0)
    bt.v.fill_(0)
    k = torch.ones((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    for case in ("page", "length", "angle"):
        table, lens, rope = bt.table.clone(), bt.seq_lens.clone(), None
        if case == "page":
            table[1, 1] = bt.k.shape[0]
        elif case == "length":
            lens[1] = 16 * table.shape[1] + 1
        else:
            lens[1] = 18
            rope = mnb.kv_rope(cos_sin_table(18, 64))
            lens[0] = lens[2] = 17
            lens[1] = 20
        bt.k.fill_(0)
        out = torch.full_like(q, 5.0)
        mnb.kv_append(bt.cache, mnb.kv_step(lens, table), q, k, k, out, rope)
        assert mnb.mnb_get_last_device_error() == CONTENT
        assert bool((out[1] == 5).all()) and not bool((out[[0, 2]] == 5).any())
        stored = int((bt.k.abs().sum(-1) > 0).sum())
        assert stored == 2
    assert mnb.mnb_get_last_device_error() == 0


def test_append_then_attention_back_to_back():
    """The cache rows that one call stores are read by the next one on the stream."""
    g = rng("backtoback")
    bt = Batch(g, [130, 64, 1], [1, 1, 1], 2, 128, 16, "bf16", new_start=False)
    bt.fill(g)
    q = torch.randn((3, 4, 128), generator=g, device="cuda")
    k, v = (torch.randn((3, 2, 128), generator=g, device="cuda") for _ in range(2))
    rope = mnb.kv_rope(cos_sin_table(130, 128))
    turned, out = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(mnb.kv_attention_workspace_size(4, 2, 128), dtype=torch.uint8, device="cuda")
    for _ in range(20):
        k.normal_(generator=g)
        v.normal_(generator=g)
        mnb.kv_append(bt.cache, bt.step, q, k, v, turned, rope)
        mnb.kv_attention(bt.cache, bt.step, turned, out, ws)
        check(bt, turned, out, None, 2, 128 ** -0.5, 0, "f32")


def test_binding_refuses_what_the_library_cannot_read():
    g = rng("refuse")
    bt = Batch(g, [5], [1], 2, 64, 8, "bf16")
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        mnb.kv_attention(bt.cache, bt.step, q.cpu(), q.clone())
    with pytest.raises(ValueError):
        mnb.kv_attention(bt.cache, bt.step, torch.zeros((2, 4, 64), dtype=q.dtype, device="cuda"), q)
    with pytest.raises(ValueError):
        mnb.kv_attention(bt.cache, bt.step, torch.zeros((1, 64, 4), dtype=q.dtype, device="cuda").transpose(1, 2), q)
    with pytest.raises(TypeError):
        mnb.kv_attention(bt.cache, bt.step, q, q.float())
    with pytest.raises(mnb.MnbError):  # fp16 queries over a bf16 cache
        mnb.kv_attention(bt.cache, bt.step, q.half(), q.half())
    with pytest.raises(mnb.MnbError):
        mnb.kv_attention(bt.cache, bt.step, q, q.clone(), scale=0.0)
    with pytest.raises(mnb.MnbError):
        mnb.kv_attention(bt.cache, bt.step, q, q.clone(), torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mnb.kv_append(bt.cache, bt.step, None, k, k, q)
    with pytest.raises(TypeError):
        mnb.kv_append(bt.cache, bt.step, q, k, k.float(), q)
    with pytest.raises(ValueError):
        mnb.kv_cache(bt.k, bt.v[:1])
    with pytest.raises(TypeError):
        mnb.kv_step(bt.seq_lens.long(), bt.table)
