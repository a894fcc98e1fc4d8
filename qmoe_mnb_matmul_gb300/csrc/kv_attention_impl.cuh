// kv_attention_impl.cuh -- attention of a step's new tokens over the paged
// key-value cache, the main kernel.
//
// Mathematics.  For row (new token i of sequence b, query head h) at position
// p: s_j = scale q.k_j over the visible cached tokens j <= p (and j > p -
// window), out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m).  The cache is read
// once, in tiles of 64 tokens, with the running maximum m and sum l of each row
// in fp32 and the exponentials in base 2; partial (m, l, O) of disjoint token
// ranges join exactly by rescaling to the larger maximum.
//
// Work.  A pair is (sequence, row tile, key-value head); the `group` query heads
// of a key-value head and the sequence's new tokens are the rows that share one
// pass over its keys and values (row = token * group + head in group).  All
// pairs' tiles form one line of units, cut into equal ranges, one per CTA (two
// CTAs per SM, one where shared memory holds no more), so that one long sequence
// or a ragged batch fills the GPU alike without the host knowing the lengths.
// A pair that lies inside one range is written out directly; the parts of a
// split pair go to the workspace (at most two per CTA: the pair that began
// before the range, and the one that goes on after it) and kv_join_kernel adds
// them in range order.
//
// Inside a CTA.  Warps 4 and 5 walk the units and load the key and the value
// tiles by TMA (4-D tensor map over the cache's own strides, 128-byte swizzle,
// boxes of as many rows as divide a page, page numbers from the page table) into
// two rings of tiles; rows past the sequence's end and page numbers outside the
// cache read as zeros (an out-of-range box).  Warps 0-3 compute, with the
// tokens (and head dimensions) on the matrix instructions' long side and the
// rows on their short one, in eights: S^T = K Q^T and O^T += V^T P^T by
// mma.sync m16n8k16.  A step has 1 .. 64 rows and is bound by HBM: a decode
// step of one to eight heads per key-value head wastes no more than it must of
// an instruction, its accumulators stay in 32 registers, and nothing goes
// through tensor memory and back.  The four warps split into WR groups along the
// rows (8 RG rows each) and 4 / WR along a tile's tokens; warps that share rows
// join through shared memory at the end of a pair.
//
// Rounding.  K and V are exact 16-bit operands.  Queries of the cache's type go
// in as they are; fp32 queries are scaled by a power of two per row and split
// in 16-bit parts (3 bf16 or 2 fp16 parts: 24 / 22 bits; fp16: of elements down to
// 2^-17 of the row's largest, smaller ones err by 2^-39 of it).  P is split
// likewise: for an fp32 output in 3 bf16 or 2 fp16 parts, for a 16-bit output
// in 2 parts of that type, so that the error of a single rounding of P (as
// large as that of the rounded output) does not add to it.  fp16 ends at 2^-24,
// but a row's output may be made of weights far below its largest one (a first
// token that draws the attention and has a value near zero).  So fp16 weights are
// 2^15 times as large (the reference lies 15 below the largest score in log2 units; 2^15
// is exact in fp16), and their second part is multiplied by 2^11 and summed apart:
// a weight w of the row's largest so far keeps 22 bits down to w = 2^-28, 16 down to
// 2^-34, and errs by 2^-51 of the largest below.  The MMAs of a tile start from zero
// and are added to the running fp32 sum outside, because the tensor core's own
// accumulation truncates: over a long cache that would drift.
//
// Measured (GB300, heads of 128, join included): 64 sequences of 1 .. 8192 tokens,
// 16 query heads over 8, 1.09 GB: 173 us, 6.3 TB/s; one sequence of 131072 tokens, 32
// over 4, 268 MB: 51 us; 777 tokens: 7.2 us, all latency (finding the range 1.5, the
// first tile 2.5, the join 2).  16 sequences with 1 .. 5 drafts, 24 .. 40 rows, 294 MB:
// 82 us in fp16 (79 without the second part's own sum), 80 in bf16, bound by the latency
// of the matrix instructions (two compute warps per scheduler, tensor pipe 31 % busy).
// Everything lives in registers there, and two CTAs per SM leave 168 of them: the 8-row
// kernels spill nothing, those of 32 and 64 rows at a width of 128 spill 184 .. 268 bytes
// (fp32 queries over an fp16 cache, 64 rows: 788).  What was slower: rows on the
// instructions' long side (187 us for the batch), one producer warp for keys and values
// (219), a page lookup that a tile waits for (344), the second parts' sum carried on into
// the first parts' (86 us for the drafts).
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "kv.h"

namespace mnb {

namespace {

constexpr int kComputeWarps = 4;
constexpr int kThreads = 32 * (kComputeWarps + 2);  // and a producer of key tiles, and one of value tiles

template <int N>
struct Int {
    static constexpr int value = N;
};

// 16-bit parts of a query and of an attention weight.
constexpr int query_parts(int dt, bool qf32) { return !qf32 ? 1 : dt == kBF16 ? 3 : 2; }
constexpr int weight_parts(int dt, bool qf32) { return !qf32 ? 2 : dt == kBF16 ? 3 : 2; }
// What the second fp16 part of an attention weight is multiplied by (see "Rounding" above).
constexpr int kF16Up = 1 << 11;

// Shared-memory plan of an instantiation for row tiles of up to ROWS rows.
template <int DP, int ROWS, bool QF32, int PARTS_Q>
struct Plan {
    static constexpr int kSlotBytes = kKvTile * DP * 2;
    // Q parts (fp32 queries, and heads or row tiles too large to keep Q in registers)
    static constexpr bool kQSmem = QF32 || DP > 128 || ROWS > 32;
    static constexpr int kQBytes = kQSmem ? PARTS_Q * ROWS * DP * 2 : 0;
    // join of the token warps: eight rows of half the columns per warp at a time,
    // rows four words apart in the banks
    static constexpr int kMergeRow = DP / 2 + 4;
    static constexpr int kMergeBytes = kComputeWarps * 8 * kMergeRow * 4;
    // 227 KB a SM, 1 KB of it reserved per CTA, 3 KB for barriers, row statistics and alignment
    static constexpr int kRoom2 = 112 * 1024 - 3072 - kQBytes - kMergeBytes;
    static constexpr int kRoom1 = 226 * 1024 - 3072 - kQBytes - kMergeBytes;
    static constexpr int kCtasPerSm = DP <= 128 && kRoom2 >= 4 * kSlotBytes ? 2 : 1;
    static constexpr int kFit = (kCtasPerSm == 2 ? kRoom2 : kRoom1) / kSlotBytes;
    static constexpr int kSlots = kFit > 8 ? 8 : kFit;
    static constexpr int kKSlots = (kSlots + 1) / 2, kVSlots = kSlots / 2;  // of key tiles, of value tiles
    static constexpr int kBytes = 1024 + kSlots * kSlotBytes + kQBytes + kMergeBytes;
    static_assert(kSlots >= 2, "a key tile and a value tile must fit");
};

template <int DT> struct Half2;
template <> struct Half2<kF16> {
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t x) {
        return __half22float2(*reinterpret_cast<const __half2*>(&x));
    }
    // bits of the values of the pair that are infinite or NaN
    static __device__ __forceinline__ uint32_t odd(uint32_t x) {
        return ((x & 0x7C00u) == 0x7C00u ? 0xFFFFu : 0u) | ((x & 0x7C000000u) == 0x7C000000u ? 0xFFFF0000u : 0u);
    }
};
template <> struct Half2<kBF16> {
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t x) {
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t odd(uint32_t x) {
        return ((x & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((x & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
    }
};

// The pair (a, b) in PARTS 16-bit parts: each the rounding of what the parts before it
// left, times UP for each part before it.
template <int DT, int PARTS, int UP = 1>
__device__ __forceinline__ void split(float a, float b, uint32_t (&out)[PARTS]) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        out[p] = Half2<DT>::pack(a, b);
        if (p + 1 < PARTS) {
            const float2 h = Half2<DT>::unpack(out[p]);
            a = (a - h.x) * UP;
            b = (b - h.y) * UP;
        }
    }
}

// d (16 x 8, fp32) += a (16 x 16) b (16 x 8).
template <int DT>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (DT == kBF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Transposes an 8 x 8 matrix of 16-bit values held one pair per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A load that is issued where it stands (the compiler would move it to its use).
__device__ __forceinline__ int load_now(const int* p) {
    int v;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

// Barrier of the compute warps (barrier 0 is __syncthreads).
__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Waits of a compute warp and its arrivals, without a branch that only one lane
// takes: every lane tries the barrier; the bounded wait follows where that fails.
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return warp_wait(bar, parity);
}
__device__ __forceinline__ void tile_free(uint64_t* bar, int lane) {
    __syncwarp();
    asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(
                     smem_u32(bar)),
                 "r"(lane)
                 : "memory");
}

// Byte offset of 16-byte chunk c of row r in a tile of `rows` rows whose
// columns are stored as 64-column (128-byte) swizzled panels.
__device__ __forceinline__ uint32_t tile_at(int rows, int r, int c) {
    return static_cast<uint32_t>((c >> 3) * rows * 128 + r * 128 + (((c ^ r) & 7) << 4));
}

// ------------------------------------------------------------- the units

// A row tile of one sequence: what its rows may see.
struct RowTile {
    int first_row;  // flat index (token * group + head) of the tile's first row
    int rows;       // rows in use
    int lo, hi;     // cached tokens that some row sees: [lo, hi)
    int lo_all, hi_all;  // cached tokens that every row sees: [lo_all, hi_all)
    int tiles;      // per key-value head, at least one
    int cost;       // units of a tile
};

struct Walk {
    int b, first, count, pos0;  // sequence, its first new token, their number, position of the first
    int rt, row_tiles;          // row tile, and how many the sequence has
    int h, tile;                // key-value head, next unit of the pair
    RowTile t;
};

// The first token that the row at position pos sees (window 0: every earlier one);
// the capacity where it sees none of the tokens that have a page.
__device__ __forceinline__ int window_start(const KvAttnArgs& a, int pos) {
    return a.window > 0 && pos >= a.window ? min(pos + 1 - a.window, a.step.capacity) : 0;
}

template <int ROWS>
__device__ __forceinline__ RowTile row_tile(const KvAttnArgs& a, int count, int pos0, int rt) {
    RowTile t;
    const int all = count * a.group;
    t.first_row = rt * ROWS;
    t.rows = min(ROWS, all - t.first_row);
    const int tok0 = a.by_group(t.first_row), tok1 = a.by_group(t.first_row + t.rows - 1);
    const int cap = a.step.capacity;
    t.hi = min(max(pos0 + tok1 + 1, 0), cap);
    t.hi_all = min(max(pos0 + tok0 + 1, 0), cap);
    t.lo = window_start(a, pos0 + tok0);
    t.lo_all = window_start(a, pos0 + tok1);
    // a tile of more than 32 rows takes about twice the time of one that HBM bounds
    // (its matrix instructions bound it: measured 4900 against 2700 cycles)
    t.cost = ROWS > 32 && t.rows > 32 ? 2 : 1;
    t.tiles = t.hi > t.lo ? (t.hi + kKvTile - 1) / kKvTile - t.lo / kKvTile : 1;
    return t;
}

// New tokens and row tiles of a sequence.
template <int ROWS>
__device__ __forceinline__ void load_sequence(const KvAttnArgs& a, Walk& w, int seq) {
    w.b = seq;
    // (beyond the page table the new tokens keep their positions, and rows see the tokens
    // that have a page; beyond any page table, there is no room for sums of positions)
    const int len = min(__ldg(a.step.seq_lens + seq), kKvMaxCapacity);
    step_tokens(a.step, seq, &w.first, &w.count);
    w.pos0 = max(len, 0) - w.count;
    w.row_tiles = (w.count * a.group + ROWS - 1) / ROWS;
}

// Units of the sequence in w over all its row tiles, for one key-value head.
template <int ROWS>
__device__ __forceinline__ int64_t sequence_units(const KvAttnArgs& a, const Walk& w) {
    int64_t n = 0;
#pragma unroll 1
    for (int rt = 0; rt < w.row_tiles; ++rt) {
        const RowTile t = row_tile<ROWS>(a, w.count, w.pos0, rt);
        n += t.tiles * t.cost;
    }
    return n;
}

// The next pair after a finished one (call only while units remain).
template <int ROWS>
__device__ __forceinline__ void next_pair(const KvAttnArgs& a, Walk& w) {
    w.tile = 0;
    if (++w.h < a.cache.heads) return;
    w.h = 0;
    if (++w.rt >= w.row_tiles) {
#pragma unroll 1
        do {
            load_sequence<ROWS>(a, w, w.b + 1);
        } while (w.row_tiles == 0);
        w.rt = 0;
    }
    w.t = row_tile<ROWS>(a, w.count, w.pos0, w.rt);
}

// The CTA's range of units.  CTA c of the `ctas` that have units takes `each` of them,
// the first `more` CTAs one more.
struct Range {
    int64_t at, end, each;
    int ctas, more;

    __device__ __forceinline__ void divide(int64_t total) {  // (a 64-bit division costs as much as a load)
        each = total < (int64_t(1) << 32) ? static_cast<uint32_t>(total) / static_cast<uint32_t>(ctas) : total / ctas;
        more = static_cast<int>(total - each * ctas);
    }
    __device__ __forceinline__ int64_t start(int c) const { return each * c + min(c, more); }
    // The CTA that unit u falls to.
    __device__ __forceinline__ int owner(int64_t u) const {
        const int64_t longer = (each + 1) * more;
        if (u < longer) return static_cast<int>(u / (each + 1));
        return more + static_cast<int>((u - longer) / each);
    }
};

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int64_t warp_scan(int64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (static_cast<int>(threadIdx.x & 31) >= o) v += x;
    }
    return v;
}

// The range and the walk's start, worked out by each warp for itself: a lane adds up
// an equal share of consecutive sequences (their loads do not wait for one another),
// and where that is more than one sequence, the warp looks through the share that
// the range begins in again.  The way from the launch to the first copy passes
// through here, so it is short rather than general: with up to 32 sequences one load
// of lengths, two 32-bit divisions (one of the units, one of the pair).
template <int ROWS>
__device__ __forceinline__ Range find_range(const KvAttnArgs& a, Walk& w) {
    const int lane = threadIdx.x & 31, batch = a.step.batch, per = (batch + 31) / 32;
    const int64_t heads = a.cache.heads;
    Walk mine = {};
    int64_t units = 0;
#pragma unroll 4
    for (int s = lane * per; s < min((lane + 1) * per, batch); ++s) {
        load_sequence<ROWS>(a, mine, s);
        units += sequence_units<ROWS>(a, mine);
    }
    units *= heads;
    int64_t incl = warp_scan(units);
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
    Range r;
    r.at = r.end = r.each = 0;
    r.more = 0;
    // a range holds a tile's first unit: as many units as the dearest tile has
    r.ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total / (ROWS > 32 ? 2 : 1)));
    if (total > 0 && r.ctas == 0) r.ctas = 1;
    const int c = blockIdx.x;
    if (c >= r.ctas) return r;  // fewer units than CTAs
    r.divide(total);
    r.at = r.start(c);
    r.end = r.start(c + 1);
    int64_t begin = incl - units;  // of this lane's share
    int src = __ffs(__ballot_sync(0xffffffffu, begin <= r.at && r.at < incl)) - 1;
    w.b = src;
    if (per > 1) {
        const int last = min((src + 1) * per, batch);
        int64_t before = __shfl_sync(0xffffffffu, begin, src);
#pragma unroll 1
        for (int s0 = src * per; s0 < last; s0 += 32) {
            units = 0;
            if (s0 + lane < last) {
                load_sequence<ROWS>(a, mine, s0 + lane);
                units = sequence_units<ROWS>(a, mine) * heads;
            }
            incl = before + warp_scan(units);
            begin = incl - units;
            const unsigned owner = __ballot_sync(0xffffffffu, begin <= r.at && r.at < incl);
            if (owner) {
                src = __ffs(owner) - 1;
                w.b = s0 + src;
                break;
            }
            before = __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    w.first = __shfl_sync(0xffffffffu, mine.first, src);
    w.count = __shfl_sync(0xffffffffu, mine.count, src);
    w.pos0 = __shfl_sync(0xffffffffu, mine.pos0, src);
    w.row_tiles = __shfl_sync(0xffffffffu, mine.row_tiles, src);
    int64_t off = r.at - __shfl_sync(0xffffffffu, begin, src);
#pragma unroll 1
    for (w.rt = 0;; ++w.rt) {
        w.t = row_tile<ROWS>(a, w.count, w.pos0, w.rt);
        const int64_t n = static_cast<int64_t>(w.t.tiles) * w.t.cost * heads;
        if (off < n) break;
        off -= n;
    }
    const int pair = w.t.tiles * w.t.cost;  // units of a pair: below 2^27
    if (off < (int64_t(1) << 31)) {
        w.h = static_cast<int>(off) / pair;
        w.tile = static_cast<int>(off) - w.h * pair;
    } else {
        w.h = static_cast<int>(off / pair);
        w.tile = static_cast<int>(off % pair);
    }
    if (ROWS > 32 && w.t.cost == 2) {
        // a tile belongs to the CTA that its first unit falls to
        r.at += w.tile & 1;
        w.tile = (w.tile + 1) >> 1;
        if (w.tile == w.t.tiles && r.at < r.end) next_pair<ROWS>(a, w);
    }
    return r;
}

// Tiles of the walk's pair that begin within the next `units`.
template <int ROWS>
__device__ __forceinline__ int part_tiles(const Walk& w, int64_t units) {
    if (ROWS > 32 && w.t.cost == 2) units = (units + 1) >> 1;
    return static_cast<int>(min(static_cast<int64_t>(w.t.tiles - w.tile), units));
}

// What the compute warps share.
struct Smem {
    uint8_t *k, *v;  // rings of tiles
    uint8_t* q;
    float* merge;
    uint64_t *k_full, *k_empty, *v_full, *v_empty;
    float2* stats;    // [4][16]: a warp's reference and sum of its rows
    float2* rows;     // [64]: the rows' reference and sum after the join
    float* row_unit;  // [64]: power of two that a row of fp32 queries was scaled down by
};

// Position in the ring of slots.
template <int SLOTS>
struct Ring {
    int slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++slot == SLOTS) {
            slot = 0;
            parity ^= 1;
        }
    }
};

// Barrier of the WR warps of token group wt; true where any thread brought true.
template <int WR>
__device__ __forceinline__ bool tokens_or(int wt, bool x) {
    if constexpr (WR == 1) {
        return __any_sync(0xffffffffu, x);
    } else {
        uint32_t y;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
            "bar.red.or.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(y)
            : "r"(2 + wt), "n"(32 * WR), "r"(x ? 1u : 0u)
            : "memory");
        return y != 0;
    }
}

// The key or the value tiles of the CTA's range, by one warp.  Lane l issues the
// box of row block l % blocks and 64-column panel l / blocks of every tile (32
// boxes at most) and looks up its page itself, one tile ahead.  This warp's own
// pace bounds how fast tiles can be asked for (a box costs some 80 cycles, a
// hand-off between warps as much again), so keys and values have a producer
// each and the loop has no division.
template <int DP, int ROWS, int SLOTS>
__device__ __forceinline__ void produce(const KvAttnArgs& a, const CUtensorMap* map, uint8_t* slots, uint64_t* full,
                                        uint64_t* empty, Walk w, const Range& r) {
    constexpr int kSlotBytes = kKvTile * DP * 2;
    asm volatile("fence.proxy.async.global;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int R = a.box_rows, blocks = kKvTile / R, ps = a.cache.page_size;
    const int panel = lane / blocks, row0 = (lane % blocks) * R;
    const int step_pages = a.by_page(kKvTile), step_rows = kKvTile - step_pages * ps;
    const bool issues = panel < DP / 64;
    const uint32_t dst = smem_u32(slots) + panel * (kKvTile * 128) + row0 * 128;
    Ring<SLOTS> ring;
    int issued = 0;
    int64_t at = r.at;
    bool ok = true, bad = false;
    while (at < r.end && ok) {
        const int nt = part_tiles<ROWS>(w, r.end - at);
        bad = bad || w.pos0 + w.count > a.step.capacity;
        int tok = (w.t.lo / kKvTile + w.tile) * kKvTile + row0;
        // page and row of the box at token tok; boxes that no row sees are asked for
        // outside the cache, which fills them with zeros and reads nothing
        const int index = a.by_page(tok);
        const int* at_page = a.step.page_table + w.b * a.step.table_stride + index;
        int row = tok - index * ps;
        auto wanted = [&] { return issues && tok < w.t.hi && tok + R > w.t.lo; };
        int page = wanted() ? load_now(at_page) : -1;
        for (int i = 0; i < nt; ++i) {
            const int cur = page, cur_row = row;
            const bool outside = wanted() && (cur < 0 || cur >= a.cache.num_pages);
            tok += kKvTile;
            row += step_rows;
            at_page += step_pages;
            if (row >= ps) {
                row -= ps;
                ++at_page;
            }
            page = i + 1 < nt && wanted() ? load_now(at_page) : -1;
            if (ok) ok = warp_wait(&empty[ring.slot], ring.parity ^ 1);  // the first round passes at once
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[ring.slot], kSlotBytes);
            __syncwarp();
            if (issues) tma_load_4d(dst + ring.slot * kSlotBytes, map, panel * 64, cur_row, w.h, cur, &full[ring.slot]);
            bad = bad || outside;
            ++issued;
            ring.next();
        }
        at += nt * w.t.cost;
        w.tile += nt;
        if (at < r.end) next_pair<ROWS>(a, w);
    }
    // a page number outside the cache: its tokens read as zeros; or a length past the page table
    if (bad) record_error(MNB_ERR_CONTENT);
    // no copy may be in flight when the CTA ends, whatever the compute warps
    // waited for: see the copies of the last slots land
    for (int n = max(0, issued - SLOTS); n < issued; ++n)
        warp_wait(&full[n % SLOTS], static_cast<uint32_t>(n / SLOTS) & 1u);
}

// Tokens [lo, hi) that row rr of the row tile sees.
__device__ __forceinline__ void row_sees(const KvAttnArgs& a, const Walk& w, int rr, int& lo, int& hi) {
    const int pos = w.pos0 + a.by_group(w.t.first_row + rr);
    hi = rr < w.t.rows ? min(pos + 1, a.step.capacity) : 0;
    lo = window_start(a, pos);
}

// Where the result of a part is stored: share (g, half) of the merge takes eight rows of
// each of WR row groups (RG eights each) and half the columns, and step k of a share
// gives this thread four columns of one row.
struct Place {
    int rr, d;  // row of the row tile, first of the four columns
};
template <int DP>
__device__ __forceinline__ Place merge_place(int rg, int g, int half, int k) {
    constexpr int HALF = DP / 2, V4 = HALF / 4;
    const int i = threadIdx.x + 32 * kComputeWarps * k;
    return {i / (8 * V4) * 8 * rg + g * 8 + i / V4 % 8, half * HALF + i % V4 * 4};
}

// An infinite value that a row sees gives that infinity, a NaN or opposite infinities
// NaN: every weight is positive, though fp32 or a weight's smaller parts may hold it
// as zero, which makes NaN of an infinity in the products.  So where a part came out
// with columns that are not finite (bits of `odd`: share 8 * (2 g + half) + step), each
// of them is looked through once more and gets the sum of its values that are not
// finite (if there are none, fp32 did not hold the sum, and it stays).  Looking at each
// stored result costs 0.1 us of a short call (777 tokens: 7.2 us); a cache that does hold
// infinities is slower (7.3 ms for 64 sequences of up to 8192 tokens with one whole row of
// them each).  Loads of eight tokens at a time made that 2.9 ms, and every other call 0.5 %
// slower by the size of the code.
template <int DT, bool QF32, int DP, int ROWS>
__device__ __forceinline__ void odd_columns(const KvAttnArgs& a, const Smem& sm, const Walk& w, int nt, bool whole,
                                            int part, int rg, uint32_t odd) {
    using H = Half2<DT>;
    const int from = (w.t.lo / kKvTile + w.tile) * kKvTile;
    const int* pages = a.step.page_table + w.b * a.step.table_stride;
#pragma unroll 1
    for (; odd != 0; odd &= odd - 1) {
        const int bit = __ffs(odd) - 1;
        const Place at = merge_place<DP>(rg, bit >> 4, bit >> 3 & 1, bit & 7);
        if (at.d >= a.cache.dim || sm.rows[at.rr].y != sm.rows[at.rr].y) continue;  // (NaN: among the scores)
        int lo, hi;
        row_sees(a, w, at.rr, lo, hi);
        hi = min(hi, from + nt * kKvTile);
        const uint16_t* values = static_cast<const uint16_t*>(a.cache.v) + w.h * a.cache.head_stride + at.d;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int j = max(lo, from); j < hi; ++j) {
            const int index = a.by_page(j), page = __ldg(pages + index);
            if (page < 0 || page >= a.cache.num_pages) continue;
            const uint2 x = __ldg(reinterpret_cast<const uint2*>(
                values + page * a.cache.page_stride + (j - index * a.cache.page_size) * a.cache.token_stride));
            const float2 v0 = H::unpack(x.x & H::odd(x.x)), v1 = H::unpack(x.y & H::odd(x.y));
            sum[0] += v0.x;
            sum[1] += v0.y;
            sum[2] += v1.x;
            sum[3] += v1.y;
        }
        const int flat = w.t.first_row + at.rr, tok = a.by_group(flat);
        const int64_t off = (w.first + tok) * a.out_stride +
                            static_cast<int64_t>(w.h * a.group + flat - tok * a.group) * a.cache.dim + at.d;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (sum[x] == 0.f) continue;
            if (!whole)
                a.part_o[(static_cast<int64_t>(part) * ROWS + at.rr) * DP + at.d + x] = sum[x];
            else
                store_from_f32(a.out, QF32 ? kF32 : DT, off + x, sum[x]);
        }
    }
}

// One pair's tiles w.tile .. w.tile + nt - 1 by the four compute warps, WR of them
// along the rows (8 RG rows each) and 4 / WR along a tile's tokens; the result goes
// to the output (`whole`) or to slot `part` of the workspace.  Returns where this
// thread's share of it is not finite (see odd_columns).
template <int DT, bool QF32, int DP, int ROWS, int WR, int RG, int KSLOTS, int VSLOTS>
__device__ __forceinline__ uint32_t run_part(const KvAttnArgs& a, const Smem& sm, const Walk& w, int nt, bool whole, int part,
                                         Ring<KSLOTS>& kring, Ring<VSLOTS>& vring, bool& ok) {
    constexpr int PQ = query_parts(DT, QF32), PP = weight_parts(DT, QF32);
    using P = Plan<DP, ROWS, QF32, PQ>;
    using H = Half2<DT>;
    constexpr int WT = kComputeWarps / WR;
    constexpr int TOK = kKvTile / WT;  // tokens of a warp in a tile
    constexpr int MT = TOK / 16;       // 16-token blocks of a warp
    constexpr int ND = DP / 16;        // 16-column blocks of the output
    constexpr int KS = DP / 16;        // steps along the head dimension of a score
    static_assert(8 * RG * WR <= ROWS, "the row groups lie within a row tile");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wr = warp % WR, wt = warp / WR;
    const int quad = lane >> 2, qc = lane & 3;
    const int dim = a.cache.dim;
    const int row0 = wr * 8 * RG;  // the warp's first row of the row tile
    const float scale2 = a.scale * 1.4426950408889634f;  // scores to log2 units
    constexpr int kShift = kv_weight_shift(DT);
    constexpr int kUp = DT == kF16 ? kF16Up : 1;  // of the weights' second part, which is then summed apart

    // ---- queries: lane holds columns 2 qc, 2 qc + 1 (+ 8) of row quad of each eight
    uint32_t qf[P::kQSmem ? 1 : KS][P::kQSmem ? 1 : RG][2];
    float c[RG][2];  // scores to log2 units, rows 2 qc and 2 qc + 1 of each eight
#pragma unroll
    for (int g = 0; g < RG; ++g) c[g][0] = c[g][1] = scale2;
    auto q_at = [&](int rr) {  // element offset of row rr's query
        const int flat = w.t.first_row + rr, tok = a.by_group(flat);
        return (w.first + tok) * a.q_stride + static_cast<int64_t>(w.h * a.group + flat - tok * a.group) * dim;
    };
    if constexpr (!P::kQSmem) {
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            const int rr = row0 + g * 8 + quad;
            const bool in = rr < w.t.rows;
            const uint16_t* q = static_cast<const uint16_t*>(a.q) + (in ? q_at(rr) : 0);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int d = ks * 16 + x * 8 + qc * 2;
                    qf[ks][g][x] = in && d < dim ? __ldg(reinterpret_cast<const unsigned*>(q + d)) : 0u;
                }
        }
    } else {
        compute_sync();  // the queries of the pair before are read
        if constexpr (QF32) {
            // a warp takes every fourth row, several at a time so that their loads overlap;
            // rows are scaled to a largest magnitude in [1, 2), over an fp16 cache in [2^14,
            // 2^15): the second fp16 part ends at 2^-24, and a row may have one element that
            // dwarfs the others and meets keys near zero
            constexpr uint32_t kUpBy = DT == kF16 ? 14 : 0;
            constexpr int PL = (DP + 63) / 64;  // element pairs per lane
            constexpr int MINE = 2 * RG * WR, AT_ONCE = MINE < 4 ? MINE : 4;
#pragma unroll 1
            for (int k0 = 0; k0 < MINE; k0 += AT_ONCE) {
                float2 v[AT_ONCE][PL];
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k) {
                    const int rr = warp + (k0 + k) * kComputeWarps;
                    const bool in = rr < w.t.rows;
                    const int64_t at = in ? q_at(rr) : 0;
#pragma unroll
                    for (int i = 0; i < PL; ++i) {
                        const int d = (i * 32 + lane) * 2;
                        v[k][i] = make_float2(0.f, 0.f);
                        if (in && d < dim)
                            v[k][i] = __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at + d));
                    }
                }
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k) {
                    const int rr = warp + (k0 + k) * kComputeWarps;
                    if (rr >= 8 * RG * WR) break;
                    float down = 1.f, big = 0.f, up = 1.f;
#pragma unroll
                    for (int i = 0; i < PL; ++i) big = fmaxf(big, fmaxf(fabsf(v[k][i].x), fabsf(v[k][i].y)));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                    // 2^(kUpBy - e) and 2^(e - kUpBy) of the largest magnitude's exponent, as
                    // far as both are normal numbers; a row with an infinity keeps its scale
                    uint32_t e = __float_as_uint(big) >> 23;
                    if (e < 255u) {
                        e = min(max(e, kUpBy + 1u), kUpBy + 253u) - kUpBy;
                        down = __uint_as_float((254u - e) << 23);
                        up = __uint_as_float(e << 23);
                    }
                    if (lane == 0) sm.row_unit[rr] = up;
#pragma unroll
                    for (int i = 0; i < PL; ++i) {
                        const int d = (i * 32 + lane) * 2;
                        uint32_t parts[PQ];
                        split<DT, PQ>(v[k][i].x * down, v[k][i].y * down, parts);
#pragma unroll
                        for (int p = 0; p < PQ; ++p)
                            *reinterpret_cast<uint32_t*>(sm.q + p * (ROWS * DP * 2) + tile_at(ROWS, rr, d >> 3) + (d & 7) * 2) =
                                parts[p];
                    }
                }
            }
        } else {
#pragma unroll 6
            for (int x = threadIdx.x; x < 8 * RG * WR * (DP / 8); x += 32 * kComputeWarps) {
                const int rr = x / (DP / 8), ch = x % (DP / 8);
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (rr < w.t.rows && ch * 8 < dim)
                    v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + q_at(rr) + ch * 8));
                *reinterpret_cast<uint4*>(sm.q + tile_at(ROWS, rr, ch)) = v;
            }
        }
        compute_sync();
        if constexpr (QF32) {
#pragma unroll
            for (int g = 0; g < RG; ++g)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    // never 0 or infinite: a score of -inf (unseen) or 0 times it stays what it is
                    const float k = c[g][x] * sm.row_unit[row0 + g * 8 + qc * 2 + x];
                    c[g][x] = fminf(fmaxf(k, __uint_as_float(1u)), 3.402823466e38f);
                }
        }
    }

    float o[ND][RG][4];  // columns quad, quad + 8 of each sixteen; rows 2 qc, 2 qc + 1 of each eight
    float m[RG][2], l[RG][2];  // weights so far are 2^(score - m), l their sum
#pragma unroll
    for (int g = 0; g < RG; ++g) {
#pragma unroll
        for (int n = 0; n < ND; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[n][g][x] = 0.f;
        m[g][0] = m[g][1] = -INFINITY;
        l[g][0] = l[g][1] = 0.f;
    }
    const bool active = row0 < w.t.rows;  // a warp whose rows are all padding only keeps the barriers
    int tok0 = (w.t.lo / kKvTile + w.tile) * kKvTile + wt * TOK;  // the warp's first token
    // This lane's ldmatrix row in a key tile, a value tile and Q.  The chunk's swizzle
    // is an XOR of address bits 4 .. 6, so chunk c + 2 i of the row is the address of
    // chunk c (0 or 1) XOR 32 i within a 128-byte panel.
    const uint32_t k_lane = tile_at(kKvTile, wt * TOK + (lane & 15), lane >> 4);
    const uint32_t v_lane = tile_at(kKvTile, wt * TOK + (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
    const uint32_t q_lane = smem_u32(sm.q) + tile_at(ROWS, row0 + (lane & 7), lane >> 3);
#pragma unroll 1
    for (int i = 0; i < nt; ++i, tok0 += kKvTile) {
        // tokens that not every row sees
        const bool edge = tok0 < w.t.lo_all || tok0 + TOK > w.t.hi_all;
        // none of them is seen by any row: the warp only keeps the rings' order (with
        // more rows the registers that this takes cost more than it saves)
        const bool none = ROWS == 8 && (tok0 >= w.t.hi || tok0 + TOK <= w.t.lo);
        // ---- scores.  With fp32 queries each product of the leading part starts from
        // zero, is added outside, and the smaller parts are added last; otherwise two
        // accumulators take turns along the head dimension where a warp has no other
        // independent work (their chains are what a decode step waits for).
        constexpr bool kTwo = !QF32 && MT * RG == 1;
        float s[MT][RG][4], s2[QF32 || kTwo ? MT : 1][QF32 || kTwo ? RG : 1][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int g = 0; g < RG; ++g)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    s[t][g][x] = 0.f;
                    if constexpr (QF32 || kTwo) s2[t][g][x] = 0.f;
                }
        if (ok) ok = tile_wait(&sm.k_full[kring.slot], kring.parity);
        if (active && !none) {
            const uint32_t kt = smem_u32(sm.k + kring.slot * P::kSlotBytes) + k_lane;
#pragma unroll
            for (int kp = 0; kp < KS / 2; ++kp) {  // two steps along the head dimension
                uint32_t qb[PQ][RG][4];
                if constexpr (P::kQSmem) {
#pragma unroll
                    for (int p = 0; p < PQ; ++p)
#pragma unroll
                        for (int g = 0; g < RG; ++g)
                            ldsm((q_lane ^ ((kp & 1) << 6)) + p * (ROWS * DP * 2) + (kp >> 1) * (ROWS * 128) + g * 1024,
                                 qb[p][g]);
                } else {
#pragma unroll
                    for (int g = 0; g < RG; ++g)
#pragma unroll
                        for (int x = 0; x < 4; ++x) qb[0][g][x] = qf[2 * kp + (x >> 1)][g][x & 1];
                }
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int ks = 2 * kp + y;
                        uint32_t ka[4];
                        ldsm((kt ^ ((ks & 3) << 5)) + (ks >> 2) * (kKvTile * 128) + t * 2048, ka);
#pragma unroll
                        for (int g = 0; g < RG; ++g) {
                            if constexpr (QF32) {
                                float z[4] = {0.f, 0.f, 0.f, 0.f};
                                mma<DT>(z, ka, qb[0][g][2 * y], qb[0][g][2 * y + 1]);
#pragma unroll
                                for (int x = 0; x < 4; ++x) s[t][g][x] += z[x];
#pragma unroll
                                for (int p = 1; p < PQ; ++p) mma<DT>(s2[t][g], ka, qb[p][g][2 * y], qb[p][g][2 * y + 1]);
                            } else if constexpr (kTwo) {
                                mma<DT>(y ? s2[t][g] : s[t][g], ka, qb[0][g][2 * y], qb[0][g][2 * y + 1]);
                            } else {
                                mma<DT>(s[t][g], ka, qb[0][g][2 * y], qb[0][g][2 * y + 1]);
                            }
                        }
                    }
            }
            if constexpr (QF32 || kTwo) {
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int g = 0; g < RG; ++g)
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[t][g][x] += s2[t][g][x];
            }
        }
        tile_free(&sm.k_empty[kring.slot], lane);
        kring.next();
        if (none) {
            if (ok) ok = tile_wait(&sm.v_full[vring.slot], vring.parity);
            tile_free(&sm.v_empty[vring.slot], lane);
            vring.next();
            continue;
        }
        // ---- mask, running maximum and sum.  s[t][g][x]: token 16 t + quad + 8 (x / 2), row 2 qc + x % 2
        if (edge) {
#pragma unroll
            for (int g = 0; g < RG; ++g)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    int lo, hi;
                    row_sees(a, w, row0 + g * 8 + qc * 2 + x, lo, hi);
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int j = tok0 + t * 16 + quad + 8 * y;
                            if (j < lo || j >= hi) s[t][g][2 * y + x] = -INFINITY;
                        }
                }
        }
        float f[RG][2];
        uint32_t pb[MT][RG][PP][2];  // P^T in 16-bit parts, as the B operand
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            float ref[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float big = -INFINITY;
#pragma unroll
                for (int t = 0; t < MT; ++t) big = fmaxf(big, fmaxf(s[t][g][x], s[t][g][2 + x]));
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, y));
                // rounded up, so that no weight passes 2^shift
                big = fmaxf(m[g][x], __fmaf_ru(big, c[g][x], -kShift));
                // a row that has seen nothing yet keeps a zero reference, so that its exponentials are 2^-inf = 0
                ref[x] = big == -INFINITY ? 0.f : big;
                f[g][x] = exp2_approx(m[g][x] - ref[x]);
                m[g][x] = big;
            }
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int t = 0; t < MT; ++t) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    s[t][g][x] = exp2_approx(fmaf(s[t][g][x], c[g][x & 1], -ref[x & 1]));
                    sum[x & 1] += s[t][g][x];
                }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t parts[PP];
                    split<DT, PP, kUp>(s[t][g][2 * y], s[t][g][2 * y + 1], parts);
#pragma unroll
                    for (int p = 0; p < PP; ++p) pb[t][g][p][y] = transpose8(parts[p]);
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) l[g][x] = fmaf(l[g][x], f[g][x], sum[x]);
        }
        if (ok) ok = tile_wait(&sm.v_full[vring.slot], vring.parity);
        uint8_t* vtile = sm.v + vring.slot * P::kSlotBytes;
        if (edge) {
            // What no row sees (past the sequence's end, before every window) counts as
            // zero whatever the cache holds: the values are cleared in the tile.  An
            // infinity or a NaN that some rows see must not reach the others as 0 * inf:
            // it is cleared too once each row that sees it has added it (its weight, a
            // positive number, changes nothing).
            // (Tokens that every row sees, [first, last) of the warp's, need neither.)
            const int first = min(max(w.t.lo_all - tok0, 0), TOK), last = min(max(w.t.hi_all - tok0, first), TOK);
            auto scan = [&](bool clear_odd) {
                bool odd = false;
#pragma unroll 1
                for (int x = wr * 32 + lane; x < (TOK - (last - first)) * (DP / 8); x += 32 * WR) {
                    const int e = x / (DP / 8) < first ? x / (DP / 8) : x / (DP / 8) + last - first, j = tok0 + e;
                    uint4* at = reinterpret_cast<uint4*>(vtile + tile_at(kKvTile, wt * TOK + e, x % (DP / 8)));
                    uint4 v = *at;
                    const bool out = j < w.t.lo || j >= w.t.hi;
                    uint32_t* y = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t bad = H::odd(y[k]);
                        odd = odd || (bad != 0 && !out);
                        y[k] = out ? 0u : y[k] & ~bad;
                    }
                    if (out || clear_odd) *at = v;
                }
                return odd;
            };
            if (tokens_or<WR>(wt, scan(false))) {
                // O = f O + what each row sees of the infinities and NaNs
#pragma unroll
                for (int g = 0; g < RG; ++g) {
                    int lo[2], hi[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) row_sees(a, w, row0 + g * 8 + qc * 2 + x, lo[x], hi[x]);
#pragma unroll
                    for (int n = 0; n < ND; ++n) {
                        float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                        for (int e = 0; e < TOK; ++e) {
                            const int j = tok0 + e;
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint32_t v = *reinterpret_cast<const uint16_t*>(
                                    vtile + tile_at(kKvTile, wt * TOK + e, 2 * n + y) + quad * 2);
                                if (H::odd(v) == 0) continue;
                                const float val = H::unpack(v).x;
                                if (j >= lo[0] && j < hi[0]) add[2 * y] += val;
                                if (j >= lo[1] && j < hi[1]) add[2 * y + 1] += val;
                            }
                        }
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[n][g][x] = fmaf(o[n][g][x], f[g][x & 1], add[x]);
                    }
                    f[g][0] = f[g][1] = 1.f;
                }
                tokens_or<WR>(wt, false);
                scan(true);
                tokens_or<WR>(wt, false);
            }
            __syncwarp();
        }
        // ---- O^T = f O^T + V^T P^T
        if (active) {
            const uint32_t vt = smem_u32(vtile) + v_lane;
            auto load_v = [&](int n, uint32_t (&va)[MT][4]) {
#pragma unroll
                for (int t = 0; t < MT; ++t) ldsm_t((vt ^ ((n & 3) << 5)) + (n >> 2) * (kKvTile * 128) + t * 2048, va[t]);
            };
            // with one block of tokens the next sixteen columns are loaded ahead of the
            // products of these (with more the registers do not allow it)
            constexpr bool kAhead = MT == 1;
            uint32_t va[2][MT][4];
            if (kAhead) load_v(0, va[0]);
#pragma unroll
            for (int n = 0; n < ND; ++n) {
                if (!kAhead)
                    load_v(n, va[n & 1]);
                else if (n + 1 < ND)
                    load_v(n + 1, va[(n + 1) & 1]);
                float z[kUp > 1 ? PP : 1][RG][4] = {};
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int p = PP - 1; p >= 0; --p)
#pragma unroll
                        for (int g = 0; g < RG; ++g)
                            mma<DT>(z[kUp > 1 ? p : 0][g], va[n & 1][t], pb[t][g][p][0], pb[t][g][p][1]);
#pragma unroll
                for (int g = 0; g < RG; ++g)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        if constexpr (kUp > 1) z[0][g][x] = fmaf(z[1][g][x], 1.f / kUp, z[0][g][x]);
                        o[n][g][x] = fmaf(o[n][g][x], f[g][x & 1], z[0][g][x]);
                    }
            }
        }
        if (edge) fence_proxy_async_smem();  // cleared values, before the slot's next copy
        tile_free(&sm.v_empty[vring.slot], lane);
        vring.next();
    }

    // ---- end of the pair's part in this CTA: the warps that share rows agree on
    // their reference and sum, and scale to it
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) l[g][x] += __shfl_xor_sync(0xffffffffu, l[g][x], y);
            if (quad == 0) sm.stats[warp * 16 + g * 8 + qc * 2 + x] = make_float2(m[g][x], l[g][x]);
        }
    compute_sync();
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int rr = g * 8 + qc * 2 + x;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int y = 0; y < WT; ++y) M = fmaxf(M, sm.stats[(y * WR + wr) * 16 + rr].x);
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int y = 0; y < WT; ++y) {
                const float2 st = sm.stats[(y * WR + wr) * 16 + rr];
                L = fmaf(st.y, exp2_approx(st.x - ref), L);
            }
            if (wt == 0 && quad == 0) sm.rows[row0 + rr] = make_float2(M, L);
            const float k = exp2_approx(m[g][x] - ref);
#pragma unroll
            for (int n = 0; n < ND; ++n) {
                o[n][g][x] *= k;
                o[n][g][2 + x] *= k;
            }
        }
    // ---- through shared memory, eight rows of each row group and half the columns
    // at a time: the token warps' shares are added in warp order, and rows come out
    // contiguous.  (Rolled loops: this runs once or twice in a launch, so that the
    // fetch of its instructions counts.  Written from the accumulators, unrolled, it
    // made a short call 0.5 us slower.)
    constexpr int V4 = DP / 8;  // steps of four columns in half of them
    static_assert(V4 * WR / 16 <= 8 && RG <= 2, "the bits of `odd`");
    uint32_t odd = 0;
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (g + half) compute_sync();  // the last share is read
            float* mine = sm.merge + warp * 8 * P::kMergeRow;
#pragma unroll
            for (int n = 0; n < ND / 2; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    mine[(qc * 2 + (x & 1)) * P::kMergeRow + n * 16 + quad + 8 * (x >> 1)] = o[half * (ND / 2) + n][g][x];
            compute_sync();
#pragma unroll 1
            for (int i = threadIdx.x, bit = 8 * (2 * g + half); i < 8 * WR * V4; i += 32 * kComputeWarps, ++bit) {
                const int d4 = i % V4, r8 = i / V4 % 8, grp = i / (8 * V4);
                const int rr = grp * 8 * RG + g * 8 + r8, d = half * (DP / 2) + d4 * 4;
                if (rr >= w.t.rows) continue;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int y = 0; y < WT; ++y) {
                    const float4 v = *reinterpret_cast<const float4*>(
                        sm.merge + ((y * WR + grp) * 8 + r8) * P::kMergeRow + d4 * 4);
                    sum.x += v.x;
                    sum.y += v.y;
                    sum.z += v.z;
                    sum.w += v.w;
                }
                // (a sum of finite numbers that overflows is looked at for nothing)
                if (!(fabsf((sum.x + sum.y) + (sum.z + sum.w)) <= 3.402823466e38f)) odd |= 1u << bit;
                const float2 ml = sm.rows[rr];
                if (whole) {
                    const int flat = w.t.first_row + rr, tok = a.by_group(flat);
                    const int64_t token = w.first + tok;
                    const int head = w.h * a.group + flat - tok * a.group;
                    const float inv = ml.y > 0.f ? 1.f / ml.y : (ml.y == 0.f ? 0.f : ml.y);  // NaN stays NaN
                    const int64_t off = token * a.out_stride + static_cast<int64_t>(head) * dim + d;
                    if (d < dim) {
                        if constexpr (QF32)
                            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + off) =
                                make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
                        else
                            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + off) =
                                make_uint2(H::pack(sum.x * inv, sum.y * inv), H::pack(sum.z * inv, sum.w * inv));
                    }
                    if (a.lse && d == 0)
                        a.lse[token * (static_cast<int64_t>(a.cache.heads) * a.group) + head] =
                            kv_log_sum(ml.x, ml.y, kShift);
                } else {
                    const int64_t at = static_cast<int64_t>(part) * ROWS + rr;
                    *reinterpret_cast<float4*>(a.part_o + at * DP + d) = sum;
                    if (d == 0) a.part_ml[at] = ml;
                }
            }
        }
    compute_sync();  // the statistics and the last share are read
    return odd;
}

template <int DT, bool QF32, int DP, int ROWS>
__global__ void __launch_bounds__(kThreads, Plan<DP, ROWS, QF32, query_parts(DT, QF32)>::kCtasPerSm)
    kv_attention_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const KvAttnArgs a) {
    using P = Plan<DP, ROWS, QF32, query_parts(DT, QF32)>;
    constexpr int KSLOTS = P::kKSlots, VSLOTS = P::kVSlots;

    extern __shared__ uint8_t raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t k_full[KSLOTS], k_empty[KSLOTS], v_full[VSLOTS], v_empty[VSLOTS];
    __shared__ float2 stats[kComputeWarps * 16], rows[64];
    __shared__ float row_unit[64];
    uint8_t* q_smem = base + P::kSlots * P::kSlotBytes;
    const Smem sm = {base,    base + KSLOTS * P::kSlotBytes,
                     q_smem,  reinterpret_cast<float*>(q_smem + P::kQBytes),
                     k_full,  k_empty,
                     v_full,  v_empty,
                     stats,   rows,
                     row_unit};

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < KSLOTS; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], kComputeWarps);
        }
        for (int s = 0; s < VSLOTS; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], kComputeWarps);
        }
        fence_barrier_init();
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();

    Walk w = {};
    const Range r = find_range<ROWS>(a, w);
    if (warp == kComputeWarps) {
        produce<DP, ROWS, KSLOTS>(a, &kmap, sm.k, k_full, k_empty, w, r);
        return;
    }
    if (warp > kComputeWarps) {
        produce<DP, ROWS, VSLOTS>(a, &vmap, sm.v, v_full, v_empty, w, r);
        return;
    }

    // --------------------------------------------------------- compute warps
    int64_t at = r.at;
    Ring<KSLOTS> kring;
    Ring<VSLOTS> vring;
    // A wait that gave up (recorded in the error word) ends the waiting but not
    // the walk: every warp still meets the others at each barrier.
    bool ok = true;
    int4 join = make_int4(-1, 0, 0, 0);
#pragma unroll 1
    while (at < r.end) {
        const int nt = part_tiles<ROWS>(w, r.end - at);
        const bool whole = w.tile == 0 && nt == w.t.tiles;
        const int slot = at == r.at ? 0 : 1, part = 2 * blockIdx.x + slot;  // (r.at is the first part's first unit)
        // the warps split along the rows only as far as the pair's rows need
        auto run = [&](auto wr, auto rg) {
            return run_part<DT, QF32, DP, ROWS, decltype(wr)::value, decltype(rg)::value>(a, sm, w, nt, whole, part, kring,
                                                                                         vring, ok);
        };
        uint32_t odd = 0;
        if (ROWS == 8 || w.t.rows <= 8) {
            odd = run(Int<1>{}, Int<1>{});
        } else if constexpr (ROWS > 8) {
            if (w.t.rows <= 16) {
                odd = run(Int<1>{}, Int<2>{});
            } else if (ROWS == 32 || w.t.rows <= 32) {
                odd = run(Int<2>{}, Int<2>{});
            } else if constexpr (ROWS > 32) {
                odd = run(Int<4>{}, Int<2>{});
            }
        }
        if (odd) odd_columns<DT, QF32, DP, ROWS>(a, sm, w, nt, whole, part, w.t.rows <= 8 ? 1 : 2, odd);
        if (w.tile == 0 && !whole) {  // the pair begins here and goes on in the next CTAs
            // (a tile belongs to the CTA that its first unit falls to)
            const int last = r.owner(at + static_cast<int64_t>(w.t.tiles - 1) * w.t.cost);
            join = make_int4(last, 2 * w.t.rows + slot, w.first * a.group + w.t.first_row, w.h);
        }
        at += nt * w.t.cost;
        w.tile += nt;
        if (at < r.end) next_pair<ROWS>(a, w);
    }
    if (warp == 0 && lane == 0) a.join[blockIdx.x] = join;
}

// ------------------------------------------------------------- host side

// Shared by the instantiations of one (cache type, query type) slice.
template <int DT, bool QF32, int DP, int ROWS>
cudaError_t launch_one(const CUtensorMap& kmap, const CUtensorMap& vmap, const KvAttnArgs& a, int sm_count, bool pdl,
                       cudaStream_t stream, int* ctas) {
    using P = Plan<DP, ROWS, QF32, query_parts(DT, QF32)>;
    const int most = sm_count * P::kCtasPerSm;
    *ctas = most < kKvMaxCtas ? most : kKvMaxCtas;
    return launch_ready<kv_attention_kernel<DT, QF32, DP, ROWS>>(dim3(static_cast<unsigned>(*ctas)), dim3(kThreads),
                                                                 P::kBytes, stream, pdl, kmap, vmap, a);
}

template <int DT, bool QF32, int DP>
cudaError_t launch_rows(const CUtensorMap& kmap, const CUtensorMap& vmap, const KvAttnArgs& a, int rows, int sm_count,
                        bool pdl, cudaStream_t stream, int* ctas) {
    if (rows == 8) return launch_one<DT, QF32, DP, 8>(kmap, vmap, a, sm_count, pdl, stream, ctas);
    if (rows == 32) return launch_one<DT, QF32, DP, 32>(kmap, vmap, a, sm_count, pdl, stream, ctas);
    return launch_one<DT, QF32, DP, 64>(kmap, vmap, a, sm_count, pdl, stream, ctas);
}

}  // namespace

// One (cache type, query type) slice of the instantiations; each slice lives in
// its own translation unit so the slices compile in parallel.
#define MNB_KV_ATTENTION_SLICE(NAME, DT, QF32)                                                                     \
    cudaError_t NAME(const CUtensorMap& kmap, const CUtensorMap& vmap, const KvAttnArgs& a, int rows, int pad,     \
                     int sm_count, bool pdl, cudaStream_t stream, int* ctas) {                                     \
        if (pad == 64) return launch_rows<DT, QF32, 64>(kmap, vmap, a, rows, sm_count, pdl, stream, ctas);         \
        if (pad == 128) return launch_rows<DT, QF32, 128>(kmap, vmap, a, rows, sm_count, pdl, stream, ctas);       \
        return launch_rows<DT, QF32, 256>(kmap, vmap, a, rows, sm_count, pdl, stream, ctas);                       \
    }                                                                                                              \
    cudaError_t NAME##_take_error(unsigned int* out) { return take_unit_error(out); }

}  // namespace mnb
