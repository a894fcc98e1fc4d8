// kv_attention_units.cuh -- what the paged attention kernels share: the line of units
// (tiles of TILE cached tokens of every sequence, row tile and key-value head) cut into
// a range per CTA, the rings of tiles, and the warp-level matrix instructions.
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

// What the second fp16 part of an attention weight is multiplied by (kv_attention_impl.cuh, "Rounding").
constexpr int kF16Up = 1 << 11;

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

// What the tiles of a pair cost, in units: of(rows in use), at most kMost, and kPair for the
// pair itself.  Over a 16-bit cache: a tile of more than 32 rows takes about twice the time
// of one that HBM bounds (its matrix instructions bound it: measured 4900 against 2700 cycles).
template <int ROWS>
struct Costs16 {
    static constexpr int kMost = ROWS > 32 ? 2 : 1, kPair = 0;
    static __device__ __forceinline__ int of(int rows) { return ROWS > 32 && rows > 32 ? 2 : 1; }
};

// Tiles that `units` reach into, at `cost` units each.
template <typename COSTS, typename N>
__device__ __forceinline__ N tiles_in(N units, int cost) {
    return COSTS::kMost == 2 ? (units + cost - 1) >> (cost - 1) : (units + cost - 1) / cost;
}

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

template <int ROWS, int TILE, typename COSTS>
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
    t.cost = COSTS::of(t.rows);
    t.tiles = t.hi > t.lo ? (t.hi + TILE - 1) / TILE - t.lo / TILE : 1;
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

// Units of the sequence in w over all its row tiles, for one key-value head: those of its
// tiles, and COSTS::kPair more ahead of each row tile's for what a pair costs by itself.
template <int ROWS, int TILE, typename COSTS>
__device__ __forceinline__ int64_t sequence_units(const KvAttnArgs& a, const Walk& w) {
    int64_t n = 0;
#pragma unroll 1
    for (int rt = 0; rt < w.row_tiles; ++rt) {
        const RowTile t = row_tile<ROWS, TILE, COSTS>(a, w.count, w.pos0, rt);
        n += t.tiles * t.cost + COSTS::kPair;
    }
    return n;
}

// The next pair after a finished one (call only while units remain).
template <int ROWS, int TILE, typename COSTS>
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
    w.t = row_tile<ROWS, TILE, COSTS>(a, w.count, w.pos0, w.rt);
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
template <int ROWS, int TILE, typename COSTS>
__device__ __forceinline__ Range find_range(const KvAttnArgs& a, Walk& w) {
    const int lane = threadIdx.x & 31, batch = a.step.batch, per = (batch + 31) / 32;
    const int64_t heads = a.cache.heads;
    Walk mine = {};
    int64_t units = 0;
#pragma unroll 4
    for (int s = lane * per; s < min((lane + 1) * per, batch); ++s) {
        load_sequence<ROWS>(a, mine, s);
        units += sequence_units<ROWS, TILE, COSTS>(a, mine);
    }
    units *= heads;
    int64_t incl = warp_scan(units);
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
    Range r;
    r.at = r.end = r.each = 0;
    r.more = 0;
    // a range holds a tile's first unit: as many units as the dearest tile has
    r.ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total / COSTS::kMost));
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
                units = sequence_units<ROWS, TILE, COSTS>(a, mine) * heads;
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
        w.t = row_tile<ROWS, TILE, COSTS>(a, w.count, w.pos0, w.rt);
        const int64_t n = (static_cast<int64_t>(w.t.tiles) * w.t.cost + COSTS::kPair) * heads;
        if (off < n) break;
        off -= n;
    }
    const int pair = w.t.tiles * w.t.cost + COSTS::kPair;  // units of a pair: below 2^31
    if (off < (int64_t(1) << 31)) {
        w.h = static_cast<int>(off) / pair;
        w.tile = static_cast<int>(off) - w.h * pair;
    } else {
        w.h = static_cast<int>(off / pair);
        w.tile = static_cast<int>(off % pair);
    }
    if (COSTS::kPair > 0) {
        // units ahead of the first tile belong to no tile
        w.tile -= COSTS::kPair;
        if (w.tile < 0) {
            r.at -= w.tile;
            w.tile = 0;
        }
    }
    if (COSTS::kMost > 1) {
        // (w.tile counts units) a tile belongs to the CTA that its first unit falls to
        const int unit = w.tile, cost = w.t.cost;
        w.tile = tiles_in<COSTS>(unit, cost);
        r.at += w.tile * cost - unit;
        if (w.tile == w.t.tiles && r.at < r.end) {
            next_pair<ROWS, TILE, COSTS>(a, w);
            r.at += COSTS::kPair;
        }
    }
    return r;
}

// Tiles of the walk's pair that begin within the next `units`.
template <typename COSTS>
__device__ __forceinline__ int part_tiles(const Walk& w, int64_t units) {
    if (COSTS::kMost > 1) {
        // (units past the pair's end do not matter: a division in 32 bits)
        const int some = static_cast<int>(min(units, static_cast<int64_t>(0x7fffffff - COSTS::kMost)));
        units = tiles_in<COSTS>(some, w.t.cost);
    }
    return static_cast<int>(min(static_cast<int64_t>(w.t.tiles - w.tile), units));
}

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

// Tokens [lo, hi) that row rr of the row tile sees.
__device__ __forceinline__ void row_sees(const KvAttnArgs& a, const Walk& w, int rr, int& lo, int& hi) {
    const int pos = w.pos0 + a.by_group(w.t.first_row + rr);
    hi = rr < w.t.rows ? min(pos + 1, a.step.capacity) : 0;
    lo = window_start(a, pos);
}

}  // namespace

}  // namespace mnb
