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
// CTAs per SM, one where heads are wider than 128), so that one long sequence
// or a ragged batch fills the GPU alike without the host knowing the lengths.  A pair that lies inside one range is written
// out directly; the parts of a split pair go to the workspace (at most two per
// CTA: the pair that began before the range, and the one that goes on after
// it) and kv_join_kernel adds them in range order.
//
// Inside a CTA.  Warp 4 walks the units and loads tiles by TMA (4-D tensor map
// over the cache's own strides, 128-byte swizzle, boxes of as many rows as
// divide a page, page numbers from the page table) into a ring of slots that
// hold a key tile or a value tile; rows past the sequence's end and page numbers
// outside the cache read as zeros (an out-of-range box).  Warps 0-3 compute:
// S = Q K^T and O += P V with mma.sync m16n8k16 (a decode step has 1 .. 64 rows;
// it is bound by HBM, and the warp-level instructions need no accumulator
// round trip through tensor memory), each warp a share of the tile's tokens
// (16 rows or fewer: 16 tokens a warp) or of the rows (64 rows: 16 a warp).
// Warps that share rows join through shared memory at the end of a pair.
//
// Rounding.  K and V are exact 16-bit operands.  Queries of the cache's type go
// in as they are; fp32 queries are scaled by a power of two per row and split
// in 16-bit parts (3 bf16 or 2 fp16 parts: 24 / 22 bits).  P is split
// likewise: for an fp32 output in 3 bf16 or 2 fp16 parts, for a 16-bit output
// in 2 parts of that type, so that the error of a single rounding of P (as
// large as that of the rounded output) does not add to it.  The MMAs of a
// tile start from zero and are added to the running fp32 sum outside, because
// the tensor core's own accumulation truncates: over a long cache that would
// drift.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "kv.h"

namespace mnb {

namespace {

constexpr int kComputeWarps = 4;
constexpr int kThreads = 32 * (kComputeWarps + 1);

// Shared-memory plan of one instantiation.
template <int DP, int WR, bool QF32, int PARTS_Q>
struct Plan {
    static constexpr int kRows = 16 * WR;
    static constexpr int kTokenWarps = kComputeWarps / WR;
    static constexpr int kSlotBytes = kKvTile * DP * 2;
    // Q parts (fp32 queries, and heads too wide to keep Q in registers)
    static constexpr bool kQSmem = QF32 || DP > 128;
    static constexpr int kQBytes = kQSmem ? PARTS_Q * kRows * DP * 2 : 0;
    static constexpr int kMergeBytes = (kTokenWarps - 1) * kRows * DP * 4;
    static constexpr int kCtasPerSm = DP > 128 ? 1 : 2;
    // 227 KB a SM, 1 KB of it reserved per CTA, 2 KB for barriers, row statistics and alignment
    static constexpr int kBudget = (kCtasPerSm == 2 ? 112 * 1024 : 226 * 1024) - 3072;
    static constexpr int kFit = (kBudget - kQBytes - kMergeBytes) / kSlotBytes;
    static constexpr int kSlots = kFit > 8 ? 8 : kFit;
    static constexpr int kBytes = 1024 + kSlots * kSlotBytes + kQBytes + kMergeBytes + 1024;
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
    // whether either value is infinite or NaN
    static __device__ __forceinline__ bool odd(uint32_t x) {
        return (x & 0x7C00u) == 0x7C00u || (x & 0x7C000000u) == 0x7C000000u;
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
    static __device__ __forceinline__ bool odd(uint32_t x) {
        return (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
    }
};

// The pair (a, b) in PARTS 16-bit parts: each the rounding of what the parts before it left.
template <int DT, int PARTS>
__device__ __forceinline__ void split(float a, float b, uint32_t (&out)[PARTS]) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        out[p] = Half2<DT>::pack(a, b);
        if (p + 1 < PARTS) {
            const float2 h = Half2<DT>::unpack(out[p]);
            a -= h.x;
            b -= h.y;
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

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
    int tiles;      // units per key-value head, at least one
};

struct Walk {
    int b, first, count, pos0;  // sequence, its first new token, their number, position of the first
    int rt, row_tiles;          // row tile, and how many the sequence has
    int h, tile;                // key-value head, next unit of the pair
    RowTile t;

    template <int ROWS>
    __device__ __forceinline__ static RowTile row_tile(const KvAttnArgs& a, int count, int pos0, int rt) {
        RowTile t;
        const int all = count * a.group;
        t.first_row = rt * ROWS;
        t.rows = min(ROWS, all - t.first_row);
        const int tok0 = t.first_row / a.group, tok1 = (t.first_row + t.rows - 1) / a.group;
        const int cap = a.step.capacity;
        t.hi = min(max(pos0 + tok1 + 1, 0), cap);
        t.hi_all = min(max(pos0 + tok0 + 1, 0), cap);
        t.lo = a.window > 0 ? max(0, pos0 + tok0 + 1 - a.window) : 0;
        t.lo_all = a.window > 0 ? max(0, pos0 + tok1 + 1 - a.window) : 0;
        t.tiles = t.hi > t.lo ? (t.hi + kKvTile - 1) / kKvTile - t.lo / kKvTile : 1;
        return t;
    }

    template <int ROWS>
    __device__ __forceinline__ void load(const KvAttnArgs& a, int seq) {
        b = seq;
        step_tokens(a.step, seq, &first, &count);
        // a length beyond the page table is cut there (the append call records it)
        const int len = min(__ldg(a.step.seq_lens + seq), a.step.capacity);
        pos0 = max(len, 0) - count;
        row_tiles = (count * a.group + ROWS - 1) / ROWS;
    }
};

template <int ROWS>
__device__ __forceinline__ int64_t sequence_units(const KvAttnArgs& a, int seq) {
    Walk w;
    w.load<ROWS>(a, seq);
    int64_t n = 0;
    for (int rt = 0; rt < w.row_tiles; ++rt) n += Walk::row_tile<ROWS>(a, w.count, w.pos0, rt).tiles;
    return n * a.cache.heads;
}

// The CTA's range of units and the walk's start, worked out by each warp for
// itself (lane l adds up the sequences l * c .. (l + 1) * c - 1).
struct Range {
    int64_t at, end, total;
    int ctas;  // CTAs that have units
};

template <int ROWS>
__device__ __forceinline__ Range find_range(const KvAttnArgs& a, Walk& w) {
    const int lane = threadIdx.x & 31;
    const int batch = a.step.batch, per = (batch + 31) / 32;
    const int s0 = min(lane * per, batch), s1 = min(s0 + per, batch);
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) mine += sequence_units<ROWS>(a, s);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    Range r;
    r.total = __shfl_sync(0xffffffffu, incl, 31);
    r.ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), r.total));
    const int c = blockIdx.x;
    if (c >= r.ctas) {
        r.at = r.end = 0;
        return r;
    }
    r.at = r.total * c / r.ctas;
    r.end = r.total * (c + 1) / r.ctas;
    const bool owner = incl - mine <= r.at && r.at < incl;
    int seq = 0;
    int64_t off = 0;
    if (owner) {
        off = r.at - (incl - mine);
        seq = s0;
        for (;;) {
            const int64_t n = sequence_units<ROWS>(a, seq);
            if (off < n) break;
            off -= n;
            ++seq;
        }
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, owner)) - 1;
    seq = __shfl_sync(0xffffffffu, seq, src);
    off = __shfl_sync(0xffffffffu, off, src);
    w.load<ROWS>(a, seq);
    for (w.rt = 0;; ++w.rt) {
        w.t = Walk::row_tile<ROWS>(a, w.count, w.pos0, w.rt);
        const int64_t n = static_cast<int64_t>(w.t.tiles) * a.cache.heads;
        if (off < n) break;
        off -= n;
    }
    w.h = static_cast<int>(off / w.t.tiles);
    w.tile = static_cast<int>(off % w.t.tiles);
    return r;
}

// The next pair after a finished one (call only while units remain).
template <int ROWS>
__device__ __forceinline__ void next_pair(const KvAttnArgs& a, Walk& w) {
    w.tile = 0;
    if (++w.h < a.cache.heads) return;
    w.h = 0;
    if (++w.rt >= w.row_tiles) {
        do {
            w.load<ROWS>(a, w.b + 1);
        } while (w.row_tiles == 0);
        w.rt = 0;
    }
    w.t = Walk::row_tile<ROWS>(a, w.count, w.pos0, w.rt);
}

// ------------------------------------------------------------- the kernel

template <int DT, bool QF32, int DP, int WR>
__global__ void __launch_bounds__(kThreads, DP > 128 ? 1 : 2)
    kv_attention_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const KvAttnArgs a) {
    constexpr int PQ = QF32 ? (DT == kBF16 ? 3 : 2) : 1;
    constexpr int PP = QF32 ? (DT == kBF16 ? 3 : 2) : 2;
    using P = Plan<DP, WR, QF32, PQ>;
    constexpr int ROWS = P::kRows, WT = P::kTokenWarps, SLOTS = P::kSlots;
    constexpr int NS = kKvTile / WT / 8;   // score column tiles of a warp
    constexpr int KB = NS / 2;             // 16-token blocks of a warp
    constexpr int NO = DP / 8;             // output column tiles
    constexpr int NOWN = NO / WT;          // output column tiles a warp owns after the join of the token warps
    constexpr int KS = DP / 16;
    using H = Half2<DT>;

    extern __shared__ uint8_t raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* qs = base + SLOTS * P::kSlotBytes;
    float* merge = reinterpret_cast<float*>(qs + P::kQBytes);
    __shared__ __align__(8) uint64_t full[SLOTS], empty[SLOTS];
    __shared__ float2 stats[kComputeWarps][16];
    __shared__ float row_unit[ROWS];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kComputeWarps);
        }
        fence_barrier_init();
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();

    Walk w;
    const Range r = find_range<ROWS>(a, w);
    int64_t at = r.at;

    if (warp == kComputeWarps) {
        // ------------------------------------------------- tile producer
        asm volatile("fence.proxy.async.global;" ::: "memory");
        const int R = a.box_rows, blocks = kKvTile / R, ps = a.cache.page_size;
        int slot = 0, issued = 0;
        uint32_t parity = 1;  // of the wait for an empty slot: the first round passes at once
        bool ok = true;
        while (at < r.end && ok) {
            const int nt = static_cast<int>(min(static_cast<int64_t>(w.t.tiles - w.tile), r.end - at));
            const int* pages = a.step.page_table + w.b * a.step.table_stride;
            const int tile0 = w.t.lo / kKvTile + w.tile;
            // lane l looks up the page of row block l of each tile, one tile ahead
            auto page_of = [&](int tile) {
                const int tok = tile * kKvTile + lane * R;
                int page = -1;
                if (lane < blocks && tok < w.t.hi && tok + R > w.t.lo) {
                    page = __ldg(pages + tok / ps);
                    if (page < 0 || page >= a.cache.num_pages) record_error(MNB_ERR_CONTENT);
                }
                return page;
            };
            int page = page_of(tile0);
            for (int i = 0; i < nt && ok; ++i) {
                const int cur = page;
                if (i + 1 < nt) page = page_of(tile0 + i + 1);
                for (int kv = 0; kv < 2; ++kv) {
                    ok = warp_wait(&empty[slot], parity);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&full[slot], P::kSlotBytes);
                    __syncwarp();
                    const uint32_t dst = smem_u32(base + slot * P::kSlotBytes);
                    for (int x0 = 0; x0 < blocks * (DP / 64); x0 += 32) {
                        const int x = x0 + lane, blk = x % blocks, panel = x / blocks;
                        const int pg = __shfl_sync(0xffffffffu, cur, blk);
                        if (panel < DP / 64) {
                            const int tok = (tile0 + i) * kKvTile + blk * R;
                            tma_load_4d(dst + panel * (kKvTile * 128) + blk * R * 128, kv ? &vmap : &kmap, panel * 64,
                                        tok % ps, w.h, pg, &full[slot]);
                        }
                    }
                    ++issued;
                    if (++slot == SLOTS) {
                        slot = 0;
                        parity ^= 1;
                    }
                }
            }
            at += nt;
            w.tile += nt;
            if (at < r.end) next_pair<ROWS>(a, w);
        }
        // no copy may be in flight when the CTA ends, whatever the compute warps
        // waited for: see the copies of the last slots land
        for (int n = max(0, issued - SLOTS); n < issued; ++n)
            warp_wait(&full[n % SLOTS], static_cast<uint32_t>(n / SLOTS) & 1u);
        return;
    }

    // --------------------------------------------------------- compute warps
    const int wr = warp % WR, wt = warp / WR;
    const int quad = lane >> 2, qc = lane & 3;
    const float scale2 = a.scale * 1.4426950408889634f;  // scores in log2 units
    int slot = 0;
    uint32_t parity = 0;
    // A wait that gave up (recorded in the error word) ends the waiting but not
    // the walk: every warp still meets the others at each barrier.
    bool ok = true;
    int join_last = -1, join_slot = 0, join_row = 0, join_rows = 0, join_head = 0;

    while (at < r.end) {
        const int nt = static_cast<int>(min(static_cast<int64_t>(w.t.tiles - w.tile), r.end - at));
        const bool whole = w.tile == 0 && nt == w.t.tiles;
        // ---- queries of the 16 rows of this warp (flat rows first_row + 16 wr ..)
        uint32_t qf[P::kQSmem ? 1 : KS][4];
        float c0 = scale2, c1 = scale2;  // score to log2 units, rows quad and quad + 8
        // visible tokens [lo, hi) of the two rows this lane holds scores of
        int row_lo[2], row_hi[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int rr = wr * 16 + quad + 8 * x;
            const int pos = w.pos0 + (w.t.first_row + rr) / a.group;
            row_hi[x] = rr < w.t.rows ? min(pos + 1, a.step.capacity) : 0;
            row_lo[x] = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
        }
        const int dim = a.cache.dim;
        auto q_at = [&](int rr) {  // element offset of row rr's query
            const int flat = w.t.first_row + rr;
            return (w.first + flat / a.group) * a.q_stride +
                   static_cast<int64_t>(w.h * a.group + flat % a.group) * dim;
        };
        if constexpr (!P::kQSmem) {
            const uint16_t* q = static_cast<const uint16_t*>(a.q);
            const int ra = wr * 16 + quad, rb = ra + 8;
            const uint16_t* qa = q + (ra < w.t.rows ? q_at(ra) : 0);
            const uint16_t* qb = q + (rb < w.t.rows ? q_at(rb) : 0);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int d = ks * 16 + x * 8 + qc * 2;
                    qf[ks][2 * x] = ra < w.t.rows && d < dim ? __ldg(reinterpret_cast<const unsigned*>(qa + d)) : 0u;
                    qf[ks][2 * x + 1] = rb < w.t.rows && d < dim ? __ldg(reinterpret_cast<const unsigned*>(qb + d)) : 0u;
                }
        } else {
            compute_sync();  // the queries of the pair before are read
            // one warp per row in turn; fp32 rows are scaled to a largest magnitude in [1, 2)
            for (int rr = warp; rr < ROWS; rr += kComputeWarps) {
                constexpr int PL = (DP + 63) / 64;  // element pairs per lane
                float2 v[PL];
                float big = 0.f;
#pragma unroll
                for (int i = 0; i < PL; ++i) {
                    const int d = (i * 32 + lane) * 2;
                    v[i] = make_float2(0.f, 0.f);
                    if (rr < w.t.rows && d < dim) {
                        if constexpr (QF32)
                            v[i] = __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + q_at(rr) + d));
                        else
                            v[i] = H::unpack(__ldg(reinterpret_cast<const unsigned*>(
                                static_cast<const uint16_t*>(a.q) + q_at(rr) + d)));
                    }
                    big = fmaxf(big, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
                }
                float down = 1.f, up = 1.f;
                if constexpr (QF32) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                    // 2^-e and 2^e of the largest magnitude's exponent, for normal numbers
                    // of moderate size; others keep their scale
                    const uint32_t e = __float_as_uint(big) >> 23;
                    if (e > 27 && e < 227) {
                        down = __uint_as_float((254u - e) << 23);
                        up = __uint_as_float(e << 23);
                    }
                    if (lane == 0) row_unit[rr] = up;
                }
#pragma unroll
                for (int i = 0; i < PL; ++i) {
                    const int d = (i * 32 + lane) * 2;
                    uint32_t part[PQ];
                    split<DT, PQ>(v[i].x * down, v[i].y * down, part);
#pragma unroll
                    for (int p = 0; p < PQ; ++p)
                        *reinterpret_cast<uint32_t*>(qs + p * (ROWS * DP * 2) + tile_at(ROWS, rr, d >> 3) +
                                                     (d & 7) * 2) = part[p];
                }
            }
            compute_sync();
            if constexpr (QF32) {
                c0 *= row_unit[wr * 16 + quad];
                c1 *= row_unit[wr * 16 + quad + 8];
            }
        }

        float o[NO][4];
#pragma unroll
        for (int n = 0; n < NO; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[n][x] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        const int tile0 = w.t.lo / kKvTile + w.tile;

        for (int i = 0; i < nt; ++i) {
            const int tok0 = (tile0 + i) * kKvTile + wt * (kKvTile / WT);  // the warp's first token
            // tokens that not every row sees need a mask
            const bool edge = tok0 < w.t.lo_all || tok0 + kKvTile / WT > w.t.hi_all;
            // ---- scores
            float s[NS][4];
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
            if (ok) ok = warp_wait(&full[slot], parity);
            {
                const uint32_t kt = smem_u32(base + slot * P::kSlotBytes);
                const int krow = wt * (kKvTile / WT) + (lane & 7) + ((lane >> 4) << 3), kchunk = (lane >> 3) & 1;
                const uint32_t qt = smem_u32(qs);
                const int qrow = wr * 16 + (lane & 15), qchunk = lane >> 4;
                float rest[QF32 ? NS : 1][4];  // the smaller parts' products, added last
                if constexpr (QF32) {
#pragma unroll
                    for (int n = 0; n < NS; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) rest[n][x] = 0.f;
                }
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t qa[PQ][4];
                    if constexpr (P::kQSmem) {
#pragma unroll
                        for (int p = 0; p < PQ; ++p)
                            ldsm(qt + p * (ROWS * DP * 2) + tile_at(ROWS, qrow, ks * 2 + qchunk), qa[p]);
                    } else {
#pragma unroll
                        for (int x = 0; x < 4; ++x) qa[0][x] = qf[ks][x];
                    }
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        uint32_t kf[4];
                        ldsm(kt + tile_at(kKvTile, krow + kb * 16, ks * 2 + kchunk), kf);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            if constexpr (QF32) {
                                float t[4] = {0.f, 0.f, 0.f, 0.f};
                                mma<DT>(t, qa[0], kf[2 * n], kf[2 * n + 1]);
#pragma unroll
                                for (int x = 0; x < 4; ++x) s[2 * kb + n][x] += t[x];
#pragma unroll
                                for (int p = 1; p < PQ; ++p) mma<DT>(rest[2 * kb + n], qa[p], kf[2 * n], kf[2 * n + 1]);
                            } else {
                                mma<DT>(s[2 * kb + n], qa[0], kf[2 * n], kf[2 * n + 1]);
                            }
                        }
                    }
                }
                if constexpr (QF32) {
#pragma unroll
                    for (int n = 0; n < NS; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[n][x] += rest[n][x];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot]);
            if (++slot == SLOTS) {
                slot = 0;
                parity ^= 1;
            }
            // ---- mask, running maximum and sum
            if (edge) {
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int j = tok0 + n * 8 + qc * 2 + (x & 1);
                        if (j < row_lo[x >> 1] || j >= row_hi[x >> 1]) s[n][x] = -INFINITY;
                    }
            }
            float b0 = m0, b1 = m1;
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                b0 = fmaxf(b0, fmaxf(s[n][0], s[n][1]));
                b1 = fmaxf(b1, fmaxf(s[n][2], s[n][3]));
            }
#pragma unroll
            for (int x = 1; x < 4; x <<= 1) {
                b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, x));
                b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, x));
            }
            // a row that has seen nothing yet keeps a zero reference, so that its exponentials are e^-inf = 0
            const float r0 = b0 == -INFINITY ? 0.f : b0 * c0, r1 = b1 == -INFINITY ? 0.f : b1 * c1;
            const float f0 = m0 == -INFINITY ? 0.f : exp2_approx(fmaf(m0, c0, -r0));
            const float f1 = m1 == -INFINITY ? 0.f : exp2_approx(fmaf(m1, c1, -r1));
            m0 = b0;
            m1 = b1;
            float t0 = 0.f, t1 = 0.f;
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                s[n][0] = exp2_approx(fmaf(s[n][0], c0, -r0));
                s[n][1] = exp2_approx(fmaf(s[n][1], c0, -r0));
                s[n][2] = exp2_approx(fmaf(s[n][2], c1, -r1));
                s[n][3] = exp2_approx(fmaf(s[n][3], c1, -r1));
                t0 += s[n][0] + s[n][1];
                t1 += s[n][2] + s[n][3];
            }
            l0 = fmaf(l0, f0, t0);
            l1 = fmaf(l1, f1, t1);
            // ---- P in 16-bit parts, as the A operand of P V
            uint32_t pf[KB][PP][4];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t part[PP];
                    split<DT, PP>(s[2 * kb + (x >> 1)][2 * (x & 1)], s[2 * kb + (x >> 1)][2 * (x & 1) + 1], part);
#pragma unroll
                    for (int p = 0; p < PP; ++p) pf[kb][p][x] = part[p];
                }
            // ---- O = f O + P V
            if (ok) ok = warp_wait(&full[slot], parity);
            {
                const uint32_t vt = smem_u32(base + slot * P::kSlotBytes);
                const int vrow = wt * (kKvTile / WT) + (lane & 15), vchunk = lane >> 4;
#pragma unroll
                for (int n = 0; n < NO; n += 2) {
                    float t[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        uint32_t vf[4];
                        ldsm_t(vt + tile_at(kKvTile, vrow + kb * 16, n + vchunk), vf);
                        bool odd = false;
                        if (edge) {
                            // tokens no row sees: whatever the cache holds there counts as zero
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const int j = tok0 + kb * 16 + (x & 1) * 8 + qc * 2;
                                uint32_t keep = 0;
                                if (j >= w.t.lo && j < w.t.hi) keep |= 0xFFFFu;
                                if (j + 1 >= w.t.lo && j + 1 < w.t.hi) keep |= 0xFFFF0000u;
                                vf[x] &= keep;
                                odd = odd || H::odd(vf[x]);
                            }
                            odd = __any_sync(0xffffffffu, odd);
                        }
                        if (!odd) {
#pragma unroll
                            for (int p = PP - 1; p >= 0; --p) {
                                mma<DT>(t[0], pf[kb][p], vf[0], vf[1]);
                                mma<DT>(t[1], pf[kb][p], vf[2], vf[3]);
                            }
                        } else {
                            // an infinity or a NaN among values that some rows see and others
                            // do not: 0 * inf would reach the others, so each row adds only what
                            // it sees (token e of the block is in lane e % 8 / 2 of the quad)
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const int src = (lane & ~3) + ((e & 7) >> 1);
                                float pa = 0.f, pb = 0.f;
#pragma unroll
                                for (int p = PP - 1; p >= 0; --p) {
                                    const float2 ua = H::unpack(__shfl_sync(0xffffffffu, pf[kb][p][2 * (e >> 3)], src));
                                    const float2 ub = H::unpack(__shfl_sync(0xffffffffu, pf[kb][p][2 * (e >> 3) + 1], src));
                                    pa += e & 1 ? ua.y : ua.x;
                                    pb += e & 1 ? ub.y : ub.x;
                                }
                                const int j = tok0 + kb * 16 + e;
                                const bool see_a = j >= row_lo[0] && j < row_hi[0];
                                const bool see_b = j >= row_lo[1] && j < row_hi[1];
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const uint8_t* at_v = base + slot * P::kSlotBytes +
                                                          tile_at(kKvTile, wt * (kKvTile / WT) + kb * 16 + e, n + y) + qc * 4;
                                    const float2 v = H::unpack(*reinterpret_cast<const uint32_t*>(at_v));
                                    if (see_a) {
                                        t[y][0] = fmaf(pa, v.x, t[y][0]);
                                        t[y][1] = fmaf(pa, v.y, t[y][1]);
                                    }
                                    if (see_b) {
                                        t[y][2] = fmaf(pb, v.x, t[y][2]);
                                        t[y][3] = fmaf(pb, v.y, t[y][3]);
                                    }
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        o[n + y][0] = fmaf(o[n + y][0], f0, t[y][0]);
                        o[n + y][1] = fmaf(o[n + y][1], f0, t[y][1]);
                        o[n + y][2] = fmaf(o[n + y][2], f1, t[y][2]);
                        o[n + y][3] = fmaf(o[n + y][3], f1, t[y][3]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot]);
            if (++slot == SLOTS) {
                slot = 0;
                parity ^= 1;
            }
        }

        // ---- end of the pair's part in this CTA
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, x);
            l1 += __shfl_xor_sync(0xffffffffu, l1, x);
        }
        // maxima to log2 units
        m0 = m0 == -INFINITY ? m0 : m0 * c0;
        m1 = m1 == -INFINITY ? m1 : m1 * c1;
        if constexpr (WT > 1) {
            // the token warps of a row group: common maximum and sum, then each
            // warp adds up its share of the columns, in warp order
            if (qc == 0) {
                stats[warp][quad] = make_float2(m0, l0);
                stats[warp][quad + 8] = make_float2(m1, l1);
            }
            compute_sync();
            float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
            for (int x = 0; x < WT; ++x) {
                M0 = fmaxf(M0, stats[x * WR + wr][quad].x);
                M1 = fmaxf(M1, stats[x * WR + wr][quad + 8].x);
            }
            const float R0 = M0 == -INFINITY ? 0.f : M0, R1 = M1 == -INFINITY ? 0.f : M1;
            float L0 = 0.f, L1 = 0.f;
#pragma unroll
            for (int x = 0; x < WT; ++x) {
                const float2 sa = stats[x * WR + wr][quad], sb = stats[x * WR + wr][quad + 8];
                L0 = fmaf(sa.y, exp2_approx(sa.x - R0), L0);
                L1 = fmaf(sb.y, exp2_approx(sb.x - R1), L1);
            }
            const float g0 = exp2_approx(m0 - R0), g1 = exp2_approx(m1 - R1);
            m0 = M0;
            m1 = M1;
            l0 = L0;
            l1 = L1;
            // region of (row group, owner, source): 16 rows of DP / WT columns, 8-column groups swizzled by row
            auto region = [&](int owner, int src) {
                return merge + ((wr * WT + owner) * (WT - 1) + (src < owner ? src : src - 1)) * (16 * (DP / WT));
            };
            auto put = [&](int row, int n) { return row * (DP / WT) + (((n ^ row) & (NOWN - 1)) << 3) + qc * 2; };
#pragma unroll
            for (int n = 0; n < NO; ++n) {
                o[n][0] *= g0;
                o[n][1] *= g0;
                o[n][2] *= g1;
                o[n][3] *= g1;
                const int owner = n / NOWN;
                if (owner != wt) {
                    float* dst = region(owner, wt);
                    *reinterpret_cast<float2*>(dst + put(quad, n)) = make_float2(o[n][0], o[n][1]);
                    *reinterpret_cast<float2*>(dst + put(quad + 8, n)) = make_float2(o[n][2], o[n][3]);
                }
            }
            compute_sync();
#pragma unroll
            for (int n = 0; n < NO; ++n) {
                if (n / NOWN != wt) continue;
                float2 sa = make_float2(0.f, 0.f), sb = sa;
#pragma unroll
                for (int x = 0; x < WT; ++x) {
                    float2 va = make_float2(o[n][0], o[n][1]), vb = make_float2(o[n][2], o[n][3]);
                    if (x != wt) {
                        const float* from = region(wt, x);
                        va = *reinterpret_cast<const float2*>(from + put(quad, n));
                        vb = *reinterpret_cast<const float2*>(from + put(quad + 8, n));
                    }
                    sa.x += va.x;
                    sa.y += va.y;
                    sb.x += vb.x;
                    sb.y += vb.y;
                }
                o[n][0] = sa.x;
                o[n][1] = sa.y;
                o[n][2] = sb.x;
                o[n][3] = sb.y;
            }
        }
        // ---- write the rows: the output, or this CTA's part of a split pair
        const int part = 2 * blockIdx.x + (at == r.at ? 0 : 1);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int rr = wr * 16 + quad + 8 * x;
            if (rr >= w.t.rows) continue;
            const float m = x ? m1 : m0, l = x ? l1 : l0;
            if (whole) {
                const int flat = w.t.first_row + rr;
                const int64_t token = w.first + flat / a.group;
                const int head = w.h * a.group + flat % a.group;
                const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays NaN
                const int64_t off = token * a.out_stride + static_cast<int64_t>(head) * dim;
#pragma unroll
                for (int n = 0; n < NO; ++n) {
                    const int d = n * 8 + qc * 2;
                    if (n / NOWN != wt || d >= dim) continue;
                    const float u = o[n][2 * x] * inv, v = o[n][2 * x + 1] * inv;
                    if constexpr (QF32)
                        *reinterpret_cast<float2*>(static_cast<float*>(a.out) + off + d) = make_float2(u, v);
                    else
                        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + off + d) = H::pack(u, v);
                }
                if (a.lse && wt == 0 && qc == 0)
                    a.lse[token * (static_cast<int64_t>(a.cache.heads) * a.group) + head] =
                        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            } else {
                float* po = a.part_o + (static_cast<int64_t>(part) * ROWS + rr) * DP;
#pragma unroll
                for (int n = 0; n < NO; ++n)
                    if (n / NOWN == wt)
                        *reinterpret_cast<float2*>(po + n * 8 + qc * 2) = make_float2(o[n][2 * x], o[n][2 * x + 1]);
                if (wt == 0 && qc == 0) a.part_ml[static_cast<int64_t>(part) * ROWS + rr] = make_float2(m, l);
            }
        }
        if (w.tile == 0 && !whole) {  // the pair begins here and goes on in the next CTAs
            join_last = static_cast<int>(((at + w.t.tiles) * r.ctas - 1) / r.total);
            join_slot = at == r.at ? 0 : 1;
            join_row = w.first * a.group + w.t.first_row;
            join_rows = w.t.rows;
            join_head = w.h;
        }
        at += nt;
        w.tile += nt;
        if (at < r.end) next_pair<ROWS>(a, w);
    }
    if (warp == 0 && lane == 0) {
        a.join[2 * blockIdx.x] = make_int4(join_last, join_slot, join_row, join_rows);
        a.join[2 * blockIdx.x + 1] = make_int4(join_head, 0, 0, 0);
    }
}

// ------------------------------------------------------------- host side

// Shared by the instantiations of one (cache type, query type) slice.
template <int DT, bool QF32, int DP, int WR>
cudaError_t launch_one(const CUtensorMap& kmap, const CUtensorMap& vmap, const KvAttnArgs& a, int sm_count, bool pdl,
                       cudaStream_t stream, int* ctas) {
    using P = Plan<DP, WR, QF32, QF32 ? (DT == kBF16 ? 3 : 2) : 1>;
    auto kern = kv_attention_kernel<DT, QF32, DP, WR>;
    cudaError_t e = set_kernel_smem(kern, P::kBytes);
    if (e != cudaSuccess) return e;
    const int most = sm_count * P::kCtasPerSm;
    *ctas = most < kKvMaxCtas ? most : kKvMaxCtas;
    return launch_ex(kern, dim3(static_cast<unsigned>(*ctas)), dim3(kThreads), P::kBytes, stream, pdl, kmap, vmap, a);
}

template <int DT, bool QF32, int DP>
cudaError_t launch_rows(const CUtensorMap& kmap, const CUtensorMap& vmap, const KvAttnArgs& a, int rows, int sm_count,
                        bool pdl, cudaStream_t stream, int* ctas) {
    if (rows == 16) return launch_one<DT, QF32, DP, 1>(kmap, vmap, a, sm_count, pdl, stream, ctas);
    if (rows == 32) return launch_one<DT, QF32, DP, 2>(kmap, vmap, a, sm_count, pdl, stream, ctas);
    return launch_one<DT, QF32, DP, 4>(kmap, vmap, a, sm_count, pdl, stream, ctas);
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
