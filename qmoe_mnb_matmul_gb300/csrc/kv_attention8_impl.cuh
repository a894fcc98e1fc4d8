// kv_attention8_impl.cuh -- attention of a step's new tokens over a paged cache of 8-bit
// codes with a scale for each block of tokens and head.
//
// Mathematics.  With codes K_j, V_j and scales a_j, b_j of token j's block: s_j = scale
// a_j (q . K_j), out = sum_j e^(s_j - m) b_j V_j / sum_j e^(s_j - m), one pass with the
// running maximum m and sum in fp32.  A scale belongs to a row of the score tile and of
// the weight tile, so neither tile of codes is ever multiplied by it: scores are
// multiplied after their products, weights before theirs.
//
// Work.  As over a 16-bit cache (kv_attention_impl.cuh): the line of tiles of all
// (sequence, row tile, key-value head) pairs is cut into a range per CTA, warps 4 and 5
// load key and value tiles by TMA, warps 0-3 compute S^T = K Q^T and O^T += V^T P^T by
// mma.sync m16n8k16, split parts go through the workspace to kv_join_kernel.  Steps of up
// to eight rows take tiles of 128 tokens, as many bytes as 64 of 16 bits, others tiles of
// 64 (their registers hold the scores of no more).
//
// Codes to operands.  e4m3 converts exactly to fp16, two codes an instruction.  A key tile
// comes by ldmatrix of 16-bit elements, that is pairs of codes: a lane gets four
// neighbouring codes of a key, where the instruction wants two pairs eight apart; the order
// of the head dimension is free as long as the queries' matches, so they are loaded as the
// codes lie (step of 16, lane qc: elements 4 qc .. 4 qc + 3).  A value tile comes by
// ldmatrix's transposed 16 x 16 matrices of bytes: a lane gets four neighbouring tokens of
// a column.  The order of a block's sixteen tokens is free likewise, as long as the
// weights' matches: row m of the score product is token_of(m), so that the lane's four
// tokens are its four places along the value product.
//
// Rounding.  Queries of every type are scaled by a power of two per row to a largest
// magnitude in [2^14, 2^15) and go in as fp16: one part for 16-bit queries (exact for
// elements down to 2^-31 of the row's largest, smaller ones err by 2^-39 of it), two for
// fp32 (22 bits, elements below 2^-17 of the largest err by 2^-39 of it).  Weights are
// 2^15 times as large and in two fp16 parts, as over an fp16 cache: 22 bits down to 2^-28
// of the row's largest so far, 16 to 2^-34, an error of 2^-51 of the largest below.  A
// warp's tokens of a tile take their weights times b_j / b (b the power of two above the
// largest of their scales; up to 16, 32 or 64 tokens share one) into the product, and the product is
// multiplied by b: a block whose scale is far below its neighbours' loses what that
// ratio takes from the 2^-51.  Sums of values of any size are finite: see kKvFarPower.
//
// Measured (GB300, heads of 128, join included): 64 sequences of 1 .. 8192 tokens, 16 query
// heads over 8, 545 MB: 95 us, 5.7 TB/s (fp32 queries 96; heads of 64, half the bytes, 73.5); 32 such
// sequences, 16 heads of 256 over 4, 274 MB: 54.6 us, 5.0 TB/s (fp32 59); one sequence of 131072
// tokens, 32 over 4, 134 MB: 33.9 us; 777 tokens: 8.0 us, all
// latency.  A tile takes 1.3 us and 0.2 us more per 4 KB of it: bound by the chain of a
// tile's steps in two compute warps per scheduler (issue slots 46 % of active cycles busy), not by the
// tensor pipe (25 %) or HBM (72 %).
// Several rows, 32 query heads over 4, 147 MB: 16 sequences of 8 .. 16 rows 50.4 us, of 8 .. 32
// rows 69 (fp32 queries 82), of 8 .. 40 rows 92 (fp32 132; over a 16-bit cache, with twice the bytes, 82:
// warps that split along the rows each convert the whole tile); of 4 .. 20 rows of heads of 80
// with a window, 57 MB: 40.3 us (fp32 44).  A prompt of 2048 tokens, 16 over 8: 265 us.  Spills, of 16-bit
// (fp32) queries at 168 registers: tiles of 32 rows 60 .. 96 (64 .. 324) bytes, of 64 rows 112 .. 436
// (256 .. 728), of eight rows none (up to 72).
// What was slower: one producer warp for keys, values and scales (153 us for the
// batch), three CTAs per SM with it (122) or with spills at 96 registers, the scores
// of the next tile among this one's products (105).
#pragma once

#include "kv_attention_units.cuh"

namespace mnb {

namespace {

// Shared-memory plan of an instantiation for row tiles of up to ROWS rows.
template <int DP, int ROWS, bool QF32>
struct Plan8 {
    static constexpr int kParts = QF32 ? 2 : 1;  // fp16 parts of a query
    static constexpr int kPad = DP <= 64 ? 64 : DP <= 128 ? 128 : 256;  // of the split parts' rows
    static constexpr int kTile = kv_tile8(ROWS, DP);
    static constexpr int kPanels = (DP + 127) / 128;  // of 128 columns (the last may be padding)
    static constexpr int kSlotBytes = kTile * kPanels * 128;
    static constexpr int kUnits = kTile / 8;  // groups of eight tokens, which share their scales
    // few rows keep their queries in registers
    static constexpr bool kQSmem = DP > 128 || ROWS > 8;
    static constexpr int kQRow = DP * 2 + 32;  // bytes; rows eight words apart in the banks
    static constexpr int kQBytes = kQSmem ? kParts * ROWS * kQRow : 0;
    static constexpr int kMergeRow = DP / 2 + 4;
    static constexpr int kMergeBytes = kComputeWarps * 8 * kMergeRow * 4;
    static constexpr int kRoom2 = 112 * 1024 - 4096 - kQBytes - kMergeBytes;
    static constexpr int kRoom1 = 226 * 1024 - 4096 - kQBytes - kMergeBytes;
    static constexpr int kCtasPerSm = (DP <= 128 || ROWS == 8) && kRoom2 >= 4 * kSlotBytes ? 2 : 1;
    static constexpr int kFit = (kCtasPerSm == 2 ? kRoom2 : kRoom1) / kSlotBytes;
    static constexpr int kSlots = kFit > 8 ? 8 : kFit;
    static constexpr int kKSlots = (kSlots + 1) / 2, kVSlots = kSlots / 2;
    static constexpr int kBytes = 1024 + kSlots * kSlotBytes + kQBytes + kMergeBytes;
    static_assert(kSlots >= 2, "a key tile and a value tile must fit");
};

// What a pair costs besides its tiles (its queries, the first tile's way, the join of the
// warps, the store), in tiles.  64 sequences of 1 .. 8192 tokens: 136 us with none, 117 with
// one, 108 with two, 100 with three, 95 with four and more; 8 of 2000 tokens 14.8 with two
// and three, 15.5 with four; 200 of 10 .. 300 48.8, 47.6, 48.5 with two, three, four.
// With more rows a tile's cost grows with them (of 64 tokens: 4 units up to 8 rows, 12 for 33 and
// more): 16 sequences of 4 .. 20 rows, heads of 80, 50 us with one unit for all, 42 with these.
// (All of it over 16-bit queries of heads of 80 and 128; fp32 queries and other widths go by the same.)
template <int ROWS>
struct Costs8 {
    static constexpr int kMost = ROWS == 8 ? 1 : ROWS == 32 ? 7 : 12, kPair = ROWS == 8 ? 4 : 16;
    static __device__ __forceinline__ int of(int rows) {
        return ROWS == 8 ? 1 : rows <= 8 ? 4 : rows <= 16 ? 5 : rows <= 32 ? 7 : 12;
    }
};

// Two codes (the low 16 bits) as fp16.
__device__ __forceinline__ uint32_t halves(uint32_t codes) {
    uint32_t h;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(codes));
    return h;
}
__device__ __forceinline__ uint32_t halves_high(uint32_t codes) {
    uint32_t h;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(h) : "r"(codes));
    return h;
}

// The token (of sixteen) in row m of a score product.
__device__ __forceinline__ int token_of(int m) { return (m & 6) * 2 + (m & 1) + (m >> 3) * 2; }

// Two transposed 16 x 16 matrices of bytes: from a 16-byte row per lane (0 .. 15 the first one's), lane
// l gets rows 4 (l % 4) .. + 3 of columns l / 4 (r[0]), l / 4 + 8 (r[1]), and the second one's.
__device__ __forceinline__ void ldsm_bytes_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Bytes of the codes among four that are NaN (0x7F, 0xFF).
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) {
    const uint32_t top = ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    return (top >> 7) * 0xFFu;
}

// Asynchronous copy of a float to shared memory (`take` false: a zero, nothing is read), and the
// arrival at a barrier once this thread's copies have landed (one of the barrier's count).
__device__ __forceinline__ void copy_float(float* dst, const float* src, bool take) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(take ? 4 : 0) : "memory");
}
__device__ __forceinline__ void arrive_with_copies(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Page and row of a token that moves on by a tile at a time.
struct Cursor {
    int tok, row;
    const int* page;
    __device__ __forceinline__ void start(const KvAttnArgs& a, const Walk& w, int token) {
        const int index = a.by_page(token);
        tok = token;
        page = a.step.page_table + w.b * a.step.table_stride + index;
        row = token - index * a.cache.page_size;
    }
    template <int TILE>
    __device__ __forceinline__ void next(const KvAttnArgs& a, int step_pages, int step_rows) {
        tok += TILE;
        row += step_rows;
        page += step_pages;
        if (row >= a.cache.page_size) {
            row -= a.cache.page_size;
            ++page;
        }
    }
};

// The key or the value tiles of the CTA's range, by one warp: lane l issues the box of
// row block l % blocks and panel l / blocks of every tile (32 boxes at most) and looks up
// its page itself, one tile ahead.  SCALES: lane l also copies the key scale (the upper
// sixteen lanes the value scale) of tokens 8 (l % 16) .. + 7 of the tile into the slot, its page
// looked up one tile ahead; both arrive with the key tile.  (Through a register, asked for one
// tile ahead, a scale's way from HBM could be a tile's time: 64 sequences of 1 .. 8192
// tokens with heads of 64 took 77 us instead of 73.)
template <int DP, int ROWS, bool QF32, int SLOTS, bool SCALES>
__device__ __forceinline__ void produce8(const KvAttnArgs& a, const CUtensorMap* map, uint8_t* slots, float* scales,
                                         uint64_t* full, uint64_t* empty, Walk w, const Range& r) {
    using P = Plan8<DP, ROWS, QF32>;
    constexpr int TILE = P::kTile;
    asm volatile("fence.proxy.async.global;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int R = a.box_rows, blocks = TILE / R, ps = a.cache.page_size;
    const int panel = lane / blocks, row0 = (lane % blocks) * R;
    const int step_pages = a.by_page(TILE), step_rows = TILE - step_pages * ps;
    const bool issues = panel < P::kPanels;
    const uint32_t dst = smem_u32(slots) + panel * (TILE * 128) + row0 * 128;
    const int unit = lane & 15;
    const bool scaled = SCALES && unit < P::kUnits;
    const float* table = lane < 16 ? a.cache.k_scale : a.cache.v_scale;
    Ring<SLOTS> ring;
    int issued = 0;
    int64_t at = r.at;
    bool ok = true, bad = false;
    while (at < r.end && ok) {
        const int nt = part_tiles<Costs8<ROWS>>(w, r.end - at);
        bad = bad || w.pos0 + w.count > a.step.capacity;
        const int first = (w.t.lo / TILE + w.tile) * TILE;
        Cursor box, mine;  // of the boxes, and of the scales
        box.start(a, w, first + row0);
        mine.start(a, w, first + unit * 8);
        // boxes that no row sees are asked for outside the cache, which fills them with
        // zeros and reads nothing; scales likewise
        auto wanted = [&] { return issues && box.tok < w.t.hi && box.tok + R > w.t.lo; };
        auto seen = [&](int tok) { return scaled && tok < w.t.hi && tok + 8 > w.t.lo; };
        int page = wanted() ? load_now(box.page) : -1;
        int scale_page = SCALES && seen(mine.tok) ? load_now(mine.page) : -1;
        for (int i = 0; i < nt; ++i) {
            const int cur = page, cur_row = box.row;
            const bool outside = wanted() && (cur < 0 || cur >= a.cache.num_pages);
            box.template next<TILE>(a, step_pages, step_rows);
            page = i + 1 < nt && wanted() ? load_now(box.page) : -1;
            const float* scale = table;
            bool scale_there = false;
            if (SCALES) {
                scale_there = scale_page >= 0 && scale_page < a.cache.num_pages;
                if (scale_there)
                    scale += scale_page * a.cache.scale_page_stride + w.h * a.cache.scale_head_stride +
                             (mine.row >> a.cache.block_shift);
                mine.template next<TILE>(a, step_pages, step_rows);
                scale_page = i + 1 < nt && seen(mine.tok) ? load_now(mine.page) : -1;
            }
            if (ok) ok = warp_wait(&empty[ring.slot], ring.parity ^ 1);  // the first round passes at once
            if (!ok) break;
            __syncwarp();  // the slot's scales were read, too
            if (issues) tma_load_4d(dst + ring.slot * P::kSlotBytes, map, panel * 128, cur_row, w.h, cur, &full[ring.slot]);
            if (SCALES) {
                copy_float(scales + ring.slot * 32 + lane, scale, scale_there);
                arrive_with_copies(&full[ring.slot]);
            }
            // (the tile may land before the barrier expects it: this arrival is still to come)
            if (lane == 0) mbar_arrive_expect_tx(&full[ring.slot], P::kSlotBytes);
            bad = bad || outside;
            ++issued;
            ring.next();
        }
        at += nt * w.t.cost;
        w.tile += nt;
        if (at < r.end) {
            next_pair<ROWS, TILE, Costs8<ROWS>>(a, w);
            at += Costs8<ROWS>::kPair;
        }
    }
    // a page number outside the cache: its tokens read as zeros; or a length past the page table
    if (bad) record_error(MNB_ERR_CONTENT);
    // no copy may be in flight when the CTA ends
    for (int n = max(0, issued - SLOTS); n < issued; ++n)
        warp_wait(&full[n % SLOTS], static_cast<uint32_t>(n / SLOTS) & 1u);
}

struct Smem8 {
    uint8_t *k, *v;   // rings of tiles
    float* scales;    // [key slots][32]: key scales of the tile's groups of eight tokens, value scales from 16 on
    uint8_t* q;
    float* merge;
    uint64_t *k_full, *k_empty, *v_full, *v_empty;
    float2* stats;    // [4][16]: a warp's reference and sum of its rows
    float2* rows;     // [64]: the rows' reference and sum after the join
    float* row_unit;  // [64]: power of two that a row of queries was scaled down by
    float* out_unit;  // [4]: what a warp's output is held times (1 or kKvFarDown)
};

// What a row of queries whose largest magnitude is `big` is multiplied by, and its
// reciprocal: powers of two that bring it to [2^14, 2^15), as far as both are normal
// numbers; a row with an infinity keeps its scale.
__device__ __forceinline__ void row_scale(float big, float& down, float& up) {
    uint32_t e = __float_as_uint(big) >> 23;
    down = up = 1.f;
    if (e < 255u) {
        e = min(max(e, 15u), 267u) - 14u;
        down = __uint_as_float((254u - e) << 23);
        up = __uint_as_float(e << 23);
    }
}

// Elements d .. d + 3 of a query (d a multiple of four below the head dimension).
__device__ __forceinline__ float4 query4(const void* q, int dtype, int64_t at) {
    if (dtype == kF32) return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(q) + at));
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(q) + at));
    const float2 a = dtype == kF16 ? Half2<kF16>::unpack(x.x) : Half2<kBF16>::unpack(x.x);
    const float2 b = dtype == kF16 ? Half2<kF16>::unpack(x.y) : Half2<kBF16>::unpack(x.y);
    return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ float largest4(float4 v) {
    return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

// This tile's value scales (exponent `be`) are the warp's first far ones (kv.h): its unit from now on,
// and what the tile's products and the outputs before it are multiplied by.  How it is
// reached is chosen by what it costs tiles without such scales (registers): within the edges'
// branch, as a call where registers spill anyway (8 .. 32 rows of heads of 128 69 us, inlined 70
// .. 75; fp32 queries 81, inlined 94), inlined up to eight rows (64 sequences 95.6, as a call 96.6).
template <int RG>
__device__ __forceinline__ void go_far(uint32_t be, float* unit, float& b, float (&f)[RG][2]) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) *unit = kKvFarDown;
    __syncwarp();
    b = __uint_as_float(be << 23) * (2.f * kKvFarDown);
#pragma unroll
    for (int g = 0; g < RG; ++g) {
        f[g][0] *= kKvFarDown;
        f[g][1] *= kKvFarDown;
    }
}
template <int RG>
__device__ __noinline__ void go_far_call(uint32_t be, float* unit, float& b, float (&f)[RG][2]) {
    go_far(be, unit, b, f);
}

// One pair's tiles w.tile .. w.tile + nt - 1 by the four compute warps, WR of them
// along the rows (8 RG rows each) and 4 / WR along a tile's tokens; the result goes
// to the output (`whole`) or to slot `part` of the workspace.
template <bool QF32, int DP, int ROWS, int WR, int RG, int KSLOTS, int VSLOTS>
__device__ __forceinline__ void run_part8(const KvAttnArgs& a, const Smem8& sm, const Walk& w, int nt, bool whole, int part,
                                          Ring<KSLOTS>& kring, Ring<VSLOTS>& vring, bool& ok) {
    using P = Plan8<DP, ROWS, QF32>;
    using H = Half2<kF16>;
    constexpr int PQ = P::kParts, PP = 2, TILE = P::kTile;
    constexpr int WT = kComputeWarps / WR;
    constexpr int TOK = TILE / WT;  // tokens of a warp in a tile
    constexpr int MT = TOK / 16;    // 16-token blocks of a warp
    constexpr int ND = DP / 16;     // 16-column blocks of the output
    constexpr int KS = DP / 16;     // steps along the head dimension of a score
    static_assert(8 * RG * WR <= ROWS, "the row groups lie within a row tile");
    constexpr bool kCall = ROWS > 8;  // of go_far
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wr = warp % WR, wt = warp / WR;
    const int quad = lane >> 2, qc = lane & 3;
    const int dim = a.cache.dim;
    const int row0 = wr * 8 * RG;  // the warp's first row of the row tile
    constexpr int kShift = kv_weight_shift(MNB_E4M3);

    // ---- queries: lane holds elements 4 qc .. 4 qc + 3 of each sixteen of row quad of each eight
    uint32_t qf[P::kQSmem ? 1 : KS][PQ][2];
    float c[RG][2];  // powers of two of the queries and the scale, rows 2 qc and 2 qc + 1 of each eight
    auto q_at = [&](int rr) {  // element offset of row rr's query
        const int flat = w.t.first_row + rr, tok = a.by_group(flat);
        return (w.first + tok) * a.q_stride + static_cast<int64_t>(w.h * a.group + flat - tok * a.group) * dim;
    };
    // (rounded towards zero: never infinite, so that a score of 0 times it stays 0)
    auto factor = [&](float up) { return __fmul_rz(a.scale_unit, up); };
    if constexpr (!P::kQSmem) {
        static_assert(P::kQSmem || (RG == 1 && WR == 1), "eight rows");
        const bool in = quad < w.t.rows;
        const int64_t at = in ? q_at(quad) : 0;
        float4 v[KS];
        float big = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int d = ks * 16 + qc * 4;
            v[ks] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in && d < dim) v[ks] = query4(a.q, QF32 ? kF32 : a.q_dtype, at + d);
            big = fmaxf(big, largest4(v[ks]));
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        float down, up;
        row_scale(big, down, up);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t lo[PQ], hi[PQ];
            split<kF16, PQ>(v[ks].x * down, v[ks].y * down, lo);
            split<kF16, PQ>(v[ks].z * down, v[ks].w * down, hi);
#pragma unroll
            for (int p = 0; p < PQ; ++p) {
                qf[ks][p][0] = lo[p];
                qf[ks][p][1] = hi[p];
            }
        }
        c[0][0] = factor(__shfl_sync(0xffffffffu, up, qc * 8));
        c[0][1] = factor(__shfl_sync(0xffffffffu, up, qc * 8 + 4));
    } else {
        compute_sync();  // the queries of the pair before are read
        // a warp takes every fourth row, two at a time so that their loads overlap
        constexpr int NV = (DP + 127) / 128, MINE = 2 * RG * WR;
#pragma unroll 1
        for (int k0 = 0; k0 < MINE; k0 += 2) {
            float4 v[2][NV];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int rr = warp + (k0 + k) * kComputeWarps;
                const bool in = rr < w.t.rows;
                const int64_t at = in ? q_at(rr) : 0;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int d = (i * 32 + lane) * 4;
                    v[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (in && d < dim) v[k][i] = query4(a.q, QF32 ? kF32 : a.q_dtype, at + d);
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int rr = warp + (k0 + k) * kComputeWarps;
                float big = 0.f, down, up;
#pragma unroll
                for (int i = 0; i < NV; ++i) big = fmaxf(big, largest4(v[k][i]));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                row_scale(big, down, up);
                if (lane == 0) sm.row_unit[rr] = up;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int d = (i * 32 + lane) * 4;
                    if (DP < 128 && d >= DP) continue;
                    uint32_t lo[PQ], hi[PQ];
                    split<kF16, PQ>(v[k][i].x * down, v[k][i].y * down, lo);
                    split<kF16, PQ>(v[k][i].z * down, v[k][i].w * down, hi);
#pragma unroll
                    for (int p = 0; p < PQ; ++p)
                        *reinterpret_cast<uint2*>(sm.q + (p * ROWS + rr) * P::kQRow + d * 2) = make_uint2(lo[p], hi[p]);
                }
            }
        }
        compute_sync();
#pragma unroll
        for (int g = 0; g < RG; ++g)
#pragma unroll
            for (int x = 0; x < 2; ++x) c[g][x] = factor(sm.row_unit[row0 + g * 8 + qc * 2 + x]);
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
    if (lane == 0) sm.out_unit[warp] = 1.f;  // (this warp's alone)
    __syncwarp();
    const bool active = row0 < w.t.rows;  // a warp whose rows are all padding only keeps the barriers
    int tok0 = (w.t.lo / TILE + w.tile) * TILE + wt * TOK;  // the warp's first token
    // This lane's ldmatrix row in a key and a value tile: 16 tokens of two 16-byte chunks.
    // Chunk c + 2 i of the row is the address of chunk c XOR 32 i within a panel.
    const uint32_t k_lane = tile_at(TILE, wt * TOK + token_of(lane & 15), lane >> 4);
    const uint32_t v_lane = tile_at(TILE, wt * TOK + (lane & 15), lane >> 4);
    const uint8_t* q_lane = sm.q + (row0 + quad) * P::kQRow + qc * 8;
#pragma unroll 1
    for (int i = 0; i < nt; ++i, tok0 += TILE) {
        // tokens that not every row sees
        const bool edge = tok0 < w.t.lo_all || tok0 + TOK > w.t.hi_all;
        // none of them is seen by any row: the warp only keeps the rings' order
        const bool none = ROWS == 8 && (tok0 >= w.t.hi || tok0 + TOK <= w.t.lo);
        // ---- scores.  With fp32 queries each product of the leading part starts from
        // zero, is added outside, and the smaller part is added last; otherwise two
        // accumulators take turns along the head dimension where a warp has little
        // other independent work.
        constexpr bool kTwo = !QF32 && MT * RG <= 2;
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
        float ka[MT], vb[MT];  // scales of keys and values: the lane's tokens of a block lie in one half of it
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const float* at = sm.scales + kring.slot * 32 + wt * (TOK / 8) + 2 * t + (quad >> 2);
            ka[t] = at[0];
            vb[t] = at[16];
        }
        if (active && !none) {
            const uint32_t kt = smem_u32(sm.k + kring.slot * P::kSlotBytes) + k_lane;
#pragma unroll
            for (int kp = 0; kp < KS / 2; ++kp) {  // two steps along the head dimension
                uint32_t qb[2][PQ][RG][2];
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int p = 0; p < PQ; ++p)
#pragma unroll
                        for (int g = 0; g < RG; ++g) {
                            if constexpr (P::kQSmem) {
                                const uint2 x = *reinterpret_cast<const uint2*>(q_lane + (p * ROWS + g * 8) * P::kQRow +
                                                                                (2 * kp + y) * 32);
                                qb[y][p][g][0] = x.x;
                                qb[y][p][g][1] = x.y;
                            } else {
                                qb[y][p][g][0] = qf[2 * kp + y][p][0];
                                qb[y][p][g][1] = qf[2 * kp + y][p][1];
                            }
                        }
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    uint32_t r[4];
                    ldsm((kt ^ ((kp & 3) << 5)) + (kp >> 2) * (TILE * 128) + t * 2048, r);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t k16[4] = {halves(r[2 * y]), halves(r[2 * y + 1]), halves_high(r[2 * y]),
                                                 halves_high(r[2 * y + 1])};
#pragma unroll
                        for (int g = 0; g < RG; ++g) {
                            if constexpr (QF32) {
                                float z[4] = {0.f, 0.f, 0.f, 0.f};
                                mma<kF16>(z, k16, qb[y][0][g][0], qb[y][0][g][1]);
#pragma unroll
                                for (int x = 0; x < 4; ++x) s[t][g][x] += z[x];
                                mma<kF16>(s2[t][g], k16, qb[y][PQ - 1][g][0], qb[y][PQ - 1][g][1]);
                            } else if constexpr (kTwo) {
                                mma<kF16>(y ? s2[t][g] : s[t][g], k16, qb[y][0][g][0], qb[y][0][g][1]);
                            } else {
                                mma<kF16>(s[t][g], k16, qb[y][0][g][0], qb[y][0][g][1]);
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int g = 0; g < RG; ++g)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        if constexpr (QF32 || kTwo) s[t][g][x] += s2[t][g][x];
                        // (the two powers first: a key's may pass 2^96, where the row's brings the score back)
                        s[t][g][x] *= __fmul_rz(ka[t], c[g][x & 1]);
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
        // ---- mask, running maximum and sum.  s[t][g][x]: token 16 t + token_of(quad + 8 (x / 2)), row 2 qc + x % 2
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
                            const int j = tok0 + t * 16 + token_of(quad + 8 * y);
                            if (j < lo || j >= hi) s[t][g][2 * y + x] = -INFINITY;
                        }
                }
        }
        // 2^(be - 126), a power of two above the warp's largest value scale, and the scales over it
        float b = 0.f;
#pragma unroll
        for (int t = 0; t < MT; ++t) b = fmaxf(b, vb[t]);
        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 16));
        const uint32_t be = min(max(__float_as_uint(b) >> 23, 1u), 254u);
        const float over = __uint_as_float((255u - be) << 23) * 0.25f;  // (subnormal for scales from 2^126 on)
#pragma unroll
        for (int t = 0; t < MT; ++t) vb[t] *= over;
        b = __uint_as_float(be << 23) * (2.f * sm.out_unit[warp]);
        float f[RG][2];
        uint32_t pb[MT][RG][PP][2];  // P^T in fp16 parts, as the B operand
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
                big = fmaxf(m[g][x], __fmaf_ru(big, a.scale_rest, -kShift));
                // a row that has seen nothing yet keeps a zero reference, so that its exponentials are 2^-inf = 0
                ref[x] = big == -INFINITY ? 0.f : big;
                f[g][x] = exp2_approx(m[g][x] - ref[x]);
                m[g][x] = big;
            }
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float& e = s[t][g][2 * y + x];
                        e = exp2_approx(fmaf(e, a.scale_rest, -ref[x]));
                        sum[x] += e;
                        e *= vb[t];
                    }
                    uint32_t parts[PP];
                    split<kF16, PP, kF16Up>(s[t][g][2 * y], s[t][g][2 * y + 1], parts);
#pragma unroll
                    for (int p = 0; p < PP; ++p) pb[t][g][p][y] = transpose8(parts[p]);
                }
#pragma unroll
            for (int x = 0; x < 2; ++x) l[g][x] = fmaf(l[g][x], f[g][x], sum[x]);
        }
        if (ok) ok = tile_wait(&sm.v_full[vring.slot], vring.parity);
        uint8_t* vtile = sm.v + vring.slot * P::kSlotBytes;
        const bool far = be > 126u + kKvFarPower, rare = edge || far;
        if (kCall ? rare : __builtin_expect(rare, 0)) {
            if (far && sm.out_unit[warp] == 1.f) {
                if constexpr (kCall)
                    go_far_call(be, sm.out_unit + warp, b, f);
                else
                    go_far(be, sm.out_unit + warp, b, f);
            }
            // What no row sees counts as zero whatever the cache holds: its codes are
            // cleared in the tile.  A NaN that some rows see must not reach the others
            // as 0 * NaN: it is cleared too once each row that sees it has added it.
            // (Tokens that every row sees, [first, last) of the warp's, need neither.)
            const int first = min(max(w.t.lo_all - tok0, 0), TOK), last = min(max(w.t.hi_all - tok0, first), TOK);
            auto scan = [&](bool clear_nan) {
                bool odd = false;
#pragma unroll 1
                for (int x = wr * 32 + lane; x < (TOK - (last - first)) * (DP / 16); x += 32 * WR) {
                    const int e = x / (DP / 16) < first ? x / (DP / 16) : x / (DP / 16) + last - first, j = tok0 + e;
                    uint4* at = reinterpret_cast<uint4*>(vtile + tile_at(TILE, wt * TOK + e, x % (DP / 16)));
                    uint4 v = *at;
                    const bool out = j < w.t.lo || j >= w.t.hi;
                    uint32_t* y = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t bad = nan_codes(y[k]);
                        odd = odd || (bad != 0 && !out);
                        y[k] = out ? 0u : y[k] & ~bad;
                    }
                    if (out || clear_nan) *at = v;
                }
                return odd;
            };
            if (tokens_or<WR>(wt, scan(false))) {
                // O = f O, NaN where a row sees one
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
                            const uint8_t* v = vtile + tile_at(TILE, wt * TOK + e, n) + quad;
                            const uint32_t bad = nan_codes(v[0] | v[8] << 8);
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                if (!(bad >> (8 * y) & 1u)) continue;
                                if (j >= lo[0] && j < hi[0]) add[2 * y] = __uint_as_float(0x7fffffffu);
                                if (j >= lo[1] && j < hi[1]) add[2 * y + 1] = __uint_as_float(0x7fffffffu);
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
        // ---- O^T = f O^T + b V^T P^T
        if (active) {
            const uint32_t vt = smem_u32(vtile) + v_lane;
#pragma unroll
            for (int np = 0; np < ND / 2; ++np) {  // 32 columns
                uint32_t r[MT][4];
#pragma unroll
                for (int t = 0; t < MT; ++t) ldsm_bytes_t((vt ^ ((np & 3) << 5)) + (np >> 2) * (TILE * 128) + t * 2048, r[t]);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float z[PP][RG][4] = {};
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const uint32_t v16[4] = {halves(r[t][2 * y]), halves(r[t][2 * y + 1]), halves_high(r[t][2 * y]),
                                                 halves_high(r[t][2 * y + 1])};
#pragma unroll
                        for (int p = PP - 1; p >= 0; --p)
#pragma unroll
                            for (int g = 0; g < RG; ++g) mma<kF16>(z[p][g], v16, pb[t][g][p][0], pb[t][g][p][1]);
                    }
#pragma unroll
                    for (int g = 0; g < RG; ++g)
#pragma unroll
                        for (int x = 0; x < 4; x += 2) {  // (packed fp32 instructions)
                            float (&to)[4] = o[2 * np + y][g];
                            const float2 sum = ffma2(make_float2(z[1][g][x], z[1][g][x + 1]),
                                                     make_float2(1.f / kF16Up, 1.f / kF16Up),
                                                     make_float2(z[0][g][x], z[0][g][x + 1]));
                            const float2 old = ffma2(make_float2(to[x], to[x + 1]), make_float2(f[g][0], f[g][1]),
                                                     make_float2(0.f, 0.f));
                            const float2 now = ffma2(sum, make_float2(b, b), old);
                            to[x] = now.x;
                            to[x + 1] = now.y;
                        }
                }
            }
        }
        if (edge) fence_proxy_async_smem();  // cleared codes, before the slot's next copy
        tile_free(&sm.v_empty[vring.slot], lane);
        vring.next();
    }

    // ---- end of the pair's part in this CTA: the warps that share rows agree on
    // their reference, sum and unit, and scale to it
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) l[g][x] += __shfl_xor_sync(0xffffffffu, l[g][x], y);
            if (quad == 0) sm.stats[warp * 16 + g * 8 + qc * 2 + x] = make_float2(m[g][x], l[g][x]);
        }
    compute_sync();
    const float unit = fminf(fminf(sm.out_unit[0], sm.out_unit[1]), fminf(sm.out_unit[2], sm.out_unit[3]));
    const float to_unit = unit < sm.out_unit[warp] ? kKvFarDown : 1.f;
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
            const float k = exp2_approx(m[g][x] - ref) * to_unit;
#pragma unroll
            for (int n = 0; n < ND; ++n) {
                o[n][g][x] *= k;
                o[n][g][2 + x] *= k;
            }
        }
    // ---- through shared memory, eight rows of each row group and half the columns
    // at a time: the token warps' shares are added in warp order, and rows come out
    // contiguous.
    constexpr int V4 = DP / 8;  // steps of four columns in half of them
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
            for (int i = threadIdx.x; i < 8 * WR * V4; i += 32 * kComputeWarps) {
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
                const float2 ml = sm.rows[rr];
                if (whole) {
                    const int flat = w.t.first_row + rr, tok = a.by_group(flat);
                    const int64_t token = w.first + tok;
                    const int head = w.h * a.group + flat - tok * a.group;
                    const float inv = (ml.y > 0.f ? 1.f / ml.y : (ml.y == 0.f ? 0.f : ml.y)) / unit;  // NaN stays NaN
                    const int64_t off = token * a.out_stride + static_cast<int64_t>(head) * dim + d;
                    sum = make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
                    if (d < dim) {
                        if constexpr (QF32)
                            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + off) = sum;
                        else
                            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + off) =
                                a.q_dtype == kF16 ? make_uint2(H::pack(sum.x, sum.y), H::pack(sum.z, sum.w))
                                                  : make_uint2(Half2<kBF16>::pack(sum.x, sum.y), Half2<kBF16>::pack(sum.z, sum.w));
                    }
                    if (a.lse && d == 0)
                        a.lse[token * (static_cast<int64_t>(a.cache.heads) * a.group) + head] =
                            kv_log_sum(ml.x, ml.y, kShift);
                } else {
                    const int64_t at = static_cast<int64_t>(part) * ROWS + rr;
                    *reinterpret_cast<float4*>(a.part_o + at * P::kPad + d) = sum;
                    if (d == 0) a.part_ml[at] = make_float2(ml.x, unit < 1.f ? -ml.y : ml.y);
                }
            }
        }
    compute_sync();  // the statistics and the last share are read
}

template <bool QF32, int DP, int ROWS>
__global__ void __launch_bounds__(kThreads, Plan8<DP, ROWS, QF32>::kCtasPerSm)
    kv_attention8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const KvAttnArgs a) {
    using P = Plan8<DP, ROWS, QF32>;
    constexpr int KSLOTS = P::kKSlots, VSLOTS = P::kVSlots, TILE = P::kTile;

    extern __shared__ uint8_t raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t k_full[KSLOTS], k_empty[KSLOTS], v_full[VSLOTS], v_empty[VSLOTS];
    __shared__ float2 stats[kComputeWarps * 16], rows[64];
    __shared__ float row_unit[64], scales[KSLOTS * 32], out_unit[kComputeWarps];
    uint8_t* q_smem = base + P::kSlots * P::kSlotBytes;
    const Smem8 sm = {base,   base + KSLOTS * P::kSlotBytes,
                      scales, q_smem,
                      reinterpret_cast<float*>(q_smem + P::kQBytes),
                      k_full, k_empty,
                      v_full, v_empty,
                      stats,  rows,
                      row_unit, out_unit};

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < KSLOTS; ++s) {
            mbar_init(&k_full[s], 1 + 32);  // the tile's, and a scale's per lane
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
    const Range r = find_range<ROWS, TILE, Costs8<ROWS>>(a, w);
    if (warp == kComputeWarps) {
        produce8<DP, ROWS, QF32, KSLOTS, true>(a, &kmap, sm.k, scales, k_full, k_empty, w, r);
        return;
    }
    if (warp > kComputeWarps) {
        produce8<DP, ROWS, QF32, VSLOTS, false>(a, &vmap, sm.v, nullptr, v_full, v_empty, w, r);
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
        const int nt = part_tiles<Costs8<ROWS>>(w, r.end - at);
        const bool whole = w.tile == 0 && nt == w.t.tiles;
        const int slot = at == r.at ? 0 : 1, part = 2 * blockIdx.x + slot;  // (r.at is the first part's first unit)
        // the warps split along the rows only as far as the pair's rows need
        auto run = [&](auto wr, auto rg) {
            run_part8<QF32, DP, ROWS, decltype(wr)::value, decltype(rg)::value>(a, sm, w, nt, whole, part, kring, vring, ok);
        };
        if (ROWS == 8 || w.t.rows <= 8) {
            run(Int<1>{}, Int<1>{});
        } else if constexpr (ROWS > 8) {
            if (w.t.rows <= 16) {
                run(Int<1>{}, Int<2>{});
            } else if (ROWS == 32 || w.t.rows <= 32) {
                run(Int<2>{}, Int<2>{});
            } else if constexpr (ROWS > 32) {
                run(Int<4>{}, Int<2>{});
            }
        }
        if (w.tile == 0 && !whole) {  // the pair begins here and goes on in the next CTAs
            // (a tile belongs to the CTA that its first unit falls to)
            const int last = r.owner(at + static_cast<int64_t>(w.t.tiles - 1) * w.t.cost);
            join = make_int4(last, 2 * w.t.rows + slot, w.first * a.group + w.t.first_row, w.h);
        }
        at += nt * w.t.cost;
        w.tile += nt;
        if (at < r.end) {
            next_pair<ROWS, TILE, Costs8<ROWS>>(a, w);
            at += Costs8<ROWS>::kPair;
        }
    }
    if (warp == 0 && lane == 0) a.join[blockIdx.x] = join;
}

// ------------------------------------------------------------- host side

template <bool QF32, int DP, int ROWS>
cudaError_t launch_one8(const CUtensorMap& kmap, const CUtensorMap& vmap, const KvAttnArgs& a, int sm_count, bool pdl,
                        cudaStream_t stream, int* ctas) {
    using P = Plan8<DP, ROWS, QF32>;
    const int most = sm_count * P::kCtasPerSm;
    *ctas = most < kKvMaxCtas ? most : kKvMaxCtas;
    return launch_ready<kv_attention8_kernel<QF32, DP, ROWS>>(dim3(static_cast<unsigned>(*ctas)), dim3(kThreads), P::kBytes,
                                                             stream, pdl, kmap, vmap, a);
}

template <bool QF32, int DP>
cudaError_t launch_rows8(const CUtensorMap& kmap, const CUtensorMap& vmap, const KvAttnArgs& a, int rows, int sm_count,
                         bool pdl, cudaStream_t stream, int* ctas) {
    if (rows == 8) return launch_one8<QF32, DP, 8>(kmap, vmap, a, sm_count, pdl, stream, ctas);
    if (rows == 32) return launch_one8<QF32, DP, 32>(kmap, vmap, a, sm_count, pdl, stream, ctas);
    return launch_one8<QF32, DP, 64>(kmap, vmap, a, sm_count, pdl, stream, ctas);
}

}  // namespace

// One slice of the instantiations (query type, padded head dimension); each slice lives
// in its own translation unit so the slices compile in parallel.
#define MNB_KV_ATTENTION8_SLICE(NAME, QF32, DP)                                                                    \
    cudaError_t NAME(const CUtensorMap& kmap, const CUtensorMap& vmap, const KvAttnArgs& a, int rows, int sm_count, \
                     bool pdl, cudaStream_t stream, int* ctas) {                                                   \
        return launch_rows8<QF32, DP>(kmap, vmap, a, rows, sm_count, pdl, stream, ctas);                           \
    }                                                                                                              \
    cudaError_t NAME##_take_error(unsigned int* out) { return take_unit_error(out); }

}  // namespace mnb
