// kv_append8.cu -- a step's keys and values into a paged cache of 8-bit codes, queries
// normed and rotated on the way.
//
// A cached element is code * scale: an e4m3 code and an fp32 scale for each block of
// 2^block_shift rows of a page and head.  With y the normed and rotated key (or the
// value) in fp32, and a the largest finite |y| among the step's tokens of a block,
//   need  = the smallest power of two s >= 2^-126 with a <= 448 s (0 for a = 0),
//   scale = need, or the old scale where the block holds older tokens and that is larger,
//   code  = y / scale to the nearest e4m3, ties to even; 0 where scale = 0; NaN for y not finite,
// and where the scale of older tokens grew, their codes become code * old / scale,
// rounded likewise.  Scales are powers of two because e4m3 keeps its precision over them:
// a finer scale gains nothing above the subnormal codes, and a grown scale that is a
// multiple of the old one by a power of two moves older codes without rounding them
// again, down to the subnormal ones (below 2^-6: 2^-14.8 of a block's largest code).
//
// Work.  A unit is a block that the step touches: sequence b's k-th one has the number
// new_start[b] / rows + 2 b + k, which no two share (n tokens touch at most n / rows + 2
// blocks), so a CTA finds its unit without a sum over the batch; numbers that no block has end
// at once.  A warp (several for long blocks) takes a block of one head of keys or
// values, a lane eight elements of a row as two runs of four that a rotation pairs, and
// holds the warp's tokens in 64 registers between the largest value and the rounding.
// Queries have CTAs of their own behind the units' (a launch of their own, with twice the
// warps on an SM, made prompts of 16920 tokens 92 us instead of 83).  The rows' angles are
// neighbours in the table: one bulk copy per block brings them to shared memory.
//
// Bound: instruction issue (63 % of active cycles, 25 instructions an element over all) and load latency for
// prompts, three dependent loads for one token.
//
// Measured: one token of 16 + 8 + 8 heads of 128 in fp32 5.0 us, 190 drafts of 64 sequences 7.5
// us where their blocks' scales stand, 6.5 and 10.4 where every block's scale grows (its older codes
// are read once the largest value is known); prompts of 16920 tokens in bf16 74 us, 3.4 TB/s (251 MB).
// The append to a 16-bit cache is faster in each (2.5, 3.6 and 56 us): it does a token's work where this one
// does a block's, and packed arithmetic.  Sixteen tokens a warp at
// 128 registers took 110 us, angles from global memory 3 us more of a short call.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv.h"
#include "kv_rows.cuh"

namespace mnb {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
// Steps of 32 / G tokens that a warp holds: 16, 8 or 8 tokens (G = 8, 16, 32), so that 16
// warps hold a block of 128.
constexpr int held_steps(int g) { return g == 32 ? 8 : 4; }

__device__ __forceinline__ float smallest_scale(float largest) {
    const uint32_t bits = __float_as_uint(largest);
    if (bits == 0) return 0.f;
    // 448 = 1.75 * 2^8
    const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
}

// Two codes, a's in the low byte.  Values past 448 do not occur but by a rounding, and become 448.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
    return c;
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) { return codes2(a, b) | codes2(c, d) << 16; }
__device__ __forceinline__ float2 values2(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// Four codes of x / scale, by the reciprocal where that is exact (the scales made here are powers of
// two).  0 where the scale is 0; what is not finite becomes NaN (t + 0 t is t or NaN).
template <bool EXACT>
__device__ __forceinline__ uint32_t quotients4(const float (&x)[4], float scale, float inv) {
    float t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t[i] = EXACT ? x[i] * inv : __fdiv_rn(x[i], scale);
        t[i] = fmaf(t[i], 0.f, t[i]);
    }
    return codes4(t[0], t[1], t[2], t[3]);
}

// The last sequence whose first new token passes `upto` (which holds up to one sequence and for
// none behind it), its first and last new token's end and its length; without new_start
// sequence n itself, with one token.  128 sequences are asked for at a time, their lengths with
// them: the way to a token's page is three loads long.
struct Located {
    int seq, start, end, len;
};
template <typename F>
__device__ __forceinline__ Located locate(const KvStep& st, int n, F upto) {
    if (st.new_start == nullptr) return {n, n, n + 1, __ldg(st.seq_lens + n)};
    const int lane = threadIdx.x & 31;
    Located r = {-1, 0, 0, 0};
    for (int b0 = 0; b0 < st.batch; b0 += 128) {
        int lo[4], hi[4], len[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = b0 + 32 * i + lane;
            const bool is = s < st.batch;
            lo[i] = is ? __ldg(st.new_start + s) : 0;
            hi[i] = is ? __ldg(st.new_start + s + 1) : 0;
            len[i] = is ? __ldg(st.seq_lens + s) : 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s0 = b0 + 32 * i;
            const unsigned yes = __ballot_sync(0xffffffffu, s0 + lane < st.batch && upto(lo[i], s0 + lane));
            if (yes == 0) return r;
            const int src = __popc(yes) - 1;
            r = {s0 + src, __shfl_sync(0xffffffffu, lo[i], src), __shfl_sync(0xffffffffu, hi[i], src),
                 __shfl_sync(0xffffffffu, len[i], src)};
            if (yes != 0xffffffffu) return r;
        }
    }
    return r;
}

// One block of one head, by the `wpb` warps from this one's `part` = 0 on: rows [from,
// to) of the page are new, [begin, from) older.  src: the lane's head of the token in
// row `from`; page: looked at once the rows are on their way; angles: the new rows' in shared
// memory, once `landed` has its copy.
template <typename TI, int G, bool INTER>
__device__ __forceinline__ void store_block(const KvAppendArgs& a, bool key, int head, const TI* src, int64_t src_step, int page,
                                            int begin, int from, int to, int part, int wpb, float* parts, const float* angles,
                                            uint64_t* landed) {
    constexpr int kPer = 32 / G, kHeldSteps = held_steps(G);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % G, group = lane / G, dim = a.cache.dim;
    const bool in = sub * 8 < dim;
    const int half = key && a.cos_sin ? a.rot_dim / 2 : 0;
    const bool turns = sub * 4 < half, apart = turns && !INTER;
    const int i0 = apart ? sub * 4 : sub * 8, i1 = apart ? half + sub * 4 : sub * 8 + 4;
    const bool norm = key && a.k_norm != nullptr;
    const int row0 = begin + part * kHeldSteps * kPer + group;  // the lane's first row
    Raw4<TI> x[kHeldSteps], y[kHeldSteps];
#pragma unroll
    for (int s = 0; s < kHeldSteps; ++s) {
        const int row = row0 + s * kPer;
        if (in && row >= from && row < to) {
            const TI* p = src + (row - from) * src_step;
            x[s].load(p + i0);
            y[s].load(p + i1);
        } else {
            x[s] = {};
            y[s] = {};
        }
    }
    if (page < 0 || page >= a.cache.num_pages) return;  // (every warp of the CTA)
    uint8_t* base = static_cast<uint8_t*>(key ? a.cache.k : a.cache.v) + page * a.cache.page_stride + head * a.cache.head_stride;
    float* scale_at = (key ? a.cache.k_scale : a.cache.v_scale) + page * a.cache.scale_page_stride +
                      head * a.cache.scale_head_stride + (begin >> a.cache.block_shift);
    const float old = from > begin ? *scale_at : 0.f;
    Run4 wu = {{1.f, 1.f, 1.f, 1.f}}, ww = wu;
    if (norm && in) {
        wu = load4(a.k_norm + i0);
        ww = load4(a.k_norm + i1);
    }
    if (half > 0) mbar_wait(landed, 0);
    float largest = 0.f;
    Run4 u[kHeldSteps], w[kHeldSteps];
#pragma unroll
    for (int s = 0; s < kHeldSteps; ++s) {
        const int row = row0 + s * kPer;
        Run4 e = x[s].widen(), f = y[s].widen();
        if (norm) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = fmaf(e.x[i], e.x[i], fmaf(f.x[i], f.x[i], sum));
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = rsqrtf(fmaf(sum, 1.f / dim, a.eps));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e.x[i] = e.x[i] * inv * wu.x[i];
                f.x[i] = f.x[i] * inv * ww.x[i];
            }
        }
        if (turns && in && row >= from && row < to) {
            const float* turn = angles + (row - from) * a.rot_dim + sub * 4;
            const float4 c4 = *reinterpret_cast<const float4*>(turn), s4 = *reinterpret_cast<const float4*>(turn + half);
            const Run4 cs = {{c4.x, c4.y, c4.z, c4.w}}, sn = {{s4.x, s4.y, s4.z, s4.w}};
            if (INTER) {  // pairs (0, 1), (2, 3) of each run
                const Run4 p = e, q = f;
                e = {{fmaf(p.x[0], cs.x[0], -p.x[1] * sn.x[0]), fmaf(p.x[1], cs.x[0], p.x[0] * sn.x[0]),
                      fmaf(p.x[2], cs.x[1], -p.x[3] * sn.x[1]), fmaf(p.x[3], cs.x[1], p.x[2] * sn.x[1])}};
                f = {{fmaf(q.x[0], cs.x[2], -q.x[1] * sn.x[2]), fmaf(q.x[1], cs.x[2], q.x[0] * sn.x[2]),
                      fmaf(q.x[2], cs.x[3], -q.x[3] * sn.x[3]), fmaf(q.x[3], cs.x[3], q.x[2] * sn.x[3])}};
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = e.x[i], q = f.x[i];
                    e.x[i] = fmaf(p, cs.x[i], -q * sn.x[i]);
                    f.x[i] = fmaf(q, cs.x[i], p * sn.x[i]);
                }
            }
        }
        u[s] = e;
        w[s] = f;
#pragma unroll
        for (int i = 0; i < 4; ++i) largest = fmaxf(largest, fmaxf(fabsf(e.x[i]), fabsf(f.x[i])));  // (drops a NaN)
    }
    if (largest > 3.402823466e38f) {  // an infinity among them: the largest of the others
        largest = 0.f;
#pragma unroll
        for (int s = 0; s < kHeldSteps; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (finite(u[s].x[i])) largest = fmaxf(largest, fabsf(u[s].x[i]));
                if (finite(w[s].x[i])) largest = fmaxf(largest, fabsf(w[s].x[i]));
            }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, o));
    if (wpb > 1) {  // (a named barrier of the block's warps; `parts` is another array in the next call)
        const int first = warp - part;
        if (lane == 0) parts[warp] = largest;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + first / wpb), "r"(wpb * 32) : "memory");
        for (int k = 0; k < wpb; ++k) largest = fmaxf(largest, parts[first + k]);
    }
    const float need = smallest_scale(largest);
    const float scale = need > old ? need : old;
    const float inv = scale > 0.f ? 1.f / scale : 0.f;
    const bool exact = (__float_as_uint(scale) & 0x7FFFFFu) == 0 && (scale == 0.f || scale >= 1.17549435e-38f);
    auto store = [&](auto by_reciprocal) {
        constexpr bool EXACT = decltype(by_reciprocal)::value;
#pragma unroll
        for (int s = 0; s < kHeldSteps; ++s) {
            const int row = row0 + s * kPer;
            if (!in || row < from || row >= to) continue;
            uint8_t* dst = base + row * a.cache.token_stride;
            *reinterpret_cast<uint32_t*>(dst + i0) = quotients4<EXACT>(u[s].x, scale, inv);
            *reinterpret_cast<uint32_t*>(dst + i1) = quotients4<EXACT>(w[s].x, scale, inv);
        }
    };
    if (exact)
        store(std::true_type{});
    else
        store(std::false_type{});
    if (scale > old && from > begin) {
        const float ratio = old * inv;  // (a scale that grew is a power of two)
#pragma unroll 2
        for (int row = row0; row < min(from, begin + (part + 1) * kHeldSteps * kPer); row += kPer) {
            if (!in) continue;
            uint2* at = reinterpret_cast<uint2*>(base + row * a.cache.token_stride + sub * 8);
            const uint2 c = *at;
            const float2 v0 = values2(c.x), v1 = values2(c.x >> 16), v2 = values2(c.y), v3 = values2(c.y >> 16);
            *at = make_uint2(codes4(v0.x * ratio, v0.y * ratio, v1.x * ratio, v1.y * ratio),
                             codes4(v2.x * ratio, v2.y * ratio, v3.x * ratio, v3.y * ratio));
        }
    }
    if (part == 0 && lane == 0) *scale_at = scale;
}

// First kv_ctas CTAs: unit blockIdx.x / shares, a share of its heads of keys and values.
// The others: a token per warp and a share of `steps` steps of its query heads.
template <typename TI, int G, bool INTER>
__global__ void __launch_bounds__(kThreads, G == 32 ? 1 : 2) kv_append8_kernel(const KvAppendArgs a, int kv_ctas, int shares, int q_shares,
                                                                int steps) {
    constexpr int kPer = 32 / G;
    extern __shared__ __align__(16) float block_angles[];
    __shared__ float parts[2][kWarps];
    __shared__ __align__(8) uint64_t landed;
    if (threadIdx.x == 0) {
        mbar_init(&landed, 1);
        fence_barrier_init();
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, dim = a.cache.dim;
    const int shift = a.cache.block_shift, rows = 1 << shift;
    const KvStep& st = a.step;
    if (static_cast<int>(blockIdx.x) < kv_ctas) {
        const int unit = blockIdx.x / shares, share = blockIdx.x % shares;
        // the sequence that the unit's number falls to
        const Located at = locate(st, unit, [&](int start, int s) { return (max(start, 0) >> shift) + 2 * s <= unit; });
        if (at.seq < 0) return;
        const int b = at.seq, k = st.new_start ? unit - (max(at.start, 0) >> shift) - 2 * b : 0;
        const int first = min(max(at.start, 0), st.tokens), count = max(min(max(at.end, 0), st.tokens) - first, 0);
        const int64_t len = at.len;
        // tokens [skip, count) have positions from pos0 on
        const int64_t before = len - count;
        const int skip = static_cast<int>(before < 0 ? -before : 0);
        const int64_t pos0 = before < 0 ? 0 : before;
        if (skip >= count || k < 0) return;
        const int64_t block = (pos0 >> shift) + k;                          // the unit's block of the sequence
        const int64_t lo = max(pos0, block << shift);
        int64_t hi = min(len, (block + 1) << shift);
        if (lo >= hi) return;
        bool bad = false;
        if (a.cos_sin && hi > a.max_pos) {  // tokens without angles
            hi = max(lo, a.max_pos);
            bad = true;
        }
        int page = -1;
        if (lo < st.capacity) page = __ldg(st.page_table + b * st.table_stride + lo / a.cache.page_size);
        if (lo >= hi) {
            if (threadIdx.x == 0) record_error(MNB_ERR_CONTENT);
            return;
        }
        const int begin = static_cast<int>((block << shift) % a.cache.page_size);
        const int from = begin + static_cast<int>(lo - (block << shift)), to = from + static_cast<int>(hi - lo);
        const int64_t token = first + skip + (lo - pos0);
        const int wpb = max(1, rows / (held_steps(G) * kPer)), slots = kWarps / wpb;
        // the new rows' angles, where this CTA has keys (positions are neighbours in the table)
        const bool turned = a.cos_sin && share * slots < a.cache.heads;
        if (turned && threadIdx.x == 0) {
            const uint32_t bytes = static_cast<uint32_t>(hi - lo) * a.rot_dim * 4;
            mbar_arrive_expect_tx(&landed, bytes);
            bulk_g2s(block_angles, a.cos_sin + lo * a.rot_dim, bytes, &landed);
        }
        const int slot = warp / wpb, part = warp % wpb, jobs = 2 * a.cache.heads;
        int pass = 0;
        for (int j0 = share * slots; j0 < jobs; j0 += shares * slots, pass ^= 1) {
            const int job = j0 + slot, head = job < a.cache.heads ? job : job - a.cache.heads;
            const bool key = job < a.cache.heads;
            if (job >= jobs) break;  // (with it the other warps of its block)
            const TI* src = static_cast<const TI*>(key ? a.k : a.v) + token * (key ? a.k_stride : a.v_stride) + int64_t(head) * dim;
            store_block<TI, G, INTER>(a, key, head, src, key ? a.k_stride : a.v_stride, page, begin, from, to, part, wpb,
                                      parts[pass], block_angles, &landed);
        }
        if (page < 0 || page >= a.cache.num_pages) bad = true;
        if (bad && threadIdx.x == 0) record_error(MNB_ERR_CONTENT);
        if (turned && threadIdx.x == 0) mbar_wait(&landed, 0);  // no copy may be in flight when the CTA ends
        return;
    }
    // ---- queries
    const int index = blockIdx.x - kv_ctas, t = index / q_shares * kWarps + warp, q_share = index % q_shares;
    if (t >= st.tokens) return;
    const Located of = locate(st, t, [&](int start, int) { return start <= t; });
    const int seq = of.seq;
    if (seq < 0 || (st.new_start && of.end <= t)) return;
    const int first = min(max(of.start, 0), st.tokens), count = max(min(max(of.end, 0), st.tokens) - first, 0);
    const int64_t pos = int64_t(of.len) - count + (t - first);
    if (pos < 0) return;
    const int sub = lane % G, group = lane / G;
    const bool in = sub * 8 < dim;
    const int half = a.cos_sin ? a.rot_dim / 2 : 0;
    const bool turns = sub * 4 < half, apart = turns && !INTER;
    const int i0 = apart ? sub * 4 : sub * 8, i1 = apart ? half + sub * 4 : sub * 8 + 4;
    if (a.cos_sin && pos >= a.max_pos) return;  // (reported with the keys)
    int page = -1;
    if (pos < st.capacity) page = __ldg(st.page_table + seq * st.table_stride + pos / a.cache.page_size);
    if (page < 0 || page >= a.cache.num_pages) return;
    Run4 cs = {{1.f, 1.f, 1.f, 1.f}}, sn = {};
    if (turns) {
        const float* angles = a.cos_sin + pos * a.rot_dim + sub * 4;
        cs = load4(angles);
        sn = load4(angles + half);
    }
    const int begin = q_share * steps * kPer, end = min(begin + steps * kPer, a.q_heads);
    const int64_t at = int64_t(begin + group) * dim, step = int64_t(kPer) * dim;
    turn_heads<INTER, G>(static_cast<const TI*>(a.q) + t * a.q_stride + at, step,
                         static_cast<TI*>(a.q_out) + t * a.q_out_stride + at, step, begin + group, end, in, i0, i1, turns,
                         a.q_norm != nullptr, make_turn<INTER>(a.q_norm, in, i0, i1, cs, sn), 1.f / dim, a.eps);
}

template <typename TI, int G, bool INTER>
cudaError_t launch_pairs(const KvAppendArgs& a, int sm_count, bool pdl, cudaStream_t stream) {
    constexpr int kPer = 32 / G;
    const int rows = 1 << a.cache.block_shift;
    const int slots = kWarps / std::max(1, rows / (held_steps(G) * kPer));
    const int64_t units = a.step.new_start ? a.step.tokens / rows + int64_t(2) * a.step.batch : a.step.batch;
    // a block's heads are shared by as many CTAs as give every SM about four: few blocks
    // are bound by latency
    const int most = cdiv(2 * a.cache.heads, slots);
    const int shares = static_cast<int>(std::min<int64_t>(most, std::max<int64_t>(1, int64_t(sm_count) * 4 / units)));
    const int64_t kv_ctas = units * shares;
    int64_t q_ctas = 0;
    int q_shares = 1, steps = 1;
    if (a.q) {
        const int all = cdiv(a.q_heads, kPer);
        const int64_t want = cdiv<int64_t>(int64_t(sm_count) * 12, a.step.tokens);
        steps = cdiv(all, static_cast<int>(std::min<int64_t>(want, all)));
        q_shares = cdiv(all, steps);
        q_ctas = cdiv<int64_t>(a.step.tokens, kWarps) * q_shares;
    }
    if (kv_ctas + q_ctas > 0x7fffffff) return cudaErrorNotSupported;
    const size_t smem = a.cos_sin ? size_t(rows) * a.rot_dim * 4 : 0;
    return launch_cluster<kv_append8_kernel<TI, G, INTER>>(dim3(static_cast<unsigned>(kv_ctas + q_ctas)), dim3(kThreads), 1, smem,
                                                           128 * 256 * 4, stream, pdl, a, static_cast<int>(kv_ctas), shares,
                                                           q_shares, steps);
}

template <typename TI, int G>
cudaError_t launch_group(const KvAppendArgs& a, int sm_count, bool pdl, cudaStream_t stream) {
    return a.interleaved ? launch_pairs<TI, G, true>(a, sm_count, pdl, stream)
                         : launch_pairs<TI, G, false>(a, sm_count, pdl, stream);
}

template <typename TI>
cudaError_t launch_lanes(const KvAppendArgs& a, int sm_count, bool pdl, cudaStream_t stream) {
    if (a.cache.dim <= 64) return launch_group<TI, 8>(a, sm_count, pdl, stream);
    if (a.cache.dim <= 128) return launch_group<TI, 16>(a, sm_count, pdl, stream);
    return launch_group<TI, 32>(a, sm_count, pdl, stream);
}

}  // namespace

cudaError_t launch_kv_append8(const KvAppendArgs& a, int sm_count, bool pdl, cudaStream_t stream) {
    if (a.in_dtype == kF32) return launch_lanes<float>(a, sm_count, pdl, stream);
    return a.in_dtype == kBF16 ? launch_lanes<__nv_bfloat16>(a, sm_count, pdl, stream)
                               : launch_lanes<__half>(a, sm_count, pdl, stream);
}

cudaError_t kv_append8_take_error(unsigned int* out) { return take_unit_error(out); }

}  // namespace mnb
