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
// again, down to the subnormal ones (448 / 2^15: 2^-14.8 of the block's largest).
//
// Work.  A unit is a block that the step touches: sequence b's k-th one has the number
// new_start[b] / rows + 2 b + k, which no two share (n tokens touch at most n / rows + 2
// blocks), so a CTA finds its unit without a sum over the batch; numbers that no block has end
// at once.  A warp (several for long blocks) takes a block of one head of keys or
// values, a lane eight elements of a row as two runs of four that a rotation pairs, and
// holds the warp's tokens in 64 registers between the largest value and the rounding.
// Queries have CTAs of their own behind the units'.
//
// Bound: HBM for prompts, three dependent loads for one token.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv.h"
#include "kv_rows.cuh"

namespace mnb {

namespace {

constexpr int kHeldSteps = 8;  // steps of 32 / G tokens that a warp holds

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

// Division by a scale: exact by its reciprocal where it is a power of two (those that
// this file makes), else a division.
struct Divide {
    float scale, inv;
    bool power;
    __device__ __forceinline__ explicit Divide(float s) {
        scale = s;
        inv = 1.f / s;
        power = (__float_as_uint(s) & 0x7FFFFFu) == 0 && s >= 1.17549435e-38f;
    }
    __device__ __forceinline__ float operator()(float x) const { return power ? x * inv : __fdiv_rn(x, scale); }
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// One block of one head, by the `wpb` warps from this one's `part` = 0 on: rows [from,
// to) of the page are new, [begin, from) older.  src: the lane's head of the token in
// row `from`; base: the page's head in the cache.  All warps of the CTA call it together
// (`on`: this one has a block) where wpb > 1.
template <typename TI, int G, bool INTER>
__device__ __forceinline__ void store_block(const KvAppendArgs& a, bool on, bool key, const TI* src, int64_t src_step,
                                            uint8_t* base, float* scale_at, int begin, int from, int to, int64_t pos,
                                            int part, int wpb, float* parts) {
    constexpr int kPer = 32 / G;
    const int lane = threadIdx.x & 31, sub = lane % G, group = lane / G, dim = a.cache.dim;
    const bool in = on && sub * 8 < dim;
    const int half = key && a.cos_sin ? a.rot_dim / 2 : 0;
    const bool turns = sub * 4 < half, apart = turns && !INTER;
    const int i0 = apart ? sub * 4 : sub * 8, i1 = apart ? half + sub * 4 : sub * 8 + 4;
    const bool norm = key && a.k_norm != nullptr;
    const float old = on && from > begin ? *scale_at : 0.f;
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
    Run4 wu = {{1.f, 1.f, 1.f, 1.f}}, ww = wu;
    if (norm && in) {
        wu = load4(a.k_norm + i0);
        ww = load4(a.k_norm + i1);
    }
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
            const float* angles = a.cos_sin + (pos + row - from) * a.rot_dim + sub * 4;
            const Run4 cs = load4(angles), sn = load4(angles + half);
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
        for (int i = 0; i < 4; ++i) {
            if (finite(e.x[i])) largest = fmaxf(largest, fabsf(e.x[i]));
            if (finite(f.x[i])) largest = fmaxf(largest, fabsf(f.x[i]));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, o));
    if (wpb > 1) {
        const int first = (threadIdx.x >> 5) - part;
        if (lane == 0) parts[threadIdx.x >> 5] = largest;
        __syncthreads();
        for (int k = 0; k < wpb; ++k) largest = fmaxf(largest, parts[first + k]);
    }
    if (!on) return;
    const float need = smallest_scale(largest);
    const float scale = need > old ? need : old;
    const Divide by(scale);
    // a value that is not finite, as NaN
    auto quotient = [&](float v) { return !finite(v) ? __uint_as_float(0x7fffffffu) : scale == 0.f ? 0.f : by(v); };
#pragma unroll
    for (int s = 0; s < kHeldSteps; ++s) {
        const int row = row0 + s * kPer;
        if (!in || row < from || row >= to) continue;
        uint8_t* dst = base + row * a.cache.token_stride;
        *reinterpret_cast<uint32_t*>(dst + i0) =
            codes4(quotient(u[s].x[0]), quotient(u[s].x[1]), quotient(u[s].x[2]), quotient(u[s].x[3]));
        *reinterpret_cast<uint32_t*>(dst + i1) =
            codes4(quotient(w[s].x[0]), quotient(w[s].x[1]), quotient(w[s].x[2]), quotient(w[s].x[3]));
    }
    if (scale > old && from > begin) {
        const float ratio = by(old);
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
template <typename TI, int G, bool INTER, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) kv_append8_kernel(const KvAppendArgs a, int kv_ctas, int shares,
                                                                          int q_shares, int steps) {
    constexpr int kPer = 32 / G, kWarps = THREADS / 32;
    __shared__ float parts[2][kWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, dim = a.cache.dim;
    const int shift = a.cache.block_shift, rows = 1 << shift;
    const KvStep& st = a.step;
    if (static_cast<int>(blockIdx.x) < kv_ctas) {
        const int unit = blockIdx.x / shares, share = blockIdx.x % shares;
        int b = unit, k = 0;
        if (st.new_start) {
            // the sequence that the unit's number falls to: the last with new_start / rows + 2 b at most that
            int upto = 0;
            for (int b0 = 0; b0 < st.batch; b0 += 32) {
                const int s = b0 + lane;
                const bool at_most = s < st.batch && (max(__ldg(st.new_start + s), 0) >> shift) + 2 * s <= unit;
                upto += __popc(__ballot_sync(0xffffffffu, at_most));
            }
            b = upto - 1;
            if (b < 0) return;
            k = unit - (max(__ldg(st.new_start + b), 0) >> shift) - 2 * b;
        }
        int first, count;
        step_tokens(st, b, &first, &count);
        // tokens [skip, count) have positions from pos0 on
        const int64_t len = __ldg(st.seq_lens + b), before = len - count;
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
        if (page < 0 || page >= a.cache.num_pages) bad = true;
        if (bad && threadIdx.x == 0) record_error(MNB_ERR_CONTENT);
        if (lo >= hi || page < 0 || page >= a.cache.num_pages) return;
        const int begin = static_cast<int>((block << shift) % a.cache.page_size);
        const int from = begin + static_cast<int>(lo - (block << shift)), to = from + static_cast<int>(hi - lo);
        const int64_t token = first + skip + (lo - pos0);
        const int wpb = max(1, rows / (kHeldSteps * kPer)), slots = kWarps / wpb;
        const int slot = warp / wpb, part = warp % wpb, jobs = 2 * a.cache.heads;
        int pass = 0;
        for (int j0 = share * slots; j0 < jobs; j0 += shares * slots, pass ^= 1) {
            const int job = j0 + slot, head = job < a.cache.heads ? job : job - a.cache.heads;
            const bool on = job < jobs, key = job < a.cache.heads;
            if (!on && wpb == 1) break;
            const TI* src = static_cast<const TI*>(key ? a.k : a.v) + token * (key ? a.k_stride : a.v_stride) + int64_t(head) * dim;
            uint8_t* base = static_cast<uint8_t*>(key ? a.cache.k : a.cache.v) + page * a.cache.page_stride +
                            head * a.cache.head_stride;
            float* scale = (key ? a.cache.k_scale : a.cache.v_scale) + page * a.cache.scale_page_stride +
                           head * a.cache.scale_head_stride + (begin >> shift);
            store_block<TI, G, INTER>(a, on, key, src, key ? a.k_stride : a.v_stride, base, scale, begin, from, to, lo, part,
                                      wpb, parts[pass]);
        }
        return;
    }
    // ---- queries
    const int index = blockIdx.x - kv_ctas, t = index / q_shares * kWarps + warp, q_share = index % q_shares;
    if (t >= st.tokens) return;
    const int seq = sequence_of(st, t);
    if (seq < 0) return;
    int first, count;
    step_tokens(st, seq, &first, &count);
    const int64_t pos = int64_t(__ldg(st.seq_lens + seq)) - count + (t - first);
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
    // blocks of up to 128 rows: eight tokens of 256 elements a warp need 16 warps
    constexpr int THREADS = G == 32 ? 512 : 256, kWarps = THREADS / 32, kPer = 32 / G;
    const int rows = 1 << a.cache.block_shift;
    const int slots = kWarps / std::max(1, rows / (kHeldSteps * kPer));
    const int64_t units = a.step.new_start ? a.step.tokens / rows + int64_t(2) * a.step.batch : a.step.batch;
    // a block's heads are shared by as many CTAs as give every SM about eight: few blocks
    // are bound by latency
    const int most = cdiv(2 * a.cache.heads, slots);
    const int shares = static_cast<int>(std::min<int64_t>(most, std::max<int64_t>(1, int64_t(sm_count) * 8 / units)));
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
    return launch_ready<kv_append8_kernel<TI, G, INTER, THREADS>>(dim3(static_cast<unsigned>(kv_ctas + q_ctas)), dim3(THREADS),
                                                                  0, stream, pdl, a, static_cast<int>(kv_ctas), shares,
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
