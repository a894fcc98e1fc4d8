// kv_append.cu -- a step's keys and values into the paged cache, with the
// per-head norm and the position rotation of queries and keys on the way.
//
// y = x / sqrt(mean(x^2) + eps) * w per head (where a norm weight is given), then
// the first rot_dim elements turn by the position's angles: a pair (a, b) becomes
// (a cos - b sin, b cos + a sin), paired half a rotation apart or interleaved.
// All of it in fp32 with one rounding at the store.
//
// Bound: HBM for prompts (each element is read once and written once), the
// launch and three dependent loads (new_start, seq_lens, page_table) for one
// token.  A group of G lanes (the power of two at or above dim / 8) holds one
// head vector, 8 elements a lane as two runs of four: in the rotated part a run
// and its partner run, so that a rotation needs no exchange between lanes.  A
// warp takes one token (or a share of its heads, where tokens are few): its
// angles, times the norm's weights, stay in registers over the heads, and those
// are read two steps at a time (at four CTAs per SM and 64 registers that spills up
// to 36 bytes; four steps spilled more and took 75 us instead of 56 for 16920 tokens
// of 32 heads).
//
// Measured: one token of 16 + 8 + 8 heads of 128 in fp32 2.5 us; prompts of 16920 tokens
// in bf16 55.6 us, 5.1 TB/s (286 MB), between instruction issue (57 %) and load latency
// at 32 warps per SM.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "kv.h"

namespace mnb {

namespace {

constexpr int kAppendThreads = 256;

// Four elements as floats, and as loaded.
struct Run4 {
    float x[4];
};
template <typename T>
struct Raw4 {
    using V = typename std::conditional<sizeof(T) == 4, float4, uint2>::type;
    V v;
    __device__ __forceinline__ void load(const T* p) { v = __ldg(reinterpret_cast<const V*>(p)); }
    __device__ __forceinline__ Run4 widen() const {
        Run4 r;
        alignas(16) T e[4];
        *reinterpret_cast<V*>(e) = v;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.x[i] = to_f32(e[i]);
        return r;
    }
};

__device__ __forceinline__ Run4 load4(const float* p) {
    Raw4<float> r;
    r.load(p);
    return r.widen();
}

__device__ __forceinline__ __half round_to(float x, __half*) { return __float2half_rn(x); }
__device__ __forceinline__ __nv_bfloat16 round_to(float x, __nv_bfloat16*) { return __float2bfloat16_rn(x); }

template <typename T>
__device__ __forceinline__ void store4(T* p, const Run4& r) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(r.x[0], r.x[1], r.x[2], r.x[3]);
    } else {
        alignas(16) T e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = round_to(r.x[i], static_cast<T*>(nullptr));
        *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(e);
    }
}

// The sequence that token t belongs to, or -1: the number of sequences that
// end at or before t, counted by the warp 32 boundaries at a time (new_start
// does not decrease).
__device__ __forceinline__ int sequence_of(const KvStep& s, int t) {
    if (s.new_start == nullptr) return t;
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int b0 = 0; b0 < s.batch; b0 += 32) {
        const int b = b0 + lane;
        const bool ended = b < s.batch && __ldg(s.new_start + b + 1) <= t;
        before += __popc(__ballot_sync(0xffffffffu, ended));
    }
    return before < s.batch && __ldg(s.new_start + before) <= t ? before : -1;
}

// What a lane does with its eight elements of every head of q or of k: the runs
// (e, f) at offsets i0 and i1, element e_j paired with f_j, become inv * (e A - f B) and
// inv * (f C + e D), where the norm's weights are folded into the angles (A = w_e cos,
// B = w_f sin, C = w_f cos, D = w_e sin) and inv is the head's reciprocal norm.
struct Turn {
    float2 A[2], B[2], C[2], D[2];
};

// Heads h, h + kPer, .. below `end` of one token, G lanes each: normed, rotated and
// rounded from `src` to `dst` (pointers to the lane's head h).
template <bool INTER, int G, typename TI, typename TO>
__device__ __forceinline__ void turn_heads(const TI* src, int64_t src_step, TO* dst, int64_t dst_step, int h, int end,
                                           bool in, int i0, int i1, bool turns, bool norm, const Turn& c, float inv_dim,
                                           float eps) {
    constexpr int kPer = 32 / G, kAtOnce = 2;
#pragma unroll 1
    for (int h0 = h; h0 - static_cast<int>(threadIdx.x & 31) / G < end; h0 += kAtOnce * kPer) {
        Raw4<TI> x[kAtOnce] = {}, y[kAtOnce] = {};
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s)
            if (in && h0 + s * kPer < end) {
                x[s].load(src + s * src_step + i0);
                y[s].load(src + s * src_step + i1);
            }
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s) {
            Run4 e = x[s].widen(), f = y[s].widen();
            if (INTER) {  // pairs (0, 1), (2, 3) of each run
                const Run4 u = e, w = f;
                e = {{u.x[0], u.x[2], w.x[0], w.x[2]}};
                f = {{u.x[1], u.x[3], w.x[1], w.x[3]}};
            }
            // pairs of elements at a time (packed fp32 instructions)
            const float2 e2[2] = {make_float2(e.x[0], e.x[1]), make_float2(e.x[2], e.x[3])};
            const float2 f2[2] = {make_float2(f.x[0], f.x[1]), make_float2(f.x[2], f.x[3])};
            float inv = 1.f;
            if (norm) {
                float2 ss = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 2; ++i) ss = ffma2(e2[i], e2[i], ffma2(f2[i], f2[i], ss));
                float sum = ss.x + ss.y;
#pragma unroll
                for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                inv = rsqrtf(fmaf(sum, inv_dim, eps));
            }
            const float2 zero = make_float2(0.f, 0.f), inv2 = make_float2(inv, inv);
            Run4 u, w;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float2 x2, y2;
                if (turns) {
                    x2 = ffma2(f2[i], c.B[i], zero);
                    x2 = ffma2(e2[i], c.A[i], make_float2(-x2.x, -x2.y));
                    y2 = ffma2(f2[i], c.C[i], ffma2(e2[i], c.D[i], zero));
                } else {  // past the rotated part: A and C alone
                    x2 = ffma2(e2[i], c.A[i], zero);
                    y2 = ffma2(f2[i], c.C[i], zero);
                }
                if (norm) {
                    x2 = ffma2(x2, inv2, zero);
                    y2 = ffma2(y2, inv2, zero);
                }
                u.x[2 * i] = x2.x;
                u.x[2 * i + 1] = x2.y;
                w.x[2 * i] = y2.x;
                w.x[2 * i + 1] = y2.y;
            }
            if (INTER) {
                e = u;
                f = w;
                u = {{e.x[0], f.x[0], e.x[1], f.x[1]}};
                w = {{e.x[2], f.x[2], e.x[3], f.x[3]}};
            }
            if (in && h0 + s * kPer < end) {
                store4(dst + s * dst_step + i0, u);
                store4(dst + s * dst_step + i1, w);
            }
        }
        src += kAtOnce * src_step;
        dst += kAtOnce * dst_step;
    }
}

// blockIdx.x: eight tokens, one per warp; blockIdx.y: a share of `steps` steps of 32 /
// G heads each, over the steps of q, then of k, then of v.
template <typename TI, typename TC, int G, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, 4) kv_append_kernel(const KvAppendArgs a, int steps) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int sub = lane % G, dim = a.cache.dim;
    constexpr int kPer = 32 / G;  // heads per step
    const int t = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.step.tokens) return;
    const int seq = sequence_of(a.step, t);
    if (seq < 0) return;  // a token of no sequence
    int first, count;
    step_tokens(a.step, seq, &first, &count);
    const int64_t pos = int64_t(__ldg(a.step.seq_lens + seq)) - count + (t - first);
    if (pos < 0) return;  // a padding token: no position, nothing to write
    // the lane's runs: (i0, i1), rotated pairs where `turns`
    const bool in = sub * 8 < dim;
    const int half = a.cos_sin ? a.rot_dim / 2 : 0;
    const bool turns = sub * 4 < half;
    const bool apart = turns && !INTER;
    const int i0 = apart ? sub * 4 : sub * 8, i1 = apart ? half + sub * 4 : sub * 8 + 4;
    const bool has_angle = a.cos_sin == nullptr || pos < a.max_pos;
    Run4 cs = {{1.f, 1.f, 1.f, 1.f}}, sn = {};
    if (turns && has_angle) {
        const float* row = a.cos_sin + pos * a.rot_dim + sub * 4;
        cs = load4(row);
        sn = load4(row + half);
    }
    // (position < 2^31: seq_lens is 32-bit)
    const int index = static_cast<int>(pos) / a.cache.page_size, row = static_cast<int>(pos) - index * a.cache.page_size;
    int page = -1;
    if (pos < a.step.capacity) page = __ldg(a.step.page_table + seq * a.step.table_stride + index);
    if (!has_angle || page < 0 || page >= a.cache.num_pages) {
        record_error(MNB_ERR_CONTENT);
        return;
    }
    const int64_t slot = page * a.cache.page_stride + row * a.cache.token_stride;
    const float inv_dim = 1.f / dim;
    const int64_t src_step = kPer * dim, dst_step = kPer * a.cache.head_stride;

    auto turn_of = [&](const float* weights) {
        Run4 wu = {{1.f, 1.f, 1.f, 1.f}}, ww = wu;
        if (weights != nullptr && in) {
            wu = load4(weights + i0);
            ww = load4(weights + i1);
        }
        if (INTER) {
            const Run4 u = wu, w = ww;
            wu = {{u.x[0], u.x[2], w.x[0], w.x[2]}};
            ww = {{u.x[1], u.x[3], w.x[1], w.x[3]}};
        }
        Turn c;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = 2 * i, k = j + 1;
            c.A[i] = make_float2(wu.x[j] * cs.x[j], wu.x[k] * cs.x[k]);
            c.B[i] = make_float2(ww.x[j] * sn.x[j], ww.x[k] * sn.x[k]);
            c.C[i] = make_float2(ww.x[j] * cs.x[j], ww.x[k] * cs.x[k]);
            c.D[i] = make_float2(wu.x[j] * sn.x[j], wu.x[k] * sn.x[k]);
        }
        return c;
    };
    // this share's steps, section by section
    const int q_steps = a.q_out ? cdiv(a.q_heads, kPer) : 0, kv_steps = cdiv(a.cache.heads, kPer);
    const int s0 = blockIdx.y * steps, s1 = s0 + steps;
    const int group = lane / G;
    auto section = [&](int before, int n, int heads, int* begin, int* end) {  // heads [begin, end) of a section
        *begin = max(s0 - before, 0) * kPer;
        *end = min(min(s1 - before, n) * kPer, heads);
        return *begin < *end;
    };
    int begin, end;
    if (section(0, q_steps, a.q_heads, &begin, &end)) {
        const int64_t at = int64_t(begin + group) * dim;
        turn_heads<INTER, G>(static_cast<const TI*>(a.q) + t * a.q_stride + at, src_step,
                             static_cast<TI*>(a.q_out) + t * a.q_out_stride + at, src_step, begin + group, end, in, i0, i1,
                             turns, a.q_norm != nullptr, turn_of(a.q_norm), inv_dim, a.eps);
    }
    if (section(q_steps, kv_steps, a.cache.heads, &begin, &end)) {
        turn_heads<INTER, G>(static_cast<const TI*>(a.k) + t * a.k_stride + int64_t(begin + group) * dim, src_step,
                             static_cast<TC*>(a.cache.k) + slot + (begin + group) * a.cache.head_stride, dst_step,
                             begin + group, end, in, i0, i1, turns, a.k_norm != nullptr, turn_of(a.k_norm), inv_dim, a.eps);
    }
    if (section(q_steps + kv_steps, kv_steps, a.cache.heads, &begin, &end) && in) {
        const TI* src = static_cast<const TI*>(a.v) + t * a.v_stride + int64_t(begin + group) * dim + sub * 8;
        TC* dst = static_cast<TC*>(a.cache.v) + slot + (begin + group) * a.cache.head_stride + sub * 8;
#pragma unroll 4
        for (int h = begin + group; h < end; h += kPer, src += src_step, dst += dst_step) {
            Raw4<TI> x, y;
            x.load(src);
            y.load(src + 4);
            store4(dst, x.widen());
            store4(dst + 4, y.widen());
        }
    }
}

template <typename TI, typename TC, int G>
cudaError_t launch_group(const KvAppendArgs& a, int sm_count, bool pdl, cudaStream_t stream) {
    // A token's heads are shared by as many warps as give every SM about 12 (one head
    // step each at most; with 24 the steps of 200 tokens took 4.6 us instead of 3.9):
    // few tokens are bound by latency, many by HBM.
    const int all = (a.q_out ? cdiv(a.q_heads, 32 / G) : 0) + 2 * cdiv(a.cache.heads, 32 / G);
    const int64_t want = cdiv<int64_t>(int64_t(sm_count) * 12, a.step.tokens);
    const int steps = cdiv(all, static_cast<int>(std::min<int64_t>(want, all)));
    const dim3 grid(static_cast<unsigned>(cdiv(a.step.tokens, kAppendThreads / 32)), static_cast<unsigned>(cdiv(all, steps)));
    if (a.interleaved)
        return launch_ready<kv_append_kernel<TI, TC, G, true>>(grid, dim3(kAppendThreads), 0, stream, pdl, a, steps);
    return launch_ready<kv_append_kernel<TI, TC, G, false>>(grid, dim3(kAppendThreads), 0, stream, pdl, a, steps);
}

template <typename TI, typename TC>
cudaError_t launch_lanes(const KvAppendArgs& a, int sm_count, bool pdl, cudaStream_t stream) {
    if (a.cache.dim <= 64) return launch_group<TI, TC, 8>(a, sm_count, pdl, stream);
    if (a.cache.dim <= 128) return launch_group<TI, TC, 16>(a, sm_count, pdl, stream);
    return launch_group<TI, TC, 32>(a, sm_count, pdl, stream);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, int sm_count, bool pdl, cudaStream_t stream) {
    const bool bf = a.cache.dtype == kBF16;
    if (a.in_dtype == kF32)
        return bf ? launch_lanes<float, __nv_bfloat16>(a, sm_count, pdl, stream)
                  : launch_lanes<float, __half>(a, sm_count, pdl, stream);
    return bf ? launch_lanes<__nv_bfloat16, __nv_bfloat16>(a, sm_count, pdl, stream)
              : launch_lanes<__half, __half>(a, sm_count, pdl, stream);
}

cudaError_t kv_append_take_error(unsigned int* out) { return take_unit_error(out); }

}  // namespace mnb
