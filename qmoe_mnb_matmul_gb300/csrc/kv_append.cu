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
// and its partner run, so that a rotation needs no exchange between lanes; the
// head's data are loaded before the chain of table lookups is waited for.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv.h"

namespace mnb {

namespace {

constexpr int kAppendThreads = 256;

struct Run4 {
    float x[4];
};

template <typename T>
__device__ __forceinline__ Run4 load4(const T* p) {
    Run4 r;
    if constexpr (sizeof(T) == 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p));
        r.x[0] = v.x; r.x[1] = v.y; r.x[2] = v.z; r.x[3] = v.w;
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        T e[4];
        *reinterpret_cast<uint2*>(e) = v;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.x[i] = to_f32(e[i]);
    }
    return r;
}

__device__ __forceinline__ __half round_to(float x, __half*) { return __float2half_rn(x); }
__device__ __forceinline__ __nv_bfloat16 round_to(float x, __nv_bfloat16*) { return __float2bfloat16_rn(x); }

template <typename T>
__device__ __forceinline__ void store4(T* p, const Run4& r) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(r.x[0], r.x[1], r.x[2], r.x[3]);
    } else {
        T e[4];
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

template <typename TI, typename TC, int G>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const KvAppendArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane % G, dim = a.cache.dim, kv_heads = a.cache.heads;
    const int first_k = a.q_heads, first_v = first_k + kv_heads, heads = first_v + kv_heads;
    constexpr int kHeadsPerWarp = 32 / G, kHeadsPerCta = kHeadsPerWarp * (kAppendThreads / 32);
    // the lane's runs: (i0, i1), a rotated pair where `turns`
    const bool in = sub * 8 < dim;
    const int half = a.cos_sin ? a.rot_dim / 2 : 0;
    const bool turns = sub * 4 < half;
    const bool apart = turns && !a.interleaved;
    const int i0 = apart ? sub * 4 : sub * 8, i1 = apart ? half + sub * 4 : sub * 8 + 4;

    for (int64_t t = blockIdx.x; t < a.step.tokens; t += gridDim.x) {
        const int seq = sequence_of(a.step, static_cast<int>(t));
        if (seq < 0) continue;  // a token of no sequence
        int first, count;
        step_tokens(a.step, seq, &first, &count);
        const int64_t pos = int64_t(__ldg(a.step.seq_lens + seq)) - count + (t - first);
        if (pos < 0) continue;  // a padding token: no position, nothing to write
        const bool has_slot = pos < a.step.capacity;
        const bool has_angle = a.cos_sin == nullptr || pos < a.max_pos;
        int page = -1;
        if (has_slot) page = __ldg(a.step.page_table + seq * a.step.table_stride + pos / a.cache.page_size);
        if (!has_angle || page < 0 || page >= a.cache.num_pages) {
            record_error(MNB_ERR_CONTENT);
            continue;
        }
        const int64_t slot = page * a.cache.page_stride + (pos % a.cache.page_size) * a.cache.token_stride;
        Run4 cs, sn;
        if (turns) {
            const float* row = a.cos_sin + pos * a.rot_dim + sub * 4;
            cs = load4(row);
            sn = load4(row + half);
        }
        for (int h0 = blockIdx.y * kHeadsPerCta + warp * kHeadsPerWarp; h0 < heads; h0 += gridDim.y * kHeadsPerCta) {
            const int h = h0 + lane / G;
            const bool live = in && h < heads && (h >= first_k || a.q_out != nullptr);
            const TI* src;
            if (h < first_k)
                src = static_cast<const TI*>(a.q) + t * a.q_stride + int64_t(h) * dim;
            else if (h < first_v)
                src = static_cast<const TI*>(a.k) + t * a.k_stride + int64_t(h - first_k) * dim;
            else
                src = static_cast<const TI*>(a.v) + t * a.v_stride + int64_t(h - first_v) * dim;
            Run4 u = {}, v = {};
            if (live) {
                u = load4(src + i0);
                v = load4(src + i1);
            }
            const float* w = h < first_k ? a.q_norm : h < first_v ? a.k_norm : nullptr;
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = fmaf(u.x[i], u.x[i], fmaf(v.x[i], v.x[i], ss));
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (!live) continue;
            if (w != nullptr) {
                const float inv = 1.f / sqrtf(ss / dim + a.eps);
                const Run4 wu = load4(w + i0), wv = load4(w + i1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u.x[i] = u.x[i] * inv * wu.x[i];
                    v.x[i] = v.x[i] * inv * wv.x[i];
                }
            }
            if (turns && h < first_v) {
                if (a.interleaved) {  // pairs (u0, u1), (u2, u3), (v0, v1), (v2, v3)
                    Run4 x = u, y = v;
                    u.x[0] = x.x[0] * cs.x[0] - x.x[1] * sn.x[0];
                    u.x[1] = x.x[1] * cs.x[0] + x.x[0] * sn.x[0];
                    u.x[2] = x.x[2] * cs.x[1] - x.x[3] * sn.x[1];
                    u.x[3] = x.x[3] * cs.x[1] + x.x[2] * sn.x[1];
                    v.x[0] = y.x[0] * cs.x[2] - y.x[1] * sn.x[2];
                    v.x[1] = y.x[1] * cs.x[2] + y.x[0] * sn.x[2];
                    v.x[2] = y.x[2] * cs.x[3] - y.x[3] * sn.x[3];
                    v.x[3] = y.x[3] * cs.x[3] + y.x[2] * sn.x[3];
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = u.x[i], y = v.x[i];
                        u.x[i] = x * cs.x[i] - y * sn.x[i];
                        v.x[i] = y * cs.x[i] + x * sn.x[i];
                    }
                }
            }
            if (h < first_k) {
                TI* dst = static_cast<TI*>(a.q_out) + t * a.q_out_stride + int64_t(h) * dim;
                store4(dst + i0, u);
                store4(dst + i1, v);
            } else {
                const bool is_k = h < first_v;
                TC* dst = static_cast<TC*>(is_k ? a.cache.k : a.cache.v) + slot +
                          (h - (is_k ? first_k : first_v)) * a.cache.head_stride;
                store4(dst + i0, u);
                store4(dst + i1, v);
            }
        }
    }
}

template <typename TI, typename TC>
cudaError_t launch_lanes(const KvAppendArgs& a, int sm_count, bool pdl, cudaStream_t stream) {
    const int runs = a.cache.dim / 8, G = runs <= 8 ? 8 : runs <= 16 ? 16 : 32;
    const int heads = (a.q_out ? a.q_heads : 0) + 2 * a.cache.heads;
    const int per_cta = (32 / G) * (kAppendThreads / 32);
    // few tokens: their heads spread over more CTAs
    const unsigned y = static_cast<unsigned>(a.step.tokens < sm_count ? cdiv(heads, per_cta) : 1);
    const unsigned x = static_cast<unsigned>(std::min<int64_t>(a.step.tokens, int64_t(sm_count) * 64));
    const dim3 grid(x, y), block(kAppendThreads);
    if (G == 8) return launch_ready<kv_append_kernel<TI, TC, 8>>(grid, block, 0, stream, pdl, a);
    if (G == 16) return launch_ready<kv_append_kernel<TI, TC, 16>>(grid, block, 0, stream, pdl, a);
    return launch_ready<kv_append_kernel<TI, TC, 32>>(grid, block, 0, stream, pdl, a);
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
