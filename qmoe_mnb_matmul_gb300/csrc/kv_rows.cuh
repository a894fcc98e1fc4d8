// kv_rows.cuh -- a token's rows of queries, keys and values: loads and stores in runs
// of four, the per-head norm and the position rotation (shared by the two appends).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "kv.h"

namespace mnb {

namespace {

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

// The angles (cs, sn) of a lane's runs with the norm's weights (null: none) folded in.
template <bool INTER>
__device__ __forceinline__ Turn make_turn(const float* weights, bool in, int i0, int i1, const Run4& cs, const Run4& sn) {
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
}

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

}  // namespace

}  // namespace mnb
