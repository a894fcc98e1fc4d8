// kv_attention.cu -- host side of the paged attention (see
// kv_attention_impl.cuh) and the kernel that joins the parts of split pairs.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "kernels.h"
#include "kv.h"
#include "tensor_map.h"

namespace mnb {

#define MNB_SLICE_DECL(NAME)                                                                                    \
    cudaError_t NAME(const CUtensorMap& kmap, const CUtensorMap& vmap, const KvAttnArgs& a, int rows, int pad,  \
                     int sm_count, bool pdl, cudaStream_t stream, int* ctas);                                   \
    cudaError_t NAME##_take_error(unsigned int* out);
MNB_SLICE_DECL(kv_attention_f16)
MNB_SLICE_DECL(kv_attention_bf16)
MNB_SLICE_DECL(kv_attention_f16_qf32)
MNB_SLICE_DECL(kv_attention_bf16_qf32)
#undef MNB_SLICE_DECL
#define MNB_SLICE_DECL(NAME)                                                                                    \
    cudaError_t NAME(const CUtensorMap& kmap, const CUtensorMap& vmap, const KvAttnArgs& a, int rows,           \
                     int sm_count, bool pdl, cudaStream_t stream, int* ctas);                                   \
    cudaError_t NAME##_take_error(unsigned int* out);
MNB_SLICE_DECL(kv_attention8_q16_64)
MNB_SLICE_DECL(kv_attention8_q16_96)
MNB_SLICE_DECL(kv_attention8_q16_128)
MNB_SLICE_DECL(kv_attention8_q16_256)
MNB_SLICE_DECL(kv_attention8_qf32_64)
MNB_SLICE_DECL(kv_attention8_qf32_96)
MNB_SLICE_DECL(kv_attention8_qf32_128)
MNB_SLICE_DECL(kv_attention8_qf32_256)
#undef MNB_SLICE_DECL

namespace {

// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over a split pair's parts in
// range order.  CTAs blockIdx.x of the grid join the pair that begins in CTA
// blockIdx.x of the main kernel: the four warps of a CTA share the parts of a row; of
// more rows than CTAs, in up to kFewParts parts, each warp joins rows by itself (40
// rows of drafts: 7 us of 85 less than with a CTA for each row; with one
// sequence's two rows in 13 parts it is the slower way, 8.9 us instead of 7.2).
// The parts come from L2 (2.5 MB in all with
// 8-row tiles); what it costs is the launch and two dependent loads (the record,
// then the first parts together with the statistics), so it is kept small: eight
// rows at a time in 256 threads took 2.4 us longer, 72 registers instead of 56 (seven CTAs per
// SM instead of nine) 3 us of 95 for drafts of 24 .. 40 rows.
constexpr int kFewParts = 16;
constexpr int kJoinGridY = 16;  // CTAs of a pair

// Writes columns d, d + 1 of a row (lane's share of it, `far` 2^-64 times as large) and the row's log-sum-exp.
__device__ __forceinline__ void join_store(const KvAttnArgs& a, int out_dtype, int flat, int head_kv, int d, float2 s,
                                           float m, float l, bool far) {
    const int tok = a.by_group(flat), head = head_kv * a.group + flat - tok * a.group;
    const int64_t token = tok;
    const float inv = (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) * (far ? 1.f / kKvFarDown : 1.f);  // NaN stays NaN
    if (d < a.cache.dim) {
        const int64_t at = token * a.out_stride + static_cast<int64_t>(head) * a.cache.dim + d;
        store_from_f32(a.out, out_dtype, at, s.x * inv);
        store_from_f32(a.out, out_dtype, at + 1, s.y * inv);
    }
    if (a.lse && d == 0)
        a.lse[token * (static_cast<int64_t>(a.cache.heads) * a.group) + head] =
            kv_log_sum(m, l, kv_weight_shift(a.cache.dtype));
}

// A part's weight.  Over 16-bit values never zero: a part with an infinite column adds that infinity
// however small its weight (2^-126 of anything finite changes nothing).  Codes have no
// infinities, and of their sums, as large as 2^119, it would change something.
__device__ __forceinline__ float part_weight(float reference, float largest, bool codes) {
    const float w = exp2f(reference - largest);
    return !codes && w < 1.17549435e-38f ? 1.17549435e-38f : w;  // (NaN stays NaN)
}

template <int DP>
__global__ void __launch_bounds__(128, DP == 128 ? 9 : 7) kv_join_kernel(const KvAttnArgs a, int rows_per_tile, int out_dtype) {
    constexpr int NV = DP / 64;    // float2 per lane
    constexpr int AHEAD = 8 / NV;  // parts of a warp asked for before their weights are known
    __shared__ float weight[kKvMaxCtas];
    __shared__ float red[2][4];
    __shared__ float2 sums[4][32 * NV];
    grid_dependency_wait();
    grid_launch_dependents();
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 j = a.join[c];
    if (j.x < 0) return;
    const int n = j.x - c + 1, rows = j.y >> 1, slot0 = 2 * c + (j.y & 1), head_kv = j.w;
    const bool codes = a.cache.dtype == MNB_E4M3;  // (a negative sum of weights: kKvFarDown)
    if (rows > kJoinGridY && n <= kFewParts) {
#pragma unroll 1
        for (int row = blockIdx.y * 4 + warp; row < rows; row += gridDim.y * 4) {
            auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? slot0 : 2 * (c + i)) * rows_per_tile + row; };
            const float2 ml = lane < n ? a.part_ml[slot(lane)] : make_float2(-INFINITY, 0.f);
            float2 acc[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) acc[v] = make_float2(0.f, 0.f);
            float m = ml.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            float w = lane < n ? part_weight(ml.x, m == -INFINITY ? 0.f : m, codes) : 0.f;
            const float l = warp_sum(w * fabsf(ml.y));
            const bool far = __any_sync(0xffffffffu, ml.y < 0.f);
            if (far && !(ml.y < 0.f)) w *= kKvFarDown;
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float2* o = reinterpret_cast<const float2*>(a.part_o + slot(i) * DP) + lane;
                const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const float2 x = o[v * 32];
                    acc[v].x = fmaf(wi, x.x, acc[v].x);
                    acc[v].y = fmaf(wi, x.y, acc[v].y);
                }
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) join_store(a, out_dtype, j.z + row, head_kv, (v * 32 + lane) * 2, acc[v], m, l, far);
        }
        return;
    }
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
        auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? slot0 : 2 * (c + i)) * rows_per_tile + row; };
        auto o_at = [&](int i) { return reinterpret_cast<const float2*>(a.part_o + slot(i) * DP) + lane; };
        float m = -INFINITY;
        float2 ml[3];
#pragma unroll
        for (int x = 0; x < 3; ++x) {  // kKvMaxCtas <= 3 * 128
            const int i = threadIdx.x + 128 * x;
            ml[x] = i < n ? a.part_ml[slot(i)] : make_float2(-INFINITY, 0.f);
        }
        float2 ahead[AHEAD][NV];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
#pragma unroll
            for (int v = 0; v < NV; ++v)
                ahead[k][v] = warp + 4 * k < n ? o_at(warp + 4 * k)[v * 32] : make_float2(0.f, 0.f);
#pragma unroll
        for (int x = 0; x < 3; ++x) m = fmaxf(m, ml[x].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) red[0][warp] = m;
        const bool far = __syncthreads_or(ml[0].y < 0.f || ml[1].y < 0.f || ml[2].y < 0.f);
        m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
        const float ref = m == -INFINITY ? 0.f : m;
        float l = 0.f;
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            const int i = threadIdx.x + 128 * x;
            if (i >= n) continue;
            const float w = part_weight(ml[x].x, ref, codes);
            weight[i] = far && !(ml[x].y < 0.f) ? w * kKvFarDown : w;
            l = fmaf(w, fabsf(ml[x].y), l);
        }
        l = warp_sum(l);
        if (lane == 0) red[1][warp] = l;
        __syncthreads();
        l = red[1][0] + red[1][1] + red[1][2] + red[1][3];
        float2 acc[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) acc[v] = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (warp + 4 * k >= n) break;
            const float w = weight[warp + 4 * k];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                acc[v].x = fmaf(w, ahead[k][v].x, acc[v].x);
                acc[v].y = fmaf(w, ahead[k][v].y, acc[v].y);
            }
        }
#pragma unroll 4
        for (int i = warp + 4 * AHEAD; i < n; i += 4) {
            const float w = weight[i];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const float2 x = o_at(i)[v * 32];
                acc[v].x = fmaf(w, x.x, acc[v].x);
                acc[v].y = fmaf(w, x.y, acc[v].y);
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) sums[warp][v * 32 + lane] = acc[v];
        __syncthreads();
        if (threadIdx.x < 32 * NV) {
            float2 s = sums[0][threadIdx.x];
#pragma unroll
            for (int x = 1; x < 4; ++x) {
                s.x += sums[x][threadIdx.x].x;
                s.y += sums[x][threadIdx.x].y;
            }
            join_store(a, out_dtype, j.z + row, head_kv, threadIdx.x * 2, s, m, l, far);
        }
        __syncthreads();
    }
}

cudaError_t encode_cache(CUtensorMap* map, void* base, const KvCache& c, int box_rows) {
    auto encode = encode_fn();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.num_pages)};
    const int es = c.dtype == MNB_E4M3 ? 1 : 2;
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.token_stride * es),
                                   static_cast<cuuint64_t>(c.head_stride * es),
                                   static_cast<cuuint64_t>(c.page_stride * es)};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box_rows), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    std::memset(map, 0, sizeof *map);
    const CUtensorMapDataType type = c.dtype == MNB_E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : c.dtype == kBF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUresult r = encode(map, type, 4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorNotSupported;
}

}  // namespace

int kv_attention_rows(int group, int64_t max_new) {
    const int64_t rows = group * max_new;
    return rows <= 8 ? 8 : rows <= 32 ? 32 : 64;
}

int kv_attention_pad(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

KvAttnSpace kv_attention_space(int rows, int pad) {
    auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    KvAttnSpace s;
    s.part_o = 0;
    s.part_ml = up(s.part_o + int64_t(2) * kKvMaxCtas * rows * pad * 4);
    s.join = up(s.part_ml + int64_t(2) * kKvMaxCtas * rows * 8);
    s.total = up(s.join + int64_t(kKvMaxCtas) * 16);
    return s;
}

cudaError_t kv_attention_take_error(unsigned int* out) {
    unsigned int first = 0;
    for (auto take : {kv_attention_f16_take_error, kv_attention_bf16_take_error, kv_attention_f16_qf32_take_error,
                      kv_attention_bf16_qf32_take_error, kv_attention8_q16_64_take_error,
                      kv_attention8_q16_128_take_error, kv_attention8_q16_256_take_error,
                      kv_attention8_qf32_64_take_error, kv_attention8_qf32_128_take_error,
                      kv_attention8_qf32_256_take_error, kv_attention8_q16_96_take_error,
                      kv_attention8_qf32_96_take_error}) {
        unsigned int v = 0;
        const cudaError_t e = take(&v);
        if (e != cudaSuccess) return e;
        if (first == 0) first = v;
    }
    *out = first;
    return cudaSuccess;
}

cudaError_t launch_kv_attention(const KvAttnArgs& in, int q_dtype, int64_t max_new, void* workspace, int sm_count,
                                bool pdl, cudaStream_t stream) {
    KvAttnArgs a = in;
    const int rows = kv_attention_rows(a.group, max_new), pad = kv_attention_pad(a.cache.dim);
    const KvAttnSpace sp = kv_attention_space(rows, pad);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.part_o = reinterpret_cast<float*>(ws + sp.part_o);
    a.part_ml = reinterpret_cast<float2*>(ws + sp.part_ml);
    a.join = reinterpret_cast<int4*>(ws + sp.join);
    a.by_group.set(static_cast<uint32_t>(a.group));
    a.by_page.set(static_cast<uint32_t>(a.cache.page_size));
    a.q_dtype = q_dtype;
    int power;
    a.scale_rest = std::frexp(a.scale, &power) * 2.f * 1.4426950408889634f;
    a.scale_unit = std::ldexp(1.f, power - 1);
    const bool codes = a.cache.dtype == MNB_E4M3;
    // a TMA box holds as many rows as divide a page (at least 8, at most a tile)
    a.box_rows = codes ? kv_tile8(rows, pad) : kKvTile;
    while (a.cache.page_size % a.box_rows) a.box_rows >>= 1;
    CUtensorMap kmap, vmap;
    cudaError_t e = encode_cache(&kmap, a.cache.k, a.cache, a.box_rows);
    if (e == cudaSuccess) e = encode_cache(&vmap, a.cache.v, a.cache, a.box_rows);
    if (e != cudaSuccess) return e;
    const bool bf = a.cache.dtype == kBF16, f32 = q_dtype == kF32;
    int ctas = 0;
    if (codes) {
        auto slice = pad == 64             ? (f32 ? kv_attention8_qf32_64 : kv_attention8_q16_64)
                     : a.cache.dim <= 96 ? (f32 ? kv_attention8_qf32_96 : kv_attention8_q16_96)
                     : pad == 128        ? (f32 ? kv_attention8_qf32_128 : kv_attention8_q16_128)
                                         : (f32 ? kv_attention8_qf32_256 : kv_attention8_q16_256);
        e = slice(kmap, vmap, a, rows, sm_count, pdl, stream, &ctas);
    } else {
        auto slice = bf ? (f32 ? kv_attention_bf16_qf32 : kv_attention_bf16) : (f32 ? kv_attention_f16_qf32 : kv_attention_f16);
        e = slice(kmap, vmap, a, rows, pad, sm_count, pdl, stream, &ctas);
    }
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(ctas),
                    static_cast<unsigned>(std::min<int64_t>(std::min<int64_t>(rows, a.group * max_new), kJoinGridY)));
    if (pad == 64) return launch_ready<kv_join_kernel<64>>(grid, dim3(128), 0, stream, pdl, a, rows, q_dtype);
    if (pad == 128) return launch_ready<kv_join_kernel<128>>(grid, dim3(128), 0, stream, pdl, a, rows, q_dtype);
    return launch_ready<kv_join_kernel<256>>(grid, dim3(128), 0, stream, pdl, a, rows, q_dtype);
}

}  // namespace mnb
