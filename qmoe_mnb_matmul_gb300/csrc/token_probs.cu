// token_probs.cu -- a step's logits to the probabilities that the next tokens are drawn
// from: penalties for repeated tokens, biases, grammar masks, temperature, softmax.
//
// For row i of sequence b and token v, in fp32 with one rounding for each operation:
//   x = logit;  where v has occurred: x = x > 0 ? x / repetition : x * repetition
//   x = x - frequency * count;  where count > 0: x = x - presence
//   x = x + bias;  where the mask forbids v: x = -inf
//   p = e^((x - m) / T) / sum e^((x - m) / T), m the row's largest x; T = 0: 1 for the first largest x
// A token has occurred in the prompt, in what was generated, or among the drafts ahead of
// the row; its count leaves the prompt out.
//
// Bound: HBM for a batch (each logit read once, each probability written once), the chain
// of loads, two block sums and one exchange for one sequence.  One cluster of CTAs per
// row: a CTA holds its run of the row in registers (20 values a thread; what a vocabulary
// over 163840 leaves is read again, from L2) between the largest value, the sum, and the
// store, and the CTAs exchange (largest, sum) through distributed shared memory.  Counts
// and biases of the run's tokens are arrays in shared memory that every CTA fills from
// the lists by itself; a count is a whole number, so the order of the additions does not
// matter, and of several biases of one token the last one in the list counts.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv.h"

namespace mnb {

namespace {

constexpr int kProbThreads = 512;
constexpr int kProbWarps = kProbThreads / 32;
constexpr int kProbGroups = 5;  // groups of four values that a thread keeps
constexpr int kProbCluster = 16;
constexpr uint32_t kInPrompt = 0x80000000u;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T> struct Four;
template <> struct Four<float> {
    using V = float4;
};
template <> struct Four<__half> {
    using V = uint2;
};
template <> struct Four<__nv_bfloat16> {
    using V = uint2;
};

// Largest of the block's values; `red` is free again after the next barrier.
__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[threadIdx.x & (kProbWarps - 1)];
#pragma unroll
    for (int o = kProbWarps / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[threadIdx.x & (kProbWarps - 1)];
#pragma unroll
    for (int o = kProbWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ int block_min(int v, int* red) {
    v = __reduce_min_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_min_sync(0xffffffffu, red[threadIdx.x & (kProbWarps - 1)]);
}

// VEC: rows may be read and written four values at a time.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kProbThreads, 2) token_probs_kernel(const ProbArgs a) {
    extern __shared__ __align__(16) uint32_t prob_smem[];
    __shared__ float red[2][kProbWarps];
    __shared__ int first_red[kProbWarps];
    __shared__ uint2 stat;  // largest value, and the sum or the first place of the largest
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int row = blockIdx.x / ctas, i = row % a.rows;
    const int64_t b = row / a.rows;
    const T* logits = static_cast<const T*>(a.logits);
    if (a.row_start) {
        const int r0 = __ldg(a.row_start + b), r1 = __ldg(a.row_start + b + 1), r = r0 + i;
        if (r0 < 0 || r >= r1 || r >= a.tokens) return;  // (the whole cluster)
        logits += r * a.logits_row;
    } else {
        logits += b * a.logits_seq + i * a.logits_row;
    }
    float* out = a.out + b * a.out_seq + i * a.out_row;
    const uint32_t* mask = a.mask ? a.mask + b * a.mask_seq + i * a.mask_row : nullptr;
    const int vocab = static_cast<int>(a.vocab);
    const int run = cdiv(cdiv(vocab, static_cast<int>(ctas)), 128) * 128;
    const int lo = min(static_cast<int>(rank) * run, vocab), hi = min(lo + run, vocab), size = hi - lo;

    // ---- the run's counts and biases
    uint32_t* counts = a.history || a.draft_tokens ? prob_smem : nullptr;
    float* bias = a.biases > 0 ? reinterpret_cast<float*>(prob_smem + (counts ? run : 0)) : nullptr;
    if (counts || bias) {
        const int words = run * ((counts ? 1 : 0) + (bias ? 1 : 0));
        for (int w = tid * 4; w < words; w += kProbThreads * 4)
            *reinterpret_cast<uint4*>(prob_smem + w) = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        if (a.history) {
            const int* past = a.history + b * a.history_stride;
            const int len = min(max(__ldg(a.history_lens + b), 0), a.history_columns);
            const int prompt = a.prompt_lens ? __ldg(a.prompt_lens + b) : 0;
#pragma unroll 4
            for (int j = tid; j < len; j += kProbThreads) {
                const unsigned at = static_cast<unsigned>(__ldg(past + j)) - lo;
                if (at >= static_cast<unsigned>(size)) continue;
                if (j < prompt)
                    atomicOr(counts + at, kInPrompt);
                else
                    atomicAdd(counts + at, 1u);
            }
        }
        if (a.draft_tokens)
            for (int j = tid; j < i; j += kProbThreads) {
                const unsigned at = static_cast<unsigned>(__ldg(a.draft_tokens + b * (a.rows - 1) + j)) - lo;
                if (at < static_cast<unsigned>(size)) atomicAdd(counts + at, 1u);
            }
        if (bias) {
            const int* tokens = a.bias_tokens + b * a.bias_stride;
            for (int e = tid; e < a.biases; e += kProbThreads) {
                const int token = __ldg(tokens + e);
                const unsigned at = static_cast<unsigned>(token) - lo;
                if (at >= static_cast<unsigned>(size)) continue;
                bool last = true;
                for (int f = e + 1; f < a.biases && last; ++f) last = __ldg(tokens + f) != token;
                if (last) bias[at] = __ldg(a.bias_values + b * a.bias_stride + e);
            }
        }
        __syncthreads();
    }
    const float repetition = a.repetition ? __ldg(a.repetition + b) : 1.f;
    const float frequency = a.frequency ? __ldg(a.frequency + b) : 0.f;
    const float presence = a.presence ? __ldg(a.presence + b) : 0.f;
    const float temperature = a.temperature ? __ldg(a.temperature + b) : 1.f;
    const bool greedy = !(temperature > 0.f);

    // ---- the row's values.  Value j of group k is token place(k, j).
    const int groups = cdiv(run, kProbThreads * 4);
    auto place = [&](int k, int j) {
        return VEC ? lo + (k * kProbThreads + tid) * 4 + j : lo + (k * 4 + j) * kProbThreads + tid;
    };
    auto read = [&](int k, float (&x)[4]) {
        if (VEC) {
            const int at = place(k, 0);
            if (at + 4 <= hi) {
                using V = typename Four<T>::V;
                alignas(16) T raw[4];
                *reinterpret_cast<V*>(raw) = *reinterpret_cast<const V*>(logits + at);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = to_f32(raw[j]);
                return;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = place(k, j) < hi ? to_f32(logits[place(k, j)]) : -INFINITY;
    };
    auto penalise = [&](uint32_t c, float& x) {
        if (c == 0) return;
        const float n = static_cast<float>(c & ~kInPrompt);
        x = x > 0.f ? __fdiv_rn(x, repetition) : __fmul_rn(x, repetition);
        x = __fsub_rn(x, __fmul_rn(frequency, n));
        if (n > 0.f) x = __fsub_rn(x, presence);
    };
    auto treat = [&](int k, float (&x)[4]) {
        if (VEC) {
            const int at = place(k, 0);
            if (at >= hi) return;
            if (counts) {
                const uint4 c = *reinterpret_cast<const uint4*>(counts + at - lo);
                if (c.x | c.y | c.z | c.w) {
                    penalise(c.x, x[0]);
                    penalise(c.y, x[1]);
                    penalise(c.z, x[2]);
                    penalise(c.w, x[3]);
                }
            }
            if (bias) {
                const float4 add = *reinterpret_cast<const float4*>(bias + at - lo);
                x[0] += add.x;
                x[1] += add.y;
                x[2] += add.z;
                x[3] += add.w;
            }
            if (mask) {
                const uint32_t bits = __ldg(mask + (at >> 5)) >> (at & 31);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (!(bits >> j & 1u)) x[j] = -INFINITY;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = place(k, j);
                if (at >= hi) continue;
                if (counts) penalise(counts[at - lo], x[j]);
                if (bias) x[j] += bias[at - lo];
                if (mask && !(__ldg(mask + (at >> 5)) >> (at & 31) & 1u)) x[j] = -INFINITY;
            }
        }
    };
    auto store = [&](int k, const float (&x)[4]) {
        if (VEC && place(k, 0) + 4 <= hi) {
            *reinterpret_cast<float4*>(out + place(k, 0)) = make_float4(x[0], x[1], x[2], x[3]);
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (place(k, j) < hi) out[place(k, j)] = x[j];
    };

    if (!a.softmax) {
        for (int k = 0; k < groups; ++k) {
            float x[4];
            read(k, x);
            treat(k, x);
            if (!greedy)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = __fdiv_rn(x[j], temperature);
            store(k, x);
        }
        return;
    }

    float x[kProbGroups][4];
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kProbGroups; ++k) {
        if (k < groups)
            read(k, x[k]);
        else
#pragma unroll
            for (int j = 0; j < 4; ++j) x[k][j] = -INFINITY;
    }
#pragma unroll
    for (int k = 0; k < kProbGroups; ++k) {
        if (k < groups) treat(k, x[k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, x[k][j]);
    }
    for (int k = kProbGroups; k < groups; ++k) {
        float y[4];
        read(k, y);
        treat(k, y);
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, y[j]);
    }
    top = block_max(top, red[0]);
    // values to log2 units; finite and not zero, so that neither 0 times it nor -inf times it is NaN
    const float scale = fminf(fmaxf(1.4426950408889634f / temperature, 1.17549435e-38f), 3.402823466e38f);
    const float ref = top == -INFINITY ? 0.f : top;
    uint32_t second;
    if (!greedy) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kProbGroups; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[k][j] = exp2_fast((x[k][j] - ref) * scale);
                sum += x[k][j];
            }
        for (int k = kProbGroups; k < groups; ++k) {
            float y[4];
            read(k, y);
            treat(k, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += exp2_fast((y[j] - ref) * scale);
        }
        second = __float_as_uint(block_sum(sum, red[1]));
    } else {
        // the first place of the largest value; a NaN anywhere shows as place -1
        int at = 0x7fffffff;
        auto look = [&](int k, const float (&y)[4]) {
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                if (place(k, j) >= hi) continue;
                if (y[j] == top && top > -INFINITY) at = min(at, place(k, j));
                if (y[j] != y[j]) at = -1;
            }
        };
#pragma unroll
        for (int k = 0; k < kProbGroups; ++k)
            if (k < groups) look(k, x[k]);
        for (int k = kProbGroups; k < groups; ++k) {
            float y[4];
            read(k, y);
            treat(k, y);
            look(k, y);
        }
        second = static_cast<uint32_t>(block_min(at, first_red));
    }
    // ---- the whole row's
    if (ctas > 1) {
        if (tid == 0) stat = make_uint2(__float_as_uint(top), second);
        cluster_arrive();
        cluster_wait();
    }
    float m = top;
    uint2 theirs = make_uint2(__float_as_uint(top), second);
    if (ctas > 1) {
        const bool in = lane < static_cast<int>(ctas);
        const uint64_t v = load_remote(reinterpret_cast<const uint64_t*>(&stat), in ? lane : 0);
        theirs = make_uint2(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32));
        cluster_arrive();  // waited for before the CTA ends
        m = in ? __uint_as_float(theirs.x) : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (!in) theirs = make_uint2(__float_as_uint(-INFINITY), greedy ? 0x7fffffffu : 0u);
    }
    if (!greedy) {
        const float base = m == -INFINITY ? 0.f : m;
        float total = __uint_as_float(second);
        if (ctas > 1) {
            const float t = __uint_as_float(theirs.x);
            total = warp_sum(__uint_as_float(theirs.y) * exp2_fast((t - base) * scale));
        }
        // a row that the masks leave empty gets zeros; NaN stays NaN
        const float part = total == 0.f ? 0.f : exp2_fast((ref - base) * scale) / total;
#pragma unroll
        for (int k = 0; k < kProbGroups; ++k) {
            if (k >= groups) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[k][j] *= part;
            store(k, x[k]);
        }
        for (int k = kProbGroups; k < groups; ++k) {
            float y[4];
            read(k, y);
            treat(k, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = exp2_fast((y[j] - ref) * scale) * part;
            store(k, y);
        }
    } else {
        int at = static_cast<int>(second);
        if (ctas > 1) {
            // (a CTA without the largest value has nothing to say but a NaN)
            const int place = static_cast<int>(theirs.y);
            at = __reduce_min_sync(0xffffffffu, __uint_as_float(theirs.x) == m || place < 0 ? place : 0x7fffffff);
        }
        for (int k = 0; k < groups; ++k) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = at < 0 ? __uint_as_float(0x7fffffffu) : place(k, j) == at ? 1.f : 0.f;
            store(k, y);
        }
    }
    if (ctas > 1) cluster_wait();
}

template <typename T>
cudaError_t launch_type(const ProbArgs& a, bool vec, dim3 grid, unsigned cluster, size_t smem, bool pdl, cudaStream_t stream) {
    if (vec)
        return launch_cluster<token_probs_kernel<T, true>>(grid, dim3(kProbThreads), cluster, smem, kProbMostSmem, stream, pdl, a);
    return launch_cluster<token_probs_kernel<T, false>>(grid, dim3(kProbThreads), cluster, smem, kProbMostSmem, stream, pdl, a);
}

}  // namespace

int64_t token_probs_smem(int64_t vocab, bool counts, bool biases, int cluster) {
    const int64_t run = cdiv<int64_t>(cdiv<int64_t>(vocab, cluster), 128) * 128;
    return run * 4 * ((counts ? 1 : 0) + (biases ? 1 : 0));
}

cudaError_t launch_token_probs(const ProbArgs& a, int dtype, bool pdl, cudaStream_t stream) {
    const size_t es = dtype == kF32 ? 4 : 2;
    const bool vec = reinterpret_cast<uintptr_t>(a.logits) % (4 * es) == 0 && a.logits_row % 4 == 0 &&
                     (a.row_start || a.logits_seq % 4 == 0) && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
                     a.out_seq % 4 == 0 && a.out_row % 4 == 0;
    // CTAs per row: as many as have a group of four for every thread
    int cluster = 1;
    while (cluster < kProbCluster && int64_t(cluster) * kProbThreads * 4 < a.vocab) cluster *= 2;
    const size_t smem = static_cast<size_t>(token_probs_smem(a.vocab, a.history || a.draft_tokens, a.biases > 0, cluster));
    const dim3 grid(static_cast<unsigned>(a.batch * a.rows * cluster));
    if (dtype == kF32) return launch_type<float>(a, vec, grid, cluster, smem, pdl, stream);
    if (dtype == kF16) return launch_type<__half>(a, vec, grid, cluster, smem, pdl, stream);
    return launch_type<__nv_bfloat16>(a, vec, grid, cluster, smem, pdl, stream);
}

cudaError_t token_probs_take_error(unsigned int* out) { return take_unit_error(out); }

}  // namespace mnb
