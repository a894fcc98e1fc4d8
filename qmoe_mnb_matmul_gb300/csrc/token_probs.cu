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
// of loads, block sums and one exchange for one sequence.  One cluster of CTAs per row: a
// thread goes over its part of the CTA's tokens with a running (largest, sum), the CTAs
// exchange theirs through distributed shared memory, and a second pass reads the logits
// again, from L2, and writes the probabilities.
//
// Few tokens of a vocabulary are listed (in the history, the drafts or the biases), and
// changing one costs as much as passing over a hundred others, so both passes leave them
// out: a bit for each of the CTA's tokens says so, like the mask's.  The listed ones
// stand in a dense array, in the order of the bits (token v's place is the number of bits
// before its own): each is read, changed and joined once, evenly over the threads, and its
// probability stored over what the second pass wrote.  Counts are whole numbers, of
// several biases of a token the largest number stays, and the array's order is that of the bits: no
// result depends on the order of the atomics.  (One word per token in the passes
// themselves, changed where a thread meets it: 165 us instead of 73 for 64 sequences of up
// to 6 rows.)  A warp takes 128 neighbouring tokens at a time and the next 128 belong
// to another CTA: a vocabulary's frequent tokens are neighbours.
//
// Measured (151936 entries): one sequence of 5 fp32 rows with 2000 tokens of history 9.8 us (one
// row without lists 6.1), 64 sequences of up to 6 bf16 rows with 3000 tokens, biases and
// masks, 208 MB: 73 us, 2.8 TB/s (all greedy 92, changed logits alone 102); 64 fp32 rows without lists, 78 MB:
// 23 us (greedy 28.5, logits 18).  A row has three phases with
// a barrier of its cluster between them, and two CTAs of 512 threads per SM do not
// cover each other's (issue 46 %, DRAM 32 %, 89 MB read for 67).  256 threads, 1024, and three or four
// CTAs per SM with fewer registers were slower, one kernel that keeps the row in registers too (245 us).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "kv.h"

namespace mnb {

namespace {

constexpr int kProbThreads = 512;
constexpr int kProbWarps = kProbThreads / 32;
constexpr int kProbCluster = 16;
// A listed token's word: bits 0 .. 19 its count, bit 20 whether the prompt holds it, from
// bit 21 on the number of its bias plus one.
constexpr uint32_t kInPrompt = 1u << 20, kCount = kInPrompt - 1;
constexpr int kBiasShift = 21;
static_assert(kProbMostHistory == kCount && kProbMostBiases == (1 << (32 - kBiasShift)) - 1, "the fields of a word");

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four logits as loaded.
template <typename T>
struct Raw {
    using V = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;
    V v;
    // -infinity for the values whose bit (of the low four) of `take` is 0: the product puts bit j on
    // top of byte j, and a byte permutation spreads a byte's top bit
    __device__ __forceinline__ void keep(uint32_t take) {
        constexpr uint32_t kNothing = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
        const uint32_t tops = (take & 0xFu) * 0x10204080u;
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int j = 0; j < static_cast<int>(sizeof(V) / 4); ++j) {
            uint32_t m;
            const uint32_t spread = sizeof(T) == 4 ? 0x8888u + 0x1111u * j : j == 0 ? 0x9988u : 0xBBAAu;
            asm("prmt.b32 %0, %1, 0, %2;" : "=r"(m) : "r"(tops), "r"(spread));
            w[j] = (w[j] & m) | (kNothing & ~m);
        }
    }
    __device__ __forceinline__ void widen(float (&x)[4]) const {
        alignas(16) T e[4];
        *reinterpret_cast<V*>(e) = v;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = to_f32(e[j]);
    }
};

template <int N>
struct Count {
    static constexpr int value = N;
};

// A running softmax: the largest value and the sum of 2^((value - largest) scale).  (One
// fused multiply-add by a reference in log2 units would do, but its rounding is 2^-24 of
// value * scale, which a low temperature makes as large as one likes.)
struct Soft {
    float top, sum;
};
__device__ __forceinline__ float reference(float top) { return top == -INFINITY ? 0.f : top; }
__device__ __forceinline__ float power(float x, float ref, float scale) { return exp2_fast((x - ref) * scale); }
// Of two values (packed fp32 instructions).
__device__ __forceinline__ float2 power2(float2 x, float2 minus_ref, float2 scale) {
    x = ffma2(x, make_float2(1.f, 1.f), minus_ref);
    x = ffma2(x, scale, make_float2(-0.f, -0.f));
    return make_float2(exp2_fast(x.x), exp2_fast(x.y));
}
// (Two products and a sum, not one fused: the same bits with a and b exchanged, so that after an
// exchange in pairs every lane and CTA of a row holds the same sum.)
__device__ __forceinline__ Soft join(const Soft& a, const Soft& b, float scale) {
    const float top = fmaxf(a.top, b.top), ref = reference(top);
    return {top, __fadd_rn(__fmul_rn(a.sum, power(a.top, ref, scale)), __fmul_rn(b.sum, power(b.top, ref, scale)))};
}
// A running argmax: the largest value and its first place; a NaN anywhere shows as place -1.
struct First {
    float top;
    int at;
};
__device__ __forceinline__ First join(const First& a, const First& b, float) {
    if (a.at < 0 || b.at < 0) return {fmaxf(a.top, b.top), -1};
    if (a.top == b.top) return {a.top, min(a.at, b.at)};
    return a.top > b.top ? a : b;
}

__device__ __forceinline__ Soft shuffle_xor(const Soft& v, int o) {
    return {__shfl_xor_sync(0xffffffffu, v.top, o), __shfl_xor_sync(0xffffffffu, v.sum, o)};
}
__device__ __forceinline__ First shuffle_xor(const First& v, int o) {
    return {__shfl_xor_sync(0xffffffffu, v.top, o), __shfl_xor_sync(0xffffffffu, v.at, o)};
}
__device__ __forceinline__ uint2 bits(const Soft& v) { return make_uint2(__float_as_uint(v.top), __float_as_uint(v.sum)); }
__device__ __forceinline__ uint2 bits(const First& v) { return make_uint2(__float_as_uint(v.top), static_cast<uint32_t>(v.at)); }
__device__ __forceinline__ void from_bits(uint2 x, Soft& v) { v = {__uint_as_float(x.x), __uint_as_float(x.y)}; }
__device__ __forceinline__ void from_bits(uint2 x, First& v) { v = {__uint_as_float(x.x), static_cast<int>(x.y)}; }

// The row's value from every thread's, in every thread: over the warp, the block (red),
// the cluster (stat).  Joined in a fixed order.  The caller waits for the cluster once
// more before it ends.
template <typename V>
__device__ __forceinline__ V whole_row(V v, float scale, uint2* red, uint2* stat, uint32_t ctas) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = join(v, shuffle_xor(v, o), scale);
    if (lane == 0) red[threadIdx.x >> 5] = bits(v);
    __syncthreads();
    from_bits(red[lane & (kProbWarps - 1)], v);
#pragma unroll
    for (int o = kProbWarps / 2; o > 0; o >>= 1) v = join(v, shuffle_xor(v, o), scale);
    if (ctas > 1) {
        if (threadIdx.x == 0) *stat = bits(v);
        cluster_arrive();
        cluster_wait();
        const uint64_t x = load_remote(reinterpret_cast<const uint64_t*>(stat), lane & (ctas - 1));
        cluster_arrive();
        from_bits(make_uint2(static_cast<uint32_t>(x), static_cast<uint32_t>(x >> 32)), v);
        for (int o = ctas >> 1; o > 0; o >>= 1) v = join(v, shuffle_xor(v, o), scale);
    }
    return v;
}

// VEC: rows may be read and written four values at a time.  FILTER: there is a mask or a list.
template <typename T, bool VEC, bool FILTER>
__global__ void __launch_bounds__(kProbThreads, 2) token_probs_kernel(const ProbArgs a, int items) {
    extern __shared__ __align__(16) uint32_t prob_smem[];
    __shared__ uint2 red[kProbWarps];
    __shared__ uint2 stat;
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int row = blockIdx.x / ctas, i = row % a.rows;
    const int64_t b = row / a.rows;
    const T* logits = static_cast<const T*>(a.logits);
    if (a.row_start) {
        const int64_t r0 = __ldg(a.row_start + b), r1 = __ldg(a.row_start + b + 1), r = r0 + i;  // (r passes 32 bits where r0 ends there)
        if (r >= r1) return;  // (the whole cluster, here and below)
        if (r0 < 0 || r >= a.tokens) {
            if (rank == 0 && tid == 0) record_error(MNB_ERR_CONTENT);
            return;
        }
        logits += r * a.logits_row;
    } else {
        logits += b * a.logits_seq + i * a.logits_row;
    }
    float* out = a.out + b * a.out_seq + i * a.out_row;
    const uint32_t* mask = a.mask ? a.mask + b * a.mask_seq + i * a.mask_row : nullptr;
    const int vocab = static_cast<int>(a.vocab);
    // The row's tokens in chunks of 128: chunk n belongs to CTA n % ctas, as its chunk n / ctas.
    // In group k warp w takes the CTA's chunk k kProbWarps + w; value j of a lane is token place(k, j).
    const int ctas_log = 31 - __clz(ctas);
    const int groups = cdiv(vocab, static_cast<int>(ctas) * kProbWarps * 128);
    auto chunk = [&](int k) { return (k * kProbWarps + warp) << ctas_log | static_cast<int>(rank); };
    auto place = [&](int k, int j) { return chunk(k) * 128 + (VEC ? lane * 4 + j : j * 32 + lane); };
    // (the row's logits on their way to L2 while the lists are read)
    for (int k = 0; k < groups; ++k) {
        const int at = chunk(k) * 128 + lane * static_cast<int>(128 / sizeof(T));
        if (lane < static_cast<int>(sizeof(T)) && at < vocab)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(logits + at));
    }

    const float temperature = a.temperature ? __ldg(a.temperature + b) : 1.f;
    const bool greedy = !(temperature > 0.f);

    // ---- the listed tokens among the CTA's
    const int bit_words = groups * kProbWarps * 4;
    uint32_t* listed = prob_smem;               // a bit per token of the CTA's
    uint32_t* before = listed + bit_words;      // bits in the words before (in the array's order)
    uint32_t* item_token = before + bit_words;
    uint32_t* item = item_token + items;        // its word, then the bits of its changed value
    int count = 0;                              // listed tokens of this CTA
    // the bit of a token of this CTA, -1 for another's or one outside the vocabulary
    auto bit_of = [&](int token) {
        const unsigned t = static_cast<unsigned>(token), n = t >> 7;
        return t < static_cast<unsigned>(vocab) && (n & (ctas - 1)) == rank ? static_cast<int>(n >> ctas_log << 7 | (t & 127u))
                                                                            : -1;
    };
    auto item_of = [&](int bit) { return before[bit >> 5] + __popc(listed[bit >> 5] & ((1u << (bit & 31)) - 1u)); };
    if (items > 0) {
        const int* past = a.history + b * a.history_stride;
        const int len = a.history ? min(max(__ldg(a.history_lens + b), 0), a.history_columns) : 0;
        const int prompt = a.prompt_lens ? __ldg(a.prompt_lens + b) : 0;
        const int drafts = a.draft_tokens ? i : 0;
        const int* draft = a.draft_tokens + b * (a.rows - 1);
        const int* bias_tokens = a.bias_tokens + b * a.bias_stride;
        for (int w = tid; w < bit_words; w += kProbThreads) listed[w] = 0u;
        __syncthreads();
        auto mark = [&](int token) {
            const int bit = bit_of(token);
            if (bit >= 0) atomicOr(listed + (bit >> 5), 1u << (bit & 31));
        };
        constexpr int kKept = 8;  // of the history, between its two passes
        int kept[kKept];
#pragma unroll
        for (int k = 0; k < kKept; ++k) {
            const int j = tid + k * kProbThreads;
            kept[k] = j < len ? __ldg(past + j) : -1;
        }
#pragma unroll
        for (int k = 0; k < kKept; ++k) mark(kept[k]);
#pragma unroll 4
        for (int j = tid + kKept * kProbThreads; j < len; j += kProbThreads) mark(__ldg(past + j));
        for (int j = tid; j < drafts; j += kProbThreads) mark(__ldg(draft + j));
        for (int e = tid; e < a.biases; e += kProbThreads) mark(__ldg(bias_tokens + e));
        __syncthreads();
        // a thread's words are kProbThreads apart: neighbours, of which many bits are set, are spread
        int mine = 0;
        for (int w = tid; w < bit_words; w += kProbThreads) mine += __popc(listed[w]);
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 31) red[warp].x = upto;
        __syncthreads();
        int first = upto - mine;
#pragma unroll
        for (int w = 0; w < kProbWarps; ++w) {
            const int n = red[w].x;
            if (w < warp) first += n;
            count += n;
        }
        for (int w = tid; w < bit_words; w += kProbThreads) {
            before[w] = first;
            const int token = ((w >> 2) << ctas_log | static_cast<int>(rank)) * 128 + (w & 3) * 32;
            for (uint32_t bits = listed[w]; bits; bits &= bits - 1) {
                item_token[first] = token + __ffs(bits) - 1;
                item[first++] = 0u;
            }
        }
        __syncthreads();
        if (a.biases > 0) {
            for (int e = tid; e < a.biases; e += kProbThreads) {
                const int bit = bit_of(__ldg(bias_tokens + e));
                if (bit >= 0) atomicMax(item + item_of(bit), static_cast<uint32_t>(e + 1) << kBiasShift);
            }
            __syncthreads();
        }
        auto tally = [&](int token, bool said) {
            const int bit = bit_of(token);
            if (bit < 0) return;
            if (said)
                atomicAdd(item + item_of(bit), 1u);
            else
                atomicOr(item + item_of(bit), kInPrompt);
        };
#pragma unroll
        for (int k = 0; k < kKept; ++k) tally(kept[k], tid + k * kProbThreads >= prompt);
#pragma unroll 4
        for (int j = tid + kKept * kProbThreads; j < len; j += kProbThreads) tally(__ldg(past + j), j >= prompt);
        for (int j = tid; j < drafts; j += kProbThreads) tally(__ldg(draft + j), true);
        __syncthreads();
        const float* bias = a.bias_values + b * a.bias_stride;
        const float repetition = a.repetition ? __ldg(a.repetition + b) : 1.f;
        const float frequency = a.frequency ? __ldg(a.frequency + b) : 0.f;
        const float presence = a.presence ? __ldg(a.presence + b) : 0.f;
#pragma unroll 2
        for (int n = tid; n < count; n += kProbThreads) {
            const int token = item_token[n];
            const uint32_t w = item[n];
            float x = to_f32(logits[token]);
            if (w & (kInPrompt | kCount)) {
                const float said = static_cast<float>(w & kCount);
                x = x > 0.f ? __fdiv_rn(x, repetition) : __fmul_rn(x, repetition);
                x = __fsub_rn(x, __fmul_rn(frequency, said));
                if (said > 0.f) x = __fsub_rn(x, presence);
            }
            if (w >> kBiasShift) x = __fadd_rn(x, __ldg(bias + (w >> kBiasShift) - 1));
            if (mask && !(__ldg(mask + (token >> 5)) >> (token & 31) & 1u)) x = -INFINITY;
            item[n] = __float_as_uint(x);  // read by this thread alone
        }
    }

    if (FILTER) {
        // the bits of the tokens that are the passes' own: allowed, and not listed
        for (int w = tid; w < bit_words; w += kProbThreads) {
            const int at = ((w >> 2) << ctas_log | static_cast<int>(rank)) * 4 + (w & 3);  // of the row's words
            uint32_t own = mask == nullptr ? ~0u : at * 32 < vocab ? __ldg(mask + at) : 0u;
            if (items > 0) own &= ~listed[w];
            listed[w] = own;
        }
        __syncthreads();
    }

    // ---- the other tokens: x[j] = -inf where the value is not the passes' own.  The first `full` groups of a warp lie within the vocabulary, `last` is its part of the
    // chunk that the vocabulary ends in.
    const int whole = vocab >> 7, step = kProbWarps << ctas_log;
    const int full = whole > chunk(0) ? (whole - chunk(0) - 1) / step + 1 : 0;
    const bool last = (vocab & 127) != 0 && chunk(full) == whole;
    const int offset = VEC ? lane * 4 : lane;
    const T* const from = logits + static_cast<int64_t>(chunk(0)) * 128 + offset;
    float* const to = out + static_cast<int64_t>(chunk(0)) * 128 + offset;
    const int64_t stride = static_cast<int64_t>(step) * 128;
    // bits of the four values that are the passes' own
    auto own_values = [&](int k) {
        const uint32_t* words = listed + (k * kProbWarps + warp) * 4;
        if (VEC) return words[lane >> 3] >> (lane * 4 & 31);
        uint32_t take = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) take |= (words[j] >> lane & 1u) << j;
        return take;
    };
    // all groups of this warp: each(x of the groups), N groups loaded at a time; `write`: what
    // it leaves in x is stored (with the listed tokens' places, which get theirs later)
    auto pass = [&](auto count_at_once, bool write, auto each) {
        constexpr int N = decltype(count_at_once)::value;
        auto some = [&](int k0, auto count_here) {
            constexpr int M = decltype(count_here)::value;
            Raw<T> raw[M];
            float x[M][4];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const T* p = from + (k0 + m) * stride;
                if (VEC) {
                    raw[m].v = *reinterpret_cast<const typename Raw<T>::V*>(p);
                } else {
                    T* e = reinterpret_cast<T*>(&raw[m].v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[j] = p[j * 32];
                }
            }
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (FILTER) raw[m].keep(own_values(k0 + m));
                raw[m].widen(x[m]);
            }
            each(k0, x);
            if (write)
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    float* p = to + (k0 + m) * stride;
                    if (VEC) {
                        *reinterpret_cast<float4*>(p) = make_float4(x[m][0], x[m][1], x[m][2], x[m][3]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) p[j * 32] = x[m][j];
                    }
                }
        };
        int k = 0;
#pragma unroll 1
        for (; k + N <= full; k += N) some(k, Count<N>{});
#pragma unroll 1
        for (; k < full; ++k) some(k, Count<1>{});
        if (last) {
            float x[1][4];
            const uint32_t take = FILTER ? own_values(full) : 0xFu;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[0][j] = place(full, j) < vocab && (take >> j & 1u) ? to_f32(logits[place(full, j)]) : -INFINITY;
            each(full, x);
            if (write)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (place(full, j) < vocab) out[place(full, j)] = x[0][j];
        }
    };
    // the listed tokens' results over what the pass stored in their places
    auto store_items = [&](auto result) {
        if (items == 0) return;
        __syncthreads();
        for (int n = tid; n < count; n += kProbThreads) out[item_token[n]] = result(__uint_as_float(item[n]));
    };

    if (!a.softmax) {
        if (items > 0) __syncthreads();  // out may be the logits, and the listed ones are read
        auto cooled = [&](float x) { return greedy ? x : __fdiv_rn(x, temperature); };
        pass(Count<2>{}, true, [&](int, auto& x) {
            for (auto& group : x)
                for (float& v : group) v = cooled(v);
        });
        store_items(cooled);
        return;
    }
    if (!greedy) {
        // values to log2 units; finite and not zero, so that neither 0 times it nor -inf times it is
        // NaN (subnormal for temperatures from 1.3e38 on, 2^-149 for an infinite one)
        const float scale = fminf(fmaxf(1.4426950408889634f / temperature, __uint_as_float(1u)), 3.402823466e38f);
        Soft mine = {-INFINITY, 0.f};
        pass(Count<4>{}, false, [&](int, auto& x) {
            float top = mine.top;
            for (auto& group : x)
                for (float& v : group) top = fmaxf(top, v);
            const float ref = reference(top);
            if (top > mine.top) {
                mine.sum *= power(mine.top, ref, scale);
                mine.top = top;
            }
            float2 sum = make_float2(0.f, 0.f);
            const float2 minus_ref = make_float2(-ref, -ref), scale2 = make_float2(scale, scale);
            for (auto& group : x)
#pragma unroll
                for (int j = 0; j < 4; j += 2)
                    sum = ffma2(power2(make_float2(group[j], group[j + 1]), minus_ref, scale2), make_float2(1.f, 1.f), sum);
            mine.sum += sum.x + sum.y;
        });
        for (int n = tid; n < count; n += kProbThreads) {
            const float x = __uint_as_float(item[n]);
            mine = join(mine, Soft{x, power(x, reference(x), scale)}, scale);
        }
        const Soft all = whole_row(mine, scale, red, &stat, ctas);
        // a row that the masks leave empty gets zeros; NaN stays NaN
        const float part = all.sum == 0.f ? 0.f : 1.f / all.sum, ref = reference(all.top);
        auto share = [&](float x) { return power(x, ref, scale) * part; };
        const float2 minus_ref = make_float2(-ref, -ref), scale2 = make_float2(scale, scale), part2 = make_float2(part, part);
        pass(Count<4>{}, true, [&](int, auto& x) {
            for (auto& group : x)
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const float2 p = ffma2(power2(make_float2(group[j], group[j + 1]), minus_ref, scale2), part2,
                                           make_float2(-0.f, -0.f));
                    group[j] = p.x;
                    group[j + 1] = p.y;
                }
        });
        store_items(share);
    } else {
        First mine = {-INFINITY, 0x7fffffff};
        auto look = [&](float x, int at) {
            if (x != x)
                mine.at = -1;
            else if (mine.at >= 0 && (x > mine.top || (x == mine.top && x > -INFINITY && at < mine.at)))
                mine = {x, at};
        };
        pass(Count<1>{}, false, [&](int k, auto& x) {
            for (int j = 0; j < 4; ++j) look(x[0][j], place(k, j));
        });
        for (int n = tid; n < count; n += kProbThreads) look(__uint_as_float(item[n]), item_token[n]);
        const First all = whole_row(mine, 0.f, red, &stat, ctas);
        pass(Count<1>{}, true, [&](int k, auto& x) {
            for (int j = 0; j < 4; ++j)
                x[0][j] = all.at < 0 ? __uint_as_float(0x7fffffffu) : place(k, j) == all.at ? 1.f : 0.f;
        });
    }
    if (ctas > 1) cluster_wait();
}

// Listed tokens that a CTA may have, and the bytes of its bits and lists (of the bits alone, for a mask).
struct ProbPlan {
    int64_t items, bytes;
};
ProbPlan plan_probs(int64_t vocab, int64_t listed, int cluster) {
    const int64_t tokens = cdiv<int64_t>(vocab, int64_t(cluster) * kProbWarps * 128) * kProbWarps * 128;
    const int64_t items = std::min(listed, tokens);
    return {items, tokens / 32 * (listed > 0 ? 8 : 4) + items * 8};
}

template <typename T, bool VEC>
cudaError_t launch_filter(const ProbArgs& a, dim3 grid, unsigned cluster, size_t smem, int items, bool pdl, cudaStream_t stream) {
    if (items > 0 || a.mask)
        return launch_cluster<token_probs_kernel<T, VEC, true>>(grid, dim3(kProbThreads), cluster, smem, kProbMostSmem, stream,
                                                                pdl, a, items);
    return launch_cluster<token_probs_kernel<T, VEC, false>>(grid, dim3(kProbThreads), cluster, smem, kProbMostSmem, stream, pdl,
                                                             a, items);
}

template <typename T>
cudaError_t launch_type(const ProbArgs& a, bool vec, dim3 grid, unsigned cluster, size_t smem, int items, bool pdl,
                        cudaStream_t stream) {
    return vec ? launch_filter<T, true>(a, grid, cluster, smem, items, pdl, stream)
               : launch_filter<T, false>(a, grid, cluster, smem, items, pdl, stream);
}

}  // namespace

bool token_probs_fits(int64_t vocab, int64_t listed) {
    return plan_probs(vocab, listed, kProbCluster).bytes <= kProbMostSmem;
}

cudaError_t launch_token_probs(const ProbArgs& a, int dtype, int sm_count, bool pdl, cudaStream_t stream) {
    const size_t es = dtype == kF32 ? 4 : 2;
    const bool vec = reinterpret_cast<uintptr_t>(a.logits) % (4 * es) == 0 && a.logits_row % 4 == 0 &&
                     (a.row_start || a.logits_seq % 4 == 0) && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
                     a.out_seq % 4 == 0 && a.out_row % 4 == 0;
    const int64_t listed = (a.history ? a.history_columns : 0) + (a.draft_tokens ? a.rows - 1 : 0) + a.biases;
    // CTAs per row: up to about three per SM in all, so that one's loads cover another's exchange (222
    // rows of 151936 entries with lists, measured side by side: 70 us in twos, 86 in fours, 113 in eights; 5 rows
    // 9.6 in sixteens, 11.3 in eights); no more than there are tokens for, and
    // more where the lists would not leave room for two on an SM
    const int64_t rows = a.row_start ? std::min(a.batch * a.rows, a.tokens) : a.batch * a.rows;
    int cluster = kProbCluster;
    while (cluster > 1 && rows * cluster * 5 > int64_t(sm_count) * 17) cluster >>= 1;
    while (cluster > 1 && int64_t(cluster >> 1) * kProbThreads * 4 >= a.vocab) cluster >>= 1;
    while (cluster < kProbCluster && plan_probs(a.vocab, listed, cluster).bytes > kProbMostSmem / 2) cluster <<= 1;
    const ProbPlan plan = plan_probs(a.vocab, listed, cluster);
    const dim3 grid(static_cast<unsigned>(a.batch * a.rows * cluster));
    const size_t smem = listed > 0 || a.mask ? static_cast<size_t>(plan.bytes) : 0;
    const int items = static_cast<int>(plan.items);
    if (dtype == kF32) return launch_type<float>(a, vec, grid, cluster, smem, items, pdl, stream);
    if (dtype == kF16) return launch_type<__half>(a, vec, grid, cluster, smem, items, pdl, stream);
    return launch_type<__nv_bfloat16>(a, vec, grid, cluster, smem, items, pdl, stream);
}

cudaError_t token_probs_take_error(unsigned int* out) { return take_unit_error(out); }

}  // namespace mnb
