// draft.cu -- verification of drafted tokens against the target's
// probabilities, from given uniform numbers.
//
// Draft i of a sequence stands while u_i q_i(x_i) < p_i(x_i) (fp32 product; a
// draft without probabilities has q_i(x_i) = 1).  At the first one that falls, r,
// the next token is drawn from the weights max(p_r - q_r, 0) (without
// probabilities: p_r with x_r left out), after the last from p_n itself.
//
// The draw.  Weights become whole numbers, floor(2^40 min(max(., 0), 1)), of
// which fewer than 2^22 add up below 2^62: whole-number sums do not depend on
// their order, so the drawn token is the same however the vocabulary is split,
// and the same as a plain left-to-right sum gives.  What 2^-40 cuts off is at most
// vocab * 2^-40 of the mass (1.4e-7 at 151936 entries, as fine as fp32 rounding).
// The token is the smallest i with w_0 + .. + w_i > floor(U total / 2^24), U =
// floor(2^24 u), and is found exactly.
//
// Work.  One cluster of CTAs per sequence; every warp finds the accepted count
// for itself (a few gathers), then sums the weights of its own run of the
// vocabulary: one pass over the one or two rows that matter, bound by HBM for a
// batch and by the chain of gather, pass, exchange and search for one sequence.
// The warps' totals are exchanged through distributed shared memory, and the one
// warp whose run holds the drawn point reads half of it again, from L2.
//
// Measured (151936 entries): one sequence of four drafts 7.4 us, 64 sequences of up to
// five 22 us (78 MB; 7 us of the chain, then 5.2 TB/s).  256 threads and at most 64
// registers, because a cluster's CTAs must fit one group of SMs together: with 512
// threads at 128 registers clusters ran eight at a time and 64 sequences took 52 us.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv.h"

namespace mnb {

namespace {

constexpr int kDraftThreads = 256;
constexpr int kDraftWarps = kDraftThreads / 32;
constexpr int kMaxCluster = 16;

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The row whose weights are drawn from: max(p - q, 0) in units of 2^-40, q null
// for p itself, entry `skip` left out (-1: none).
struct Weights {
    const float* p;
    const float* q;
    int skip;
};

// floor(2^40 w) of w = min(max(x, 0), 1) (fmaxf drops a NaN), in two parts of 20 bits:
// adding 8 to w with rounding toward zero leaves floor(2^20 w) in the sum's low
// bits, and adding 2^-17 to what that cut off leaves the next 20 bits likewise.  Both
// parts still carry the bits of the number added (kHi, kLo), taken off once per sum.
// (The conversion to 64-bit integers runs at a small fraction of the rate of these
// adds: with it the 64-sequence case took 37 us.)
constexpr uint32_t kHi = 0x41000000u, kLo = 0x37000000u;  // 8.0f, 2^-17
__device__ __forceinline__ void weigh(float x, uint32_t& hi, uint32_t& lo) {
    const float w = fminf(fmaxf(x, 0.f), 1.f);
    const float h = __fadd_rz(w, 8.f);
    hi = __float_as_uint(h);
    lo = __float_as_uint(__fadd_rz(w - (h - 8.f), 7.62939453125e-6f));
}
// The sum of n weights from the sums of their parts (modulo 2^32: parts are below 2^20 + 1, n is at most 4).
__device__ __forceinline__ uint64_t join(uint32_t hi, uint32_t lo, uint32_t n) {
    return (static_cast<uint64_t>(hi - n * kHi) << 20) + (lo - n * kLo);
}

// p - q of entries i .. i + 3 (zero from `end` on), i a multiple of four; VEC: both
// rows may be read 16 bytes at a time.
template <bool VEC>
__device__ __forceinline__ void four(const Weights& w, int i, int end, float (&x)[4]) {
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    x[0] = x[1] = x[2] = x[3] = 0.f;
    if (VEC && i + 4 <= end) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(w.p + i));
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        if (w.q) {
            const float4 u = __ldg(reinterpret_cast<const float4*>(w.q + i));
            y[0] = u.x; y[1] = u.y; y[2] = u.z; y[3] = u.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < end) {
                x[e] = __ldg(w.p + i + e);
                if (w.q) y[e] = __ldg(w.q + i + e);
            }
    }
    if (w.q) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] -= y[e];
    } else if (static_cast<unsigned>(w.skip) - static_cast<unsigned>(i) < 4u) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (w.skip == i + e) x[e] = 0.f;
    }
}

__device__ __forceinline__ uint64_t sum4(const float (&x)[4]) {
    uint32_t h = 0, l = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t hi, lo;
        weigh(x[e], hi, lo);
        h += hi;
        l += lo;
    }
    return join(h, l, 4);
}

// This lane's share of the weights of [lo, hi), and what it had added up before the
// second half of the run's steps (128 entries a step): the search starts at a half.
template <bool VEC>
__device__ __forceinline__ uint64_t run_sum(const Weights& w, int lo, int hi, int half, uint64_t& mark) {
    const int lane = threadIdx.x & 31, steps = cdiv(hi - lo, 128);
    uint64_t sum = 0;
    mark = 0;
#pragma unroll 4
    for (int s = 0; s < steps; ++s) {
        float x[4];
        four<VEC>(w, lo + s * 128 + lane * 4, hi, x);
        if (s == half) mark = sum;
        sum += sum4(x);
    }
    if (half >= steps) mark = sum;
    return sum;
}

// The smallest entry of [lo, hi) whose inclusive sum from lo exceeds `goal` (there is
// one: the run's total does), given the mark of run_sum.
template <bool VEC>
__device__ __forceinline__ int run_search(const Weights& w, int lo, int hi, int half, uint64_t goal, uint64_t mark) {
    const int lane = threadIdx.x & 31;
    int at = lo;
    mark = warp_sum64(mark);
    if (mark <= goal) {
        goal -= mark;
        at = lo + half * 128;
    }
    constexpr int kAtOnce = 4;  // steps read together
    for (; at < hi; at += kAtOnce * 128) {
        float x[kAtOnce][4];
        uint64_t mine[kAtOnce], all = 0;
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s) four<VEC>(w, at + s * 128 + lane * 4, hi, x[s]);
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s) {
            mine[s] = sum4(x[s]);
            all += mine[s];
        }
        all = warp_sum64(all);
        if (all <= goal) {
            goal -= all;
            continue;
        }
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s) {
            uint64_t incl = mine[s];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, incl > goal);
            if (past) {
                int k = 0;
                uint64_t sum = incl - mine[s];
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    uint32_t h, l;
                    weigh(x[s][e], h, l);
                    sum += join(h, l, 1);
                    if (sum <= goal && k == e) ++k;
                }
                const int src = __ffs(past) - 1;
                return at + s * 128 + src * 4 + __shfl_sync(0xffffffffu, k, src);
            }
            goal -= __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    return hi - 1;  // not reached
}

template <bool VEC>
__global__ void __launch_bounds__(kDraftThreads, 4) draft_verify_kernel(const DraftArgs a) {
    __shared__ uint64_t totals[2][kDraftWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int64_t b = blockIdx.x / ctas;
    const int* x = a.draft_tokens + b * a.drafts;
    const float* u = a.uniforms + b * (a.drafts + 1);
    const float* target = a.target + b * a.target_seq;
    const float* draft = a.draft ? a.draft + b * a.draft_seq : nullptr;
    int tok = lane < a.drafts ? __ldg(x + lane) : -1;
    float chance = lane < a.drafts ? __ldg(u + lane) : 0.f;
    const int given = a.n_drafts ? min(max(__ldg(a.n_drafts + b), 0), a.drafts) : a.drafts;

    // ---- how many drafts stand
    const float u_last = __ldg(u + a.drafts);
    int count = 0;
    for (int i0 = 0; i0 < given; i0 += 32) {
        const int i = i0 + lane;
        if (i0 > 0) {  // (the first 32 were asked for together with their number)
            tok = i < given ? __ldg(x + i) : -1;
            chance = i < given ? __ldg(u + i) : 0.f;
        }
        bool ok = false;
        if (i < given && tok >= 0 && tok < a.vocab) {
            const float p = __ldg(target + i * a.target_row + tok);
            const float q = draft ? __ldg(draft + i * a.draft_row + tok) : 1.f;
            ok = __fmul_rn(chance, q) < p;
        }
        const unsigned fell = ~__ballot_sync(0xffffffffu, ok);
        count = i0 + (fell ? __ffs(fell) - 1 : 32);
        if (fell) break;
    }
    count = min(count, given);

    // ---- draw the next token
    Weights w;
    w.p = target + count * a.target_row;
    w.q = nullptr;
    w.skip = -1;
    if (count < given) {
        if (draft)
            w.q = draft + count * a.draft_row;
        else
            w.skip = __ldg(x + count);
    }
    const int warps = static_cast<int>(ctas) * kDraftWarps, mine = static_cast<int>(rank) * kDraftWarps + warp;
    const int vocab = static_cast<int>(a.vocab), run = cdiv(cdiv(vocab, warps), 128) * 128, half = cdiv(run / 128, 2);
    const int lo = min(mine * run, vocab), hi = min(lo + run, vocab);
    uint64_t mark, part[kMaxCluster * kDraftWarps / 32], total = 0;
    // Where the weights that a fallen draft leaves are all zero (p <= q
    // everywhere), the second pass draws from p itself.
    int pass = 0;
    for (;; ++pass) {
        const uint64_t sum = warp_sum64(run_sum<VEC>(w, lo, hi, half, mark));
        if (lane == 0) totals[pass][warp] = sum;
        cluster_arrive();
        cluster_wait();
        total = 0;
#pragma unroll
        for (int k = 0; k < kMaxCluster * kDraftWarps / 32; ++k) {
            const int g = k * 32 + lane;
            part[k] = g < warps ? load_remote(&totals[pass][g % kDraftWarps], g / kDraftWarps) : 0ull;
            total += part[k];
        }
        total = warp_sum64(total);
        if (total != 0 || pass == 1 || (w.q == nullptr && w.skip < 0)) break;
        w.q = nullptr;
        w.skip = -1;
    }
    cluster_arrive();  // the totals are read; waited for before the CTA ends

    const float scaled = u_last * 16777216.f;
    const uint64_t U = scaled > 0.f ? static_cast<uint64_t>(fminf(scaled, 16777215.f)) : 0ull;
    const uint64_t goal = (total >> 24) * U + (((total & 0xFFFFFFull) * U) >> 24);
    // sum of the runs before this warp's
    uint64_t before = 0;
#pragma unroll
    for (int k = 0; k < kMaxCluster * kDraftWarps / 32; ++k)
        if (k * 32 + lane < mine) before += part[k];
    before = warp_sum64(before);
    uint64_t own = 0;
#pragma unroll
    for (int k = 0; k < kMaxCluster * kDraftWarps / 32; ++k) {
        const uint64_t v = __shfl_sync(0xffffffffu, part[k], mine & 31);
        if (k == (mine >> 5)) own = v;
    }
    int* out = a.tokens + b * (a.drafts + 1);
    if (before <= goal && goal < before + own) {
        const int token = run_search<VEC>(w, lo, hi, half, goal - before, mark);
        if (lane == 0) out[count] = token;
    }
    if (rank == 0 && warp == 0) {
        for (int i = lane; i <= a.drafts; i += 32)
            if (i != count) out[i] = i < count ? __ldg(x + i) : -1;
        if (lane == 0) {
            a.accepted[b] = count;
            if (total == 0) {  // no probability anywhere in the row
                out[count] = -1;
                record_error(MNB_ERR_CONTENT);
            }
            if (count < given && (__ldg(x + count) < 0 || __ldg(x + count) >= a.vocab)) record_error(MNB_ERR_CONTENT);
        }
    }
    cluster_wait();
}

}  // namespace

cudaError_t launch_draft_verify(const DraftArgs& a, int sm_count, bool pdl, cudaStream_t stream) {
    auto rows16 = [](const float* p, int64_t seq, int64_t row) {
        return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && seq % 4 == 0 && row % 4 == 0;
    };
    const bool vec = rows16(a.target, a.target_seq, a.target_row) && (!a.draft || rows16(a.draft, a.draft_seq, a.draft_row));
    auto kern = vec ? draft_verify_kernel<true> : draft_verify_kernel<false>;
    cudaError_t e = set_max_carveout(kern);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    // CTAs per sequence: as many as give every SM about four, at most 16
    int cluster = kMaxCluster;
    while (cluster > 1 && a.batch * cluster > int64_t(sm_count) * 4) cluster >>= 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.batch * cluster));
    cfg.blockDim = dim3(kDraftThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

cudaError_t draft_take_error(unsigned int* out) { return take_unit_error(out); }

}  // namespace mnb
