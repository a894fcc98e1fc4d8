// kv_plan.cu -- a step's lengths, starts, pages and slots from what each sequence
// keeps in the cache and adds to it.
//
// With k kept and n added tokens a sequence needs w = ceil((k + n) / page_size) pages
// and holds h: it takes max(w - h, 0) from the stack of free pages or gives max(h - w,
// 0) back.  What is given back lies on the stack before anything is taken, the first
// sequence's first page on top, and the first sequence takes first: a step that takes
// pages and a step that gives the same ones back undo each other.  A sequence that asks
// for more than the pool, the table or the step has left is refused, and every later
// one that asks for the same resource; so the sums of what is asked for decide, and
// both passes are prefix sums.
//
// Bound: latency (a step of 64 sequences moves 3 KB).  Every CTA of one cluster works
// out the sums of all sequences for itself (shared memory, 28 bytes a sequence); after the
// cluster's barrier no input is read any more that an output may stand on, and pages and
// slots are shared out over its threads, each found by a binary search among the sums.
// Many slots (the map of a batch of prompts) have a grid of their own behind it.
//
// Measured: 64 sequences with 1 .. 5 new tokens 5.8 us (5.1 without slots), 4.6 where nothing is asked for;
// 1000 sequences and 31000 pages 9.3 us, with 500000 slots 13.8 (the slots' grid took 6.9 with a
// search for every token and stores eight bytes apart per lane).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv.h"

namespace mnb {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;          // the largest cluster
constexpr int kAtOnce = 4;               // pages that a thread looks for together
constexpr int kSlotRun = 8;              // tokens of a thread in the slot map's own grid
constexpr uint32_t kMost = 0x7fffffffu;  // sums stay there once they reach it

// Sums of non-negative numbers that stop at kMost: the order does not matter.
__device__ __forceinline__ uint32_t add_up(uint32_t a, uint32_t b) { return min(a + b, kMost); }

struct Sums {
    uint32_t a, b, c;
};
__device__ __forceinline__ Sums operator+(const Sums& x, const Sums& y) {
    return {add_up(x.a, y.a), add_up(x.b, y.b), add_up(x.c, y.c)};
}

// The sums of the threads before this one; `total` those of all.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* warps, Sums* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
    Sums in = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums x = {__shfl_up_sync(0xffffffffu, in.a, o), __shfl_up_sync(0xffffffffu, in.b, o),
                        __shfl_up_sync(0xffffffffu, in.c, o)};
        if (lane >= o) in = in + x;
    }
    if (lane == 31) warps[warp] = in;
    Sums before = {__shfl_up_sync(0xffffffffu, in.a, 1), __shfl_up_sync(0xffffffffu, in.b, 1),
                   __shfl_up_sync(0xffffffffu, in.c, 1)};
    if (lane == 0) before = {0, 0, 0};
    __syncthreads();
    Sums w = lane < n ? warps[lane] : Sums{0, 0, 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums x = {__shfl_up_sync(0xffffffffu, w.a, o), __shfl_up_sync(0xffffffffu, w.b, o),
                        __shfl_up_sync(0xffffffffu, w.c, o)};
        if (lane >= o) w = w + x;
    }
    *total = {__shfl_sync(0xffffffffu, w.a, 31), __shfl_sync(0xffffffffu, w.b, 31), __shfl_sync(0xffffffffu, w.c, 31)};
    const int src = max(warp - 1, 0);
    const Sums front = {__shfl_sync(0xffffffffu, w.a, src), __shfl_sync(0xffffffffu, w.b, src),
                        __shfl_sync(0xffffffffu, w.c, src)};
    __syncthreads();  // `warps` may be written again
    return warp > 0 ? front + before : before;
}

// The last of n ascending numbers that is at most i (the first one is).
__device__ __forceinline__ int last_at_most(const uint32_t* first, int n, uint32_t i) {
    int lo = 0;
    for (int hi = n; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const KvPlanArgs a, bool with_slots) {
    extern __shared__ uint32_t plan_smem[];
    __shared__ Sums warps[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, threads = blockDim.x, batch = a.batch;
    uint32_t* start = plan_smem;           // first new token
    uint32_t* keep = start + batch;
    uint32_t* held = keep + batch;         // pages before the step
    uint32_t* target = held + batch;       // pages after it
    uint32_t* takes = target + batch;      // pages that the sequences before take
    uint32_t* gives = takes + batch;       // pages that they give back
    uint32_t* adds = gives + batch;        // new tokens, bit 31: more than the table has columns for
    bool bad = false;
    const int raw_free = __ldg(a.free_count);
    const uint32_t free_count = min(max(raw_free, 0), a.num_pages);
    if (static_cast<int>(free_count) != raw_free) bad = true;
    for (int b = tid; b < batch; b += threads) {
        const int h0 = __ldg(a.held + b), k0 = __ldg(a.keep + b), n0 = __ldg(a.add + b);
        const int h = min(max(h0, 0), a.max_pages);
        const int64_t has = static_cast<int64_t>(h) * a.page_size;
        const int k = static_cast<int>(min(static_cast<int64_t>(max(k0, 0)), has)), n = max(n0, 0);
        if (h != h0 || k != k0 || n != n0) bad = true;
        const int64_t len = static_cast<int64_t>(k) + n;
        const int64_t want = (len + a.page_size - 1) / a.page_size;
        const bool too_long = n > 0 && (want > a.max_pages || len > kKvMaxCapacity);
        keep[b] = k;
        held[b] = h;
        target[b] = too_long ? h : static_cast<uint32_t>(want);
        adds[b] = too_long ? 0x80000000u : static_cast<uint32_t>(n);
    }
    __syncthreads();
    // a thread takes consecutive sequences
    const int per = (batch + threads - 1) / threads, b0 = min(tid * per, batch), b1 = min(b0 + per, batch);
    auto asked = [&](int b) -> Sums {
        const uint32_t h = held[b], t = target[b];
        return {t > h ? t - h : 0u, h > t ? h - t : 0u, adds[b] & kMost};
    };
    Sums mine = {0, 0, 0}, total;
    for (int b = b0; b < b1; ++b) mine = mine + asked(b);
    Sums at = block_scan(mine, warps, &total);
    const uint32_t back = total.b;  // pages given back
    const int64_t room = static_cast<int64_t>(free_count) + back;
    mine = {0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        const Sums x = asked(b);
        gives[b] = at.b;
        at = at + x;
        const bool refused = (adds[b] >> 31) || (x.c > 0 && ((x.a > 0 && at.a > room) || at.c > a.max_tokens));
        if (refused) {
            adds[b] = 0x80000000u;
            if (x.a > 0) target[b] = held[b];
        } else {
            mine = mine + Sums{x.a, x.c, 0u};
        }
    }
    at = block_scan(mine, warps, &total);
    const uint32_t taken = total.a, tokens = total.b;
    for (int b = b0; b < b1; ++b) {
        takes[b] = at.a;
        start[b] = at.b;
        const uint32_t h = held[b], t = target[b];
        at = at + Sums{t > h ? t - h : 0u, adds[b] & kMost, 0u};
    }
    // every input that an output may stand on has been read by every CTA
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    }
    __syncthreads();

    if (rank == 0) {
        for (int b = tid; b < batch; b += threads) {
            const uint32_t n = adds[b] & kMost;
            a.seq_lens[b] = keep[b] + n;
            a.new_start[b] = start[b];
            a.held_out[b] = target[b];
            if (a.refused) a.refused[b] = adds[b] >> 31;
        }
        if (tid == 0) {
            a.new_start[batch] = tokens;
            const int64_t left = room - taken;
            if (left > a.num_pages) bad = true;
            *a.free_count_out = static_cast<int>(min(left, static_cast<int64_t>(a.num_pages)));
        }
    }
    const int64_t g0 = static_cast<int64_t>(rank) * threads + tid, step = static_cast<int64_t>(ctas) * threads;
    // page number r of those given back; it stands at room - 1 - r of the stack
    auto given = [&](uint32_t r) {
        const int b = last_at_most(gives, batch, r);
        return a.page_table[b * a.table_stride + target[b] + (r - gives[b])];
    };
    auto popped = [&](uint32_t i) { return i < back ? given(i) : a.free_pages[room - 1 - i]; };
    for (int64_t i = g0; i < taken; i += kAtOnce * step) {  // (several at a time: their loads do not wait for one another)
        int b[kAtOnce], page[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int64_t p = i + k * step;
            if (p >= taken) break;
            page[k] = popped(static_cast<uint32_t>(p));
            b[k] = last_at_most(takes, batch, static_cast<uint32_t>(p));
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int64_t p = i + k * step;
            if (p >= taken) break;
            if (page[k] < 0 || page[k] >= a.num_pages) bad = true;
            a.page_table[b[k] * a.table_stride + held[b[k]] + (static_cast<uint32_t>(p) - takes[b[k]])] = page[k];
        }
    }
    for (int64_t r = taken + g0; r < back; r += step) {
        const int64_t place = room - 1 - r;
        if (place < a.num_pages)
            a.free_pages[place] = given(static_cast<uint32_t>(r));
        else
            bad = true;
    }
    if (with_slots)
        for (int64_t t = g0; t < tokens; t += step) {
            const int b = last_at_most(start, batch, static_cast<uint32_t>(t));
            const int pos = static_cast<int>(keep[b] + (static_cast<uint32_t>(t) - start[b]));
            const int column = a.by_page(pos);
            const int page = column < static_cast<int>(held[b]) ? a.page_table[b * a.table_stride + column]
                                                                : popped(takes[b] + column - held[b]);
            const bool out = page < 0 || page >= a.num_pages;
            if (out) bad = true;
            a.slots[t] = out ? -1 : static_cast<int64_t>(page) * a.page_size + (pos - column * a.page_size);
        }
    if (bad) record_error(MNB_ERR_CONTENT);
}

// The slot map of a large step, from the plan that the kernel ahead wrote: a warp takes 32
// kSlotRun neighbouring tokens, finds the first one's sequence (the starts are in shared
// memory) and goes on from there, a lane with every 32nd token.
__global__ void __launch_bounds__(256) kv_slots_kernel(const KvPlanArgs a) {
    extern __shared__ uint32_t starts[];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tokens = a.new_start[a.batch];
    if (static_cast<int64_t>(blockIdx.x) * 256 * kSlotRun >= tokens) return;
    for (int b = threadIdx.x; b <= a.batch; b += 256) starts[b] = a.new_start[b];
    __syncthreads();
    bool bad = false;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * 8 + warp) * 32 * kSlotRun; t0 < tokens;
         t0 += static_cast<int64_t>(gridDim.x) * 256 * kSlotRun) {
        int b = last_at_most(starts, a.batch, static_cast<uint32_t>(t0));
        int page[kSlotRun], row[kSlotRun];
#pragma unroll
        for (int k = 0; k < kSlotRun; ++k) {
            const int64_t t = t0 + 32 * k + lane;
            if (t >= tokens) break;
            while (starts[b + 1] <= static_cast<uint32_t>(t)) ++b;  // (ends: starts[batch] = tokens > t)
            const int pos = a.seq_lens[b] - static_cast<int>(starts[b + 1]) + static_cast<int>(t), column = a.by_page(pos);
            row[k] = pos - column * a.page_size;
            page[k] = a.page_table[b * a.table_stride + column];
        }
#pragma unroll
        for (int k = 0; k < kSlotRun; ++k) {
            const int64_t t = t0 + 32 * k + lane;
            if (t >= tokens) break;
            const bool out = page[k] < 0 || page[k] >= a.num_pages;
            if (out) bad = true;
            a.slots[t] = out ? -1 : static_cast<int64_t>(page[k]) * a.page_size + row[k];
        }
    }
    if (bad) record_error(MNB_ERR_CONTENT);
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& in, int sm_count, bool pdl, cudaStream_t stream) {
    KvPlanArgs a = in;
    a.by_page.set(static_cast<uint32_t>(a.page_size));
    // Slots: inside the plan's cluster up to 16 a thread, else in a grid of their own.
    const bool own_grid = a.slots && a.max_tokens > 16 * kPlanThreads;
    const bool inside = a.slots && !own_grid;
    // CTAs: a thread's share of pages and slots stays small (at most four of each, until the cluster is full).
    const int64_t pages = std::min(int64_t(a.batch) * a.max_pages, int64_t(a.num_pages));
    const int64_t work = std::max(pages / 4, inside ? a.max_tokens : int64_t(0));
    int ctas = 1;
    while (ctas < kPlanCluster && int64_t(ctas) * kPlanThreads * 4 < work) ctas *= 2;
    const int threads = ctas == 1 && a.batch <= 256 && work <= 1024 ? 256 : kPlanThreads;
    const size_t smem = size_t(7) * sizeof(uint32_t) * std::max(a.batch, 1);
    const cudaError_t e = launch_cluster<kv_plan_kernel>(dim3(static_cast<unsigned>(ctas)), dim3(static_cast<unsigned>(threads)),
                                                         static_cast<unsigned>(ctas), smem,
                                                         size_t(7) * sizeof(uint32_t) * kKvPlanMaxBatch, stream, pdl, a, inside);
    if (e != cudaSuccess || !own_grid) return e;
    const int64_t grid = std::min<int64_t>(cdiv<int64_t>(a.max_tokens, 256 * kSlotRun), int64_t(sm_count) * 4);
    return launch_cluster<kv_slots_kernel>(dim3(static_cast<unsigned>(grid)), dim3(256), 1, size_t(a.batch + 1) * 4,
                                           size_t(kKvPlanMaxBatch + 1) * 4, stream, pdl, a);
}

cudaError_t kv_plan_take_error(unsigned int* out) { return take_unit_error(out); }

}  // namespace mnb
