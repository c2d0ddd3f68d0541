// Tokens sorted by expert and back.
//
// Slot i = t * k + j holds token t's j-th expert id.  The sort is a stable
// counting sort:
//   offsets[e]  = number of valid slots with an id below e
//   slot_row[i] = offsets[id_i] + number of valid slots before i with id_i
//   row_slot    = its inverse, -1 past the last row that holds a slot
// Slots are placed kSortThreads at a time: lanes of a warp with the same id
// find their rank with one match, the warps' counts per expert are summed in
// warp order, so no atomic decides an order.  Up to kSortThreads slots (a
// decoding step) every CTA of the gather sorts them by itself and the whole
// dispatch is one launch.  Up to kClusterSlots one cluster of 8 CTAs sorts them
// (their counts meet through distributed shared memory), above that a count
// kernel and a place kernel; the gather follows as their programmatic
// dependent.
//
// The row movements are bound by memory: the gather reads a token's row once
// and writes it to its k rows, the combine reads the k rows and writes one,
// the combine's gradient reads dout and the k rows and writes k rows and k dot
// products.  A group of 1 to 8 warps owns a token.  Rows on 16-byte boundaries
// move in 16-byte vectors, BF16 rows of even widths in pairs, others element by
// element, several in flight: 4096 x 8 rows of 2046 BF16 are combined in 36.9 us
// by pairs, 53.4 by elements.  (Odd rows read as two aligned vectors and a shift
// along the boundaries of the row that is written were slower than elements:
// 4096 x 8 x 2047 combined in 70 us instead of 53, its gradient with k = 4 in 92
// instead of 49, because the warps that hold a row's ends go both ways.)
#include <algorithm>
#include <type_traits>
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "tcgen05.cuh"

namespace bsq {
namespace {

constexpr int kSortThreads = 1024;     // slots per step: one per thread

// Slots of one CTA: whole steps, so that at most kSortCtas CTAs cover them.
constexpr int kSortCtas = 128;
inline int64_t sort_chunk(int64_t slots) {
    const int64_t steps = (slots + kSortThreads - 1) / kSortThreads;
    return (steps + kSortCtas - 1) / kSortCtas * kSortThreads;
}

struct SortArgs {
    const void* ids;
    int64_t slots, chunk;
    int ids64, experts, chunks;
    int32_t* counts;               // [chunks][experts]
    int64_t* offsets;
    int32_t* slot_row;
    int32_t* row_slot;
};

__device__ __forceinline__ int load_id(const SortArgs& a, int64_t i) {
    const int64_t id = a.ids64 ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
    return id >= 0 && id < a.experts ? (int)id : -1;
}

// Exclusive scan over the threads of a CTA; `all` is the sum.
template <int THREADS>
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t& all) {
    __shared__ int32_t warp_sum[THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += u;
    }
    if (lane == 31) warp_sum[warp] = s;
    __syncthreads();
    int32_t w = lane < THREADS / 32 ? warp_sum[lane] : 0;
#pragma unroll
    for (int d = 1; d < THREADS / 32; d <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += u;
    }
    all = __shfl_sync(0xffffffffu, w, THREADS / 32 - 1);
    const int32_t before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return s - v + (warp > 0 ? before : 0);
}

// counts[w] of `warps` warps, `pitch` apart: each becomes the sum of those
// before it; returns the sum of all.
__device__ __forceinline__ int32_t scan_warps(uint16_t* counts, int pitch, int warps) {
    int32_t sum = 0;
    for (int w0 = 0; w0 < warps; w0 += 8) {
        int n[8];
#pragma unroll
        for (int w = 0; w < 8; w++) n[w] = w0 + w < warps ? counts[(w0 + w) * pitch] : 0;
#pragma unroll
        for (int w = 0; w < 8; w++) {
            if (w0 + w < warps) counts[(w0 + w) * pitch] = (uint16_t)sum;
            sum += n[w];
        }
    }
    return sum;
}

// One step: this thread's slot (expert e, -1 for none).  wcount[warps][experts]
// receives, per warp, the slots of each expert in the warps before it; returns
// the slot's rank in its warp.  `sum` (thread x < experts): the step's slots of
// expert x.  Ends with the counts visible to the CTA.
template <int THREADS>
__device__ __forceinline__ int step_ranks(int e, int experts, int warps, uint16_t* wcount, int32_t& sum) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int x = tid; x < warps * experts; x += THREADS) wcount[x] = 0;
    __syncthreads();
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1));
    if (e >= 0 && rank == 0) wcount[warp * experts + e] = (uint16_t)__popc(same);
    __syncthreads();
    sum = tid < experts ? scan_warps(wcount + tid, experts, warps) : 0;
    return rank;
}

// counts[b][e]: valid slots of chunk b with expert e
__global__ void __launch_bounds__(kSortThreads) moe_count_kernel(const SortArgs a) {
    extern __shared__ int32_t sm[];
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads) sm[e] = 0;
    __syncthreads();
    pdl_launch_dependents();
    const int64_t lo = blockIdx.x * a.chunk, hi = min(a.slots, lo + a.chunk);
    for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads) {
        const int e = load_id(a, i);
        if (e >= 0) atomicAdd(&sm[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads)
        a.counts[(int64_t)blockIdx.x * a.experts + e] = sm[e];
}

// Places the slots of one chunk.  Shared memory: total[experts], base[experts]
// (the next free row of each expert for this chunk) and wcount[32][experts].
__global__ void __launch_bounds__(kSortThreads) moe_place_kernel(const SortArgs a) {
    extern __shared__ int32_t sm[];
    const int E = a.experts, tid = threadIdx.x;
    int32_t* total = sm;
    int32_t* base = sm + E;
    uint16_t* wcount = reinterpret_cast<uint16_t*>(sm + 2 * E);
    for (int e = tid; e < 2 * E; e += kSortThreads) sm[e] = 0;
    const int64_t lo = blockIdx.x * a.chunk, hi = min(a.slots, lo + a.chunk);
    int e = lo + tid < hi ? load_id(a, lo + tid) : -1;         // ids are inputs: read before the counts are done
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    // totals and this chunk's start within each expert: integer sums, any order
    for (int i = tid; i < a.chunks * E; i += kSortThreads) {
        const int b = i / E, x = i - b * E;
        const int32_t c = a.counts[i];
        if (c) {
            atomicAdd(&total[x], c);
            if (b < (int)blockIdx.x) atomicAdd(&base[x], c);
        }
    }
    __syncthreads();
    int32_t all;
    const int32_t first = block_scan<kSortThreads>(tid < E ? total[tid] : 0, all);
    if (tid < E) {
        base[tid] += first;
        if (blockIdx.x == 0) a.offsets[tid] = first;
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[E] = all;
    for (int64_t i = max(lo, (int64_t)all) + tid; i < hi; i += kSortThreads) a.row_slot[i] = -1;
    for (int64_t s = lo; s < hi; s += kSortThreads) {
        const int64_t i = s + tid;
        if (s > lo) e = i < hi ? load_id(a, i) : -1;
        int32_t sum;
        const int rank = step_ranks<kSortThreads>(e, E, 32, wcount, sum);
        __syncthreads();
        const int32_t row = e >= 0 ? base[e] + wcount[(tid >> 5) * E + e] + rank : -1;
        __syncthreads();
        if (tid < E) base[tid] += sum;
        if (i < hi) {
            a.slot_row[i] = row;
            if (row >= 0) a.row_slot[row] = (int32_t)i;
        }
    }
}

// One cluster sorts up to kClusterSlots slots, one a thread: a CTA's counts per
// expert meet the other CTAs' through distributed shared memory.  (With 2 to 8
// slots a thread it also sorted 65536, but 8 SMs write the plan too slowly then:
// 32768 slots took 4 us longer than the two launches below.)
constexpr int kCluster = 8;
constexpr int64_t kClusterSlots = (int64_t)kCluster * kSortThreads;

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSortThreads) moe_cluster_sort_kernel(const SortArgs a) {
    extern __shared__ int32_t sm[];
    const int E = a.experts, tid = threadIdx.x;
    int32_t* mine = sm;                                     // [E] this CTA's slots of each expert
    int32_t* base = sm + E;                                 // [E] first row of each expert for this CTA
    uint16_t* wcount = reinterpret_cast<uint16_t*>(sm + 2 * E);    // [32][E]
    const int64_t slot = (int64_t)blockIdx.x * kSortThreads + tid;
    pdl_launch_dependents();
    const int e = slot < a.slots ? load_id(a, slot) : -1;
    int32_t sum;
    const int rank = step_ranks<kSortThreads>(e, E, 32, wcount, sum);
    if (tid < E) mine[tid] = sum;
    tc::cluster_sync();
    int32_t total = 0, before = 0;
    if (tid < E) {
        const uint32_t at = tc::smem_u32(mine + tid);
#pragma unroll
        for (int c = 0; c < kCluster; c++) {
            const int32_t n = tc::ld_cluster_s32(tc::mapa(at, c));
            if (c < (int)blockIdx.x) before += n;
            total += n;
        }
    }
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");      // done with the other CTAs' counts
    int32_t all;
    const int32_t first = block_scan<kSortThreads>(total, all);
    if (tid < E) {
        base[tid] = first + before;
        if (blockIdx.x == 0) a.offsets[tid] = first;
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[E] = all;
    __syncthreads();
    const int32_t row = e >= 0 ? base[e] + wcount[(tid >> 5) * E + e] + rank : -1;
    if (slot < a.slots) {
        a.slot_row[slot] = row;
        if (row >= 0) a.row_slot[row] = (int32_t)slot;
        if (slot >= all) a.row_slot[slot] = -1;
    }
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");        // a CTA's counts outlive their readers
}

struct RowArgs {
    const void* src;
    int64_t ld_src;
    void* dst;
    int64_t ld_dst;
    int64_t tokens;
    int32_t nvec;                  // vectors (or elements) of a row
    int32_t k;
    const int32_t* slot_row;
    const int64_t* total;          // offsets[num_experts]: rows that hold a slot
    const float* weights;
    const void* rows;              // combine gradient
    int64_t ld_rows;
    float* dweights;
};

// The rows from `total` on hold no slot: token t's group clears those among
// rows t k .. t k + k - 1.
template <typename T, int VEC>
__device__ __forceinline__ void clear_rows(const RowArgs& a, int64_t t, int64_t total, int v0, int step) {
    Pack<T, VEC> z;
    z.zero();
    for (int64_t r = max(t * a.k, total); r < (t + 1) * a.k; r++) {
        T* out = static_cast<T*>(a.dst) + r * a.ld_dst;
        for (int v = v0; v < a.nvec; v += step) z.store(out + (int64_t)v * VEC);
    }
}

// The vectors of a row that a thread copies at a time
template <typename T, int VEC>
struct Copied {
    static constexpr int UN = 4;
    Pack<T, VEC> p[UN];
    __device__ __forceinline__ void load(const RowArgs& a, int64_t t, int v, int step) {
        const T* in = static_cast<const T*>(a.src) + t * a.ld_src;
#pragma unroll
        for (int u = 0; u < UN; u++)
            if (v + u * step < a.nvec) p[u].load(in + (int64_t)(v + u * step) * VEC);
    }
};
// Copies token t's row to its rows; rows_of(j) is slot j's row.  `loaded`: the
// first vectors are in `held` already.
template <typename T, int VEC, typename F>
__device__ __forceinline__ void copy_row(const RowArgs& a, int64_t t, F rows_of, int v0, int step, Copied<T, VEC>& held,
                                         bool loaded) {
    constexpr int UN = Copied<T, VEC>::UN;
    for (int v = v0; v < a.nvec; v += UN * step, loaded = false) {
        if (!loaded) held.load(a, t, v, step);
        for (int j = 0; j < a.k; j++) {
            const int32_t r = rows_of(j);
            if (r < 0) continue;
            T* out = static_cast<T*>(a.dst) + r * a.ld_dst;
#pragma unroll
            for (int u = 0; u < UN; u++)
                if (v + u * step < a.nvec) held.p[u].store(out + (int64_t)(v + u * step) * VEC);
        }
    }
}

constexpr int kRowThreads = 256;

// Token of this thread's group of WPT warps, its first vector and its step
struct Place {
    int64_t t;
    int v0, step;
};
template <int WPT>
__device__ __forceinline__ Place place() {
    constexpr int PER = kRowThreads / 32 / WPT;
    const int g = threadIdx.x / (32 * WPT), at = threadIdx.x % (32 * WPT);
    return {(int64_t)blockIdx.x * PER + g, at + (int)blockIdx.y * 32 * WPT, 32 * WPT * (int)gridDim.y};
}

// Bound by the writes: 32768 rows of 7168 BF16 from 4096 in 80 us, 6.6 TB/s; with
// the sort before it the dispatch takes 87.9 us (0.90 of a copy's rate; 89.4 when x
// was read only after the sort).
template <typename T, int VEC, int WPT>
__global__ void __launch_bounds__(kRowThreads) moe_gather_kernel(const RowArgs a) {
    const Place at = place<WPT>();
    if (at.t >= a.tokens) return;
    const int32_t* rows = a.slot_row + at.t * a.k;
    Copied<T, VEC> held;
    held.load(a, at.t, at.v0, at.step);            // x does not depend on the sort
    pdl_wait();
    copy_row<T, VEC>(a, at.t, [&](int j) { return rows[j]; }, at.v0, at.step, held, true);
    clear_rows<T, VEC>(a, at.t, *a.total, at.v0, at.step);
}

// Sort and gather of at most THREADS slots over at most THREADS experts in one
// launch: every CTA sorts all slots in shared memory (they are few) and moves
// its own pieces of rows; CTA 0 writes the plan.  The first piece of a row is
// read before the sort, so the two wait for memory together.  With a.src null
// it only sorts.  Bound by latency: one token to 8 of 64 experts, 7168 BF16, in
// 4.1 us, which is what a launch takes.
template <typename T, int VEC, int THREADS>
__global__ void __launch_bounds__(THREADS) moe_small_kernel(const SortArgs s, const RowArgs a, int pieces) {
    extern __shared__ int32_t sm[];
    const int E = s.experts, n = (int)s.slots, tid = threadIdx.x, warps = (n + 31) >> 5;
    int32_t* row_of = sm;                                        // [THREADS]
    int32_t* base = sm + THREADS;                                // [E]
    uint16_t* wcount = reinterpret_cast<uint16_t*>(base + E);    // [warps][E]
    const int e = tid < n ? load_id(s, tid) : -1;
    // a piece: 128 threads' share of one token's row
    const int at = tid & 127, step = pieces * 128;
    const int64_t all_pieces = a.tokens * pieces, ahead = (int64_t)gridDim.x * (THREADS / 128);
    int64_t w = (int64_t)blockIdx.x * (THREADS / 128) + (tid >> 7);
    const auto token = [&] { return w / pieces; };
    const auto first_vec = [&] { return (int)(w - token() * pieces) * 128 + at; };
    Copied<T, VEC> held;
    if (a.src && w < all_pieces) held.load(a, token(), first_vec(), step);
    int32_t sum, all;
    const int rank = step_ranks<THREADS>(e, E, warps, wcount, sum);
    const int32_t first = block_scan<THREADS>(sum, all);
    if (tid < E) base[tid] = first;
    __syncthreads();
    const int32_t row = e >= 0 ? base[e] + wcount[(tid >> 5) * E + e] + rank : -1;
    row_of[tid] = row;
    if (blockIdx.x == 0) {
        if (tid < E) s.offsets[tid] = first;
        if (tid == 0) s.offsets[E] = all;
        if (tid < n) {
            s.slot_row[tid] = row;
            if (row >= 0) s.row_slot[row] = tid;
            if (tid >= all) s.row_slot[tid] = -1;
        }
    }
    if (!a.src) return;
    __syncthreads();
    for (bool loaded = true; w < all_pieces; w += ahead, loaded = false) {
        const int64_t t = token();
        copy_row<T, VEC>(a, t, [&](int j) { return row_of[t * a.k + j]; }, first_vec(), step, held, loaded);
        clear_rows<T, VEC>(a, t, all, first_vec(), step);
    }
}

// Slots of a token handled together: 8 vectors (the usual k in one pass), or 4
// single elements of 4 columns each.  (Odd combine of 1021 x 3 x 2047: 9.3 us
// with 4, 12.3 with 8.)
template <int VEC>
constexpr int kSlots = VEC <= 2 ? 4 : 8;

// out[t] = sum_j weights[t, j] rows[slot_row[t, j]], in the order of j.  Bound by
// reading the rows: 4096 x 8 x 7168 BF16 in 85.3 us, 6.2 TB/s (0.93 of a copy's
// rate); 1021 x 3 x 2047 element by element in 8.2 us, two thirds of it latency.
template <typename T, int VEC, int WPT, bool WEIGHTED>
__global__ void __launch_bounds__(kRowThreads) moe_combine_kernel(const RowArgs a) {
    constexpr int UN = VEC <= 2 ? 4 : 1, S = kSlots<VEC>;
    const Place at = place<WPT>();
    if (at.t >= a.tokens) return;
    const T* src = static_cast<const T*>(a.src);
    T* out = static_cast<T*>(a.dst) + at.t * a.ld_dst;
    int32_t row[S];
    float w[S];
    auto slots = [&](int j0) {
#pragma unroll
        for (int j = 0; j < S; j++) {
            row[j] = j0 + j < a.k ? a.slot_row[at.t * a.k + j0 + j] : -1;
            w[j] = WEIGHTED && row[j] >= 0 ? a.weights[at.t * a.k + j0 + j] : 1.0f;
        }
    };
    slots(0);
    for (int v = at.v0; v < a.nvec; v += UN * at.step) {
        float acc[UN][VEC] = {};
        for (int j0 = 0; j0 < a.k; j0 += S) {
            if (a.k > S) slots(j0);
            Pack<T, VEC> p[UN][S];
#pragma unroll
            for (int j = 0; j < S; j++)
#pragma unroll
                for (int u = 0; u < UN; u++)
                    if (row[j] >= 0 && v + u * at.step < a.nvec)
                        p[u][j].load(src + row[j] * a.ld_src + (int64_t)(v + u * at.step) * VEC);
#pragma unroll
            for (int j = 0; j < S; j++)
                if (row[j] >= 0)
#pragma unroll
                    for (int u = 0; u < UN; u++) {
                        float f[VEC];
                        p[u][j].unpack(f);
#pragma unroll
                        for (int i = 0; i < VEC; i++)
                            acc[u][i] = WEIGHTED ? fmaf(w[j], f[i], acc[u][i]) : acc[u][i] + f[i];
                    }
        }
#pragma unroll
        for (int u = 0; u < UN; u++)
            if (v + u * at.step < a.nvec) {
                Pack<T, VEC> o;
                o.pack(acc[u]);
                o.store(out + (int64_t)(v + u * at.step) * VEC);
            }
    }
}

// drows[row] = weights[slot] dout[t], dweights[slot] = dout[t] . rows[row].  Bound
// by memory: 4096 x 8 x 7168 BF16 in 155 us, 6.4 TB/s (0.95 of a copy's rate).
// Three CTAs per SM (80 registers): the batch of 32768 x 7168 takes 156 us,
// with two (98 registers) 209, with four (spills) 176.
template <typename T, int VEC, int WPT, bool DOT>
__global__ void __launch_bounds__(kRowThreads, 3) moe_combine_backward_kernel(const RowArgs a) {
    constexpr int UN = VEC <= 2 ? 4 : 1, S = kSlots<VEC>;
    __shared__ float part[kRowThreads / 32][S];
    const Place at = place<WPT>();
    const bool live = at.t < a.tokens;
    const T* dout = static_cast<const T*>(a.src) + (live ? at.t : 0) * a.ld_src;
    const T* rows = static_cast<const T*>(a.rows);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int j0 = 0; j0 < a.k; j0 += S) {
        int32_t row[S];
        float w[S], dot[S];
#pragma unroll
        for (int j = 0; j < S; j++) {
            row[j] = live && j0 + j < a.k ? a.slot_row[at.t * a.k + j0 + j] : -1;
            w[j] = row[j] >= 0 ? a.weights[at.t * a.k + j0 + j] : 0.0f;
            dot[j] = 0.0f;
        }
        for (int v = live ? at.v0 : a.nvec; v < a.nvec; v += UN * at.step) {
            Pack<T, VEC> d[UN], p[UN][S];
#pragma unroll
            for (int u = 0; u < UN; u++) {
                if (v + u * at.step >= a.nvec) continue;
                d[u].load(dout + (int64_t)(v + u * at.step) * VEC);
                if (DOT)
#pragma unroll
                    for (int j = 0; j < S; j++)
                        if (row[j] >= 0) p[u][j].load(rows + row[j] * a.ld_rows + (int64_t)(v + u * at.step) * VEC);
            }
#pragma unroll
            for (int u = 0; u < UN; u++) {
                if (v + u * at.step >= a.nvec) continue;
                float f[VEC];
                d[u].unpack(f);
#pragma unroll
                for (int j = 0; j < S; j++) {
                    if (row[j] < 0) continue;
                    float o[VEC];
                    if (DOT) {
                        p[u][j].unpack(o);
#pragma unroll
                        for (int i = 0; i < VEC; i++) dot[j] = fmaf(f[i], o[i], dot[j]);
                    }
#pragma unroll
                    for (int i = 0; i < VEC; i++) o[i] = w[j] * f[i];
                    Pack<T, VEC> g;
                    g.pack(o);
                    g.store(static_cast<T*>(a.dst) + row[j] * a.ld_dst + (int64_t)(v + u * at.step) * VEC);
                }
            }
        }
        if (DOT) {
#pragma unroll
            for (int j = 0; j < S; j++)
#pragma unroll
                for (int d = 16; d; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
            __syncthreads();
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < S; j++) part[warp][j] = dot[j];
            __syncthreads();
            const int j = threadIdx.x % (32 * WPT);
            if (live && j < S && j0 + j < a.k) {
                float s = 0.0f;
#pragma unroll
                for (int x = 0; x < WPT; x++) s += part[warp / WPT * WPT + x][j];
                a.dweights[at.t * a.k + j0 + j] = s;
            }
        }
    }
    if (live) clear_rows<T, VEC>(a, at.t, *a.total, at.v0, at.step);
}

// ------------------------------------------------------------------- launches
SortArgs sort_args(const MoePlanArgs& p, const void* ids, bool ids64, void* ws) {
    SortArgs a{};
    a.ids = ids;
    a.slots = p.tokens * p.k;
    a.chunk = sort_chunk(a.slots);
    a.chunks = (int)((a.slots + a.chunk - 1) / a.chunk);
    a.ids64 = ids64;
    a.experts = p.num_experts;
    a.counts = static_cast<int32_t*>(ws);
    a.offsets = p.offsets;
    a.slot_row = p.slot_row;
    a.row_slot = p.row_slot;
    return a;
}

RowArgs row_args(const MoePlanArgs& p, const MoeRowsArgs& m, int vec) {
    RowArgs a{};
    a.src = m.src;
    a.ld_src = m.ld_src;
    a.dst = m.dst;
    a.ld_dst = m.ld_dst;
    a.tokens = p.tokens;
    a.nvec = (int32_t)(m.cols / vec);
    a.k = p.k;
    a.slot_row = p.slot_row;
    a.total = p.offsets + p.num_experts;
    a.weights = m.weights;
    a.rows = m.rows;
    a.ld_rows = m.ld_rows;
    a.dweights = m.dweights;
    return a;
}

// vectors of so many bytes only where every matrix of the call allows them
bool vectors(const MoeRowsArgs& m, int bytes) {
    const int e = m.bf16 ? 2 : 4;
    return rows_vec(m.src, m.ld_src, m.cols, e, bytes) && rows_vec(m.dst, m.ld_dst, m.cols, e, bytes) &&
           (!m.rows || rows_vec(m.rows, m.ld_rows, m.cols, e, bytes));
}
// f(element, vector length): 16 bytes, else pairs of BF16, else single elements
template <typename F>
cudaError_t by_vector(const MoeRowsArgs& m, F f) {
    using std::integral_constant;
    if (!m.bf16) return vectors(m, 16) ? f(0.0f, integral_constant<int, 4>()) : f(0.0f, integral_constant<int, 1>());
    if (vectors(m, 16)) return f(__nv_bfloat16(), integral_constant<int, 8>());
    return vectors(m, 4) ? f(__nv_bfloat16(), integral_constant<int, 2>()) : f(__nv_bfloat16(), integral_constant<int, 1>());
}

// warps per token: about 64 vectors each, so that a warp has several in flight
int warps_per_token(int nvec) {
    int w = 1;
    while (w < 8 && nvec > 64 * w) w *= 2;
    return w;
}

// Tokens along x; with few tokens their rows are cut along y as well (where
// the kernel allows it), until two CTAs per SM have work.
dim3 row_grid(const RowArgs& a, int wpt, bool split, int num_sms) {
    const int per = kRowThreads / 32 / wpt;
    const int64_t x = (a.tokens + per - 1) / per;
    const int64_t most = (a.nvec + 32 * wpt - 1) / (32 * wpt);
    const int64_t y = split ? std::min(most, std::max<int64_t>(1, 2 * num_sms / x)) : 1;
    return dim3((unsigned)x, (unsigned)y);
}

template <typename T, int VEC>
cudaError_t gather_t(const MoePlanArgs& p, const MoeRowsArgs& m, bool dependent, cudaStream_t st) {
    const RowArgs a = row_args(p, m, VEC);
    const int w = warps_per_token(a.nvec);
    const dim3 g = row_grid(a, w, true, p.num_sms);
    switch (w) {
    case 1: return launch_k(dependent, moe_gather_kernel<T, VEC, 1>, g, kRowThreads, 0, st, a);
    case 2: return launch_k(dependent, moe_gather_kernel<T, VEC, 2>, g, kRowThreads, 0, st, a);
    case 4: return launch_k(dependent, moe_gather_kernel<T, VEC, 4>, g, kRowThreads, 0, st, a);
    default: return launch_k(dependent, moe_gather_kernel<T, VEC, 8>, g, kRowThreads, 0, st, a);
    }
}

template <typename T, int VEC, bool WEIGHTED>
cudaError_t combine_w(const MoePlanArgs& p, const RowArgs& a, cudaStream_t st) {
    const int w = warps_per_token(a.nvec);
    const dim3 g = row_grid(a, w, true, p.num_sms);
    switch (w) {
    case 1: moe_combine_kernel<T, VEC, 1, WEIGHTED><<<g, kRowThreads, 0, st>>>(a); break;
    case 2: moe_combine_kernel<T, VEC, 2, WEIGHTED><<<g, kRowThreads, 0, st>>>(a); break;
    case 4: moe_combine_kernel<T, VEC, 4, WEIGHTED><<<g, kRowThreads, 0, st>>>(a); break;
    default: moe_combine_kernel<T, VEC, 8, WEIGHTED><<<g, kRowThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}
template <typename T, int VEC>
cudaError_t combine_t(const MoePlanArgs& p, const MoeRowsArgs& m, cudaStream_t st) {
    const RowArgs a = row_args(p, m, VEC);
    return m.weights ? combine_w<T, VEC, true>(p, a, st) : combine_w<T, VEC, false>(p, a, st);
}

template <typename T, int VEC, bool DOT>
cudaError_t backward_d(const MoePlanArgs& p, const RowArgs& a, cudaStream_t st) {
    const int w = warps_per_token(a.nvec);
    const dim3 g = row_grid(a, w, !DOT, p.num_sms);         // a dot product stays in one CTA
    switch (w) {
    case 1: moe_combine_backward_kernel<T, VEC, 1, DOT><<<g, kRowThreads, 0, st>>>(a); break;
    case 2: moe_combine_backward_kernel<T, VEC, 2, DOT><<<g, kRowThreads, 0, st>>>(a); break;
    case 4: moe_combine_backward_kernel<T, VEC, 4, DOT><<<g, kRowThreads, 0, st>>>(a); break;
    default: moe_combine_backward_kernel<T, VEC, 8, DOT><<<g, kRowThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}
template <typename T, int VEC>
cudaError_t backward_t(const MoePlanArgs& p, const MoeRowsArgs& m, cudaStream_t st) {
    const RowArgs a = row_args(p, m, VEC);
    return m.dweights ? backward_d<T, VEC, true>(p, a, st) : backward_d<T, VEC, false>(p, a, st);
}

template <typename T, int VEC, int THREADS>
cudaError_t small_n(const MoePlanArgs& p, const SortArgs& s, const MoeRowsArgs* m, cudaStream_t st) {
    RowArgs a{};
    int pieces = 1;
    int64_t ctas = 1;
    if (m) {
        a = row_args(p, *m, VEC);
        // a token's row in pieces of at least 128 vectors, about as many pieces as there is room for
        constexpr int PER = THREADS / 128;
        const int64_t room = (int64_t)p.num_sms * PER;
        pieces = (int)std::max<int64_t>(1, std::min<int64_t>((a.nvec + 127) / 128, room / p.tokens));
        ctas = std::min<int64_t>(p.num_sms, (p.tokens * pieces + PER - 1) / PER);
    }
    const size_t smem = (THREADS + s.experts) * sizeof(int32_t) +
                        (size_t)((s.slots + 31) / 32) * s.experts * sizeof(uint16_t);
    if (smem > 40 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(moe_small_kernel<T, VEC, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             80 * 1024);
        if (e != cudaSuccess) return e;
    }
    moe_small_kernel<T, VEC, THREADS><<<(unsigned)ctas, THREADS, smem, st>>>(s, a, pieces);
    return cudaGetLastError();
}
template <typename T, int VEC>
cudaError_t small_t(const MoePlanArgs& p, const SortArgs& s, const MoeRowsArgs* m, cudaStream_t st) {
    constexpr int FEW = 256;           // a smaller CTA starts and synchronizes sooner
    return s.slots <= FEW && s.experts <= FEW ? small_n<T, VEC, FEW>(p, s, m, st) : small_n<T, VEC, kSortThreads>(p, s, m, st);
}

// more than kSortThreads slots: the plan by one cluster, or in two launches
cudaError_t sort_large(const SortArgs& s, cudaStream_t st) {
    const size_t smem = 2 * s.experts * sizeof(int32_t) + (size_t)32 * s.experts * sizeof(uint16_t);
    const auto allow = [&](const void* k) {
        return smem > 40 * 1024 ? cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 80 * 1024)
                                : cudaSuccess;
    };
    if (s.slots <= kClusterSlots) {
        cudaError_t e = allow(reinterpret_cast<const void*>(moe_cluster_sort_kernel));
        if (e != cudaSuccess) return e;
        moe_cluster_sort_kernel<<<kCluster, kSortThreads, smem, st>>>(s);
        return cudaGetLastError();
    }
    cudaError_t e = allow(reinterpret_cast<const void*>(moe_place_kernel));
    if (e != cudaSuccess) return e;
    moe_count_kernel<<<s.chunks, kSortThreads, s.experts * sizeof(int32_t), st>>>(s);
    return launch_k(true, moe_place_kernel, dim3(s.chunks), kSortThreads, smem, st, s);
}

}  // namespace

size_t moe_sort_workspace(int64_t tokens, int k, int num_experts) {
    const int64_t slots = tokens * k, chunk = sort_chunk(slots);
    return slots <= kSortThreads ? 0 : (size_t)((slots + chunk - 1) / chunk) * num_experts * sizeof(int32_t);
}

cudaError_t run_moe_sort(const MoePlanArgs& p, const void* ids, bool ids64, void* ws, cudaStream_t st) {
    const SortArgs s = sort_args(p, ids, ids64, ws);
    return s.slots <= kSortThreads ? small_t<float, 4>(p, s, nullptr, st) : sort_large(s, st);
}

cudaError_t run_moe_dispatch(const MoePlanArgs& p, const MoeRowsArgs& m, const void* ids, bool ids64, void* ws,
                             cudaStream_t st) {
    const SortArgs s = sort_args(p, ids, ids64, ws);
    if (s.slots <= kSortThreads)
        return by_vector(m, [&](auto t, auto v) { return small_t<decltype(t), decltype(v)::value>(p, s, &m, st); });
    cudaError_t e = sort_large(s, st);
    if (e != cudaSuccess) return e;
    return by_vector(m, [&](auto t, auto v) { return gather_t<decltype(t), decltype(v)::value>(p, m, true, st); });
}

cudaError_t run_moe_gather(const MoePlanArgs& p, const MoeRowsArgs& m, cudaStream_t st) {
    return by_vector(m, [&](auto t, auto v) { return gather_t<decltype(t), decltype(v)::value>(p, m, false, st); });
}
cudaError_t run_moe_combine(const MoePlanArgs& p, const MoeRowsArgs& m, cudaStream_t st) {
    return by_vector(m, [&](auto t, auto v) { return combine_t<decltype(t), decltype(v)::value>(p, m, st); });
}
cudaError_t run_moe_combine_backward(const MoePlanArgs& p, const MoeRowsArgs& m, cudaStream_t st) {
    return by_vector(m, [&](auto t, auto v) { return backward_t<decltype(t), decltype(v)::value>(p, m, st); });
}

}  // namespace bsq
