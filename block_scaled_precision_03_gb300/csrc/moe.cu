// Tokens sorted by expert and back.
//
// Slot i = t * k + j holds token t's j-th expert id.  The sort is a stable
// counting sort:
//   offsets[e]  = number of valid slots with an id below e
//   slot_row[i] = offsets[id_i] + number of valid slots before i with id_i
//   row_slot    = its inverse, -1 past the last row that holds a slot
// The gather copies each token's row to its slots' rows; the combine sums a
// token's expert rows with its routing weights (the gather's gradient with
// weights 1); the combine's gradient scales dout into the expert rows and
// takes one dot product per slot.
#include "common.cuh"
#include "internal.h"

namespace bsq {
namespace {

constexpr int kSortThreads = 1024;     // slots per step: one per thread

// Slots of one CTA: whole steps, so that at most kSortCtas CTAs cover them.
constexpr int kSortCtas = 128;
__host__ __device__ inline int64_t sort_chunk(int64_t slots) {
    const int64_t steps = (slots + kSortThreads - 1) / kSortThreads;
    return (steps + kSortCtas - 1) / kSortCtas * kSortThreads;
}

__device__ __forceinline__ int load_id(const void* ids, bool ids64, int64_t i, int experts) {
    const int64_t id = ids64 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
    return id >= 0 && id < experts ? (int)id : -1;
}

// counts[b][e]: valid slots of chunk b with expert e
__global__ void __launch_bounds__(kSortThreads) moe_count_kernel(const void* ids, bool ids64, int64_t slots,
                                                                 int64_t chunk, int experts, int32_t* counts) {
    extern __shared__ int32_t hist[];
    for (int e = threadIdx.x; e < experts; e += kSortThreads) hist[e] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * chunk, hi = min(slots, lo + chunk);
    for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads) {
        const int e = load_id(ids, ids64, i, experts);
        if (e >= 0) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += kSortThreads) counts[(int64_t)blockIdx.x * experts + e] = hist[e];
}

// Places the slots of one chunk.  Shared memory: base[experts + 1] (the next
// free row of each expert for this chunk; its last entry the total) and
// wcount[32][experts], the slots of each expert in each warp of a step.
__global__ void __launch_bounds__(kSortThreads) moe_place_kernel(const void* ids, bool ids64, int64_t slots,
                                                                 int64_t chunk, int experts, const int32_t* counts,
                                                                 int chunks, int64_t* offsets, int32_t* slot_row,
                                                                 int32_t* row_slot) {
    extern __shared__ int32_t sm[];
    int32_t* base = sm;
    uint16_t* wcount = reinterpret_cast<uint16_t*>(sm + experts + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ int32_t carry[33];
    // totals and this chunk's start within each expert, then an exclusive scan over the experts
    int32_t total = 0, before = 0;
    if (tid < experts)
        for (int b = 0; b < chunks; b++) {
            const int32_t c = counts[(int64_t)b * experts + tid];
            if (b < (int)blockIdx.x) before += c;
            total += c;
        }
    int32_t scan = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += u;
    }
    if (lane == 31) carry[warp + 1] = scan;
    if (tid == 0) carry[0] = 0;
    __syncthreads();
    if (tid == 0)
        for (int w = 1; w <= 32; w++) carry[w] += carry[w - 1];
    __syncthreads();
    const int32_t first = carry[warp] + scan - total;      // rows of the experts before this one
    if (tid < experts) {
        base[tid] = first + before;
        if (blockIdx.x == 0) offsets[tid] = first;
    }
    const int32_t all = carry[32];
    if (blockIdx.x == 0 && tid == 0) offsets[experts] = all;
    const int64_t lo = blockIdx.x * chunk, hi = min(slots, lo + chunk);
    for (int64_t i = max(lo, (int64_t)all) + tid; i < hi; i += kSortThreads) row_slot[i] = -1;
    for (int64_t s = lo; s < hi; s += kSortThreads) {
        for (int x = tid; x < 32 * experts; x += kSortThreads) wcount[x] = 0;
        __syncthreads();
        const int64_t i = s + tid;
        const int e = i < hi ? load_id(ids, ids64, i, experts) : -1;
        // slots of the same expert in this warp: the lanes before this one give its rank
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1));
        if (e >= 0 && rank == 0) wcount[warp * experts + e] = (uint16_t)__popc(same);
        __syncthreads();
        int32_t row = -1;
        if (e >= 0) {
            row = base[e] + rank;
            for (int w = 0; w < warp; w++) row += wcount[w * experts + e];
        }
        __syncthreads();
        if (tid < experts) {
            int32_t n = 0;
            for (int w = 0; w < 32; w++) n += wcount[w * experts + tid];
            base[tid] += n;
        }
        if (i < hi) {
            slot_row[i] = row;
            if (row >= 0) row_slot[row] = (int32_t)i;
        }
        __syncthreads();
    }
}

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(float v) { return v; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }

constexpr int kRowThreads = 256;

// rows[r] = src[slot / k] (times weights[slot]), 0 where row r holds no slot
template <typename T>
__global__ void __launch_bounds__(kRowThreads) moe_gather_kernel(const T* src, int64_t ld_src, T* dst, int64_t ld_dst,
                                                                 int64_t cols, int k, const float* weights,
                                                                 const int32_t* row_slot) {
    const int64_t r = blockIdx.x;
    const int32_t slot = row_slot[r];
    T* out = dst + r * ld_dst;
    if (slot < 0) {
        for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) out[c] = from_float<T>(0.0f);
        return;
    }
    const T* in = src + (int64_t)(slot / k) * ld_src;
    if (weights) {
        const float w = weights[slot];
        for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) out[c] = from_float<T>(w * to_float(in[c]));
    } else {
        for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) out[c] = in[c];
    }
}

// out[t] = sum_j weights[t, j] rows[slot_row[t, j]]
template <typename T>
__global__ void __launch_bounds__(kRowThreads) moe_combine_kernel(const T* rows, int64_t ld_rows, T* dst,
                                                                  int64_t ld_dst, int64_t cols, int k,
                                                                  const float* weights, const int32_t* slot_row) {
    const int64_t t = blockIdx.x;
    for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) {
        float acc = 0.0f;
        for (int j = 0; j < k; j++) {
            const int32_t r = slot_row[t * k + j];
            if (r < 0) continue;
            const float v = to_float(rows[r * ld_rows + c]);
            acc = weights ? fmaf(weights[t * k + j], v, acc) : acc + v;
        }
        dst[t * ld_dst + c] = from_float<T>(acc);
    }
}

// dweights[slot] = dout[slot / k] . rows[slot_row[slot]], one warp per slot
template <typename T>
__global__ void __launch_bounds__(kRowThreads) moe_dweights_kernel(const T* dout, int64_t ldd, const T* rows,
                                                                   int64_t ld_rows, int64_t cols, int64_t slots, int k,
                                                                   const int32_t* slot_row, float* dweights) {
    const int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= slots) return;
    const int32_t r = slot_row[i];
    float acc = 0.0f;
    if (r >= 0) {
        const T* a = dout + i / k * ldd;
        const T* b = rows + r * ld_rows;
        for (int64_t c = lane; c < cols; c += 32) acc = fmaf(to_float(a[c]), to_float(b[c]), acc);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
    if (lane == 0) dweights[i] = acc;
}

template <typename T>
cudaError_t gather(const MoePlanArgs& p, const MoeRowsArgs& a, cudaStream_t st) {
    moe_gather_kernel<T><<<(unsigned)(p.tokens * p.k), kRowThreads, 0, st>>>(
        static_cast<const T*>(a.src), a.ld_src, static_cast<T*>(a.dst), a.ld_dst, a.cols, p.k, a.weights, p.row_slot);
    return cudaGetLastError();
}

template <typename T>
cudaError_t combine(const MoePlanArgs& p, const MoeRowsArgs& a, cudaStream_t st) {
    moe_combine_kernel<T><<<(unsigned)p.tokens, kRowThreads, 0, st>>>(
        static_cast<const T*>(a.src), a.ld_src, static_cast<T*>(a.dst), a.ld_dst, a.cols, p.k, a.weights, p.slot_row);
    return cudaGetLastError();
}

template <typename T>
cudaError_t combine_backward(const MoePlanArgs& p, const MoeRowsArgs& a, cudaStream_t st) {
    cudaError_t e = gather<T>(p, a, st);
    if (e != cudaSuccess || !a.dweights) return e;
    const int64_t slots = p.tokens * p.k, per = kRowThreads / 32;
    moe_dweights_kernel<T><<<(unsigned)((slots + per - 1) / per), kRowThreads, 0, st>>>(
        static_cast<const T*>(a.src), a.ld_src, static_cast<const T*>(a.rows), a.ld_rows, a.cols, slots, p.k,
        p.slot_row, a.dweights);
    return cudaGetLastError();
}

}  // namespace

size_t moe_sort_workspace(int64_t tokens, int k, int num_experts) {
    const int64_t slots = tokens * k, chunk = sort_chunk(slots);
    return (size_t)((slots + chunk - 1) / chunk) * num_experts * sizeof(int32_t);
}

cudaError_t run_moe_sort(const MoePlanArgs& p, const void* ids, bool ids64, void* ws, cudaStream_t st) {
    const int64_t slots = p.tokens * p.k, chunk = sort_chunk(slots);
    const int chunks = (int)((slots + chunk - 1) / chunk), E = p.num_experts;
    int32_t* counts = static_cast<int32_t*>(ws);
    moe_count_kernel<<<chunks, kSortThreads, E * sizeof(int32_t), st>>>(ids, ids64, slots, chunk, E, counts);
    const size_t smem = (E + 1) * sizeof(int32_t) + (size_t)32 * E * sizeof(uint16_t);
    cudaError_t e = cudaFuncSetAttribute(moe_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 80 * 1024);
    if (e != cudaSuccess) return e;
    moe_place_kernel<<<chunks, kSortThreads, smem, st>>>(ids, ids64, slots, chunk, E, counts, chunks, p.offsets,
                                                         p.slot_row, p.row_slot);
    return cudaGetLastError();
}

cudaError_t run_moe_gather(const MoePlanArgs& p, const MoeRowsArgs& a, cudaStream_t st) {
    return a.bf16 ? gather<__nv_bfloat16>(p, a, st) : gather<float>(p, a, st);
}
cudaError_t run_moe_combine(const MoePlanArgs& p, const MoeRowsArgs& a, cudaStream_t st) {
    return a.bf16 ? combine<__nv_bfloat16>(p, a, st) : combine<float>(p, a, st);
}
cudaError_t run_moe_combine_backward(const MoePlanArgs& p, const MoeRowsArgs& a, cudaStream_t st) {
    return a.bf16 ? combine_backward<__nv_bfloat16>(p, a, st) : combine_backward<float>(p, a, st);
}

}  // namespace bsq
