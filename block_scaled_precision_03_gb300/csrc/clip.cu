// Global norm of many gradients, and their clipped copies:
//   norm = sqrt(sum g^2), out = g min(1, max_norm / (norm + eps)).
//
// The list of tensors travels in the kernels' parameters.  Tensors are cut
// into chunks of 32 KB, eight 16-byte vectors a thread; CTA b takes the chunks
// b, b + grid, ... of the whole list, so every sum has a fixed order.  The
// first kernel leaves one FP64 partial sum per CTA; every CTA of the second,
// its programmatic dependent, loads its first chunk, waits, and adds all of
// them up in the same order, which saves a launch in between.  Bound by
// memory: the gradients are read twice and written once.  The second kernel
// walks the list backwards, so it starts with what the first left in L2.
#include <algorithm>
#include "../../include/bsq.h"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace bsq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxCtas = 1216;         // partial sums per launch: 8 CTAs on each of 152 SMs
constexpr int kVectors = 8;            // of a thread per chunk
constexpr int64_t kChunkBytes = (int64_t)kThreads * kVectors * 16;
template <typename T>
constexpr int64_t kChunk = kChunkBytes / (int64_t)sizeof(T);

template <int CAP>
struct Table {
    const void* in[CAP];
    void* out[CAP];
    int64_t n[CAP];
    int32_t first[CAP + 1];            // chunks before each tensor
    uint8_t bf16[CAP];
    int32_t count;
};
// the smallest table that holds the list travels: its bytes are copied at every launch
constexpr int kSmall = 16, kMiddle = 128, kLarge = 1024;
static_assert(sizeof(Table<kLarge>) + 64 <= 32764, "kernel parameters");

template <int CAP>
__device__ __forceinline__ int find(const Table<CAP>& t, int chunk) {
    int lo = 0, hi = t.count - 1;                       // the last tensor whose first chunk is <= chunk
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Sum over the CTA, known to warp 0.  The SM has few FP64 lanes (a warp's
// addition takes some 16 cycles of them), so one warp adds: 13 additions
// instead of the 104 of a tree in every warp.  Once per CTA.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double all[kThreads];
    all[threadIdx.x] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x < 32) {
#pragma unroll
        for (int w = 0; w < kThreads / 32; w++) s += all[w * 32 + threadIdx.x];
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    }
    return s;
}

// elements before the first 16-byte boundary
template <typename T>
__device__ __forceinline__ int64_t head_of(const T* p, int64_t n) {
    return min(n, (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int64_t)sizeof(T));
}

// A thread's share of the sum of squares of g[0, n), n <= kChunk
template <typename T>
__device__ __forceinline__ float squares(const T* g, int64_t n) {
    constexpr int VEC = kVec<T>;
    const int64_t head = head_of(g, n), nv = (n - head) / VEC;
    float s[2] = {0.0f, 0.0f};
    Pack<T, VEC> p[kVectors];
#pragma unroll
    for (int u = 0; u < kVectors; u++) {
        p[u].zero();
        if (threadIdx.x + u * kThreads < nv) p[u].load(g + head + (int64_t)(threadIdx.x + u * kThreads) * VEC);
    }
    // at most 15 + 7 elements lie outside the vectors
    const int64_t tail = head + nv * VEC;
    Pack<T, 1> e;
    e.zero();
    if (threadIdx.x < head) e.load(g + threadIdx.x);
    else if (threadIdx.x >= 32 && tail + threadIdx.x - 32 < n) e.load(g + tail + threadIdx.x - 32);
    float x[1];
    e.unpack(x);
    s[0] = x[0] * x[0];
#pragma unroll
    for (int u = 0; u < kVectors; u++) {
        float f[VEC];
        p[u].unpack(f);
#pragma unroll
        for (int i = 0; i < VEC; i++) s[i & 1] = fmaf(f[i], f[i], s[i & 1]);
    }
    return s[0] + s[1];
}

// One read of the gradients: 480 MB in 71 us, 6.8 TB/s (a copy's rate).
template <int CAP>
__global__ void __launch_bounds__(kThreads) square_sum_kernel(const __grid_constant__ Table<CAP> t, double* partial) {
    double sum = 0.0;
    for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        const int i = find(t, c);
        const int64_t at = c - t.first[i];
        if (t.bf16[i]) {
            constexpr int64_t K = kChunk<__nv_bfloat16>;
            sum += (double)squares(static_cast<const __nv_bfloat16*>(t.in[i]) + at * K, min(K, t.n[i] - at * K));
        } else {
            constexpr int64_t K = kChunk<float>;
            sum += (double)squares(static_cast<const float*>(t.in[i]) + at * K, min(K, t.n[i] - at * K));
        }
    }
    pdl_launch_dependents();
    sum = block_sum(sum);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__device__ __forceinline__ float total_norm(const double* partial, int parts) {
    double s = 0.0;
    __shared__ float norm;
    for (int i = threadIdx.x; i < parts; i += kThreads) s += partial[i];
    s = block_sum(s);
    if (threadIdx.x == 0) norm = (float)sqrt(s);
    __syncthreads();
    return norm;
}

__global__ void __launch_bounds__(kThreads) norm_out_kernel(const double* partial, int parts, float* norm) {
    pdl_wait();
    const float n = total_norm(partial, parts);
    if (threadIdx.x == 0) *norm = n;
}

// The factor, computed by a CTA when it first needs it
struct Factor {
    const double* partial;
    int parts;
    float max_norm, eps;
    float* norm;
    float value;
    bool known;
    __device__ __forceinline__ float get() {
        if (!known) {
            pdl_wait();
            const float n = total_norm(partial, parts);
            if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
            const float f = max_norm / (n + eps);
            value = f > 1.0f ? 1.0f : f;                // NaN stays NaN
            known = true;
        }
        return value;
    }
};

template <typename T>
__device__ __forceinline__ void scale_chunk(const T* g, T* o, int64_t n, Factor& factor) {
    constexpr int VEC = kVec<T>;
    if (((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(o)) & 15) != 0) {
        // input and output lie differently to 16-byte boundaries: element by element
        const float f = factor.get();
#pragma unroll 4
        for (int64_t i = threadIdx.x; i < n; i += kThreads) {
            Pack<T, 1> p;
            float x[1];
            p.load(g + i);
            p.unpack(x);
            x[0] *= f;
            p.pack(x);
            p.store(o + i);
        }
        return;
    }
    const int64_t head = head_of(g, n), nv = (n - head) / VEC, tail = head + nv * VEC;
    Pack<T, VEC> p[kVectors];
#pragma unroll
    for (int u = 0; u < kVectors; u++)
        if (threadIdx.x + u * kThreads < nv) p[u].load(g + head + (int64_t)(threadIdx.x + u * kThreads) * VEC);
    const int64_t one = threadIdx.x < head ? threadIdx.x : threadIdx.x >= 32 ? tail + threadIdx.x - 32 : n;
    Pack<T, 1> e;
    e.zero();
    if (one < n) e.load(g + one);
    const float f = factor.get();
#pragma unroll
    for (int u = 0; u < kVectors; u++) {
        if (threadIdx.x + u * kThreads >= nv) continue;
        float x[VEC];
        p[u].unpack(x);
#pragma unroll
        for (int i = 0; i < VEC; i++) x[i] *= f;
        p[u].pack(x);
        p[u].store(o + head + (int64_t)(threadIdx.x + u * kThreads) * VEC);
    }
    if (one < n) {
        float x[1];
        e.unpack(x);
        x[0] *= f;
        e.pack(x);
        e.store(o + one);
    }
}

// A second read and the write: 480 MB in 146 us, 6.6 TB/s (0.98 of a copy's rate);
// both kernels on one layer's 610 MB 281 us.  The second read finds next to nothing
// in the 129 MB of L2: there, reading forwards took 284 us, and keeping the first
// read's lines with an evict-last policy 278.  Short lists are bound by the two launches (61 tensors,
// 200003 elements: 8.2 us; one cluster that does it all in one launch took 18).
template <int CAP>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<CAP> t, Factor factor) {
    factor.known = false;
    const int chunks = t.first[t.count];
    for (int k = blockIdx.x; k < chunks; k += gridDim.x) {
        const int c = chunks - 1 - k, i = find(t, c);
        const int64_t at = c - t.first[i];
        if (t.bf16[i]) {
            constexpr int64_t K = kChunk<__nv_bfloat16>;
            scale_chunk(static_cast<const __nv_bfloat16*>(t.in[i]) + at * K, static_cast<__nv_bfloat16*>(t.out[i]) + at * K,
                        min(K, t.n[i] - at * K), factor);
        } else {
            constexpr int64_t K = kChunk<float>;
            scale_chunk(static_cast<const float*>(t.in[i]) + at * K, static_cast<float*>(t.out[i]) + at * K,
                        min(K, t.n[i] - at * K), factor);
        }
    }
    factor.get();                                       // a list without elements still has a norm
}

// Table of grads[at ...]: at most CAP non-empty tensors; returns the first
// gradient that did not fit.  (2^40 elements in 2^20 tensors, the most a call
// takes, are fewer than 2^28 chunks.)
template <int CAP>
int fill(Table<CAP>& t, const bsq_grad* grads, int at, int count, bool scale) {
    t.count = 0;
    t.first[0] = 0;
    for (; at < count; at++) {
        const bsq_grad& g = grads[at];
        if (g.n == 0) continue;
        if (t.count == CAP) break;
        const int64_t chunk = g.type == BSQ_OUT_BF16 ? kChunk<__nv_bfloat16> : kChunk<float>;
        const int i = t.count++;
        t.in[i] = g.grad;
        t.out[i] = scale ? g.out : nullptr;
        t.n[i] = g.n;
        t.bf16[i] = g.type == BSQ_OUT_BF16;
        t.first[i + 1] = t.first[i] + (int32_t)((g.n + chunk - 1) / chunk);
    }
    return at;
}

template <int CAP>
cudaError_t run(const ClipArgs& a, cudaStream_t st) {
    const bsq_grad* grads = static_cast<const bsq_grad*>(a.grads);
    const int most = std::min(a.num_sms * 8, kMaxCtas);
    Table<CAP> t;
    const auto grid = [most](const Table<CAP>& t) { return dim3((unsigned)std::max(1, std::min(t.first[t.count], most))); };
    int parts = 0, last = 0;
    cudaError_t e = cudaSuccess;
    for (int at = 0; at < a.count && e == cudaSuccess;) {
        last = at;
        at = fill(t, grads, at, a.count, a.scale);
        const dim3 g = grid(t);
        e = launch_k(false, square_sum_kernel<CAP>, g, kThreads, 0, st, t, a.ws + parts);
        parts += (int)g.x;
    }
    if (e != cudaSuccess) return e;
    if (!a.scale) return launch_k(true, norm_out_kernel, dim3(1), kThreads, 0, st, a.ws, parts, a.norm);
    Factor f{a.ws, parts, a.max_norm, a.eps, a.norm, 0.0f, false};
    // a list of one table goes again as it is; the first of several launches writes the norm
    for (int at = 0; at < a.count && e == cudaSuccess;) {
        const bool first = at == 0;
        if (last > 0) at = fill(t, grads, at, a.count, a.scale);
        else at = a.count;
        f.norm = first ? a.norm : nullptr;
        e = launch_k(first, scale_kernel<CAP>, grid(t), kThreads, 0, st, t, f);
    }
    return e;
}

}  // namespace

size_t clip_workspace(int count, int) {
    return (size_t)((count + kLarge - 1) / kLarge + 1) * kMaxCtas * sizeof(double);
}

cudaError_t run_clip(const ClipArgs& a, cudaStream_t st) {
    if (a.count <= kSmall) return run<kSmall>(a, st);
    return a.count <= kMiddle ? run<kMiddle>(a, st) : run<kLarge>(a, st);
}

}  // namespace bsq
