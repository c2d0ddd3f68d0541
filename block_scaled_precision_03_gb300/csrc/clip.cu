// Global norm of many gradients, and their clipped copies:
//   norm = sqrt(sum g^2), out = g min(1, max_norm / (norm + eps)).
// The list of tensors travels in the kernel's parameters.  Tensors are cut
// into chunks of kChunk elements; CTA b takes the chunks b, b + grid, ... of
// the whole list, so every sum has a fixed order.  The first kernel leaves
// one FP64 partial sum per CTA; every CTA of the second adds all of them up
// (in the same order), which saves a launch in between.
#include "../../include/bsq.h"
#include "common.cuh"
#include "internal.h"

namespace bsq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxCtas = 1216;         // partial sums per launch: 8 CTAs on each of 152 SMs
constexpr int64_t kChunk = 16384;

template <int CAP>
struct Table {
    const void* in[CAP];
    void* out[CAP];
    int64_t n[CAP];
    int32_t first[CAP + 1];            // chunks before each tensor
    uint8_t bf16[CAP];
    int32_t count;
};
constexpr int kSmall = 32, kLarge = 1024;
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

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[kThreads / 32];
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) s += part[w];
    return s;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) square_sum_kernel(const __grid_constant__ Table<CAP> t, double* partial) {
    double sum = 0.0;
    for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        const int i = find(t, c);
        const int64_t lo = (int64_t)(c - t.first[i]) * kChunk, hi = min(t.n[i], lo + kChunk);
        float s = 0.0f;
        if (t.bf16[i]) {
            const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(t.in[i]);
            for (int64_t e = lo + threadIdx.x; e < hi; e += kThreads) {
                const float v = __bfloat162float(g[e]);
                s = fmaf(v, v, s);
            }
        } else {
            const float* g = static_cast<const float*>(t.in[i]);
            for (int64_t e = lo + threadIdx.x; e < hi; e += kThreads) s = fmaf(g[e], g[e], s);
        }
        sum += (double)s;
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__device__ __forceinline__ float total_norm(const double* partial, int parts) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) s += partial[i];
    return (float)sqrt(block_sum(s));
}

__global__ void __launch_bounds__(kThreads) norm_out_kernel(const double* partial, int parts, float* norm) {
    const float n = total_norm(partial, parts);
    if (threadIdx.x == 0) *norm = n;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<CAP> t, const double* partial,
                                                         int parts, float max_norm, float eps, float* norm) {
    const float n = total_norm(partial, parts);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    const float f = max_norm / (n + eps);
    const float factor = f > 1.0f ? 1.0f : f;           // NaN stays NaN
    for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        const int i = find(t, c);
        const int64_t lo = (int64_t)(c - t.first[i]) * kChunk, hi = min(t.n[i], lo + kChunk);
        if (t.bf16[i]) {
            const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(t.in[i]);
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(t.out[i]);
            for (int64_t e = lo + threadIdx.x; e < hi; e += kThreads)
                o[e] = __float2bfloat16_rn(__bfloat162float(g[e]) * factor);
        } else {
            const float* g = static_cast<const float*>(t.in[i]);
            float* o = static_cast<float*>(t.out[i]);
            for (int64_t e = lo + threadIdx.x; e < hi; e += kThreads) o[e] = g[e] * factor;
        }
    }
}

// Table of grads[at ...]: at most CAP non-empty tensors; returns the first
// gradient that did not fit.  (2^40 elements in 2^20 tensors, the most a call
// takes, are fewer than 2^27 chunks.)
template <int CAP>
int fill(Table<CAP>& t, const bsq_grad* grads, int at, int count, bool scale) {
    t.count = 0;
    t.first[0] = 0;
    for (; at < count; at++) {
        const bsq_grad& g = grads[at];
        if (g.n == 0) continue;
        const int64_t chunks = (g.n + kChunk - 1) / kChunk;
        if (t.count == CAP) break;
        const int i = t.count++;
        t.in[i] = g.grad;
        t.out[i] = scale ? g.out : nullptr;
        t.n[i] = g.n;
        t.bf16[i] = g.type == BSQ_OUT_BF16;
        t.first[i + 1] = t.first[i] + (int32_t)chunks;
    }
    return at;
}

template <int CAP>
cudaError_t run(const ClipArgs& a, cudaStream_t st) {
    const bsq_grad* grads = static_cast<const bsq_grad*>(a.grads);
    const int most = a.num_sms * 8 < kMaxCtas ? a.num_sms * 8 : kMaxCtas;
    Table<CAP> t;
    int parts = 0;
    for (int at = 0; at < a.count;) {
        at = fill(t, grads, at, a.count, a.scale);
        const int grid = t.first[t.count] < most ? (t.first[t.count] > 0 ? t.first[t.count] : 1) : most;
        square_sum_kernel<CAP><<<grid, kThreads, 0, st>>>(t, a.ws + parts);
        parts += grid;
    }
    if (!a.scale) {
        norm_out_kernel<<<1, kThreads, 0, st>>>(a.ws, parts, a.norm);
        return cudaGetLastError();
    }
    for (int at = 0; at < a.count;) {
        const bool first = at == 0;
        at = fill(t, grads, at, a.count, a.scale);
        const int grid = t.first[t.count] < most ? (t.first[t.count] > 0 ? t.first[t.count] : 1) : most;
        scale_kernel<CAP><<<grid, kThreads, 0, st>>>(t, a.ws, parts, a.max_norm, a.eps, first ? a.norm : nullptr);
    }
    return cudaGetLastError();
}

}  // namespace

size_t clip_workspace(int count, int) {
    return (size_t)((count + kLarge - 1) / kLarge + 1) * kMaxCtas * sizeof(double);
}

cudaError_t run_clip(const ClipArgs& a, cudaStream_t st) {
    return a.count <= kSmall ? run<kSmall>(a, st) : run<kLarge>(a, st);
}

}  // namespace bsq
