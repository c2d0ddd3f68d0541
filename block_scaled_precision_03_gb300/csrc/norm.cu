// Layer norm, forward and backward.
//
// Forward, per row: mean = sum x / C, var = sum (x - mean)^2 / C,
// rstd = 1 / sqrt(var + eps), y = (x - mean) rstd w + b.  The variance is
// taken of the centred values, so a large mean costs no precision.
// Backward, with xh = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum(g) / C - xh sum(g xh) / C),
//   dw = sum over the rows of dy xh, db = sum over the rows of dy.
// Column sums go through one partial row per CTA and a second kernel, in a
// fixed order.
#include "common.cuh"
#include "internal.h"

namespace bsq {
namespace {

constexpr int kThreads = 256;
constexpr int kPartials = 128;         // row groups of the column sums

template <typename T>
__device__ __forceinline__ float ld(const T* p);
template <>
__device__ __forceinline__ float ld(const float* p) { return *p; }
template <>
__device__ __forceinline__ float ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st(float* p, float v) { *p = v; }
__device__ __forceinline__ void st(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float param(const void* p, int bf16, int64_t c) {
    return bf16 ? ld(static_cast<const __nv_bfloat16*>(p) + c) : static_cast<const float*>(p)[c];
}

__device__ __forceinline__ float block_sum(float v) {
    __shared__ float part[kThreads / 32];
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) s += part[w];
    return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_kernel(const NormArgs a) {
    const int64_t r = blockIdx.x, C = a.cols;
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    T* y = static_cast<T*>(a.y) + r * a.ldy;
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < C; c += kThreads) s += ld(x + c);
    const float mean = block_sum(s) / (float)C;
    s = 0.0f;
    for (int64_t c = threadIdx.x; c < C; c += kThreads) {
        const float d = ld(x + c) - mean;
        s = fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(block_sum(s) / (float)C + a.eps);
    for (int64_t c = threadIdx.x; c < C; c += kThreads) {
        const float w = a.weight ? param(a.weight, a.param_bf16, c) : 1.0f;
        const float b = a.bias ? param(a.bias, a.param_bf16, c) : 0.0f;
        st(y + c, (ld(x + c) - mean) * rstd * w + b);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
}

// column sums of one group of rows: partial[group][0][c] of dy xh, [1][c] of dy
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_columns_kernel(const NormArgs a) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.cols) return;
    const int64_t per = (a.rows + gridDim.y - 1) / gridDim.y;
    const int64_t lo = blockIdx.y * per, hi = min(a.rows, lo + per);
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = lo; r < hi; r++) {
        const float d = ld(static_cast<const T*>(a.dy) + r * a.ld_dy + c);
        const float xh = (ld(static_cast<const T*>(a.x) + r * a.ldx + c) - a.mean[r]) * a.rstd[r];
        dw = fmaf(d, xh, dw);
        db += d;
    }
    a.ws[((int64_t)blockIdx.y * 2) * a.cols + c] = dw;
    a.ws[((int64_t)blockIdx.y * 2 + 1) * a.cols + c] = db;
}

__global__ void __launch_bounds__(kThreads) norm_reduce_kernel(const float* ws, int groups, int64_t cols,
                                                               float* dweight, float* dbias) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= cols) return;
    float dw = 0.0f, db = 0.0f;
    for (int g = 0; g < groups; g++) {
        dw += ws[(int64_t)g * 2 * cols + c];
        db += ws[((int64_t)g * 2 + 1) * cols + c];
    }
    if (dweight) dweight[c] = dw;
    if (dbias) dbias[c] = db;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_dx_kernel(const NormArgs a) {
    const int64_t r = blockIdx.x, C = a.cols;
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.ld_dy;
    T* dx = static_cast<T*>(a.y) + r * a.ldy;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < C; c += kThreads) {
        const float w = a.weight ? param(a.weight, a.param_bf16, c) : 1.0f;
        const float g = ld(dy + c) * w;
        s1 += g;
        s2 = fmaf(g, (ld(x + c) - mean) * rstd, s2);
    }
    s1 = block_sum(s1) / (float)C;
    s2 = block_sum(s2) / (float)C;
    for (int64_t c = threadIdx.x; c < C; c += kThreads) {
        const float w = a.weight ? param(a.weight, a.param_bf16, c) : 1.0f;
        const float xh = (ld(x + c) - mean) * rstd;
        st(dx + c, rstd * (ld(dy + c) * w - s1 - xh * s2));
    }
}

template <typename T>
cudaError_t backward(const NormArgs& a, cudaStream_t stream) {
    if (a.dweight || a.dbias) {
        const int groups = (int)(a.rows < kPartials ? a.rows : kPartials);
        const unsigned blocks = (unsigned)((a.cols + kThreads - 1) / kThreads);
        norm_columns_kernel<T><<<dim3(blocks, groups), kThreads, 0, stream>>>(a);
        norm_reduce_kernel<<<blocks, kThreads, 0, stream>>>(a.ws, groups, a.cols, a.dweight, a.dbias);
    }
    norm_dx_kernel<T><<<(unsigned)a.rows, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t norm_workspace(int64_t rows, int64_t cols, int) {
    return (size_t)(rows < kPartials ? rows : kPartials) * 2 * cols * sizeof(float);
}

cudaError_t run_layer_norm(const NormArgs& a, cudaStream_t stream) {
    if (a.bf16) norm_kernel<__nv_bfloat16><<<(unsigned)a.rows, kThreads, 0, stream>>>(a);
    else norm_kernel<float><<<(unsigned)a.rows, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t run_layer_norm_backward(const NormArgs& a, cudaStream_t stream) {
    return a.bf16 ? backward<__nv_bfloat16>(a, stream) : backward<float>(a, stream);
}

}  // namespace bsq
