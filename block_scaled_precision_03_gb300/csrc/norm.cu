// Layer norm, forward and backward.
//
// Forward, per row: mean = sum x / C, var = sum (x - mean)^2 / C,
// rstd = 1 / sqrt(var + eps), y = (x - mean) rstd w + b.  The variance is
// taken of the centred values, so a large mean costs no precision.
// Backward, with xh = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum(g) / C - xh sum(g xh) / C),
//   dw = sum over the rows of dy xh, db = sum over the rows of dy.
//
// Both are bound by memory.  A group of threads owns a row and holds it in
// registers as packed 16-byte vectors (elements where rows are not aligned),
// so the input is read once; the grid is persistent, so weight, bias and the
// column sums of the backward pass stay in registers over all rows of a
// group, and the next row is loaded before the current one is worked on.
// The column sums leave as one partial row per CTA, which a second kernel
// (its programmatic dependent) adds up in a fixed order.  Rows too wide for a
// group's registers take kernels that read them again from cache.
#include <algorithm>
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace bsq {
namespace {

constexpr int kMaxThreads = 512;       // of a row's group: 128 registers each
constexpr int kMinThreads = 128;       // of a CTA
constexpr int kMaxParts = 608;         // partial rows of the column sums: 4 CTAs on each of 152 SMs
constexpr int kWide = 512;             // threads of the kernels for wide rows
constexpr int kWideParts = 128;

__device__ __forceinline__ float param(const void* p, int bf16, int64_t c) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]) : static_cast<const float*>(p)[c];
}

// Sum over a row's group of `tpr` threads, the same bits in every thread.
// part: one float2 per warp of the CTA, not the one of the group's previous
// sum (its readers may still be at it).
__device__ __forceinline__ float2 group_sum(float2 v, int tpr, float2* part) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
    }
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, wpr = tpr >> 5, g = warp / wpr;
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    asm volatile("bar.sync %0, %1;" :: "r"(g + 1), "r"(tpr) : "memory");
    float2 s = make_float2(0.0f, 0.0f);
    for (int w = 0; w < wpr; w++) {
        const float2 u = part[g * wpr + w];
        s.x += u.x;
        s.y += u.y;
    }
    return s;
}

// A row's vectors of one thread: v = at + i * tpr
template <typename T, int VEC, int NV>
struct Row {
    Pack<T, VEC> p[NV];
    __device__ __forceinline__ void load(const T* row, int at, int tpr, int nvec) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            p[i].zero();
            if (at + i * tpr < nvec) p[i].load(row + (int64_t)(at + i * tpr) * VEC);
        }
    }
};

template <int VEC, int NV>
__device__ __forceinline__ void load_params(float (&f)[NV][VEC], const void* p, int bf16, float none, int at, int tpr,
                                            int nvec) {
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < VEC; e++)
            f[i][e] = p && at + i * tpr < nvec ? param(p, bf16, (int64_t)(at + i * tpr) * VEC + e) : none;
}

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormArgs a, int tpr) {
    __shared__ float2 part[2][kMaxThreads / 32];
    const int g = threadIdx.x / tpr, at = threadIdx.x % tpr, nvec = (int)(a.cols / VEC);
    const int64_t step = (int64_t)gridDim.x * (blockDim.x / tpr);
    int64_t r = (int64_t)blockIdx.x * (blockDim.x / tpr) + g;
    if (r >= a.rows) return;
    const float C = (float)a.cols;
    Row<T, VEC, NV> next;
    next.load(static_cast<const T*>(a.x) + r * a.ldx, at, tpr, nvec);
    float w[NV][VEC], b[NV][VEC];
    load_params<VEC, NV>(w, a.weight, a.param_bf16, 1.0f, at, tpr, nvec);
    load_params<VEC, NV>(b, a.bias, a.param_bf16, 0.0f, at, tpr, nvec);
    for (; r < a.rows; r += step) {
        const Row<T, VEC, NV> x = next;
        if (r + step < a.rows) next.load(static_cast<const T*>(a.x) + (r + step) * a.ldx, at, tpr, nvec);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float f[VEC];
            x.p[i].unpack(f);
#pragma unroll
            for (int e = 0; e < VEC; e++) s += f[e];
        }
        const float mean = group_sum(make_float2(s, 0.0f), tpr, part[0]).x / C;
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (at + i * tpr >= nvec) continue;
            float f[VEC];
            x.p[i].unpack(f);
#pragma unroll
            for (int e = 0; e < VEC; e++) s = fmaf(f[e] - mean, f[e] - mean, s);
        }
        const float rstd = 1.0f / sqrtf(group_sum(make_float2(s, 0.0f), tpr, part[1]).x / C + a.eps);
        T* y = static_cast<T*>(a.y) + r * a.ldy;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (at + i * tpr >= nvec) continue;
            float f[VEC];
            x.p[i].unpack(f);
#pragma unroll
            for (int e = 0; e < VEC; e++) f[e] = (f[e] - mean) * rstd * w[i][e] + b[i][e];
            Pack<T, VEC> o;
            o.pack(f);
            o.store(y + (int64_t)(at + i * tpr) * VEC);
        }
        if (at == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

// COLS: also the column sums, one partial row [2][cols] per CTA
template <typename T, int VEC, int NV, bool PREFETCH, bool COLS>
__global__ void __launch_bounds__(kMaxThreads) norm_backward_kernel(const NormArgs a, int tpr) {
    __shared__ float2 part[2][kMaxThreads / 32];
    extern __shared__ float merged[];              // [groups - 1][2][cols]
    const int groups = blockDim.x / tpr, g = threadIdx.x / tpr, at = threadIdx.x % tpr, nvec = (int)(a.cols / VEC);
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t r = (int64_t)blockIdx.x * groups + g;
    const float C = (float)a.cols;
    const T* X = static_cast<const T*>(a.x);
    const T* DY = static_cast<const T*>(a.dy);
    Row<T, VEC, NV> nx, nd;
    float nmean = 0.0f, nrstd = 0.0f;
    auto fetch = [&](int64_t row) {
        nx.load(X + row * a.ldx, at, tpr, nvec);
        nd.load(DY + row * a.ld_dy, at, tpr, nvec);
        nmean = a.mean[row];
        nrstd = a.rstd[row];
    };
    if (PREFETCH && r < a.rows) fetch(r);
    float w[NV][VEC];
    load_params<VEC, NV>(w, a.weight, a.param_bf16, 1.0f, at, tpr, nvec);
    float dw[NV][VEC] = {}, db[NV][VEC] = {};
    for (int n = 0; r < a.rows; r += step, n ^= 1) {
        if (!PREFETCH) fetch(r);
        const Row<T, VEC, NV> x = nx, d = nd;
        const float mean = nmean, rstd = nrstd;
        if (PREFETCH && r + step < a.rows) fetch(r + step);
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (at + i * tpr >= nvec) continue;
            float fx[VEC], fd[VEC];
            x.p[i].unpack(fx);
            d.p[i].unpack(fd);
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                const float xh = (fx[e] - mean) * rstd, gr = fd[e] * w[i][e];
                s.x += gr;
                s.y = fmaf(gr, xh, s.y);
                if (COLS) {
                    dw[i][e] = fmaf(fd[e], xh, dw[i][e]);
                    db[i][e] += fd[e];
                }
            }
        }
        s = group_sum(s, tpr, part[n]);
        s.x /= C;
        s.y /= C;
        T* dx = static_cast<T*>(a.y) + r * a.ldy;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (at + i * tpr >= nvec) continue;
            float fx[VEC], fd[VEC];
            x.p[i].unpack(fx);
            d.p[i].unpack(fd);
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                const float xh = (fx[e] - mean) * rstd;
                fd[e] = rstd * (fd[e] * w[i][e] - s.x - xh * s.y);
            }
            Pack<T, VEC> o;
            o.pack(fd);
            o.store(dx + (int64_t)(at + i * tpr) * VEC);
        }
    }
    if (!COLS) return;
    pdl_launch_dependents();
    // the CTA's groups meet in shared memory; group 0 adds them in order and writes the partial row
    const int64_t c0 = a.cols;
    if (g > 0) {
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (at + i * tpr < nvec)
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    const int64_t c = (int64_t)(at + i * tpr) * VEC + e;
                    merged[(g - 1) * 2 * c0 + c] = dw[i][e];
                    merged[((g - 1) * 2 + 1) * c0 + c] = db[i][e];
                }
    }
    if (groups > 1) __syncthreads();
    if (g > 0) return;
    float* out = a.ws + (int64_t)blockIdx.x * 2 * c0;
#pragma unroll
    for (int i = 0; i < NV; i++)
        if (at + i * tpr < nvec)
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                const int64_t c = (int64_t)(at + i * tpr) * VEC + e;
                for (int k = 1; k < groups; k++) {
                    dw[i][e] += merged[(k - 1) * 2 * c0 + c];
                    db[i][e] += merged[((k - 1) * 2 + 1) * c0 + c];
                }
                out[c] = dw[i][e];
                out[c0 + c] = db[i][e];
            }
}

// Adds the partial rows: 32 columns a CTA, the parts dealt to 32 threads each
// (blockIdx.y: 0 dweight, 1 dbias).
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* ws, int parts, int64_t cols, float* dweight,
                                                           float* dbias) {
    __shared__ float sum[32][33];
    float* out = blockIdx.y ? dbias : dweight;
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    pdl_wait();
    if (!out) return;
    float s = 0.0f;
    if (c < cols)
#pragma unroll 4
        for (int i = g; i < parts; i += 32) s += ws[((int64_t)i * 2 + blockIdx.y) * cols + c];
    sum[g][lane] = s;
    __syncthreads();
    s = sum[lane][g];                              // warp g: the parts of column g
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const int64_t col = (int64_t)blockIdx.x * 32 + g;
    if (lane == 0 && col < cols) out[col] = s;
}

// ------------------------------------------------------------------ wide rows
__device__ __forceinline__ float2 block_sum(float2 v) {
    __shared__ float2 part[kWide / 32];
    __syncthreads();
    return group_sum(v, kWide, part);
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kWide) norm_wide_kernel(const NormArgs a) {
    const int64_t r = blockIdx.x, n = a.cols / VEC;
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    T* y = static_cast<T*>(a.y) + r * a.ldy;
    const float C = (float)a.cols;
    float s = 0.0f;
#pragma unroll 4
    for (int64_t v = threadIdx.x; v < n; v += kWide) {
        Pack<T, VEC> p;
        float f[VEC];
        p.load(x + v * VEC);
        p.unpack(f);
#pragma unroll
        for (int e = 0; e < VEC; e++) s += f[e];
    }
    const float mean = block_sum(make_float2(s, 0.0f)).x / C;
    s = 0.0f;
#pragma unroll 4
    for (int64_t v = threadIdx.x; v < n; v += kWide) {
        Pack<T, VEC> p;
        float f[VEC];
        p.load(x + v * VEC);
        p.unpack(f);
#pragma unroll
        for (int e = 0; e < VEC; e++) s = fmaf(f[e] - mean, f[e] - mean, s);
    }
    const float rstd = 1.0f / sqrtf(block_sum(make_float2(s, 0.0f)).x / C + a.eps);
#pragma unroll 2
    for (int64_t v = threadIdx.x; v < n; v += kWide) {
        Pack<T, VEC> p;
        float f[VEC];
        p.load(x + v * VEC);
        p.unpack(f);
#pragma unroll
        for (int e = 0; e < VEC; e++) {
            const float w = a.weight ? param(a.weight, a.param_bf16, v * VEC + e) : 1.0f;
            const float b = a.bias ? param(a.bias, a.param_bf16, v * VEC + e) : 0.0f;
            f[e] = (f[e] - mean) * rstd * w + b;
        }
        p.pack(f);
        p.store(y + v * VEC);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
}

// column sums of one group of rows (blockIdx.y), VEC columns a thread
template <typename T, int VEC>
__global__ void __launch_bounds__(128) norm_columns_kernel(const NormArgs a) {
    const int64_t c = ((int64_t)blockIdx.x * 128 + threadIdx.x) * VEC;
    if (c >= a.cols) return;
    const int64_t per = (a.rows + gridDim.y - 1) / gridDim.y;
    const int64_t lo = blockIdx.y * per, hi = min(a.rows, lo + per);
    float dw[VEC] = {}, db[VEC] = {};
#pragma unroll 4
    for (int64_t r = lo; r < hi; r++) {
        Pack<T, VEC> d, x;
        float fd[VEC], fx[VEC];
        d.load(static_cast<const T*>(a.dy) + r * a.ld_dy + c);
        x.load(static_cast<const T*>(a.x) + r * a.ldx + c);
        d.unpack(fd);
        x.unpack(fx);
        const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
        for (int e = 0; e < VEC; e++) {
            dw[e] = fmaf(fd[e], (fx[e] - mean) * rstd, dw[e]);
            db[e] += fd[e];
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; e++) {
        a.ws[((int64_t)blockIdx.y * 2) * a.cols + c + e] = dw[e];
        a.ws[((int64_t)blockIdx.y * 2 + 1) * a.cols + c + e] = db[e];
    }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kWide) norm_wide_dx_kernel(const NormArgs a) {
    const int64_t r = blockIdx.x, n = a.cols / VEC;
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.ld_dy;
    T* dx = static_cast<T*>(a.y) + r * a.ldy;
    const float mean = a.mean[r], rstd = a.rstd[r], C = (float)a.cols;
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll 2
    for (int64_t v = threadIdx.x; v < n; v += kWide) {
        Pack<T, VEC> d, p;
        float fd[VEC], fx[VEC];
        d.load(dy + v * VEC);
        p.load(x + v * VEC);
        d.unpack(fd);
        p.unpack(fx);
#pragma unroll
        for (int e = 0; e < VEC; e++) {
            const float g = fd[e] * (a.weight ? param(a.weight, a.param_bf16, v * VEC + e) : 1.0f);
            s.x += g;
            s.y = fmaf(g, (fx[e] - mean) * rstd, s.y);
        }
    }
    s = block_sum(s);
    s.x /= C;
    s.y /= C;
#pragma unroll 2
    for (int64_t v = threadIdx.x; v < n; v += kWide) {
        Pack<T, VEC> d, p;
        float fd[VEC], fx[VEC];
        d.load(dy + v * VEC);
        p.load(x + v * VEC);
        d.unpack(fd);
        p.unpack(fx);
#pragma unroll
        for (int e = 0; e < VEC; e++) {
            const float w = a.weight ? param(a.weight, a.param_bf16, v * VEC + e) : 1.0f;
            fd[e] = rstd * (fd[e] * w - s.x - (fx[e] - mean) * rstd * s.y);
        }
        d.pack(fd);
        d.store(dx + v * VEC);
    }
}

// ------------------------------------------------------------------- launches
// Threads of a row's group, of a CTA, and CTAs, for NV vectors a thread.
struct Shape {
    int tpr, threads, groups;
    unsigned ctas;
};
template <typename K>
Shape shape(K kernel, const NormArgs& a, int vec, int nv, size_t smem_per_group, int per_sm) {
    const int64_t nvec = a.cols / vec;
    Shape s;
    s.tpr = (int)((nvec + 32 * nv - 1) / (32 * nv)) * 32;
    if (s.tpr < kMinThreads) {                     // several rows a CTA
        int t = 32;
        while (t < s.tpr) t *= 2;
        s.tpr = t;
        s.threads = kMinThreads;
    } else {
        s.threads = s.tpr;
    }
    s.groups = s.threads / s.tpr;
    int occ = 1;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, s.threads, smem_per_group * (s.groups - 1)) !=
            cudaSuccess || occ < 1)
        occ = 1;
    const int64_t most = (int64_t)a.num_sms * std::min(occ, per_sm), want = (a.rows + s.groups - 1) / s.groups;
    s.ctas = (unsigned)std::min(most, want);
    return s;
}

template <typename T, int VEC, int NV>
cudaError_t forward(const NormArgs& a, cudaStream_t st) {
    const Shape s = shape(norm_kernel<T, VEC, NV>, a, VEC, NV, 0, 16);
    norm_kernel<T, VEC, NV><<<s.ctas, s.threads, 0, st>>>(a, s.tpr);
    return cudaGetLastError();
}

template <typename T, int VEC, int NV, bool PREFETCH>
cudaError_t backward(const NormArgs& a, cudaStream_t st) {
    if (!a.dweight && !a.dbias) {
        const Shape s = shape(norm_backward_kernel<T, VEC, NV, PREFETCH, false>, a, VEC, NV, 0, 16);
        norm_backward_kernel<T, VEC, NV, PREFETCH, false><<<s.ctas, s.threads, 0, st>>>(a, s.tpr);
        return cudaGetLastError();
    }
    const size_t per = 2 * a.cols * sizeof(float);
    Shape s = shape(norm_backward_kernel<T, VEC, NV, PREFETCH, true>, a, VEC, NV, per, 4);
    s.ctas = std::min<unsigned>(s.ctas, kMaxParts);
    norm_backward_kernel<T, VEC, NV, PREFETCH, true><<<s.ctas, s.threads, per * (s.groups - 1), st>>>(a, s.tpr);
    return launch_k(true, norm_reduce_kernel, dim3((unsigned)((a.cols + 31) / 32), 2), 1024, 0, st, a.ws, (int)s.ctas,
                    a.cols, a.dweight, a.dbias);
}

template <typename T, int VEC>
cudaError_t forward_wide(const NormArgs& a, cudaStream_t st) {
    norm_wide_kernel<T, VEC><<<(unsigned)a.rows, kWide, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t backward_wide(const NormArgs& a, cudaStream_t st) {
    if (a.dweight || a.dbias) {
        const int groups = (int)std::min<int64_t>(a.rows, kWideParts);
        norm_columns_kernel<T, VEC><<<dim3((unsigned)((a.cols / VEC + 127) / 128), groups), 128, 0, st>>>(a);
        norm_reduce_kernel<<<dim3((unsigned)((a.cols + 31) / 32), 2), 1024, 0, st>>>(a.ws, groups, a.cols, a.dweight,
                                                                                   a.dbias);
    }
    norm_wide_dx_kernel<T, VEC><<<(unsigned)a.rows, kWide, 0, st>>>(a);
    return cudaGetLastError();
}

bool vectors(const NormArgs& a) {
    const int e = a.bf16 ? 2 : 4;
    return rows_vec(a.x, a.ldx, a.cols, e) && rows_vec(a.y, a.ldy, a.cols, e) &&
           (!a.dy || rows_vec(a.dy, a.ld_dy, a.cols, e));
}

// Vectors a thread: one where few rows leave SMs idle (a row's latency counts),
// two where many rows stream through (fewer threads share a row's sums).
template <typename T>
cudaError_t forward_t(const NormArgs& a, cudaStream_t st) {
    constexpr int VEC = kVec<T>;
    if (vectors(a)) {
        const int64_t n = a.cols / VEC;
        if (n <= kMaxThreads && a.rows <= 2 * a.num_sms) return forward<T, VEC, 1>(a, st);
        if (n <= 2 * kMaxThreads) return forward<T, VEC, 2>(a, st);
        if (n <= 4 * kMaxThreads) return forward<T, VEC, 4>(a, st);
        return forward_wide<T, VEC>(a, st);
    }
    if (a.cols <= 4 * kMaxThreads) return forward<T, 1, 4>(a, st);
    if (a.cols <= 16 * kMaxThreads) return forward<T, 1, 16>(a, st);
    return forward_wide<T, 1>(a, st);
}

template <typename T>
cudaError_t backward_t(const NormArgs& a, cudaStream_t st) {
    constexpr int VEC = kVec<T>;
    if (vectors(a)) {
        const int64_t n = a.cols / VEC;
        if (n <= kMaxThreads && a.rows <= 2 * a.num_sms) return backward<T, VEC, 1, true>(a, st);
        if (n <= 2 * kMaxThreads) return backward<T, VEC, 2, true>(a, st);
        return backward_wide<T, VEC>(a, st);
    }
    if (a.cols <= 4 * kMaxThreads) return backward<T, 1, 4, true>(a, st);
    if (a.cols <= 16 * kMaxThreads) return backward<T, 1, 16, false>(a, st);
    return backward_wide<T, 1>(a, st);
}

}  // namespace

size_t norm_workspace(int64_t rows, int64_t cols, int) {
    return (size_t)std::min<int64_t>(rows, kMaxParts) * 2 * cols * sizeof(float);
}

cudaError_t run_layer_norm(const NormArgs& a, cudaStream_t st) {
    return a.bf16 ? forward_t<__nv_bfloat16>(a, st) : forward_t<float>(a, st);
}

cudaError_t run_layer_norm_backward(const NormArgs& a, cudaStream_t st) {
    return a.bf16 ? backward_t<__nv_bfloat16>(a, st) : backward_t<float>(a, st);
}

}  // namespace bsq
