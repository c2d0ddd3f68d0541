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
// group.  The rows ahead are copied into shared memory (cp.async, each thread
// its own vectors, so no barrier): DEPTH rows of every group in flight, about
// 100 KB per SM, what the memory's latency asks for at its rate.
// The column sums leave as one partial row per CTA, which a second kernel
// (its programmatic dependent) adds up in a fixed order.  Rows too wide for a
// group's registers take kernels that read them again from cache.
#include <algorithm>
#include <atomic>
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

// The rows ahead of a group: a ring of DEPTH slots in shared memory that each
// thread fills and reads by itself (DEPTH 0: rows whose vectors are single
// elements; the next row waits in registers instead).
template <typename T, int VEC, int NV, int DEPTH>
struct Ahead {
    Row<T, VEC, NV> next;
    uint32_t slot0;                // this thread's first vector of slot 0
    int32_t pitch;                 // bytes between its vectors
    __device__ __forceinline__ void init(void* ring) {
        slot0 = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16;
        pitch = blockDim.x * 16;
    }
    __device__ __forceinline__ void issue(const T* row, bool there, int slot, int at, int tpr, int nvec) {
        if (DEPTH == 0) {
            if (there) next.load(row, at, tpr, nvec);
        } else if (there) {
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (at + i * tpr < nvec)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                 :: "r"(slot0 + (slot * NV + i) * pitch), "l"(row + (int64_t)(at + i * tpr) * VEC) : "memory");
        }
    }
    __device__ __forceinline__ void read(Row<T, VEC, NV>& r, int slot, int at, int tpr, int nvec) {
        if (DEPTH == 0) {
            r = next;
            return;
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            r.p[i].zero();
            if (at + i * tpr < nvec) {
                uint4 u;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(slot0 + (slot * NV + i) * pitch) : "memory");
                if constexpr (VEC > 1) r.p[i].v = *reinterpret_cast<const decltype(r.p[i].v)*>(&u);
            }
        }
    }
};
__device__ __forceinline__ void ahead_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the youngest N groups of this thread have landed
template <int N>
__device__ __forceinline__ void ahead_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

template <int VEC, int NV>
__device__ __forceinline__ void load_params(float (&f)[NV][VEC], const void* p, int bf16, float none, int at, int tpr,
                                            int nvec) {
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < VEC; e++)
            f[i][e] = p && at + i * tpr < nvec ? param(p, bf16, (int64_t)(at + i * tpr) * VEC + e) : none;
}

template <typename T, int VEC, int NV, int DEPTH>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormArgs a, int tpr) {
    extern __shared__ uint4 ring[];                // [DEPTH][NV][threads]
    __shared__ float2 part[2][kMaxThreads / 32];
    constexpr int AHEAD = DEPTH == 0 ? 1 : DEPTH;
    const int g = threadIdx.x / tpr, at = threadIdx.x % tpr, nvec = (int)(a.cols / VEC);
    const int64_t step = (int64_t)gridDim.x * (blockDim.x / tpr);
    int64_t r = (int64_t)blockIdx.x * (blockDim.x / tpr) + g;
    if (r >= a.rows) return;
    const float C = (float)a.cols;
    const T* X = static_cast<const T*>(a.x);
    Ahead<T, VEC, NV, DEPTH> ahead;
    ahead.init(ring);
#pragma unroll
    for (int d = 0; d < AHEAD; d++) {
        ahead.issue(X + (r + d * step) * a.ldx, r + d * step < a.rows, d, at, tpr, nvec);
        ahead_commit();
    }
    float w[NV][VEC], b[NV][VEC];
    load_params<VEC, NV>(w, a.weight, a.param_bf16, 1.0f, at, tpr, nvec);
    load_params<VEC, NV>(b, a.bias, a.param_bf16, 0.0f, at, tpr, nvec);
    for (int slot = 0; r < a.rows; r += step, slot = slot + 1 == AHEAD ? 0 : slot + 1) {
        Row<T, VEC, NV> x;
        ahead_wait<AHEAD - 1>();
        ahead.read(x, slot, at, tpr, nvec);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float f[VEC];
            x.p[i].unpack(f);
#pragma unroll
            for (int e = 0; e < VEC; e++) s += f[e];
        }
        const float mean = group_sum(make_float2(s, 0.0f), tpr, part[0]).x / C;
        // the slot has been read (its values are summed): the row AHEAD steps on takes it
        ahead.issue(X + (r + AHEAD * step) * a.ldx, r + AHEAD * step < a.rows, slot, at, tpr, nvec);
        ahead_commit();
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
template <typename T, int VEC, int NV, int DEPTH, bool COLS>
__global__ void __launch_bounds__(kMaxThreads) norm_backward_kernel(const NormArgs a, int tpr) {
    extern __shared__ uint4 ring[];                // x and dy [DEPTH][NV][threads] each; then the sums' meeting
    __shared__ float2 part[2][kMaxThreads / 32];
    constexpr int AHEAD = DEPTH == 0 ? 1 : DEPTH;
    const int groups = blockDim.x / tpr, g = threadIdx.x / tpr, at = threadIdx.x % tpr, nvec = (int)(a.cols / VEC);
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t r = (int64_t)blockIdx.x * groups + g;
    const float C = (float)a.cols;
    const T* X = static_cast<const T*>(a.x);
    const T* DY = static_cast<const T*>(a.dy);
    Ahead<T, VEC, NV, DEPTH> ax, ad;
    ax.init(ring);
    ad.init(ring + (size_t)DEPTH * NV * blockDim.x);
    auto issue = [&](int64_t row, int slot) {
        ax.issue(X + row * a.ldx, row < a.rows, slot, at, tpr, nvec);
        ad.issue(DY + row * a.ld_dy, row < a.rows, slot, at, tpr, nvec);
        ahead_commit();
    };
#pragma unroll
    for (int d = 0; d < AHEAD; d++) issue(r + d * step, d);
    float nmean = r < a.rows ? a.mean[r] : 0.0f, nrstd = r < a.rows ? a.rstd[r] : 0.0f;
    float w[NV][VEC];
    load_params<VEC, NV>(w, a.weight, a.param_bf16, 1.0f, at, tpr, nvec);
    float dw[NV][VEC] = {}, db[NV][VEC] = {};
    for (int n = 0, slot = 0; r < a.rows; r += step, n ^= 1, slot = slot + 1 == AHEAD ? 0 : slot + 1) {
        Row<T, VEC, NV> x, d;
        ahead_wait<AHEAD - 1>();
        ax.read(x, slot, at, tpr, nvec);
        ad.read(d, slot, at, tpr, nvec);
        const float mean = nmean, rstd = nrstd;
        if (r + step < a.rows) {
            nmean = a.mean[r + step];
            nrstd = a.rstd[r + step];
        }
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
        issue(r + AHEAD * step, slot);                     // the slot has been read
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
    // the CTA's groups meet in shared memory, [groups - 1][2][cols]; group 0 adds them in order and
    // writes the partial row
    const int64_t c0 = a.cols;
    float* merged = reinterpret_cast<float*>(ring);
    ahead_wait<0>();
    if (groups > 1) __syncthreads();
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
// Threads of a row's group, of a CTA, CTAs and shared memory
struct Shape {
    int tpr, threads, groups;
    size_t smem;
    unsigned ctas;
};
template <typename K>
cudaError_t shape(Shape& s, K kernel, const NormArgs& a, int vec, int nv, int slots, bool cols, int per_sm) {
    const int64_t nvec = a.cols / vec;
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
    s.smem = (size_t)slots * nv * s.threads * 16;
    if (cols) s.smem = std::max(s.smem, (size_t)(s.groups - 1) * 2 * a.cols * sizeof(float));
    if (s.smem > 40 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
        if (e != cudaSuccess) return e;
    }
    // resident CTAs, asked once per kernel and size
    static std::atomic<uint64_t> known[kMaxThreads / 32 + 1];
    const uint64_t key = known[s.threads / 32].load(std::memory_order_relaxed);
    int occ = (int)(key >> 32);
    if (occ == 0 || (uint32_t)key != (uint32_t)s.smem) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, s.threads, s.smem) != cudaSuccess || occ < 1)
            occ = 1;
        known[s.threads / 32].store((uint64_t)occ << 32 | (uint32_t)s.smem, std::memory_order_relaxed);
    }
    const int64_t most = (int64_t)a.num_sms * std::min(occ, per_sm), want = (a.rows + s.groups - 1) / s.groups;
    s.ctas = (unsigned)std::min(most, want);
    return cudaSuccess;
}

template <typename T, int VEC, int NV, int DEPTH>
cudaError_t forward(const NormArgs& a, cudaStream_t st) {
    Shape s;
    cudaError_t e = shape(s, norm_kernel<T, VEC, NV, DEPTH>, a, VEC, NV, DEPTH, false, 16);
    if (e != cudaSuccess) return e;
    norm_kernel<T, VEC, NV, DEPTH><<<s.ctas, s.threads, s.smem, st>>>(a, s.tpr);
    return cudaGetLastError();
}

template <typename T, int VEC, int NV, int DEPTH>
cudaError_t backward(const NormArgs& a, cudaStream_t st) {
    Shape s;
    if (!a.dweight && !a.dbias) {
        cudaError_t e = shape(s, norm_backward_kernel<T, VEC, NV, DEPTH, false>, a, VEC, NV, 2 * DEPTH, false, 16);
        if (e != cudaSuccess) return e;
        norm_backward_kernel<T, VEC, NV, DEPTH, false><<<s.ctas, s.threads, s.smem, st>>>(a, s.tpr);
        return cudaGetLastError();
    }
    cudaError_t e = shape(s, norm_backward_kernel<T, VEC, NV, DEPTH, true>, a, VEC, NV, 2 * DEPTH, true, 4);
    if (e != cudaSuccess) return e;
    s.ctas = std::min<unsigned>(s.ctas, kMaxParts);
    norm_backward_kernel<T, VEC, NV, DEPTH, true><<<s.ctas, s.threads, s.smem, st>>>(a, s.tpr);
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
        if (n <= kMaxThreads && a.rows <= 2 * a.num_sms) return forward<T, VEC, 1, 2>(a, st);
        if (n <= 2 * kMaxThreads) return forward<T, VEC, 2, 4>(a, st);
        if (n <= 4 * kMaxThreads) return forward<T, VEC, 4, 2>(a, st);
        return forward_wide<T, VEC>(a, st);
    }
    if (a.cols <= 4 * kMaxThreads) return forward<T, 1, 4, 0>(a, st);
    if (a.cols <= 16 * kMaxThreads) return forward<T, 1, 16, 0>(a, st);
    return forward_wide<T, 1>(a, st);
}

template <typename T>
cudaError_t backward_t(const NormArgs& a, cudaStream_t st) {
    constexpr int VEC = kVec<T>;
    if (vectors(a)) {
        const int64_t n = a.cols / VEC;
        if (n <= kMaxThreads && a.rows <= 2 * a.num_sms) return backward<T, VEC, 1, 2>(a, st);
        if (n <= 2 * kMaxThreads) return backward<T, VEC, 2, 3>(a, st);
        return backward_wide<T, VEC>(a, st);
    }
    if (a.cols <= 4 * kMaxThreads) return backward<T, 1, 4, 0>(a, st);
    if (a.cols <= 12 * kMaxThreads) return backward<T, 1, 12, 0>(a, st);
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
