// Layer norm, forward and backward.
//
// Forward, per row: mean = sum x / C, var = sum (x - mean)^2 / C,
// rstd = 1 / sqrt(var + eps), y = (x - mean) rstd w + b.  The variance is
// taken of the centred values, so a large mean costs no precision.
// Backward, with xh = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum(g) / C - xh sum(g xh) / C),
//   dw = sum over the rows of dy xh, db = sum over the rows of dy.
//
// Both read a row once and hold it in registers as packed 16-byte vectors; the
// floor is memory: two passes of the matrix forward, three backward.  With one
// to four warps per scheduler, what holds the kernels above it is the
// instructions per row and the latency of its two sums, so most of the choices
// below save instructions: packed FP32 (two elements an instruction), kernels
// without tests for the usual widths, and as few threads to a row as its
// registers allow.
//
// EVEN rows start on 16-byte boundaries and hold whole vectors, in every matrix
// of the call.  Other rows are walked along the boundaries of x: whole vectors,
// and the few elements outside them one by one.
//
// Forward: a group of lanes owns a row, as few as its registers allow, and many
// independent rows per SM hide the latency of their sums.  (A block of 256
// threads per row, two barriers each, took 46 us on 8192 x 4096 whatever was
// prefetched.)
//
// Backward with column sums: a thread keeps its columns' weight and sums in
// registers over all rows of a persistent CTA; the rows ahead are copied into shared memory
// (cp.async, each thread its own vectors, so no barrier there).  Each CTA
// leaves one partial row, and a second kernel (its programmatic dependent)
// adds them up in a fixed order.  Where columns and threads do not line up
// (rows that start off 16-byte boundaries) or are too many for the registers,
// the column sums take a pass of their own.  (Whole blocks of rows for one
// CTA of 1024 threads, copied in bulk and reduced together, took 49 us instead
// of 45 on 8192 x 4096: its warps add, reduce and wait all at the same time.)
//
// Measured, BF16, of the copy rate: 8192 x 4096 forward 24.7 us (0.81), backward
// 43.1 us (0.70); FP32 8192 x 2048 26.4 and 39.4 us; 8192 x 2047 24.7 and 50.9;
// 2048 x 14336 28.7 and 57.5; one row of 7168 4.1 us (a launch).
#include <algorithm>
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace bsq {
namespace {

constexpr int kMaxThreads = 512;       // of a CTA: 128 registers each
constexpr int kCta = 128;              // of a CTA of several rows
// of many odd rows, whose weight and bias are in shared memory once a CTA: the more rows share
// them, the less a CTA spends on filling it (1704 x 5746: 24.6 us, 42.9 with 128)
constexpr int kOddCta = 512;
constexpr int kMaxParts = 608;         // partial rows of the column sums: 4 CTAs on each of 152 SMs
constexpr int kWide = 512;             // threads of the kernels for wide rows
constexpr int kWideParts = 128;
constexpr int kMaxOddCols = 16384;     // weight and bias in shared memory

__device__ __forceinline__ float param(const void* p, int bf16, int64_t c) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]) : static_cast<const float*>(p)[c];
}
// VEC parameters from column c.  The loads are volatile: they do not change
// from row to row, and the compiler would otherwise keep a whole row's worth of
// them in registers (NV 16 spilled 1.3 KB); they come from L1.
template <int VEC>
__device__ __forceinline__ void params(float (&f)[VEC], const void* p, int bf16, float none, int64_t c) {
    if (!p) {
#pragma unroll
        for (int e = 0; e < VEC; e++) f[e] = none;
    } else if (!bf16 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4)
            asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(f[e]), "=f"(f[e + 1]), "=f"(f[e + 2]), "=f"(f[e + 3])
                         : "l"(static_cast<const float*>(p) + c + e));
    } else if (VEC == 8 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        uint32_t w[4];
        asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(static_cast<const __nv_bfloat16*>(p) + c));
#pragma unroll
        for (int e = 0; e < VEC; e++) f[e] = e & 1 ? bf16hi(w[(e >> 1) & 3]) : bf16lo(w[(e >> 1) & 3]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e++) f[e] = param(p, bf16, c + e);
    }
}

// A row's group of `tpr` threads (a power of two below 32, or whole warps) and
// where its warps' sums meet in shared memory: `part` holds [2][N][kPart]
// floats, a group's warps side by side from a multiple of 4, zero where it has
// none.  (At most 32: a CTA is one group of up to 16 warps, or 512 threads in
// groups of 2 warps or more.)
constexpr int kPart = 32;
struct Group {
    int tpr, g, at, slot, base, quads;
    __device__ __forceinline__ Group(int lanes_per_row, float* part, int floats) : tpr(lanes_per_row) {
        g = threadIdx.x / tpr;
        at = threadIdx.x - g * tpr;
        const int wpr = tpr >> 5;
        quads = (wpr + 3) >> 2;
        base = g * quads * 4;
        slot = base + (at >> 5);
        for (int i = threadIdx.x; i < floats; i += blockDim.x) part[i] = 0.0f;
        __syncthreads();
    }
};
// Sums over the group, the same bits in every thread.  `turn` alternates: the
// readers of the sum before may still be at its half of `part`.
// WARPS: the group is known to be whole warps.
template <bool WARPS = false, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], const Group& q, float* part, int turn) {
    float* mine = part + turn * N * kPart;
    if (WARPS && N == 2 && q.tpr > 32) {
        // the lanes' halves take one sum each: 5 shuffles for the two
        const bool upper = threadIdx.x & 16;
        float s = upper ? v[N - 1] : v[0];
        s += __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[N - 1], 16);
#pragma unroll
        for (int d = 8; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if ((threadIdx.x & 15) == 0) mine[(upper ? kPart : 0) + q.slot] = s;
    } else {
#pragma unroll
        for (int d = 16; d; d >>= 1)
            if (WARPS || d < q.tpr)
#pragma unroll
                for (int i = 0; i < N; i++) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
        if (q.tpr <= 32) return;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; i++) mine[i * kPart + q.slot] = v[i];
    }
    asm volatile("bar.sync %0, %1;" :: "r"(q.g + 1), "r"(q.tpr) : "memory");
    mine += q.base;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float4 t = *reinterpret_cast<const float4*>(mine + i * kPart);
        v[i] = (t.x + t.y) + (t.z + t.w);
    }
    if (q.quads > 1) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float4 t = *reinterpret_cast<const float4*>(mine + i * kPart + 4);
            v[i] += (t.x + t.y) + (t.z + t.w);
        }
        for (int k = 2; k < q.quads; k++)
#pragma unroll
            for (int i = 0; i < N; i++) {
                const float4 t = *reinterpret_cast<const float4*>(mine + i * kPart + 4 * k);
                v[i] += (t.x + t.y) + (t.z + t.w);
            }
    }
}

// Where a thread's part of a row lies.  Its vectors lie on 16-byte boundaries of x
// (whatever the other matrices do, so that the sums do not depend on them), the
// first at column `c0`, the next `step` columns further, all of them whole; the
// up to 2 VEC - 2 elements of the row outside whole vectors go to the group's
// first lanes, one each (column `edge`, -1 for none).  EVEN calls, whose rows
// start on a boundary and hold whole vectors, have none.
template <typename T, bool EVEN>
struct Part {
    static constexpr int VEC = kVec<T>;
    int shift, first, c0, step, edge;
    __device__ __forceinline__ Part(const T* row, int at, int tpr, int cols) {
        shift = EVEN ? 0 : row_shift(row);
        first = shift ? 1 : 0;                     // vector 0 holds columns -shift ...
        c0 = (first + at) * VEC - shift;
        step = tpr * VEC;
        edge = -1;
        if (!EVEN) {
            const int head = min(cols, first * VEC - shift), tail = cols - (cols - head) % VEC;
            edge = at < head ? at : tail + at - head < cols ? tail + at - head : -1;
        }
    }
    __device__ __forceinline__ int column(int i) const { return c0 + i * step; }
};

template <typename T, int NV, bool EVEN>
struct Row {
    static constexpr int VEC = kVec<T>;
    Pack<T, VEC> p[NV];
    float edge;
    // `alike`: the row lies to 16-byte boundaries as the vectors do
    __device__ __forceinline__ void load(const T* row, bool alike, const Part<T, EVEN>& at, int cols) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            p[i].zero();
            if (alike && at.column(i) + VEC <= cols) p[i].load(row + at.column(i));
        }
        if (!alike)
#pragma unroll 1
            for (int i = 0; i < NV; i++)
                if (at.column(i) + VEC <= cols) {
                    Pack<T, VEC> q;
                    load_each(q, row + at.column(i));
#pragma unroll
                    for (int k = 0; k < NV; k++)
                        if (k == i) p[k] = q;
                }
        edge = at.edge < 0 ? 0.0f : element(row, at.edge);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < NV; i++) p[i].zero();
        edge = 0.0f;
    }
    __device__ __forceinline__ static float element(const T* row, int c) {
        Pack<T, 1> e;
        float f[1];
        e.load(row + c);
        e.unpack(f);
        return f[0];
    }
    __device__ __forceinline__ static void put(T* row, int c, float v) {
        Pack<T, 1> e;
        const float f[1] = {v};
        e.pack(f);
        e.store(row + c);
    }
    __device__ __forceinline__ static void store(T* row, bool alike, int c, const F2 (&f)[VEC / 2]) {
        Pack<T, VEC> o;
        pack2(o, f);
        if (alike) o.store(row + c);
        else store_each(o, row + c);
    }
    // Between two passes over the row: the compiler may not keep the unpacked
    // values of the first for the second (twice the registers).
    __device__ __forceinline__ void again() {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            uint32_t* u = reinterpret_cast<uint32_t*>(&p[i].v);
            asm volatile("" : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]));
        }
    }
};

// Kernels of up to 2 vectors a thread run where rows are few
__host__ __device__ constexpr bool staged(int nv) { return nv > 2; }

// Weight and bias of odd rows: column c at [c % VEC][c / VEC], so that lanes
// whose columns lie VEC apart read neighbouring words.  The last word of every
// line is zero, and so is what columns outside the row find there.
// Not STAGED (a CTA has one or two rows): they are read from global memory (7 x 4692 in 8.2 us, 8.9 staged).
template <int VEC, bool STAGED>
struct OddParams {
    float* w;
    int pitch, off[VEC];
    __device__ __forceinline__ void fill(float* smem, const NormArgs& a, bool bias) {
        if (!STAGED) return;
        pitch = (int)((a.cols + VEC - 1) / VEC) + 1;
        w = smem;
        for (int i = threadIdx.x; i < (bias ? 2 : 1) * VEC * pitch; i += blockDim.x) w[i] = 0.0f;
        __syncthreads();
#pragma unroll 8
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float* at = w + c % VEC * pitch + c / VEC;
            at[0] = a.weight ? param(a.weight, a.param_bf16, c) : 1.0f;
            if (bias) at[VEC * pitch] = a.bias ? param(a.bias, a.param_bf16, c) : 0.0f;
        }
        __syncthreads();
    }
    // for a row whose vectors are shifted: where element e of vector v is, off[e] + v
    __device__ __forceinline__ void row(int shift) {
#pragma unroll
        for (int e = 0; e < VEC; e++) off[e] = ((e - shift) & (VEC - 1)) * pitch + ((e - shift) >> (VEC == 8 ? 3 : 2));
    }
    // of vector v, whose first column is c
    __device__ __forceinline__ void get(F2 (&f)[VEC / 2], const float* from, const void* p, int bf16, float none, int v, int c) const {
#pragma unroll
        for (int e = 0; e < VEC; e += 2)
            f[e / 2] = STAGED ? F2(from[off[e] + v], from[off[e + 1] + v])
                         : p ? F2(param(p, bf16, c + e), param(p, bf16, c + e + 1)) : F2(none);
    }
    __device__ __forceinline__ void weights(F2 (&f)[VEC / 2], const NormArgs& a, int v, int c) const {
        get(f, w, a.weight, a.param_bf16, 1.0f, v, c);
    }
    __device__ __forceinline__ void biases(F2 (&f)[VEC / 2], const NormArgs& a, int v, int c) const {
        get(f, w + VEC * pitch, a.bias, a.param_bf16, 0.0f, v, c);
    }
    __device__ __forceinline__ static float weight(const NormArgs& a, int c) {
        return a.weight ? param(a.weight, a.param_bf16, c) : 1.0f;
    }
    __device__ __forceinline__ static float bias(const NormArgs& a, int c) {
        return a.bias ? param(a.bias, a.param_bf16, c) : 0.0f;
    }
};

// VEC parameters from column c as pairs
template <int VEC>
__device__ __forceinline__ void params2(F2 (&f)[VEC / 2], const void* p, int bf16, float none, int64_t c) {
    float x[VEC];
    params<VEC>(x, p, bf16, none, c);
#pragma unroll
    for (int e = 0; e < VEC / 2; e++) f[e] = F2(x[2 * e], x[2 * e + 1]);
}

// Forward of odd rows and of very wide ones.  8192 x 2047 BF16: 24.7 us, 2.7 TB/s,
// of which the weight and bias, read from shared memory element by element
// because their place shifts from row to row, are the larger part.  (With a test
// per element it was 46.5 us and four times the instructions of even rows.)
template <typename T, int NV, bool EVEN>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormArgs a, int tpr) {
    constexpr int VEC = kVec<T>, H = VEC / 2;
    using R = Row<T, NV, EVEN>;
    extern __shared__ float odd_smem[];
    __shared__ __align__(16) float part[2 * kPart];
    const Group q(tpr, part, 2 * kPart);
    const int groups = blockDim.x / tpr, g = q.g, at = q.at, cols = (int)a.cols;
    const float per_col = 1.0f / (float)cols;
    OddParams<VEC, staged(NV)> odd;
    if (!EVEN) odd.fill(odd_smem, a, true);
    for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < a.rows; r0 += (int64_t)gridDim.x * groups) {
        const int64_t r = r0 + g;
        const bool live = r < a.rows;              // lanes of a warp stay together for the sums
        T* y = static_cast<T*>(a.y) + (live ? r : 0) * a.ldy;
        const T* row = static_cast<const T*>(a.x) + (live ? r : 0) * a.ldx;
        const Part<T, EVEN> mine(row, at, tpr, cols);
        const bool alike = EVEN || row_shift(y) == mine.shift;
        if (!EVEN) odd.row(mine.shift);
        R x;
        if (live) x.load(row, true, mine, cols);
        else x.zero();
        F2 sum(0.0f);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            F2 f[H];
            unpack2(x.p[i], f);
#pragma unroll
            for (int e = 0; e < H; e++) sum = sum + f[e];
        }
        float s[1] = {sum.get().x + sum.get().y + x.edge};
        group_sum(s, q, part, 0);
        const float mean = s[0] * per_col;
        const F2 minus(-mean);
        F2 sq(0.0f);
        x.again();
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (mine.column(i) + VEC > cols) continue;
            F2 f[H];
            unpack2(x.p[i], f);
#pragma unroll
            for (int e = 0; e < H; e++) {
                f[e] = f[e] + minus;
                sq = fma2(f[e], f[e], sq);
            }
        }
        s[0] = sq.get().x + sq.get().y;
        if (!EVEN && mine.edge >= 0) s[0] = fmaf(x.edge - mean, x.edge - mean, s[0]);
        group_sum(s, q, part, 1);
        const float rstd = rsqrtf(fmaf(s[0], per_col, a.eps));
        if (!live) continue;
        const F2 scale(rstd);
        x.again();
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = mine.column(i);
            if (c + VEC > cols) continue;
            F2 f[H], w[H], b[H];
            unpack2(x.p[i], f);
            if (EVEN) {
                params2<VEC>(w, a.weight, a.param_bf16, 1.0f, c);
                params2<VEC>(b, a.bias, a.param_bf16, 0.0f, c);
            } else {
                odd.weights(w, a, mine.first + at + i * tpr, c);
                odd.biases(b, a, mine.first + at + i * tpr, c);
            }
#pragma unroll
            for (int e = 0; e < H; e++) f[e] = fma2((f[e] + minus) * scale, w[e], b[e]);
            R::store(y, alike, c, f);
        }
        if (!EVEN && mine.edge >= 0)
            R::put(y, mine.edge, fmaf((x.edge - mean) * rstd, odd.weight(a, mine.edge), odd.bias(a, mine.edge)));
        if (at == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

// dx alone, a group of lanes per row as above: odd rows, after the pass for the
// column sums (8192 x 2047 BF16, both: 50.9 us; x and dy are read twice).  It runs
// beside the sum of the partial rows, which lets it start once the column pass is
// done: dx may be written over dy.
template <typename T, int NV, bool EVEN>
__global__ void __launch_bounds__(kMaxThreads) norm_dx_kernel(const NormArgs a, int tpr) {
    constexpr int VEC = kVec<T>, H = VEC / 2;
    using R = Row<T, NV, EVEN>;
    extern __shared__ float odd_smem[];
    __shared__ __align__(16) float part[2 * 2 * kPart];
    const Group q(tpr, part, 2 * 2 * kPart);
    const int groups = blockDim.x / tpr, g = q.g, at = q.at, cols = (int)a.cols;
    const float per_col = 1.0f / (float)cols;
    OddParams<VEC, staged(NV)> odd;
    if (!EVEN) odd.fill(odd_smem, a, false);
    int n = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < a.rows; r0 += (int64_t)gridDim.x * groups, n ^= 1) {
        const int64_t r = r0 + g;
        const bool live = r < a.rows;
        T* dx = static_cast<T*>(a.y) + (live ? r : 0) * a.ldy;
        const T* row = static_cast<const T*>(a.x) + (live ? r : 0) * a.ldx;
        const Part<T, EVEN> mine(row, at, tpr, cols);
        const bool alike = EVEN || row_shift(dx) == mine.shift;
        if (!EVEN) odd.row(mine.shift);
        R x, d;
        float mean = 0.0f, rstd = 0.0f;
        if (live) {
            const T* dy = static_cast<const T*>(a.dy) + r * a.ld_dy;
            x.load(row, true, mine, cols);
            d.load(dy, EVEN || row_shift(dy) == mine.shift, mine, cols);
            mean = a.mean[r];
            rstd = a.rstd[r];
        } else {
            x.zero();
            d.zero();
        }
        const F2 minus(-mean), scale(rstd);
        const auto weights = [&](F2 (&w)[H], int i) {
            if (EVEN) params2<VEC>(w, a.weight, a.param_bf16, 1.0f, mine.column(i));
            else odd.weights(w, a, mine.first + at + i * tpr, mine.column(i));
        };
        F2 s0(0.0f), s1(0.0f);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (mine.column(i) + VEC > cols) continue;
            F2 fx[H], fd[H], w[H];
            unpack2(x.p[i], fx);
            unpack2(d.p[i], fd);
            weights(w, i);
#pragma unroll
            for (int e = 0; e < H; e++) {
                const F2 gr = fd[e] * w[e];
                s0 = s0 + gr;
                s1 = fma2(gr, (fx[e] + minus) * scale, s1);
            }
        }
        float s[2] = {s0.get().x + s0.get().y, s1.get().x + s1.get().y};
        float we = 0.0f;
        if (!EVEN && mine.edge >= 0) {
            we = odd.weight(a, mine.edge);
            s[0] = fmaf(d.edge, we, s[0]);
            s[1] = fmaf(d.edge * we, (x.edge - mean) * rstd, s[1]);
        }
        group_sum(s, q, part, n);
        if (!live) continue;
        const float t0 = -(s[0] * per_col), t1 = -(s[1] * per_col);
        const F2 m0(t0), m1(t1);
        x.again();
        d.again();
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = mine.column(i);
            if (c + VEC > cols) continue;
            F2 fx[H], fd[H], w[H];
            unpack2(x.p[i], fx);
            unpack2(d.p[i], fd);
            weights(w, i);
#pragma unroll
            for (int e = 0; e < H; e++) fd[e] = fma2(fd[e], w[e], fma2((fx[e] + minus) * scale, m1, m0)) * scale;
            R::store(dx, alike, c, fd);
        }
        if (!EVEN && mine.edge >= 0)
            R::put(dx, mine.edge, fmaf(d.edge, we, fmaf((x.edge - mean) * rstd, t1, t0)) * rstd);
    }
    pdl_wait();                                    // the kernel beside which this one ran is done, too
}

__device__ __forceinline__ void ahead_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the youngest N groups of this thread have landed
template <int N>
__device__ __forceinline__ void ahead_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// Rows ahead of a CTA's groups in shared memory: a ring of slots, each
// [MATS matrices][NV][threads] of 16 bytes, that every thread fills and reads
// by itself.
template <int NV, int MATS>
struct Ring {
    uint32_t mine, pitch;
    __device__ __forceinline__ Ring(void* base)
        : mine((uint32_t)__cvta_generic_to_shared(base) + threadIdx.x * 16), pitch(blockDim.x * 16) {}
    __device__ __forceinline__ uint32_t slot(int s) const { return mine + (uint32_t)(s * MATS * NV) * pitch; }
    template <typename T>
    __device__ __forceinline__ void copy(uint32_t slot, int mat, int i, const T* src) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(slot + (mat * NV + i) * pitch), "l"(src) : "memory");
    }
    template <typename P>
    __device__ __forceinline__ void read(P& p, uint32_t slot, int mat, int i) const {
        uint4 u;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(slot + (mat * NV + i) * pitch) : "memory");
        p.v = *reinterpret_cast<const decltype(p.v)*>(&u);
    }
};

// A thread's parameters as pairs; `none` where it has no columns or there is no parameter
template <int VEC, int NV>
__device__ __forceinline__ void pair_params(F2 (&f)[NV][VEC / 2], const void* p, int bf16, float none, int at, int tpr,
                                            int nvec) {
#pragma unroll
    for (int i = 0; i < NV; i++) {
        float x[VEC];
#pragma unroll
        for (int e = 0; e < VEC; e++) x[e] = none;
        if (at + i * tpr < nvec) params<VEC>(x, p, bf16, none, (int64_t)(at + i * tpr) * VEC);
#pragma unroll
        for (int e = 0; e < VEC / 2; e++) f[i][e] = F2(x[2 * e], x[2 * e + 1]);
    }
}

// The two kernels below are bound by the instructions they issue and their
// latency (issue slots 47 and 50% busy with 4 warps a scheduler), so the usual
// widths get a version without tests: FULL says that every lane of every group
// has all its NV vectors and that groups are whole warps (each then leaves the
// loop by itself).

// Forward of EVEN rows where many stream through: weight and bias stay in
// registers.  8192 x 4096 BF16: 24.7 us, 5.4 TB/s (0.81 of a copy's rate).
template <typename T, int NV, int DEPTH, bool FULL>
__global__ void __launch_bounds__(kMaxThreads) norm_stream_kernel(const NormArgs a, int tpr) {
    constexpr int VEC = kVec<T>, H = VEC / 2;
    extern __shared__ uint4 ring_smem[];
    __shared__ __align__(16) float part[2 * kPart];
    const Group q(tpr, part, 2 * kPart);
    const int groups = blockDim.x / tpr, at = q.at, nvec = (int)(a.cols / VEC);
    const float per_col = 1.0f / (float)a.cols;
    const int64_t step = (int64_t)gridDim.x * groups;
    const Ring<NV, 1> ring(ring_smem);
    int64_t r = (int64_t)blockIdx.x * groups + q.g;
    const int64_t end = FULL ? a.rows : a.rows + q.g;      // not FULL: the CTA's groups make the same steps
    // the next row to be copied, and where this thread's part of it lies
    int64_t ra = r;
    const T* xa = static_cast<const T*>(a.x) + r * a.ldx + at * VEC;
    T* y = static_cast<T*>(a.y) + r * a.ldy + at * VEC;
    const int64_t x_step = step * a.ldx, y_step = step * a.ldy;
    const auto issue = [&](int slot) {
        const uint32_t to = ring.slot(slot);
        if (ra < a.rows)
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (FULL || at + i * tpr < nvec) ring.copy(to, 0, i, xa + i * tpr * VEC);
        ahead_commit();
        ra += step;
        xa += x_step;
    };
#pragma unroll
    for (int d = 0; d < DEPTH; d++) issue(d);
    F2 w[NV][H], b[NV][H];
    pair_params<VEC, NV>(w, a.weight, a.param_bf16, 1.0f, at, tpr, nvec);
    pair_params<VEC, NV>(b, a.bias, a.param_bf16, 0.0f, at, tpr, nvec);
    for (int slot = 0; r < end; r += step, y += y_step, slot = slot + 1 == DEPTH ? 0 : slot + 1) {
        const bool live = FULL || r < a.rows;
        ahead_wait<DEPTH - 1>();
        F2 x[NV][H], sum(0.0f);
        const uint32_t from = ring.slot(slot);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            Pack<T, VEC> p;
            if (!FULL) p.zero();
            if (FULL || (live && at + i * tpr < nvec)) ring.read(p, from, 0, i);
            unpack2(p, x[i]);
#pragma unroll
            for (int e = 0; e < H; e++) sum = sum + x[i][e];
        }
        float s[1] = {sum.get().x + sum.get().y};
        group_sum<FULL>(s, q, part, 0);
        issue(slot);                                       // the slot's values have been summed
        const float mean = s[0] * per_col;
        const F2 minus(-mean);
        F2 sq(0.0f);
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (FULL || at + i * tpr < nvec)
#pragma unroll
                for (int e = 0; e < H; e++) {
                    x[i][e] = x[i][e] + minus;
                    sq = fma2(x[i][e], x[i][e], sq);
                }
        s[0] = sq.get().x + sq.get().y;
        group_sum<FULL>(s, q, part, 1);
        const float rstd = rsqrtf(fmaf(s[0], per_col, a.eps));
        if (!live) continue;
        const F2 scale(rstd);
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (FULL || at + i * tpr < nvec) {
                F2 o[H];
#pragma unroll
                for (int e = 0; e < H; e++) o[e] = fma2(x[i][e] * scale, w[i][e], b[i][e]);
                Pack<T, VEC> p;
                pack2(p, o);
                p.store(y + i * tpr * VEC);
            }
        if (at == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

// dx and the column sums of EVEN rows.  COLS: one partial row [2][cols] per CTA.
// 8192 x 4096 BF16: 43.1 us with the sum of the partial rows (about 5 of them),
// 4.7 TB/s (0.70).  The registers of the column sums allow 16 warps per SM, and
// a row's instructions (some 330 per warp and 16 columns) take most of their time.
// Two rows ahead: three left room for one CTA fewer per SM.
template <typename T, int NV, int DEPTH, bool COLS, bool FULL>
__global__ void __launch_bounds__(kMaxThreads) norm_backward_kernel(const NormArgs a, int tpr) {
    constexpr int VEC = kVec<T>, H = VEC / 2;
    extern __shared__ uint4 ring_smem[];           // the ring; then the sums' meeting
    __shared__ __align__(16) float part[2 * 2 * kPart];
    const Group q(tpr, part, 2 * 2 * kPart);
    const int groups = blockDim.x / tpr, g = q.g, at = q.at, nvec = (int)(a.cols / VEC);
    const float per_col = 1.0f / (float)a.cols;
    const int64_t step = (int64_t)gridDim.x * groups, last = a.rows - 1;
    const Ring<NV, 2> ring(ring_smem);
    int64_t r = (int64_t)blockIdx.x * groups + g;
    const int64_t end = FULL ? a.rows : a.rows + g;
    int64_t ra = r;
    const T* xa = static_cast<const T*>(a.x) + r * a.ldx + at * VEC;
    const T* da = static_cast<const T*>(a.dy) + r * a.ld_dy + at * VEC;
    T* dx = static_cast<T*>(a.y) + r * a.ldy + at * VEC;
    const int64_t x_step = step * a.ldx, d_step = step * a.ld_dy, y_step = step * a.ldy;
    const auto issue = [&](int slot) {
        const uint32_t to = ring.slot(slot);
        if (ra < a.rows)
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (FULL || at + i * tpr < nvec) {
                    ring.copy(to, 0, i, xa + i * tpr * VEC);
                    ring.copy(to, 1, i, da + i * tpr * VEC);
                }
        ahead_commit();
        ra += step;
        xa += x_step;
        da += d_step;
    };
#pragma unroll
    for (int d = 0; d < DEPTH; d++) issue(d);
    // the next row's statistics; volatile, so that they are loaded a whole step ahead of their use
    float nmean, nrstd;
    const auto statistics = [&](int64_t row) {
        row = min(row, last);
        asm volatile("ld.global.f32 %0, [%1];" : "=f"(nmean) : "l"(a.mean + row));
        asm volatile("ld.global.f32 %0, [%1];" : "=f"(nrstd) : "l"(a.rstd + row));
    };
    statistics(r);
    F2 w[NV][H], dw[NV][H], db[NV][H];
    pair_params<VEC, NV>(w, a.weight, a.param_bf16, 1.0f, at, tpr, nvec);
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < H; e++) dw[i][e] = db[i][e] = F2(0.0f);
    for (int n = 0, slot = 0; r < end; r += step, dx += y_step, n ^= 1, slot = slot + 1 == DEPTH ? 0 : slot + 1) {
        const bool live = FULL || r < a.rows;
        ahead_wait<DEPTH - 1>();
        F2 xh[NV][H], s0(0.0f), s1(0.0f);
        Pack<T, VEC> d[NV];
        const float mean = nmean, rstd = nrstd;
        statistics(r + step);
        const F2 minus(-mean), scale(rstd);
        const uint32_t from = ring.slot(slot);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            Pack<T, VEC> x;
            if (!FULL) {
                x.zero();
                d[i].zero();                       // dy is zero outside the rows and columns
            }
            if (FULL || (live && at + i * tpr < nvec)) {
                ring.read(x, from, 0, i);
                ring.read(d[i], from, 1, i);
            }
            F2 dy[H];
            unpack2(x, xh[i]);
            unpack2(d[i], dy);
#pragma unroll
            for (int e = 0; e < H; e++) {
                xh[i][e] = (xh[i][e] + minus) * scale;
                const F2 gr = dy[e] * w[i][e];
                s0 = s0 + gr;
                s1 = fma2(gr, xh[i][e], s1);
                if (COLS && live) {
                    dw[i][e] = fma2(dy[e], xh[i][e], dw[i][e]);
                    db[i][e] = db[i][e] + dy[e];
                }
            }
        }
        float s[2] = {s0.get().x + s0.get().y, s1.get().x + s1.get().y};
        group_sum<FULL>(s, q, part, n);
        issue(slot);                                       // the slot's values have been summed
        if (!live) continue;
        const F2 m0(-(s[0] * per_col)), m1(-(s[1] * per_col));
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (FULL || at + i * tpr < nvec) {
                F2 dy[H];
                unpack2(d[i], dy);
#pragma unroll
                for (int e = 0; e < H; e++) dy[e] = fma2(dy[e], w[i][e], fma2(xh[i][e], m1, m0)) * scale;
                Pack<T, VEC> o;
                pack2(o, dy);
                o.store(dx + i * tpr * VEC);
            }
    }
    if (!COLS) return;
    pdl_launch_dependents();
    // the CTA's groups meet in shared memory, [groups - 1][2][cols]; group 0 adds them in order and
    // writes the partial row
    const int64_t c0 = a.cols;
    float* merged = reinterpret_cast<float*>(ring_smem);
    ahead_wait<0>();
    if (groups > 1) __syncthreads();
    const auto column = [&](float* f, int i, int e) { return f + (at + i * tpr) * VEC + 2 * e; };
    if (g > 0) {
        float* mine = merged + (int64_t)(g - 1) * 2 * c0;
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (at + i * tpr < nvec)
#pragma unroll
                for (int e = 0; e < H; e++) {
                    *reinterpret_cast<float2*>(column(mine, i, e)) = dw[i][e].get();
                    *reinterpret_cast<float2*>(column(mine + c0, i, e)) = db[i][e].get();
                }
    }
    if (groups > 1) __syncthreads();
    if (g > 0) return;
    float* out = a.ws + (int64_t)blockIdx.x * 2 * c0;
#pragma unroll
    for (int i = 0; i < NV; i++)
        if (at + i * tpr < nvec) {
            for (int k = 0; k < groups - 1; k++) {
                float* other = merged + (int64_t)k * 2 * c0;
#pragma unroll
                for (int e = 0; e < H; e++) {
                    const float2 x = *reinterpret_cast<const float2*>(column(other, i, e));
                    const float2 y = *reinterpret_cast<const float2*>(column(other + c0, i, e));
                    dw[i][e] = dw[i][e] + F2(x.x, x.y);
                    db[i][e] = db[i][e] + F2(y.x, y.y);
                }
            }
#pragma unroll
            for (int e = 0; e < H; e += 2) {
                const float2 x = dw[i][e].get(), x1 = dw[i][e + 1].get(), y = db[i][e].get(), y1 = db[i][e + 1].get();
                *reinterpret_cast<float4*>(column(out, i, e)) = make_float4(x.x, x.y, x1.x, x1.y);
                *reinterpret_cast<float4*>(column(out + c0, i, e)) = make_float4(y.x, y.y, y1.x, y1.y);
            }
        }
}

// The same for rows of up to 32 columns a thread (BF16, kLongCols): the column
// sums alone are 64 registers, so nothing else stays in them.  The weight lies in
// shared memory as FP32, and dx's pass reads x and dy from the ring again, whose
// slot is free only after it.  One row at a time and CTA.  2048 x 14336: 57.5 us
// (3.0 TB/s; 99.0 with the column sums in a pass of their own).
constexpr int kLongVecs = 4, kLongDepth = 2;
constexpr int64_t kLongCols = 8 * kLongVecs * kMaxThreads;
template <bool COLS>
__global__ void __launch_bounds__(kMaxThreads) norm_backward_long_kernel(const NormArgs a) {
    using T = __nv_bfloat16;
    constexpr int NV = kLongVecs, VEC = 8, H = 4;
    extern __shared__ uint4 ring_smem[];           // the ring, then the weight: [2][nvec] of four columns
    __shared__ __align__(16) float part[2 * 2 * kPart];
    const int tpr = blockDim.x, at = threadIdx.x, nvec = (int)(a.cols / VEC);
    const Group q(tpr, part, 2 * 2 * kPart);
    const float per_col = 1.0f / (float)a.cols;
    const Ring<NV, 2> ring(ring_smem);
    float4* weight = reinterpret_cast<float4*>(ring_smem + kLongDepth * 2 * NV * tpr);
    int64_t ra = blockIdx.x;
    const auto issue = [&](int slot) {
        const uint32_t to = ring.slot(slot);
        if (ra < a.rows) {
            const T* x = static_cast<const T*>(a.x) + ra * a.ldx + at * VEC;
            const T* d = static_cast<const T*>(a.dy) + ra * a.ld_dy + at * VEC;
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (at + i * tpr < nvec) {
                    ring.copy(to, 0, i, x + i * tpr * VEC);
                    ring.copy(to, 1, i, d + i * tpr * VEC);
                }
        }
        ahead_commit();
        ra += gridDim.x;
    };
#pragma unroll
    for (int d = 0; d < kLongDepth; d++) issue(d);
    for (int v = at; v < nvec; v += tpr) {         // each thread its own columns: no barrier
        float f[VEC];
        params<VEC>(f, a.weight, a.param_bf16, 1.0f, (int64_t)v * VEC);
        weight[v] = make_float4(f[0], f[1], f[2], f[3]);
        weight[nvec + v] = make_float4(f[4], f[5], f[6], f[7]);
    }
    F2 dw[NV][H], db[NV][H];
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < H; e++) dw[i][e] = db[i][e] = F2(0.0f);
    int n = 0, slot = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, n ^= 1, slot = slot + 1 == kLongDepth ? 0 : slot + 1) {
        const float mean = a.mean[r], rstd = a.rstd[r];
        const F2 minus(-mean), scale(rstd);
        const uint32_t from = ring.slot(slot);
        F2 x[H], dy[H], w[H], s0(0.0f), s1(0.0f);
        const auto read = [&](int i) {
            Pack<T, VEC> px, pd;
            ring.read(px, from, 0, i);
            ring.read(pd, from, 1, i);
            const float4 w0 = weight[at + i * tpr], w1 = weight[nvec + at + i * tpr];
            unpack2(px, x);
            unpack2(pd, dy);
            w[0] = F2(w0.x, w0.y);
            w[1] = F2(w0.z, w0.w);
            w[2] = F2(w1.x, w1.y);
            w[3] = F2(w1.z, w1.w);
#pragma unroll
            for (int e = 0; e < H; e++) x[e] = (x[e] + minus) * scale;
        };
        ahead_wait<kLongDepth - 1>();
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (at + i * tpr >= nvec) continue;
            read(i);
#pragma unroll
            for (int e = 0; e < H; e++) {
                const F2 gr = dy[e] * w[e];
                s0 = s0 + gr;
                s1 = fma2(gr, x[e], s1);
                if (COLS) {
                    dw[i][e] = fma2(dy[e], x[e], dw[i][e]);
                    db[i][e] = db[i][e] + dy[e];
                }
            }
        }
        float s[2] = {s0.get().x + s0.get().y, s1.get().x + s1.get().y};
        group_sum<true>(s, q, part, n);
        const F2 m0(-(s[0] * per_col)), m1(-(s[1] * per_col));
        T* dx = static_cast<T*>(a.y) + r * a.ldy + at * VEC;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (at + i * tpr >= nvec) continue;
            read(i);
#pragma unroll
            for (int e = 0; e < H; e++) dy[e] = fma2(dy[e], w[e], fma2(x[e], m1, m0)) * scale;
            Pack<T, VEC> o;
            pack2(o, dy);
            o.store(dx + i * tpr * VEC);
        }
        issue(slot);                               // this thread has read the slot twice
    }
    ahead_wait<0>();
    if (!COLS) return;
    pdl_launch_dependents();
    float* out = a.ws + (int64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        if (at + i * tpr >= nvec) continue;
#pragma unroll
        for (int e = 0; e < H; e += 2) {
            const float2 u = dw[i][e].get(), u1 = dw[i][e + 1].get(), v = db[i][e].get(), v1 = db[i][e + 1].get();
            float* to = out + (at + i * tpr) * VEC + 2 * e;
            *reinterpret_cast<float4*>(to) = make_float4(u.x, u.y, u1.x, u1.y);
            *reinterpret_cast<float4*>(to + a.cols) = make_float4(v.x, v.y, v1.x, v1.y);
        }
    }
}

// Adds the partial rows (10 MB of 304 CTAs at 4096 columns: about 5 us from L2):
// 32 columns a CTA, the parts dealt to 32 threads each
// (blockIdx.y: 0 dweight, 1 dbias).
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* ws, int parts, int64_t cols, float* dweight,
                                                           float* dbias) {
    __shared__ float sum[32][33];
    float* out = blockIdx.y ? dbias : dweight;
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    pdl_wait();
    pdl_launch_dependents();                       // only now: see norm_dx_kernel
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
// Rows that no group of 512 threads holds in registers: a CTA per row, read again
// for each pass (from L2, mostly).
__device__ __forceinline__ float2 block_sum(float2 v) {
    __shared__ __align__(16) float part[2 * 2 * kPart];
    __syncthreads();
    const Group q(kWide, part, 2 * 2 * kPart);
    float s[2] = {v.x, v.y};
    group_sum(s, q, part, 0);
    return make_float2(s[0], s[1]);
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

// Column sums of one group of rows (blockIdx.y), VEC columns a thread, where the
// kernels above cannot keep them: x and dy are read once more (8192 x 2047 BF16:
// 22 us of the 50.9)
template <typename T, int VEC>
__global__ void __launch_bounds__(128) norm_columns_kernel(const NormArgs a) {
    const int64_t c = ((int64_t)blockIdx.x * 128 + threadIdx.x) * VEC;
    if (c >= a.cols) return;
    const int64_t per = (a.rows + gridDim.y - 1) / gridDim.y;
    const int64_t lo = blockIdx.y * per, hi = min(a.rows, lo + per);
    float dw[VEC] = {}, db[VEC] = {};
#pragma unroll 8
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
    pdl_launch_dependents();
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
// `tpr` lanes a row; CTAs of about `cta` threads unless one row takes more.
// smem(s): bytes that a CTA of s.threads needs.
template <typename K, typename S>
cudaError_t shape(Shape& s, K kernel, const NormArgs& a, int tpr, S smem, int per_sm, int cta = kCta) {
    s.tpr = tpr;
    s.threads = tpr >= cta ? tpr : cta / tpr * tpr;
    s.groups = s.threads / tpr;
    s.smem = smem(s);
    if (s.smem > 40 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
        if (e != cudaSuccess) return e;
    }
    int occ = 1;
    if (a.rows > (int64_t)a.num_sms * s.groups) {
        cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, s.threads, s.smem);
        if (e != cudaSuccess) return e;
        occ = std::max(1, std::min(occ, per_sm));
    }
    s.ctas = (unsigned)std::min((int64_t)a.num_sms * occ, (a.rows + s.groups - 1) / s.groups);
    return cudaSuccess;
}

// Lanes for n vectors, at most nv each: a power of two (`least` or more) below a warp, else whole warps.
int lanes(int64_t n, int nv, int least = 4) {
    const int64_t want = (n + nv - 1) / nv;
    if (want > 32) return (int)((want + 31) / 32 * 32);
    int t = least;
    while (t < want) t *= 2;
    return t;
}

int row_cta(const NormArgs& a, bool even) { return even || a.rows < 4 * (int64_t)a.num_sms ? kCta : kOddCta; }
size_t odd_bytes(const NormArgs& a, int nv, bool even) {
    const int64_t vec = a.bf16 ? 8 : 4;
    return even || !staged(nv) ? 0 : (size_t)(2 * vec * ((a.cols + vec - 1) / vec + 1)) * sizeof(float);
}

template <typename T, int NV, bool EVEN>
cudaError_t forward(const NormArgs& a, int64_t n, cudaStream_t st) {
    Shape s;
    cudaError_t e = shape(s, norm_kernel<T, NV, EVEN>, a, lanes(n, NV, EVEN ? 4 : 16), [&](const Shape&) { return odd_bytes(a, NV, EVEN); }, 16, row_cta(a, EVEN));
    if (e != cudaSuccess) return e;
    norm_kernel<T, NV, EVEN><<<s.ctas, s.threads, s.smem, st>>>(a, s.tpr);
    return cudaGetLastError();
}

// every lane has nv vectors, and a row takes whole warps
bool full(int64_t n, int nv) { return n % (32 * nv) == 0; }

template <typename T, int NV, int DEPTH, bool FULL>
cudaError_t stream_f(const NormArgs& a, cudaStream_t st) {
    Shape s;
    const auto ring = [](const Shape& x) { return (size_t)DEPTH * NV * x.threads * 16; };
    cudaError_t e = shape(s, norm_stream_kernel<T, NV, DEPTH, FULL>, a, lanes(a.cols / kVec<T>, NV), ring, 16);
    if (e != cudaSuccess) return e;
    norm_stream_kernel<T, NV, DEPTH, FULL><<<s.ctas, s.threads, s.smem, st>>>(a, s.tpr);
    return cudaGetLastError();
}
template <typename T, int NV, int DEPTH>
cudaError_t stream(const NormArgs& a, cudaStream_t st) {
    return full(a.cols / kVec<T>, NV) ? stream_f<T, NV, DEPTH, true>(a, st) : stream_f<T, NV, DEPTH, false>(a, st);
}

template <typename T, int NV, bool EVEN>
cudaError_t dx_only(const NormArgs& a, int64_t n, cudaStream_t st) {
    Shape s;
    cudaError_t e = shape(s, norm_dx_kernel<T, NV, EVEN>, a, lanes(n, NV, EVEN ? 4 : 16), [&](const Shape&) { return odd_bytes(a, NV, EVEN); }, 16, row_cta(a, EVEN));
    if (e != cudaSuccess) return e;
    return launch_k(a.dweight || a.dbias, norm_dx_kernel<T, NV, EVEN>, dim3(s.ctas), (unsigned)s.threads, s.smem, st, a, s.tpr);
}

template <typename T, int NV, int DEPTH, bool FULL>
cudaError_t backward_f(const NormArgs& a, cudaStream_t st) {
    const int tpr = lanes(a.cols / kVec<T>, NV);
    const auto ring = [](const Shape& s) { return (size_t)DEPTH * 2 * NV * s.threads * 16; };
    Shape s;
    if (!a.dweight && !a.dbias) {
        cudaError_t e = shape(s, norm_backward_kernel<T, NV, DEPTH, false, FULL>, a, tpr, ring, 16);
        if (e != cudaSuccess) return e;
        norm_backward_kernel<T, NV, DEPTH, false, FULL><<<s.ctas, s.threads, s.smem, st>>>(a, s.tpr);
        return cudaGetLastError();
    }
    cudaError_t e = shape(s, norm_backward_kernel<T, NV, DEPTH, true, FULL>, a, tpr, [&](const Shape& x) {
        return std::max(ring(x), (size_t)(x.groups - 1) * 2 * a.cols * sizeof(float));
    }, 4);
    if (e != cudaSuccess) return e;
    s.ctas = std::min<unsigned>(s.ctas, kMaxParts);
    norm_backward_kernel<T, NV, DEPTH, true, FULL><<<s.ctas, s.threads, s.smem, st>>>(a, s.tpr);
    return launch_k(true, norm_reduce_kernel, dim3((unsigned)((a.cols + 31) / 32), 2), 1024, 0, st, a.ws, (int)s.ctas,
                    a.cols, a.dweight, a.dbias);
}
template <typename T, int NV, int DEPTH>
cudaError_t backward(const NormArgs& a, cudaStream_t st) {
    return full(a.cols / kVec<T>, NV) ? backward_f<T, NV, DEPTH, true>(a, st) : backward_f<T, NV, DEPTH, false>(a, st);
}

template <bool COLS>
cudaError_t backward_long_c(const NormArgs& a, cudaStream_t st) {
    const int64_t nvec = a.cols / 8;
    const int threads = lanes(nvec, kLongVecs);
    const size_t smem = (size_t)kLongDepth * 2 * kLongVecs * threads * 16 + (size_t)a.cols * 4;
    cudaError_t e = cudaFuncSetAttribute(norm_backward_long_kernel<COLS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         200 * 1024);
    if (e != cudaSuccess) return e;
    const unsigned ctas = (unsigned)std::min<int64_t>({a.num_sms, a.rows, kMaxParts});
    norm_backward_long_kernel<COLS><<<ctas, threads, smem, st>>>(a);
    if (!COLS) return cudaGetLastError();
    return launch_k(true, norm_reduce_kernel, dim3((unsigned)((a.cols + 31) / 32), 2), 1024, 0, st, a.ws, (int)ctas,
                    a.cols, a.dweight, a.dbias);
}

template <typename T, int VEC>
cudaError_t columns(const NormArgs& a, cudaStream_t st) {
    // row groups: enough CTAs for every SM to hold several, at least 8 rows each
    const int64_t blocks = (a.cols + 128 * VEC - 1) / (128 * VEC);
    const int64_t want = std::max<int64_t>(kWideParts, (int64_t)a.num_sms * 8 / blocks);
    const int groups = (int)std::max<int64_t>(1, std::min<int64_t>({want, (a.rows + 7) / 8, kMaxParts}));
    norm_columns_kernel<T, VEC><<<dim3((unsigned)blocks, groups), 128, 0, st>>>(a);
    return launch_k(true, norm_reduce_kernel, dim3((unsigned)((a.cols + 31) / 32), 2), 1024, 0, st, a.ws, groups, a.cols,
                    a.dweight, a.dbias);
}

// rows on 16-byte boundaries that hold whole vectors, in every matrix of the call
bool even_rows(const NormArgs& a) {
    const int e = a.bf16 ? 2 : 4;
    return rows_vec(a.x, a.ldx, a.cols, e) && rows_vec(a.y, a.ldy, a.cols, e) &&
           (!a.dy || rows_vec(a.dy, a.ld_dy, a.cols, e));
}

template <typename T>
cudaError_t forward_t(const NormArgs& a, cudaStream_t st) {
    const int64_t n = a.cols / kVec<T>;
    if (even_rows(a)) {
        // few rows: one or two vectors a thread and one slot ahead, for the latency of a row; many:
        // as few threads share a row's sums as the registers allow
        if (a.rows <= a.num_sms && n <= kMaxThreads) return stream<T, 1, 1>(a, st);
        if (a.rows <= a.num_sms && n <= 2 * kMaxThreads) return stream<T, 2, 1>(a, st);
        if (n <= 4 * kMaxThreads) return stream<T, 4, 2>(a, st);
        if (n <= 16 * kMaxThreads) return forward<T, 16, true>(a, n, st);
        norm_wide_kernel<T, kVec<T>><<<(unsigned)a.rows, kWide, 0, st>>>(a);
        return cudaGetLastError();
    }
    if (a.cols <= kMaxOddCols) {
        const int64_t odd = a.cols / kVec<T>;                          // whole vectors, at most
        if (a.rows <= 2 * a.num_sms && odd <= kMaxThreads) return forward<T, 1, false>(a, odd, st);
        if (a.rows <= 2 * a.num_sms && odd <= 2 * kMaxThreads) return forward<T, 2, false>(a, odd, st);
        return odd <= 4 * 32 ? forward<T, 4, false>(a, odd, st) : forward<T, 8, false>(a, odd, st);
    }
    norm_wide_kernel<T, 1><<<(unsigned)a.rows, kWide, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dx_odd(const NormArgs& a, cudaStream_t st) {
    const int64_t n = a.cols / kVec<T>;
    if (a.rows <= 2 * a.num_sms && n <= 2 * kMaxThreads) return dx_only<T, 2, false>(a, n, st);
    if (n <= 4 * 32) return dx_only<T, 4, false>(a, n, st);
    return dx_only<T, 8, false>(a, n, st);
}
template <typename T>
cudaError_t backward_t(const NormArgs& a, cudaStream_t st) {
    constexpr int VEC = kVec<T>;
    const bool even = even_rows(a);
    const int64_t n = a.cols / VEC;
    if (even) {
        if (n <= kMaxThreads && a.rows <= 2 * a.num_sms) return backward<T, 1, 2>(a, st);
        // 16 columns a thread: more would not leave room for their sums
        constexpr int NV = 16 / VEC;
        if (n <= NV * kMaxThreads) return backward<T, NV, 2>(a, st);
        if constexpr (VEC == 8)
            if (a.cols <= kLongCols)
                return a.dweight || a.dbias ? backward_long_c<true>(a, st) : backward_long_c<false>(a, st);
    }
    // the column sums first: dx may be written over dy
    if (a.dweight || a.dbias) {
        cudaError_t e = even ? columns<T, VEC>(a, st) : columns<T, 1>(a, st);
        if (e != cudaSuccess) return e;
    }
    if (even && n <= 8 * kMaxThreads) return dx_only<T, 8, true>(a, n, st);
    if (!even && a.cols <= kMaxOddCols) return dx_odd<T>(a, st);
    if (even) norm_wide_dx_kernel<T, kVec<T>><<<(unsigned)a.rows, kWide, 0, st>>>(a);
    else norm_wide_dx_kernel<T, 1><<<(unsigned)a.rows, kWide, 0, st>>>(a);
    return cudaGetLastError();
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
