// Products of block-scaled operands with one token or two, with the epilogue of
// bsq_gemm_linear or bsq_gemm_gated: the single tokens of a decoding step.
//
// On the CUDA cores, as linear_gemv_kernel, with no set-up before the first loads.  Bound
// by decoding (some 3 instructions a code) as much as by streaming the weights' codes:
// 14336 -> 4096 of one token in 17.5 us (the tensor cores' way 27.5), gated 4096 -> 14336
// 26.5 (40; NVFP4 24.7); of two 22 and 33, of four 45 and 62, where the tensor cores take 29 and 41.  A
// lane takes 16 codes of a row at a time, decodes them to FP32, and multiplies the sum of
// their products, which lie in one scale block of either operand, by both scales.  A
// warp's four rows of w are 32 apart, in one 128-row band: in the 128 x 4 tiles of the
// scales the four scales of each of those rows are 16 neighbouring bytes, one load for
// four rows and four blocks.  `parts` warps of a CTA share a row's columns.
#include <algorithm>
#include "common.cuh"
#include "fused.cuh"
#include "internal.h"
#include "launch.cuh"

namespace bsq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 4;                            // of each matrix, 32 apart
enum { kFP8, kNV, kMX4 };

struct ScaledGemv {
    const uint8_t *x, *x_scales;   // codes [T][row_bytes], scales in tiles
    const uint8_t *w[2], *w_scales[2];
    const float* ts_x;             // NVFP4: tensor scales
    const float* ts_w[2];
    int64_t N, row_bytes;
    int64_t vectors, part;         // 16 codes each: of a row, and of one of its parts
    int64_t atoms;                 // scale tiles of a band
    int32_t T, parts, x_e5m2, w_e5m2;
    Fused f;
};

template <int KIND>
struct Codes {
    uint4 v;
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const uint8_t* p) {
        if (KIND == kFP8) v = *reinterpret_cast<const uint4*>(p);
        else {
            const uint2 a = *reinterpret_cast<const uint2*>(p);
            v = make_uint4(a.x, a.y, 0, 0);
        }
    }
    // (not .nc: the kernel runs already while the one before it writes the weights)
    __device__ __forceinline__ void stream(const uint8_t* p) {
        if (KIND == kFP8)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
        else {
            asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
            v.z = v.w = 0;
        }
    }
    __device__ __forceinline__ void decode(int e5m2, F2 (&f)[8]) const {
        uint32_t h[8];
        if (KIND == kFP8) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (e5m2) {
#pragma unroll
                for (int i = 0; i < 8; i++) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h[i]) : "h"((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[i]) : "h"((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
            }
        } else {
            const uint32_t w[2] = {v.x, v.y};
#pragma unroll
            for (int i = 0; i < 2; i++)
                asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\tmov.b32 {t0, t1, t2, t3}, %4;\n\t"
                    "cvt.rn.f16x2.e2m1x2 %0, t0;\n\tcvt.rn.f16x2.e2m1x2 %1, t1;\n\t"
                    "cvt.rn.f16x2.e2m1x2 %2, t2;\n\tcvt.rn.f16x2.e2m1x2 %3, t3;\n\t}"
                    : "=r"(h[4 * i]), "=r"(h[4 * i + 1]), "=r"(h[4 * i + 2]), "=r"(h[4 * i + 3])
                    : "r"(w[i]));
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
            f[i] = F2(a.x, a.y);
        }
    }
};
// sum times both scales.  E8M0: the exponents' sum is applied in two halves, so that one large and one small scale
// neither overflow nor underflow on the way; 255 is NaN.
template <int KIND>
__device__ __forceinline__ float scaled(float sum, uint32_t a, uint32_t b) {
    if (KIND == kNV) return sum * e4m3_to_float(a) * e4m3_to_float(b);
    const uint32_t e = a + b, half = e >> 1;       // 2^(e - 254)
    const float s = sum * __uint_as_float(half << 23) * __uint_as_float((e - half) << 23);
    return max(a, b) == 255 ? __uint_as_float(0x7FFFFFFFu) : s;
}

template <int KIND, int TOK, bool GATED>
__global__ void __launch_bounds__(kThreads, TOK == 1 ? 3 : 2) scaled_gemv_kernel(const __grid_constant__ ScaledGemv p) {
    constexpr int MATS = GATED ? 2 : 1, AHEAD = GATED ? 1 : 2, BYTES = KIND == kFP8 ? 16 : 8;
    __shared__ float sums[kWarps][MATS * kRows * TOK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / p.parts, part = warp - group * p.parts, groups = kWarps / p.parts;
    const int64_t task = (int64_t)blockIdx.x * groups + group, band = task >> 5;
    const int j = (int)(task & 31);
    const uint8_t* row[MATS][kRows];
#pragma unroll
    for (int m = 0; m < MATS; m++)
#pragma unroll
        for (int r = 0; r < kRows; r++)            // rows past the last read the last one and are not written
            row[m][r] = p.w[m] + min(p.N - 1, band * 128 + j + 32 * r) * p.row_bytes;
    // (a CTA's last tasks may lie past the last band: they read its scales)
    const int64_t scale0 = min(band, (p.N - 1) >> 7) * p.atoms * 512 + j * 16;
    float acc[MATS][kRows][TOK] = {};
    pdl_launch_dependents();
    pdl_wait();
    const int64_t end = min(p.vectors, (part + 1) * p.part);
    for (int64_t k = part * p.part + lane; k < end; k += 32 * AHEAD) {
        Codes<KIND> w[AHEAD][MATS][kRows], x[AHEAD][TOK];
        uint4 ws[AHEAD][MATS];
        uint32_t xs[AHEAD][TOK];
#pragma unroll
        for (int a = 0; a < AHEAD; a++) {
            const int64_t v = k + 32 * a, block = KIND == kNV ? v : v >> 1, tile = (block >> 2) * 512;
            const bool in = v < end;
#pragma unroll
            for (int m = 0; m < MATS; m++) {
#pragma unroll
                for (int r = 0; r < kRows; r++) {
                    w[a][m][r].zero();
                    if (in) w[a][m][r].stream(row[m][r] + v * BYTES);
                }
                ws[a][m] = make_uint4(0, 0, 0, 0);
                if (in) ws[a][m] = *reinterpret_cast<const uint4*>(p.w_scales[m] + scale0 + tile);
            }
#pragma unroll
            for (int t = 0; t < TOK; t++) {
                x[a][t].zero();
                xs[a][t] = 0;
                if (in && t < p.T) {
                    x[a][t].load(p.x + t * p.row_bytes + v * BYTES);
                    xs[a][t] = p.x_scales[tile + t * 16 + (block & 3)];
                }
            }
        }
#pragma unroll
        for (int a = 0; a < AHEAD; a++) {
            F2 f[TOK][8];
#pragma unroll
            for (int t = 0; t < TOK; t++) x[a][t].decode(p.x_e5m2, f[t]);
            const int64_t v = k + 32 * a;
            const int shift = 8 * (int)((KIND == kNV ? v : v >> 1) & 3);
#pragma unroll
            for (int m = 0; m < MATS; m++) {
                const uint32_t s[kRows] = {ws[a][m].x, ws[a][m].y, ws[a][m].z, ws[a][m].w};
#pragma unroll
                for (int r = 0; r < kRows; r++) {
                    F2 g[8];
                    w[a][m][r].decode(p.w_e5m2, g);
#pragma unroll
                    for (int t = 0; t < TOK; t++) {
                        F2 d = g[0] * f[t][0];
#pragma unroll
                        for (int i = 1; i < 8; i++) d = fma2(g[i], f[t][i], d);
                        const float2 q = d.get();
                        acc[m][r][t] += scaled<KIND>(q.x + q.y, s[r] >> shift & 0xFF, xs[a][t]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MATS; m++)
#pragma unroll
        for (int r = 0; r < kRows; r++)
#pragma unroll
            for (int t = 0; t < TOK; t++) {
                float s = acc[m][r][t];
#pragma unroll
                for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                if (lane == 0) sums[warp][(m * kRows + r) * TOK + t] = s;
            }
    __syncthreads();
    // one output a thread, the parts of a row in their order
    const int i = threadIdx.x;
    if (i >= groups * kRows * TOK) return;
    const int t = i / (groups * kRows), g = i - t * groups * kRows, mine = g / kRows, r = g - mine * kRows;
    const int64_t at = (int64_t)blockIdx.x * groups + mine, feature = (at >> 5) * 128 + (at & 31) + 32 * r;
    if (t >= p.T || feature >= p.N) return;
    const auto sum = [&](int m) {
        float s = 0.0f;
        for (int k = 0; k < p.parts; k++) s += sums[mine * p.parts + k][(m * kRows + r) * TOK + t];
        // the tensor scales one after the other: their product may underflow
        return KIND == kNV ? s * *p.ts_x * *p.ts_w[m] : s;
    };
    finish_one<GATED>(sum(0), GATED ? sum(MATS - 1) : 1.0f, p.f, t, feature);
}

template <int KIND, bool GATED>
cudaError_t launch(const ScaledGemv& p, dim3 grid, cudaStream_t st) {
    if (p.T == 1) return launch_k(true, scaled_gemv_kernel<KIND, 1, GATED>, grid, kThreads, 0, st, p);
    return launch_k(true, scaled_gemv_kernel<KIND, 2, GATED>, grid, kThreads, 0, st, p);
}

}  // namespace

cudaError_t run_scaled_gemv(const GemmArgs& a, const GemmArgs& up, const LinearArgs& l, bool gated, cudaStream_t st) {
    const int kind = a.fmt_a == kNVFP4 ? kNV : a.fmt_a == kMXFP4 ? kMX4 : kFP8;
    ScaledGemv p{};
    p.x = a.a_codes;
    p.x_scales = a.a_scales;
    p.w[0] = a.b_codes;
    p.w[1] = up.b_codes;
    p.w_scales[0] = a.b_scales;
    p.w_scales[1] = up.b_scales;
    p.ts_x = a.ts_a;
    p.ts_w[0] = a.ts_b;
    p.ts_w[1] = up.ts_b;
    p.N = a.N;
    p.row_bytes = kind == kFP8 ? a.K : a.K / 2;
    p.vectors = a.K / 16;
    p.atoms = (a.K / (kind == kNV ? 16 : 32) + 3) / 4;
    p.T = (int32_t)a.M;
    p.x_e5m2 = a.fmt_a == kE5M2;
    p.w_e5m2 = a.fmt_b == kE5M2;
    fused_args(p.f, l);
    const int64_t tasks = (a.N + 127) / 128 * 32;
    p.parts = 1;
    while (p.parts < kWarps && tasks * p.parts * p.T < (int64_t)a.num_sms * 64 && p.vectors > 32 * p.parts) p.parts *= 2;
    p.part = ((p.vectors + p.parts - 1) / p.parts + 31) / 32 * 32;
    const dim3 grid((unsigned)((tasks * p.parts + kWarps - 1) / kWarps));
    if (kind == kNV) return gated ? launch<kNV, true>(p, grid, st) : launch<kNV, false>(p, grid, st);
    if (kind == kMX4) return gated ? launch<kMX4, true>(p, grid, st) : launch<kMX4, false>(p, grid, st);
    return gated ? launch<kFP8, true>(p, grid, st) : launch<kFP8, false>(p, grid, st);
}

}  // namespace bsq
