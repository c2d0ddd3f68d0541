// What the epilogue of a product does with its sums besides storing them:
//   linear  z = sum + bias, y = act(z) + residual
//   gated   h = act(gate) * up
// for the BF16 products (linear.cu) and the block-scaled ones (gemm2.cu).
// Everything is FP32 until the store, which rounds once.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "launch.cuh"
#include "pair_gemm.cuh"
#include "tcgen05.cuh"

namespace bsq {

enum { kActIdentity, kActRelu, kActSilu, kActGelu, kActGeluTanh, kActs };

// A TMA store does not cut a row inside 16 bytes: where a row ends there, the box with its end is written otherwise.
enum { kNone, kPart, kWhole };

struct Fused {
    int32_t act;
    int32_t y_bf16;                // y (and the residual): BF16 or FP32
    int32_t bias_bf16;
    int32_t y_tma, z_tma, u_tma;   // the output's rows suit TMA stores (kWhole, kPart), or not (0)
    int32_t res_vec, bias_vec;     // 16-byte loads
    const void* bias;              // [N] or nullptr
    const void* residual;          // or nullptr
    int64_t ld_res;
    void* y;
    int64_t ldy;
    __nv_bfloat16* z;              // linear: the pre-activation; gated: the gate's; or nullptr
    int64_t ldz;
    __nv_bfloat16* u;              // gated: the other projection; or nullptr
    int64_t ldu;
};

// ------------------------------------------------------------- activations
// Two values at a time, in packed instructions: the epilogue's instructions compete with those of the thread that
// issues the MMAs.  ex2 and rcp are good to 2^-22 each; exp(-x) = inf gives 0.
constexpr float kLog2eF = 1.44269504088896340736f;
constexpr float kGeluC = 0.79788456080286535588f;      // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
__device__ __forceinline__ F2 exp2_two(F2 x) {
    const float2 v = x.get();
    return F2(pair::exp2_fast(v.x), pair::exp2_fast(v.y));
}
__device__ __forceinline__ F2 rcp_two(F2 x) {
    const float2 v = x.get();
    float a, b;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(v.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(v.y));
    return F2(a, b);
}
__device__ __forceinline__ F2 sigmoid(F2 x) { return rcp_two(F2(1.0f) + exp2_two(x * F2(-kLog2eF))); }
// 0.5 (1 + tanh(t)) is the sigmoid of 2 t, without the cancellation at negative t; 2 t = z (2 c + 2 c a z^2)
__device__ __forceinline__ F2 gelu_gate(F2 z) {
    const F2 t = z * fma2(z * z, F2(-2.0f * kGeluC * kGeluA * kLog2eF), F2(-2.0f * kGeluC * kLog2eF));
    return rcp_two(F2(1.0f) + exp2_two(t));
}
// The normal distribution's value at z, and e = exp(-z^2 / 2).  With x = |z| / sqrt(2) and t = 1 / (1 + 0.45 x) the
// tail beyond |z| is e / 2 times t P(t), a polynomial fitted to exp(x^2) erfc(x) for a small relative error (3.9e-7 up to x = 10);
// no part of it cancels, so it keeps its relative error as far as e does.  A third of erfcf's instructions, which
// were most of a gelu epilogue.
__device__ __forceinline__ F2 normal_cdf(F2 z, F2& e) {
    const float2 v = z.get();
    const F2 a(fabsf(v.x), fabsf(v.y));
    e = exp2_two(z * z * F2(-0.72134752044448170368f));
    const F2 t = rcp_two(fma2(F2(0.31819805153394638598f), a, F2(1.0f)));
    F2 q(0.5f * 0.06687701493501663f);
    q = fma2(q, t, F2(0.5f * -0.2403355836868286f));
    q = fma2(q, t, F2(0.5f * 0.20899593830108643f));
    q = fma2(q, t, F2(0.5f * 0.040100302547216415f));
    q = fma2(q, t, F2(0.5f * 0.18878303468227386f));
    q = fma2(q, t, F2(0.5f * 0.22802451252937317f));
    q = fma2(q, t, F2(0.5f * 0.25364693999290466f));
    q = fma2(q, t, F2(0.5f * 0.2539081275463104f));
    const F2 tail = q * t * e;
    const float2 lo = tail.get(), hi = fma2(tail, F2(-1.0f), F2(1.0f)).get();
    return F2(v.x < 0.0f ? lo.x : hi.x, v.y < 0.0f ? lo.y : hi.y);
}

template <int ACT>
__device__ __forceinline__ F2 act_two(F2 z) {
    if (ACT == kActRelu) {
        const float2 v = z.get();                                      // NaN stays NaN
        return F2(v.x > 0.0f || v.x != v.x ? v.x : 0.0f, v.y > 0.0f || v.y != v.y ? v.y : 0.0f);
    }
    if (ACT == kActSilu) return z * sigmoid(z);
    if (ACT == kActGelu) {
        F2 e;
        return z * normal_cdf(z, e);
    }
    if (ACT == kActGeluTanh) return z * gelu_gate(z);
    return z;
}
// act'(z), and act(z) beside it
template <int ACT>
__device__ __forceinline__ F2 act_slope(F2 z, F2& value) {
    value = z;
    if (ACT == kActRelu) {
        value = act_two<kActRelu>(z);
        const float2 v = z.get();
        return F2(v.x > 0.0f ? 1.0f : v.x != v.x ? v.x : 0.0f, v.y > 0.0f ? 1.0f : v.y != v.y ? v.y : 0.0f);
    }
    if (ACT == kActSilu) {
        const F2 s = sigmoid(z);
        value = z * s;
        return s * fma2(z, fma2(s, F2(-1.0f), F2(1.0f)), F2(1.0f));
    }
    if (ACT == kActGelu) {
        F2 e;
        const F2 c = normal_cdf(z, e);
        value = z * c;
        return fma2(z * F2(0.39894228040143267794f), e, c);            // + z exp(-z^2 / 2) / sqrt(2 pi)
    }
    if (ACT == kActGeluTanh) {
        const F2 s = gelu_gate(z);
        value = z * s;
        const float2 q = (z * z).get();                                // (finite: 0 times it is 0)
        const F2 p = fma2(F2(3.0f * kGeluA), F2(fminf(q.x, 1e30f), fminf(q.y, 1e30f)), F2(1.0f));
        return fma2(value * fma2(s, F2(-1.0f), F2(1.0f)) * F2(2.0f * kGeluC), p, s);
    }
    return F2(1.0f);
}
// f<ACT>() for the activation `act`
#define BSQ_WITH_ACT(act, F)                                 \
    switch (act) {                                           \
        case kActRelu: F(kActRelu); break;                   \
        case kActSilu: F(kActSilu); break;                   \
        case kActGelu: F(kActGelu); break;                   \
        case kActGeluTanh: F(kActGeluTanh); break;           \
        default: F(kActIdentity); break;                     \
    }

template <int N>
__device__ __forceinline__ void activate(int act, float (&v)[N]) {
    if (act == kActIdentity) return;
#define F(A)                                                                  \
    _Pragma("unroll") for (int j = 0; j < N; j += 2) {                        \
        const float2 y = act_two<A>(F2(v[j], v[j + 1 < N ? j + 1 : j])).get(); \
        v[j] = y.x;                                                           \
        if (j + 1 < N) v[j + 1 < N ? j + 1 : j] = y.y;                        \
    }
    BSQ_WITH_ACT(act, F)
#undef F
}

__device__ __forceinline__ float load_as_float(const void* p, int64_t i, int bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// ------------------------------------------------- chunks of 32 rows by 32 columns
__device__ __forceinline__ void add_two(float* v, F2 x) {
    const float2 s = (F2(v[0], v[1]) + x).get();
    v[0] = s.x;
    v[1] = s.y;
}
// v += p[0 .. 32), the first `n` of them (32 or more: all), 16 bytes at a time where `vec`
__device__ __forceinline__ void add_row(float (&v)[32], const void* p, int64_t at, int bf16, int vec, int64_t n) {
    if (vec && n >= 32) {
        if (bf16) {
            const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(p) + at;
            Pack<__nv_bfloat16, 8> k[4];
#pragma unroll
            for (int i = 0; i < 4; i++) k[i].load(from + 8 * i);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                F2 f[4];
                unpack2(k[i], f);
#pragma unroll
                for (int e = 0; e < 4; e++) add_two(v + 8 * i + 2 * e, f[e]);
            }
        } else {
            const float* from = static_cast<const float*>(p) + at;
            float4 k[8];
#pragma unroll
            for (int i = 0; i < 8; i++) k[i] = *reinterpret_cast<const float4*>(from + 4 * i);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                add_two(v + 4 * i, F2(k[i].x, k[i].y));
                add_two(v + 4 * i + 2, F2(k[i].z, k[i].w));
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 32; j++)
        if (j < n) v[j] += load_as_float(p, at + j, bf16);
}

// A warp's staging: BUFS buffers of 2 KB, used in turn; `n` counts the chunks.  Every chunk is a bulk group, an empty one
// where no TMA store reads it, so that the groups before the last BUFS - 1 are the buffer's own store too.
template <int BUFS>
struct Staging {
    uint32_t base;
    int n;
    __device__ __forceinline__ uint32_t next(int lane) {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" :: "n"(BUFS - 1) : "memory");
        __syncwarp();
        return base + (uint32_t)(n++ % BUFS) * 2048u;
    }
};

// The warp's chunk (lane: row row0 + lane, its columns col ..) leaves as BF16 or FP32: through a staging
// buffer and a TMA store, or (rows off 16-byte boundaries) from the buffer with neighbouring lanes on
// neighbouring columns.  Rows from M and columns from N on are not written.
template <int BUFS>
__device__ __forceinline__ void store_chunk(const float (&v)[32], int bf16, int tma, const void* tmap, void* out, int64_t ld,
                                            int64_t row0, int64_t col, int64_t M, int64_t N, Staging<BUFS>& st, int lane) {
    if (bf16) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; j++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        const uint32_t buf = st.next(lane);
        if (tma == kWhole || (tma && col + 32 <= N)) {
            pair::stage_chunk(w, buf, lane);
            if (lane == 0) {
                tc::tma_store_2d(tmap, (int)col, (int)row0, buf);
                tc::bulk_commit();
            }
            return;
        }
        // (not through the asynchronous proxy, whose fence would wait for the stores of the chunk before)
        pair::put_chunk(w, buf, lane);
        __syncwarp();
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + row0 * ld + col + lane;
        const int rows = (int)min((int64_t)32, M - row0);
        const bool in = col + lane < N;
        // where the lane's column is in rows 0 and 1, 2 and 3, 4 and 5, 6 and 7 of every eight
        uint32_t at[4];
#pragma unroll
        for (int k = 0; k < 4; k++) at[k] = buf + ((((uint32_t)lane >> 3) ^ k) << 4) + ((uint32_t)lane & 7u) * 2u;
#pragma unroll 1
        for (int r = 0; r < rows; r += 8) {
            uint16_t x[8];
#pragma unroll
            for (int k = 0; k < 8; k++)
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x[k]) : "r"(at[k >> 1] + (uint32_t)(r + k) * 64u) : "memory");
#pragma unroll
            for (int k = 0; k < 8; k++) {
                if (in && r + k < rows) *o = __ushort_as_bfloat16(x[k]);
                o += ld;
            }
        }
        if (lane == 0) tc::bulk_commit();
        __syncwarp();
        return;
    }
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; j++) w[j] = __float_as_uint(v[c + j]);
        const uint32_t buf = st.next(lane);
        if (tma == kWhole || (tma && col + c + 16 <= N)) {
            pair::stage_chunk(w, buf, lane);
            if (lane == 0) {
                tc::tma_store_2d(tmap, (int)col + c, (int)row0, buf);
                tc::bulk_commit();
            }
            continue;
        }
        pair::put_chunk(w, buf, lane);
        __syncwarp();
        const int k0 = lane & 15, r0 = lane >> 4;
        float* o = static_cast<float*>(out) + (row0 + r0) * ld + col + c + k0;
        const int rows = (int)min((int64_t)32, M - row0);
        const bool in = col + c + k0 < N;
        uint32_t at[4];                            // rows 2 k and 2 k + 1 of every eight
#pragma unroll
        for (int k = 0; k < 4; k++) at[k] = buf + (uint32_t)r0 * 64u + ((((uint32_t)k0 >> 2) ^ k) << 4) + ((uint32_t)k0 & 3u) * 4u;
#pragma unroll 1
        for (int r = 0; r < rows; r += 8) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; k++)
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x[k]) : "r"(at[k] + (uint32_t)(r + 2 * k) * 64u) : "memory");
#pragma unroll
            for (int k = 0; k < 4; k++) {
                if (in && r + 2 * k + r0 < rows) *o = x[k];
                o += 2 * ld;
            }
        }
        if (lane == 0) tc::bulk_commit();
        __syncwarp();
    }
}

// v += the chunk of `p` (lane: row row0 + lane, its columns col ..) where its rows are off 16-byte boundaries or end in
// it: read with neighbouring lanes on neighbouring columns and turned in a staging buffer.  (Each lane its own row,
// an element at a time, the residual was most of the time of 660 x 160 -> 481: MXFP8 41 us, 18 now, 11 without
// one; BF16 with gelu and z 12.8 us, 7.5 now.)
template <int BUFS>
__device__ __forceinline__ void add_chunk(float (&v)[32], const void* p, int bf16, int64_t ld, int64_t row0, int64_t col, int64_t M,
                                          int64_t N, Staging<BUFS>& st, int lane) {
    const int rows = (int)min((int64_t)32, M - row0);
    if (bf16) {
        const uint32_t buf = st.next(lane);
        const uint16_t* from = static_cast<const uint16_t*>(p) + row0 * ld + col + lane;
        const bool in = col + lane < N;
        uint32_t at[4];
#pragma unroll
        for (int k = 0; k < 4; k++) at[k] = buf + ((((uint32_t)lane >> 3) ^ k) << 4) + ((uint32_t)lane & 7u) * 2u;
#pragma unroll 1
        for (int r = 0; r < rows; r += 16) {
            uint16_t x[16];
#pragma unroll
            for (int k = 0; k < 16; k++) x[k] = in && r + k < rows ? from[(r + k) * ld] : (uint16_t)0;
#pragma unroll
            for (int k = 0; k < 16; k++)
                asm volatile("st.shared.u16 [%0], %1;" :: "r"(at[(k & 7) >> 1] + (uint32_t)(r + k) * 64u), "h"(x[k]) : "memory");
        }
        __syncwarp();
        uint32_t w[16];
        pair::get_chunk(w, buf, lane);
#pragma unroll
        for (int j = 0; j < 16; j++) {
            v[2 * j] += __uint_as_float(w[j] << 16);
            v[2 * j + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
        }
        if (lane == 0) tc::bulk_commit();
        __syncwarp();
        return;
    }
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
        const uint32_t buf = st.next(lane);
        const int k0 = lane & 15, r0 = lane >> 4;
        const float* from = static_cast<const float*>(p) + (row0 + r0) * ld + col + c + k0;
        const bool in = col + c + k0 < N;
        uint32_t at[4];                            // rows 2 k and 2 k + 1 of every eight
#pragma unroll
        for (int k = 0; k < 4; k++) at[k] = buf + (uint32_t)r0 * 64u + ((((uint32_t)k0 >> 2) ^ k) << 4) + ((uint32_t)k0 & 3u) * 4u;
#pragma unroll 1
        for (int r = 0; r < rows; r += 16) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; k++) x[k] = in && r + 2 * k + r0 < rows ? from[(r + 2 * k) * ld] : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; k++)
                asm volatile("st.shared.f32 [%0], %1;" :: "r"(at[k & 3] + (uint32_t)(r + 2 * k) * 64u), "f"(x[k]) : "memory");
        }
        __syncwarp();
        uint32_t w[16];
        pair::get_chunk(w, buf, lane);
#pragma unroll
        for (int j = 0; j < 16; j++) v[c + j] += __uint_as_float(w[j]);
        if (lane == 0) tc::bulk_commit();
        __syncwarp();
    }
}

// One element, of one token: sum (and of a gated layer up's) becomes z and y, or gate, up and h
template <bool GATED>
__device__ __forceinline__ void finish_one(float z, float u, const Fused& f, int64_t t, int64_t feature) {
    if (!GATED && f.bias) z += load_as_float(f.bias, feature, f.bias_bf16);
    if (f.z) {
        f.z[t * f.ldz + feature] = __float2bfloat16_rn(z);
        if (GATED) f.u[t * f.ldu + feature] = __float2bfloat16_rn(u);
    }
    float v[1] = {z};
    activate(f.act, v);
    float y = GATED ? v[0] * u : v[0];
    if (!GATED && f.residual) y += load_as_float(f.residual, t * f.ld_res + feature, f.y_bf16);
    if (f.y_bf16) static_cast<__nv_bfloat16*>(f.y)[t * f.ldy + feature] = __float2bfloat16_rn(y);
    else static_cast<float*>(f.y)[t * f.ldy + feature] = y;
}

// 32 columns of a linear layer's sums become z, y
template <int BUFS>
__device__ __forceinline__ void finish_linear(float (&v)[32], const Fused& f, const void* tm_y, const void* tm_z, int64_t row0,
                                              int64_t col, int64_t M, int64_t N, Staging<BUFS>& st, int lane) {
    if (f.bias) add_row(v, f.bias, col, f.bias_bf16, f.bias_vec, N - col);
    if (f.z) store_chunk(v, 1, f.z_tma, tm_z, f.z, f.ldz, row0, col, M, N, st, lane);
    activate(f.act, v);
    if (f.residual) {
        if (f.res_vec && col + 32 <= N) {
            if (row0 + lane < M) add_row(v, f.residual, (row0 + lane) * f.ld_res + col, f.y_bf16, 1, N - col);
        } else {
            add_chunk(v, f.residual, f.y_bf16, f.ld_res, row0, col, M, N, st, lane);
        }
    }
    store_chunk(v, f.y_bf16, f.y_tma, tm_y, f.y, f.ldy, row0, col, M, N, st, lane);
}
// 32 columns of both projections become h
template <int BUFS>
__device__ __forceinline__ void finish_gated(float (&v)[32], const float (&u)[32], const Fused& f, const void* tm_y,
                                             const void* tm_z, const void* tm_u, int64_t row0, int64_t col, int64_t M, int64_t N,
                                             Staging<BUFS>& st, int lane) {
    if (f.z) {
        store_chunk(v, 1, f.z_tma, tm_z, f.z, f.ldz, row0, col, M, N, st, lane);
        store_chunk(u, 1, f.u_tma, tm_u, f.u, f.ldu, row0, col, M, N, st, lane);
    }
    activate(f.act, v);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const float2 h = (F2(v[j], v[j + 1]) * F2(u[j], u[j + 1])).get();
        v[j] = h.x;
        v[j + 1] = h.y;
    }
    store_chunk(v, f.y_bf16, f.y_tma, tm_y, f.y, f.ldy, row0, col, M, N, st, lane);
}

// The column of column c of a gated layer's gate among its parts of a sum; up's is 128 further
__device__ __forceinline__ int64_t gate_col(int64_t c) { return (c >> 7) * 256 + (c & 127); }

struct LinearArgs;
// the epilogue of a call (without the tensor maps' part)
void fused_args(Fused& f, const LinearArgs& a);
// Parts of a split sum over K are FP32 [part][row][fused_acc_cols]: gated, 128 columns of the gate's sums, then up's
// of the same columns, and so on.
int64_t fused_acc_cols(int64_t N, bool gated);
// the parts that get any of `stages`, dealt to n
int fused_parts(int64_t stages, int64_t n);
// What `n` parts of each tile's sum cost: the busiest pair's time, and the join's, its launch and the parts written and
// read (tile_us: what a tile costs besides its stages; part_us: the least for a part's)
double split_us(int64_t tiles, int64_t stages, int64_t n, double stage_us, double tile_us, double part_us, double part_bytes, int pairs);
// How many parts: more than one where there are fewer tiles than pairs, or few in the last wave
int fused_splits(int64_t tiles, int64_t stages, double stage_us, double tile_us, double part_us, double part_bytes, int pairs);
// adds the parts in their order and does the epilogue; starts beside the kernel before it
cudaError_t run_linear_join(const float* acc, int splits, int64_t M, int64_t N, bool gated, const LinearArgs& a, cudaStream_t st);

// Tensor map of an output for 32 x 64-byte stores, if its rows suit them
inline int fused_map(CUtensorMap* m, void* p, int64_t rows, int64_t cols, int64_t ld, bool bf16) {
    const int64_t e = bf16 ? 2 : 4;
    if (!p || reinterpret_cast<uintptr_t>(p) % 16 || ld * e % 16 || !tmap::out_2d(m, p, rows, cols, ld, bf16)) return kNone;
    return cols * e % 16 ? kPart : kWhole;
}

}  // namespace bsq
