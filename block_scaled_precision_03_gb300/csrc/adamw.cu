// One AdamW step over many tensors:
//   g' = g f                       f = min(1, max_norm / (norm + eps)), or 1
//   m' = beta1 m + (1 - beta1) g'
//   v' = beta2 v + ((1 - beta2) g') g'
//   p' = decay p - size (m' / (sqrt(v') root + eps))
// with decay = 1 - lr weight_decay, size = lr / (1 - beta1^step), root = 1 /
// sqrt(1 - beta2^step).  Every operation is one FP32 operation rounded to
// nearest, in this order (no contraction: the packed instructions and the
// _rn intrinsics), so that a result can be recomputed bit for bit.
//
// Moments in 8 bits: E4M3 codes with one E8M0 scale for 32 elements of a tensor,
// the format of the MXFP8 tensors, m as it is and v as its root r (an 8-bit v
// would have to span the square of the range).  The scale is the power of two
// that keeps the block's largest magnitude between 224 and 448.  E4M3 has 3
// bits of mantissa, so rounded to nearest a moment that moves by less than 3% of
// itself, as v does by 0.1% a step, would stand still; with a seed the codes (and
// BF16 weights) are rounded stochastically, up with the probability of what is
// cut off, and move as they should on average.
//
// The list travels in the kernel's parameters; tensors are cut into chunks of
// 2048 elements, 8 neighbours a thread: a block of 32 is four lanes.
#include <algorithm>
#include <cmath>
#include "../../include/bsq.h"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace bsq {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                             // elements of a thread
constexpr int64_t kChunk = (int64_t)kThreads * kPer;

struct Entry {
    void* p;
    const void* g;
    void *m, *v;                   // FP32, or codes
    uint8_t *m_scales, *v_scales;
    __nv_bfloat16* copy;
    int64_t n;
    int32_t index;                 // in the caller's list
    int8_t p_bf16, g_bf16, bits8, vec;
};
template <int CAP>
struct Table {
    Entry e[CAP];
    int32_t first[CAP + 1];        // chunks before each tensor
    int32_t count;
};
constexpr int kSmall = 16, kLarge = 384;
struct Options {
    float beta1, beta2, c1, c2;    // c: 1 - beta
    float decay, size, root, eps;
    const float* norm;
    float max_norm, clip_eps;
    uint32_t seed_lo, seed_hi;
    int64_t step;
    const int64_t* step_at;        // on the device: the step, and then the scalars that depend on it
    const float* lr_at;
    float lr, weight_decay, log_beta1, log_beta2;
};
static_assert(sizeof(Table<kLarge>) + sizeof(Options) <= 32764, "kernel parameters");

// A permutation of the 32-bit integers that leaves no visible order (multiply and
// xor-shift; the constants are those of C. Wellons' lowbias32)
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x7FEB352Du;
    x ^= x >> 15;
    x *= 0x846CA68Bu;
    return x ^ (x >> 16);
}
// 2^(byte - 127)
__device__ __forceinline__ float power(uint32_t byte) { return __uint_as_float(byte == 0 ? 1u << 22 : byte << 23); }

// 8 magnitudes, already scaled to at most 448 (a little more is cut), to the E4M3 grid: 16 random bits each.
// Below 2^-6 the grid's steps are 2^-9: with 2^-6 added they are those of the next binade.
__device__ __forceinline__ float stochastic_e4m3(float y, uint32_t bits16) {
    const float low = y < 0.015625f ? 0.015625f : 0.0f;
    const uint32_t w = __float_as_uint(__fadd_rn(y, low)) + (bits16 << 4);
    return __fsub_rn(__uint_as_float(w & ~0xFFFFFu), low);
}

// The 8 moments x of a thread (their block: four neighbouring lanes) as codes and a scale byte
template <bool RANDOM, bool ROOT>
__device__ __forceinline__ uint2 encode(const float (&x)[kPer], const uint32_t (&bits)[kPer], uint32_t& byte) {
    // bits of the largest magnitude: NaN and infinity above all others
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kPer; i++) most = max(most, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
    if (most >= 0x7F800000u) {
        byte = 0xFF;
        return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    }
    const int e = (int)(__float_as_uint(__fmul_rn(__uint_as_float(most), 8.0f / 7.0f)) >> 23) - 8;
    byte = (uint32_t)max(e, 0);
    const float up = power(254 - byte);
    float y[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const float a = __fmul_rn(fabsf(x[i]), up);
        const float s = fminf(RANDOM ? stochastic_e4m3(a, ROOT ? bits[i] >> 16 : bits[i] & 0xFFFFu) : a, 448.0f);
        // a second moment that is not 0 stays so (2^-9 is the smallest code)
        if (ROOT) y[i] = x[i] != 0.0f ? fmaxf(s, 0.001953125f) : 0.0f;
        else y[i] = x[i] < 0.0f ? -s : s;
    }
    return pack8_fp8<kE4M3>(y);
}
__device__ __forceinline__ void decode(uint2 codes, uint32_t byte, float (&x)[kPer]) {
    const float s = power(byte);
    const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t h2;
        const uint16_t in = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(in));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        x[2 * i] = __fmul_rn(f.x, s);
        x[2 * i + 1] = __fmul_rn(f.y, s);
    }
}

// 8 elements at p[at ..), the first n of them; 16-byte (codes: 8-byte) accesses where `vec`
__device__ __forceinline__ void get(const void* p, int64_t at, int bf16, bool vec, int n, float (&x)[kPer]) {
    if (bf16) {
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p) + at;
        if (vec) {
            Pack<__nv_bfloat16, 8> k;
            k.load(q);
            k.unpack(x);
            return;
        }
#pragma unroll
        for (int i = 0; i < kPer; i++) x[i] = i < n ? __bfloat162float(q[i]) : 0.0f;
        return;
    }
    const float* q = static_cast<const float*>(p) + at;
    if (vec) {
        const float4 a = reinterpret_cast<const float4*>(q)[0], b = reinterpret_cast<const float4*>(q)[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        return;
    }
#pragma unroll
    for (int i = 0; i < kPer; i++) x[i] = i < n ? q[i] : 0.0f;
}
__device__ __forceinline__ void put(void* p, int64_t at, int bf16, bool vec, int n, const float (&x)[kPer]) {
    if (bf16) {
        __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p) + at;
        if (vec) {
            Pack<__nv_bfloat16, 8> k;
            k.pack(x);
            k.store(q);
            return;
        }
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (i < n) q[i] = __float2bfloat16_rn(x[i]);
        return;
    }
    float* q = static_cast<float*>(p) + at;
    if (vec) {
        reinterpret_cast<float4*>(q)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(q)[1] = make_float4(x[4], x[5], x[6], x[7]);
        return;
    }
#pragma unroll
    for (int i = 0; i < kPer; i++)
        if (i < n) q[i] = x[i];
}
__device__ __forceinline__ uint2 get_codes(const void* p, int64_t at, bool vec, int n) {
    const uint8_t* q = static_cast<const uint8_t*>(p) + at;
    if (vec) return *reinterpret_cast<const uint2*>(q);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kPer; i++)
        if (i < n) w[i >> 2] |= (uint32_t)q[i] << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void put_codes(void* p, int64_t at, bool vec, int n, uint2 c) {
    uint8_t* q = static_cast<uint8_t*>(p) + at;
    if (vec) {
        *reinterpret_cast<uint2*>(q) = c;
        return;
    }
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < kPer; i++)
        if (i < n) q[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
}

// What a step with its number (or its learning rate) on the device computes itself, once a CTA: 1 - beta^t as
// -expm1(t log beta), which loses nothing at small t
__device__ __forceinline__ void step_scalars(Options& o) {
    __shared__ float shared[3];
    __shared__ int64_t step;
    if (threadIdx.x == 0) {
        const int64_t t = o.step_at ? *o.step_at : o.step;
        const float lr = o.lr_at ? *o.lr_at : o.lr;
        shared[0] = 1.0f - lr * o.weight_decay;
        shared[1] = lr / -expm1f((float)t * o.log_beta1);
        shared[2] = 1.0f / sqrtf(-expm1f((float)t * o.log_beta2));
        step = t;
    }
    __syncthreads();
    o.decay = shared[0];
    o.size = shared[1];
    o.root = shared[2];
    o.step = step;
}

template <int CAP, bool RANDOM>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<CAP> t, Options o) {
    if (o.step_at || o.lr_at) step_scalars(o);
    float factor = 1.0f;
    if (o.norm) {
        const float f = __fdiv_rn(o.max_norm, __fadd_rn(*o.norm, o.clip_eps));
        factor = f > 1.0f ? 1.0f : f;               // NaN stays NaN
    }
    for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        int lo = 0, hi = t.count - 1;               // the last tensor whose first chunk is <= c
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (t.first[mid] <= c) lo = mid; else hi = mid - 1;
        }
        const Entry& e = t.e[lo];
        const int64_t at = (int64_t)(c - t.first[lo]) * kChunk + threadIdx.x * kPer;
        const int n = (int)max((int64_t)0, min((int64_t)kPer, e.n - at));
        const bool vec = e.vec && n == kPer;
        float p[kPer], g[kPer], m[kPer] = {}, v[kPer] = {};
        uint2 mc = make_uint2(0, 0), vc = mc;
        uint32_t mb = 0, vb = 0;
        get(e.p, at, e.p_bf16, vec, n, p);
        get(e.g, at, e.g_bf16, vec, n, g);
        if (e.bits8) {
            mc = get_codes(e.m, at, vec, n);
            vc = get_codes(e.v, at, vec, n);
            if (n > 0) {
                mb = e.m_scales[at >> 5];
                vb = e.v_scales[at >> 5];
            }
            decode(mc, mb, m);
            decode(vc, vb, v);
#pragma unroll
            for (int i = 0; i < kPer; i++) v[i] = __fmul_rn(v[i], v[i]);
        } else {
            get(e.m, at, 0, vec, n, m);
            get(e.v, at, 0, vec, n, v);
        }
        uint32_t bits[kPer] = {};
        if (RANDOM) {
            uint32_t key = mix((uint32_t)e.index ^ o.seed_lo);
            key = mix(key ^ o.seed_hi);
            key = mix(key ^ (uint32_t)o.step) + (uint32_t)(at >> 32) * 0x9E3779B9u;
#pragma unroll
            for (int i = 0; i < kPer; i++) bits[i] = mix((uint32_t)(at + i) ^ key);
        }
        float r[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const float x = o.norm ? __fmul_rn(g[i], factor) : g[i];
            m[i] = __fadd_rn(__fmul_rn(o.beta1, m[i]), __fmul_rn(o.c1, x));
            v[i] = __fadd_rn(__fmul_rn(o.beta2, v[i]), __fmul_rn(__fmul_rn(o.c2, x), x));
            r[i] = __fsqrt_rn(v[i]);
            const float d = __fadd_rn(__fmul_rn(r[i], o.root), o.eps);
            p[i] = __fsub_rn(__fmul_rn(o.decay, p[i]), __fmul_rn(o.size, __fdiv_rn(m[i], d)));
        }
        if (e.bits8) {
            // elements past the end are 0 and change no scale; every lane takes part in the block's maximum
#pragma unroll
            for (int i = 0; i < kPer; i++)
                if (i >= n) m[i] = r[i] = 0.0f;
            mc = encode<RANDOM, false>(m, bits, mb);
            vc = encode<RANDOM, true>(r, bits, vb);
            put_codes(e.m, at, vec, n, mc);
            put_codes(e.v, at, vec, n, vc);
            if (n > 0 && (threadIdx.x & 3) == 0) {
                e.m_scales[at >> 5] = (uint8_t)mb;
                e.v_scales[at >> 5] = (uint8_t)vb;
            }
        } else {
            put(e.m, at, 0, vec, n, m);
            put(e.v, at, 0, vec, n, v);
        }
        if (e.copy) put(e.copy, at, 1, vec, n, p);
        if (RANDOM && e.p_bf16) {
#pragma unroll
            for (int i = 0; i < kPer; i++) {
                const uint32_t w = __float_as_uint(p[i]);
                if ((w & 0x7F800000u) != 0x7F800000u)       // not infinite, not NaN
                    p[i] = __uint_as_float((w + (bits[i] * 0x9E3779B1u >> 16)) & 0xFFFF0000u);
            }
        }
        put(e.p, at, e.p_bf16, vec, n, p);
    }
}

template <int CAP>
cudaError_t run(const AdamwArgs& a, const Options& o, bool random, cudaStream_t st) {
    const bsq_adamw_tensor* list = static_cast<const bsq_adamw_tensor*>(a.tensors);
    cudaError_t e = cudaSuccess;
    for (int at = 0; at < a.count && e == cudaSuccess;) {
        Table<CAP> t;
        t.count = 0;
        t.first[0] = 0;
        for (; at < a.count && t.count < CAP; at++) {
            const bsq_adamw_tensor& x = list[at];
            if (x.n == 0) continue;
            const int i = t.count++;
            const auto on = [](const void* p, uintptr_t k) { return reinterpret_cast<uintptr_t>(p) % k == 0; };
            const bool bits8 = x.state == BSQ_MOMENTS_8BIT;
            t.e[i] = {x.param, x.grad, x.m, x.v, x.m_scales, x.v_scales, static_cast<__nv_bfloat16*>(x.copy), x.n, at,
                      (int8_t)(x.param_type == BSQ_OUT_BF16), (int8_t)(x.grad_type == BSQ_OUT_BF16), (int8_t)bits8,
                      (int8_t)(on(x.param, 16) && on(x.grad, 16) && on(x.copy, 16) && on(x.m, bits8 ? 8 : 16) &&
                               on(x.v, bits8 ? 8 : 16))};
            t.first[i + 1] = t.first[i] + (int32_t)((x.n + kChunk - 1) / kChunk);
        }
        if (t.count == 0) break;
        const unsigned grid = (unsigned)std::min(t.first[t.count], a.num_sms * 16);
        e = random ? launch_k(false, adamw_kernel<CAP, true>, dim3(grid), kThreads, 0, st, t, o)
                   : launch_k(false, adamw_kernel<CAP, false>, dim3(grid), kThreads, 0, st, t, o);
    }
    return e;
}

}  // namespace

cudaError_t run_adamw(const AdamwArgs& a, cudaStream_t st) {
    const bsq_adamw_options& x = *static_cast<const bsq_adamw_options*>(a.options);
    Options o{};
    o.beta1 = (float)x.beta1;
    o.beta2 = (float)x.beta2;
    o.c1 = (float)(1.0 - x.beta1);
    o.c2 = (float)(1.0 - x.beta2);
    o.eps = (float)x.eps;
    o.decay = (float)(1.0 - x.lr * x.weight_decay);
    o.size = (float)(x.lr / (1.0 - std::pow(x.beta1, (double)x.step)));
    o.root = (float)(1.0 / std::sqrt(1.0 - std::pow(x.beta2, (double)x.step)));
    o.norm = x.norm;
    o.max_norm = (float)x.max_norm;
    o.clip_eps = (float)x.clip_eps;
    o.seed_lo = (uint32_t)x.seed;
    o.seed_hi = (uint32_t)(x.seed >> 32);
    o.step = x.step;
    o.step_at = x.step_device;
    o.lr_at = x.lr_device;
    o.lr = (float)x.lr;
    o.weight_decay = (float)x.weight_decay;
    o.log_beta1 = (float)std::log(x.beta1);
    o.log_beta2 = (float)std::log(x.beta2);
    return a.count <= kSmall ? run<kSmall>(a, o, x.stochastic != 0, st) : run<kLarge>(a, o, x.stochastic != 0, st);
}

}  // namespace bsq
