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
// 1024 elements, 8 neighbours a thread: a block of 32 is four lanes.
#include <algorithm>
#include <cmath>
#include "../../include/bsq.h"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace bsq {
namespace {

constexpr int kThreads = 128;
constexpr int kPer = 8;                             // elements of a thread
constexpr int kCtas = 32;                           // at most, of an SM
constexpr int64_t kChunk = (int64_t)kThreads * kPer;

struct Entry {
    void* p;
    const void* g;
    void *m, *v;                   // FP32, or codes
    uint8_t *m_scales, *v_scales;
    __nv_bfloat16* copy;
    int64_t n;
    uint32_t key;                  // of its random bits, before the step's number
    int8_t p_bf16, g_bf16;
    int8_t vec, p_vec, g_vec, copy_vec;    // on 16-byte boundaries: the moments (codes: 8), and the others
};
template <int CAP>
struct Table {
    Entry e[CAP];
    int32_t first[CAP + 1];        // chunks before each tensor
    int32_t count;
};
constexpr int kSmall = 16, kMiddle = 96, kLarge = 384;   // the smallest that holds the list travels
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
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x7FEB352Du;
    x ^= x >> 15;
    x *= 0x846CA68Bu;
    return x ^ (x >> 16);
}
// mix((at + i) ^ key) for the 8 elements from `at` on, a multiple of 8: i stays in the lowest bits
__device__ __forceinline__ void random_bits(uint32_t at, uint32_t key, uint32_t (&bits)[kPer]) {
    uint32_t x = at ^ key;
    x ^= x >> 16;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        uint32_t b = (x ^ (uint32_t)i) * 0x7FEB352Du;
        b = (b ^ (b >> 15)) * 0x846CA68Bu;
        bits[i] = b ^ (b >> 16);
    }
}
// The largest and smallest of 8 floats that are not negative, by their bits, which are in the same order: NaN is above
// infinity, and a NaN with its sign set is below 0.
__device__ __forceinline__ int32_t bits_of(float x) { return __float_as_int(x); }
__device__ __forceinline__ int32_t largest(const float (&x)[kPer]) {
    const int32_t a = __vimax3_s32(bits_of(x[0]), bits_of(x[1]), bits_of(x[2])), b = __vimax3_s32(bits_of(x[3]), bits_of(x[4]), bits_of(x[5]));
    return max(__vimax3_s32(a, b, bits_of(x[6])), bits_of(x[7]));
}
__device__ __forceinline__ int32_t smallest(const float (&x)[kPer]) {
    const int32_t a = __vimin3_s32(bits_of(x[0]), bits_of(x[1]), bits_of(x[2])), b = __vimin3_s32(bits_of(x[3]), bits_of(x[4]), bits_of(x[5]));
    return min(__vimin3_s32(a, b, bits_of(x[6])), bits_of(x[7]));
}
// Of 8 magnitudes the largest (NaN if one is) and the smallest
__device__ __forceinline__ float largest_magnitude(const float (&x)[kPer]) {
    float a, b;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(x[0]), "f"(x[1]), "f"(x[2]));
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(b) : "f"(x[3]), "f"(x[4]), "f"(x[5]));
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(a), "f"(b), "f"(x[6]));
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(a), "f"(x[7]), "f"(x[7]));
    return a;
}
__device__ __forceinline__ float smallest_magnitude(const float (&x)[kPer]) {
    float a, b;
    asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(x[0]), "f"(x[1]), "f"(x[2]));
    asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(b) : "f"(x[3]), "f"(x[4]), "f"(x[5]));
    asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(a), "f"(b), "f"(x[6]));
    asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(a), "f"(x[7]), "f"(x[7]));
    return a;
}
// 2^(byte - 127)
__device__ __forceinline__ float power(uint32_t byte) { return __uint_as_float(byte == 0 ? 1u << 22 : byte << 23); }

// The 8 moments x of a thread (their block: four neighbouring lanes) as codes and a scale byte.
//
// Stochastically a value, already scaled, goes to the E4M3 grid by 16 random bits added below the three bits of
// mantissa that stay, sign and magnitude apart by themselves.  Below 2^-6 the grid's steps are 2^-9: with 2^-6 added
// they are those of the next binade.  A thread with such a value (one in some 10000 moments) takes the longer way,
// on which a second moment that is not 0 is kept from becoming so.
template <bool RANDOM, bool ROOT>
__device__ __forceinline__ uint2 encode(const float (&x)[kPer], uint32_t most, const uint32_t (&bits)[kPer], uint32_t& byte) {
    // `most`: bits of the largest magnitude; those of NaN and infinity are above all others
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
    if (most >= 0x7F800000u) {
        byte = 0xFF;
        return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    }
    const int e = (int)(__float_as_uint(__fmul_rn(__uint_as_float(most), 8.0f / 7.0f)) >> 23) - 8;
    byte = (uint32_t)max(e, 0);
    const F2 up(power(254 - byte));
    float y[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
        const float2 a = (F2(x[i], x[i + 1]) * up).get();
        y[i] = a.x;
        y[i + 1] = a.y;
    }
    // (16 random bits four places up: their half of the word times 16, by a product of halves and bytes)
    const auto cut = [&](float a, int i) {
        const uint32_t c = __dp2a_lo(bits[i], ROOT ? 0x1000u : 0x0010u, __float_as_uint(a));
        return __uint_as_float(c & 0xFFF00000u);
    };
    if (smallest_magnitude(y) >= 0.015625f) {
        if (RANDOM)
#pragma unroll
            for (int i = 0; i < kPer; i++) y[i] = cut(y[i], i);
        return pack8_fp8<kE4M3>(y);
    }
    uint2 c;
    if (RANDOM) {
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const float a = fabsf(y[i]), low = a < 0.015625f ? 0.015625f : 0.0f;
            y[i] = copysignf(__fsub_rn(cut(__fadd_rn(a, low), i), low), x[i]);
        }
    }
    c = pack8_fp8<kE4M3>(y);
    if (ROOT)
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            uint32_t& w = i < 4 ? c.x : c.y;
            if (x[i] != 0.0f && (w >> (8 * (i & 3)) & 0xFF) == 0) w |= 1u << (8 * (i & 3));
        }
    return c;
}
__device__ __forceinline__ void decode(uint2 codes, uint32_t byte, F2 (&x)[kPer / 2]) {
    const F2 s(power(byte));
    const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t h2;
        const uint16_t in = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(in));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        x[i] = F2(f.x, f.y) * s;
    }
}

// 8 BF16 elements off 16-byte boundaries as four words, read and written two at a time where those lie on 4-byte boundaries
__device__ __forceinline__ void get_pairs(const uint16_t* q, uint32_t (&w)[4]) {
    if (reinterpret_cast<uintptr_t>(q) & 2) {
        const uint32_t* k = reinterpret_cast<const uint32_t*>(q + 1);
        const uint32_t first = q[0], a = k[0], b = k[1], c = k[2], last = q[7];
        w[0] = first | a << 16;
        w[1] = __funnelshift_l(a, b, 16);
        w[2] = __funnelshift_l(b, c, 16);
        w[3] = c >> 16 | last << 16;
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = reinterpret_cast<const uint32_t*>(q)[i];
    }
}
__device__ __forceinline__ void put_pairs(uint16_t* q, const uint32_t (&w)[4]) {
    if (reinterpret_cast<uintptr_t>(q) & 2) {
        uint32_t* k = reinterpret_cast<uint32_t*>(q + 1);
        q[0] = (uint16_t)w[0];
#pragma unroll
        for (int i = 0; i < 3; i++) k[i] = __funnelshift_l(w[i], w[i + 1], 16);
        q[7] = (uint16_t)(w[3] >> 16);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) reinterpret_cast<uint32_t*>(q)[i] = w[i];
    }
}
// 8 elements at p[at ..), the first n of them; 16-byte (codes: 8-byte) accesses where `vec`
__device__ __forceinline__ void put(void* p, int64_t at, int bf16, bool vec, int n, const float (&x)[kPer]) {
    if (bf16) {
        __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p) + at;
        if (vec || n == kPer) {
            Pack<__nv_bfloat16, 8> k;
            k.pack(x);
            if (vec) k.store(q);
            else {
                const uint32_t w[4] = {k.v.x, k.v.y, k.v.z, k.v.w};
                put_pairs(reinterpret_cast<uint16_t*>(q), w);
            }
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

// The moments of 8 elements.  A packed product and the addition behind it came out as one fused instruction, in spite
// of their .rn, so a product that is added is two single ones.
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    const float2 x = a.get(), y = b.get();
    return F2(__fmul_rn(x.x, y.x), __fmul_rn(x.y, y.y));
}
__device__ __forceinline__ void moments(const float (&g)[kPer], float (&m)[kPer], float (&v)[kPer], const Options& o, float factor) {
    const F2 b1(o.beta1), b2(o.beta2), c1(o.c1), c2(o.c2), f(factor);
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
        const F2 x = F2(g[i], g[i + 1]) * f;                // (times 1 without clipping)
        const float2 ms = (mul2(b1, F2(m[i], m[i + 1])) + mul2(c1, x)).get();
        const float2 vs = (mul2(b2, F2(v[i], v[i + 1])) + mul2(c2 * x, x)).get();
        m[i] = ms.x; m[i + 1] = ms.y;
        v[i] = vs.x; v[i + 1] = vs.y;
    }
}
// Their parameters; r: the root of v.
//
// The root and the quotient are correctly rounded by Newton steps with a fused
// multiply-add (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990): from y = 1 / sqrt(v) to some 23 bits, g = v y and h = y
// / 2 are brought to full precision by one step, and the exact remainder v - g^2 rounds
// g; for m / d the remainder m - d q does.  In packed instructions that is 4.5 and 3.5
// of them an element, a third of the library's IEEE functions.  The remainders are exact
// and the quotient is neither infinite nor below 2^-126 while r lies in 2^-45 .. 2^25, |m|
// in 2^-90 .. 2^80 or is 0, 1 / sqrt(1 - beta2^step) is at most 2^10 and eps at most 2^34:
// d lies in 2^-45 .. 2^36, m / d is at most 2^125, and its remainder a multiple of 2^-149
// (in_range, usual; a v of 0, an infinite one and NaN leave an r that is not in range).
// Elsewhere the library's functions.  (The ranges are looked at behind the update, where
// the largest r and |m| are what the 8-bit codes' scales take too; before it, those of v
// and m, 243 M weights in 12 tensors took 513 us to nearest, 487 now.)
struct Largest {
    uint32_t m, r;                 // bits of the largest magnitudes
};
__device__ __forceinline__ Largest largest_of(const float (&m)[kPer], const float (&r)[kPer]) {
    return {__float_as_uint(largest_magnitude(m)), (uint32_t)largest(r)};
}
__device__ __forceinline__ bool in_range(const float (&m)[kPer], const float (&r)[kPer], const Largest& most) {
    constexpr int32_t least = (127 - 45) << 23;
    bool in = smallest(r) >= least && most.r <= (127u + 25) << 23 && most.m <= (127u + 80) << 23;
    if (smallest_magnitude(m) < 0x1p-90f) {        // 0, or too small
#pragma unroll
        for (int i = 0; i < kPer; i++) in = in && (fabsf(m[i]) >= 0x1p-90f || m[i] == 0.0f);
    }
    return in;
}
__device__ __forceinline__ bool usual(const Options& o) { return o.root <= 1024.0f && o.eps <= 0x1p34f; }
__device__ __forceinline__ void update(float (&p)[kPer], const float (&m)[kPer], const float (&v)[kPer], float (&r)[kPer],
                                       const Options& o) {
    const F2 minus(-1.0f);
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
        const F2 vv(v[i], v[i + 1]);
        float y0, y1;
        asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y0) : "f"(v[i]));
        asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y1) : "f"(v[i + 1]));
        const F2 y(y0, y1);
        F2 q = vv * y, h = y * F2(-0.5f);                  // h: -1 / (2 sqrt(v))
        const F2 e = fma2(q, h, F2(0.5f));
        q = fma2(q, e, q);
        h = fma2(h, e, h);
        q = fma2(fma2(q, q, vv * minus), h, q);
        const float2 root = q.get();
        r[i] = root.x; r[i + 1] = root.y;
        // (k: -1 / d and n: -m, so that a quotient of 0 has m's sign)
        const F2 d = mul2(q, F2(o.root)) + F2(o.eps), n = F2(m[i], m[i + 1]) * minus;
        const float2 ds = d.get();
        float i0, i1;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(i0) : "f"(-ds.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(i1) : "f"(-ds.y));
        F2 k(i0, i1);
        k = fma2(k, fma2(d, k, F2(1.0f)), k);
        F2 t = n * k;
        t = fma2(fma2(d, t, n), k, t);
        const float2 x = (mul2(F2(o.decay), F2(p[i], p[i + 1])) + mul2(F2(-o.size), t)).get();
        p[i] = x.x; p[i + 1] = x.y;
    }
}
__device__ __forceinline__ void update_any(float (&p)[kPer], const float (&m)[kPer], const float (&v)[kPer], float (&r)[kPer],
                                           const Options& o) {
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        r[i] = __fsqrt_rn(v[i]);
        const float d = __fadd_rn(__fmul_rn(r[i], o.root), o.eps);
        p[i] = __fsub_rn(__fmul_rn(o.decay, p[i]), __fmul_rn(o.size, __fdiv_rn(m[i], d)));
    }
}

struct Last {
    int tensor, first, next;       // and its chunks
};
// Chunk c of the list: its tensor, and where this thread's elements start
template <int CAP>
struct Place {
    const Entry* e;
    int64_t at;
    int n;                         // of the 8 elements
    bool whole;                    // the warp's elements are all there, and their moments lie on 16-byte boundaries
    // (`last`: where the chunk before was; mostly it is the same tensor)
    __device__ __forceinline__ Place(const Table<CAP>& t, int c, Last& last) {
        if (c >= last.next) {
            int lo = last.tensor, hi = t.count - 1;  // the last tensor whose first chunk is <= c
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (t.first[mid] <= c) lo = mid; else hi = mid - 1;
            }
            last = {lo, t.first[lo], t.first[lo + 1]};
        }
        e = &t.e[last.tensor];
        const int64_t start = (int64_t)(c - last.first) * kChunk;
        const int own = threadIdx.x * kPer, rest = (int)min(kChunk, e->n - start);
        at = start + own;
        n = max(0, min(kPer, rest - own));
        whole = e->vec && rest >= (int)(threadIdx.x & ~31u) * kPer + 32 * kPer;
    }
};
// What a chunk reads, as it lies in memory (elements off 16-byte boundaries put together)
struct Words {
    uint4 v[2];
    __device__ __forceinline__ void load(const void* p, int64_t at, int bf16, bool vec, int n) {
        v[0] = v[1] = make_uint4(0, 0, 0, 0);
        if (bf16) {
            const uint16_t* q = static_cast<const uint16_t*>(p) + at;
            if (vec) {
                v[0] = *reinterpret_cast<const uint4*>(q);
                return;
            }
            uint32_t w[4] = {0, 0, 0, 0};
            if (n == kPer) get_pairs(q, w);
            else
#pragma unroll
                for (int i = 0; i < kPer; i++)
                    if (i < n) w[i >> 1] |= (uint32_t)q[i] << (16 * (i & 1));
            v[0] = make_uint4(w[0], w[1], w[2], w[3]);
            return;
        }
        const uint32_t* q = static_cast<const uint32_t*>(p) + at;
        if (vec) {
            v[0] = reinterpret_cast<const uint4*>(q)[0];
            v[1] = reinterpret_cast<const uint4*>(q)[1];
            return;
        }
        uint32_t w[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i++) w[i] = i < n ? q[i] : 0u;
        v[0] = make_uint4(w[0], w[1], w[2], w[3]);
        v[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    __device__ __forceinline__ void get(int bf16, float (&x)[kPer]) const {
        if (bf16) {
            Pack<__nv_bfloat16, 8> k;
            k.v = v[0];
            k.unpack(x);
            return;
        }
        const uint32_t w[kPer] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int i = 0; i < kPer; i++) x[i] = __uint_as_float(w[i]);
    }
};
template <bool BITS8>
struct Moments;
template <>
struct Moments<false> {
    Words m, v;
    __device__ __forceinline__ void load(const Entry& e, int64_t at, bool vec, int n) {
        m.load(e.m, at, 0, vec, n);
        v.load(e.v, at, 0, vec, n);
    }
    __device__ __forceinline__ void get(float (&a)[kPer], float (&b)[kPer]) const {
        m.get(0, a);
        v.get(0, b);
    }
};
template <>
struct Moments<true> {
    uint2 m, v;
    uint32_t mb, vb;
    __device__ __forceinline__ void load(const Entry& e, int64_t at, bool vec, int n) {
        m = get_codes(e.m, at, vec, n);
        v = get_codes(e.v, at, vec, n);
        mb = n > 0 ? e.m_scales[at >> 5] : 0;
        vb = n > 0 ? e.v_scales[at >> 5] : 0;
    }
    __device__ __forceinline__ void get(float (&a)[kPer], float (&b)[kPer]) const {
        F2 x[kPer / 2], y[kPer / 2];
        decode(m, mb, x);
        decode(v, vb, y);
#pragma unroll
        for (int i = 0; i < kPer / 2; i++) {
            const float2 f = x[i].get(), r = (y[i] * y[i]).get();
            a[2 * i] = f.x;
            a[2 * i + 1] = f.y;
            b[2 * i] = r.x;
            b[2 * i + 1] = r.y;
        }
    }
};

// What a thread holds of a chunk becomes its new state
template <bool RANDOM, bool BITS8, bool ANY>
__device__ __forceinline__ void leave(const Entry& e, int64_t at, int n, bool vec, const Options& o, const float (&m)[kPer],
                                      const float (&v)[kPer], const float (&r)[kPer], const Largest& most, float (&p)[kPer]) {
    const bool p_vec = vec && (!ANY || e.p_vec), copy_vec = vec && (!ANY || e.copy_vec);
    uint32_t bits[kPer] = {};
    if (RANDOM) {
        const uint32_t key = mix(e.key ^ (uint32_t)o.step) + (uint32_t)(at >> 32) * 0x9E3779B9u;
        random_bits((uint32_t)at, key, bits);
    }
    if (BITS8) {
        uint32_t mb, vb;
        const uint2 mc = encode<RANDOM, false>(m, most.m, bits, mb), vc = encode<RANDOM, true>(r, most.r, bits, vb);
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
    if (e.copy) put(e.copy, at, 1, copy_vec, n, p);
    if (RANDOM && e.p_bf16) {
        uint32_t w[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i++)
            w[i] = __dp2a_lo(bits[i] * 0x9E3779B1u, 0x0100u, __float_as_uint(p[i]));
        if (n == kPer && largest_magnitude(p) < INFINITY) {
            // the upper halves are the results
            const uint32_t h[4] = {__byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632), __byte_perm(w[4], w[5], 0x7632),
                                   __byte_perm(w[6], w[7], 0x7632)};
            if (p_vec) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(e.p) + at) = make_uint4(h[0], h[1], h[2], h[3]);
            else put_pairs(static_cast<uint16_t*>(e.p) + at, h);
            return;
        }
        // (NaN and infinity stay as they are: the random bits would carry a NaN over into the sign)
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (fabsf(p[i]) < INFINITY) p[i] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    put(e.p, at, e.p_bf16, p_vec, n, p);
}

// A warp's part of a chunk, 256 elements, is a unit of its own.  The first loop takes those that are whole, with moments
// on 16-byte boundaries, with the next one's loads under way, and stores what was in the range of update(); the rest the
// second loop takes.  ANY: parameters, gradients or copies off those boundaries, a few elements at a time (118 M weights
// in BF16, 8-bit moments, stochastic: 441 us, 944 in the second loop, 292 where all are on them).
// (One loop with both ways in it held its values twice over: 92 instructions an element of 8-bit moments, 78 with two then;
// 81 now, with the ranges of m.)
constexpr int kMost = 2048;                         // chunks of a CTA
template <int CAP, bool RANDOM, bool BITS8, bool ANY>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<CAP> t, Options o) {
    __shared__ uint32_t left[kThreads / 32][kMost / 32];
    uint32_t* mine = left[threadIdx.x >> 5];
    const int lane = threadIdx.x & 31, chunks = t.first[t.count];
    pdl_launch_dependents();
    pdl_wait();
    if (o.step_at || o.lr_at) step_scalars(o);
    float factor = 1.0f;
    if (o.norm) {
        const float f = __fdiv_rn(o.max_norm, __fadd_rn(*o.norm, o.clip_eps));
        factor = f > 1.0f ? 1.0f : f;               // NaN stays NaN
    }
    const bool fast = usual(o);
    struct Chunk {
        Words p, g;
        Moments<BITS8> s;
        __device__ __forceinline__ void load(const Place<CAP>& a, bool vec) {
            p.load(a.e->p, a.at, a.e->p_bf16, vec && (!ANY || a.e->p_vec), a.n);
            g.load(a.e->g, a.at, a.e->g_bf16, vec && (!ANY || a.e->g_vec), a.n);
            s.load(*a.e, a.at, vec, a.n);
        }
    };
    {
        Last last{0, 0, 0};
        Place<CAP> ahead(t, blockIdx.x, last);
        Chunk words;
        if (ahead.whole) words.load(ahead, true);
        uint32_t some = 0;
        int k = 0;
        for (int c = blockIdx.x; c < chunks; k++) {
            const Place<CAP> at = ahead;
            const Entry& e = *at.e;
            float p[kPer], g[kPer], m[kPer], v[kPer], r[kPer];
            words.p.get(e.p_bf16, p);
            words.g.get(e.g_bf16, g);
            words.s.get(m, v);
            c += gridDim.x;
            if (c < chunks) {
                ahead = Place<CAP>(t, c, last);
                if (ahead.whole) words.load(ahead, true);
            }
            if (k > 0 && (k & 31) == 0) {
                if (lane == 0) mine[(k >> 5) - 1] = some;
                some = 0;
            }
            if (at.whole && fast) {
                moments(g, m, v, o, factor);
                update(p, m, v, r, o);
                const Largest most = largest_of(m, r);
                if (__all_sync(0xffffffffu, in_range(m, r, most))) {
                    leave<RANDOM, BITS8, ANY>(e, at.at, kPer, true, o, m, v, r, most, p);
                    continue;
                }
            }
            some |= 1u << (k & 31);
        }
        if (k > 0 && lane == 0) mine[(k - 1) >> 5] = some;
        __syncwarp();
    }
    Last last{0, 0, 0};
    for (int k = 0, c = blockIdx.x; c < chunks; k++, c += gridDim.x) {
        if (!(mine[k >> 5] >> (k & 31) & 1)) continue;
        const Place<CAP> at(t, c, last);
        const Entry& e = *at.e;
        Chunk words;
        words.load(at, at.whole);
        float p[kPer], g[kPer], m[kPer], v[kPer], r[kPer];
        words.p.get(e.p_bf16, p);
        words.g.get(e.g_bf16, g);
        words.s.get(m, v);
        moments(g, m, v, o, factor);
        // elements past the end change no scale; every lane takes part in the block's maximum
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (i >= at.n) {
                m[i] = 0.0f;
                v[i] = 1.0f;
            }
        float q[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i++) q[i] = p[i];
        update(q, m, v, r, o);
        if (!fast || !in_range(m, r, largest_of(m, r))) update_any(p, m, v, r, o);
        else
#pragma unroll
            for (int i = 0; i < kPer; i++) p[i] = q[i];
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (i >= at.n) r[i] = 0.0f;
        leave<RANDOM, BITS8, ANY>(e, at.at, at.n, at.whole, o, m, v, r, largest_of(m, r), p);
    }
}

// The tensors with 8-bit moments or the others: a launch for every CAP of them
template <int CAP, bool RANDOM, bool BITS8>
cudaError_t run(const AdamwArgs& a, const Options& o, cudaStream_t st) {
    const bsq_adamw_tensor* list = static_cast<const bsq_adamw_tensor*>(a.tensors);
    cudaError_t e = cudaSuccess;
    for (int at = 0; at < a.count && e == cudaSuccess;) {
        Table<CAP> t;
        t.count = 0;
        t.first[0] = 0;
        bool any = false;
        for (; at < a.count && t.count < CAP; at++) {
            const bsq_adamw_tensor& x = list[at];
            if (x.n == 0 || (x.state == BSQ_MOMENTS_8BIT) != BITS8) continue;
            const int i = t.count++;
            const auto on = [](const void* p, uintptr_t k) { return reinterpret_cast<uintptr_t>(p) % k == 0; };
            constexpr uintptr_t state = BITS8 ? 8 : 16;
            t.e[i] = {x.param, x.grad, x.m, x.v, x.m_scales, x.v_scales, static_cast<__nv_bfloat16*>(x.copy), x.n,
                      mix(mix((uint32_t)at ^ o.seed_lo) ^ o.seed_hi),
                      (int8_t)(x.param_type == BSQ_OUT_BF16), (int8_t)(x.grad_type == BSQ_OUT_BF16),
                      (int8_t)(on(x.m, state) && on(x.v, state)), (int8_t)on(x.param, 16), (int8_t)on(x.grad, 16), (int8_t)on(x.copy, 16)};
            any |= t.e[i].vec && !(t.e[i].p_vec && t.e[i].g_vec && t.e[i].copy_vec);
            t.first[i + 1] = t.first[i] + (int32_t)((x.n + kChunk - 1) / kChunk);
        }
        if (t.count == 0) break;
        const int n = t.first[t.count];
        const unsigned grid = (unsigned)std::max(std::min(n, a.num_sms * kCtas), (n + kMost - 1) / kMost);
        e = any ? launch_k(true, adamw_kernel<CAP, RANDOM, BITS8, true>, dim3(grid), kThreads, 0, st, t, o)
                : launch_k(true, adamw_kernel<CAP, RANDOM, BITS8, false>, dim3(grid), kThreads, 0, st, t, o);
    }
    return e;
}
template <int CAP>
cudaError_t run(const AdamwArgs& a, const Options& o, bool random, cudaStream_t st) {
    const cudaError_t e = random ? run<CAP, true, false>(a, o, st) : run<CAP, false, false>(a, o, st);
    if (e != cudaSuccess) return e;
    return random ? run<CAP, true, true>(a, o, st) : run<CAP, false, true>(a, o, st);
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
    if (a.count <= kSmall) return run<kSmall>(a, o, x.stochastic != 0, st);
    return a.count <= kMiddle ? run<kMiddle>(a, o, x.stochastic != 0, st) : run<kLarge>(a, o, x.stochastic != 0, st);
}

}  // namespace bsq
