// Programmatic dependent launch and 16-byte vector access, shared by the
// operators around the layer.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace bsq {

// A kernel launched with launch_k(true, ...) may start while the kernel before
// it on the stream still runs.  Such a kernel calls pdl_wait() before its
// first access to global memory; the kernel before it may let it start early
// with pdl_launch_dependents().  Only pdl_wait() makes visible what kernels
// before it wrote, so whoever may follow any kernel waits first, always.  A few
// kernels behind another one of the same call (norm_dx_kernel, moe_place_kernel,
// moe_gather_kernel, scale_kernel, the head's) read before it what that kernel does
// not write, and say so: inputs, as the call's first kernel is launched without this
// attribute, when all the stream's work before the call is done; and, in the head's
// gradient, what a kernel wrote for which the one in between has waited, from L2
// (TMA, __ldcg).  (Waits there cost it 1 to 8%: 2048 tokens of 16384 x 1024 171 us, 159
// without; 8192 of 65536 x 4096 7.9 ms either way.)
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
inline cudaError_t launch_k(bool dependent, void (*k)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st,
                            A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, static_cast<P>(args)...);
}

// N elements of T held packed, as they lie in memory (16 bytes, or one element)
template <typename T, int N>
struct Pack;
template <>
struct Pack<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void pack(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Pack<float, 4> {
    float4 v;
    __device__ __forceinline__ void zero() { v = make_float4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
    __device__ __forceinline__ void unpack(float (&f)[4]) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
    __device__ __forceinline__ void pack(const float (&f)[4]) { v = make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Pack<__nv_bfloat16, 2> {
    uint32_t v;
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint32_t*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint32_t*>(p) = v; }
    __device__ __forceinline__ void unpack(float (&f)[2]) const {
        f[0] = __uint_as_float(v << 16);
        f[1] = __uint_as_float(v & 0xFFFF0000u);
    }
    __device__ __forceinline__ void pack(const float (&f)[2]) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[0], f[1]);
        v = *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <>
struct Pack<__nv_bfloat16, 1> {
    __nv_bfloat16 v;
    __device__ __forceinline__ void zero() { v = __ushort_as_bfloat16(0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *p; }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *p = v; }
    __device__ __forceinline__ void unpack(float (&f)[1]) const { f[0] = __bfloat162float(v); }
    __device__ __forceinline__ void pack(const float (&f)[1]) { v = __float2bfloat16_rn(f[0]); }
};
template <>
struct Pack<float, 1> {
    float v;
    __device__ __forceinline__ void zero() { v = 0.0f; }
    __device__ __forceinline__ void load(const float* p) { v = *p; }
    __device__ __forceinline__ void store(float* p) const { *p = v; }
    __device__ __forceinline__ void unpack(float (&f)[1]) const { f[0] = v; }
    __device__ __forceinline__ void pack(const float (&f)[1]) { v = f[0]; }
};
// Two FP32 values in a register pair, for the packed FP32 instructions (two
// IEEE operations each)
struct F2 {
    unsigned long long v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit F2(float a) : F2(a, a) {}
    __device__ __forceinline__ float2 get() const {
        float2 f;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
        return f;
    }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ void unpack2(const Pack<__nv_bfloat16, 8>& p, F2 (&f)[4]) {
    const uint32_t w[4] = {p.v.x, p.v.y, p.v.z, p.v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = F2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack2(const Pack<float, 4>& p, F2 (&f)[2]) {
    f[0] = F2(p.v.x, p.v.y);
    f[1] = F2(p.v.z, p.v.w);
}
__device__ __forceinline__ void pack2(Pack<__nv_bfloat16, 8>& p, const F2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 x = f[i].get();
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    p.v = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack2(Pack<float, 4>& p, const F2 (&f)[2]) {
    const float2 a = f[0].get(), b = f[1].get();
    p.v = make_float4(a.x, a.y, b.x, b.y);
}

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// ---- rows that start anywhere.  Such a row is walked along the 16-byte
// boundaries of memory: vector v of a row holds its columns v VEC - shift ...,
// shift the elements between the boundary at or before the row's start and
// that start.
template <typename T>
__device__ __forceinline__ int row_shift(const T* row) {
    return (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}
// A vector's elements one by one, for a row that lies to 16-byte boundaries otherwise than the vectors
template <typename T>
__device__ __forceinline__ void load_each(Pack<T, kVec<T>>& p, const T* at) {
    T e[kVec<T>];
#pragma unroll
    for (int i = 0; i < kVec<T>; i++) e[i] = at[i];
    memcpy(&p.v, e, 16);
}
template <typename T>
__device__ __forceinline__ void store_each(const Pack<T, kVec<T>>& p, T* at) {
    T e[kVec<T>];
    memcpy(e, &p.v, 16);
#pragma unroll
    for (int i = 0; i < kVec<T>; i++) at[i] = e[i];
}

// rows of a matrix start on boundaries of `vector` bytes and hold whole vectors
inline bool rows_vec(const void* p, int64_t ld, int64_t cols, int bytes, int vector = 16) {
    return reinterpret_cast<uintptr_t>(p) % vector == 0 && ld * bytes % vector == 0 && cols * bytes % vector == 0;
}

}  // namespace bsq
