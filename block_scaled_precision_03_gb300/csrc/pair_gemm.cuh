// BF16 products on CTA pairs (tcgen05 cta_group::2, M = N = 256, K = 16 per MMA),
// shared by the linear head and the feed-forward layers: operand descriptors
// and tensor maps (K-major and MN-major, 128-byte swizzle), the order of the
// tiles, bounded waits, and the epilogue's reads of tensor memory and stores.
#pragma once
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include "tcgen05.cuh"
#include "tmap.h"

namespace bsq {
namespace pair {

constexpr int kTile = 256;                          // output rows and columns of a pair
constexpr int kSubK = 64;                           // K of one 128-byte sub-step
constexpr int kSub = 2;                             // sub-steps per stage
constexpr int64_t kL2Resident = 40ll << 20;         // operand bytes that stay in L2 while others stream past

// Operand descriptors as two words: only the lower one, with the address, changes.
struct Desc {
    uint32_t lo, hi;
    __device__ __forceinline__ explicit Desc(uint64_t d) : lo((uint32_t)d), hi((uint32_t)(d >> 32)) {}
    __device__ __forceinline__ Desc(uint32_t l, uint32_t h) : lo(l), hi(h) {}
    __device__ __forceinline__ Desc operator+(uint32_t n) const { return {lo + n, hi}; }
};
template <bool ACC>
__device__ __forceinline__ void mma_bf16(uint32_t d, Desc a, Desc b, uint32_t idesc, uint32_t acc) {
    if (ACC)
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
                     "setp.eq.b32 p, 0, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t}"
                     :: "r"(d), "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
                     "setp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t}"
                     :: "r"(d), "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(acc) : "memory");
}
// tcgen05 instruction descriptor of kind::f16: bits 4-5 FP32 accumulator,
// 7-9 and 10-12 BF16 operands, 15 and 16 MN-major A and B, 17-22 N>>3 (left
// 0 here), 24-28 M>>4.
__host__ __device__ constexpr uint32_t idesc_bf16(bool amn, bool bmn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((amn ? 1u : 0u) << 15) | ((bmn ? 1u : 0u) << 16) |
           ((uint32_t)(kTile >> 4) << 24);
}
// Descriptor of an MN-major operand tile with 128-byte swizzle: rows of 64
// contiguous M (or N) elements, one per k; 8 of them 1024 bytes apart, the
// next 64 elements a box of 64 rows (8192 bytes) further.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.s32 [%0], %1;" :: "r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool ADD>
__device__ __forceinline__ void tma_store_3d(const void* tmap, int32_t x, int32_t y, int32_t z, uint32_t src) {
    if (ADD)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                     :: "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];"
                     :: "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
}

// Epilogue stores.  A warp's 32 rows leave in chunks of 64 bytes a row (32
// BF16 or 16 FP32 columns) through two 2 KB staging buffers laid out with the
// 64-byte swizzle (16-byte unit u of row r at unit u ^ ((r >> 1) & 3)), one
// TMA tile store each; `n` counts the warp's chunks.
__device__ __forceinline__ void put_chunk(const uint32_t (&w)[16], uint32_t buf, int lane) {
    const uint32_t row = buf + (uint32_t)lane * 64u, sw = (uint32_t)((lane >> 1) & 3);
#pragma unroll
    for (int u = 0; u < 4; u++)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                     :: "r"(row + ((u ^ sw) << 4)), "r"(w[4 * u]), "r"(w[4 * u + 1]), "r"(w[4 * u + 2]), "r"(w[4 * u + 3])
                     : "memory");
}
__device__ __forceinline__ void get_chunk(uint32_t (&w)[16], uint32_t buf, int lane) {
    const uint32_t row = buf + (uint32_t)lane * 64u, sw = (uint32_t)((lane >> 1) & 3);
#pragma unroll
    for (int u = 0; u < 4; u++)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * u]), "=r"(w[4 * u + 1]), "=r"(w[4 * u + 2]), "=r"(w[4 * u + 3])
                     : "r"(row + ((u ^ sw) << 4)) : "memory");
}
__device__ __forceinline__ void stage_chunk(const uint32_t (&w)[16], uint32_t buf, int lane) {
    put_chunk(w, buf, lane);
    tc::fence_async_smem();
    __syncwarp();
}
// the buffer of chunk n may be written again: at most one store still reads its own
__device__ __forceinline__ uint32_t chunk_buffer(uint32_t base, int n, int lane) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
    return base + (uint32_t)(n & 1) * 2048u;
}
__device__ __forceinline__ void store_bf16(const float (&v)[32], float alpha, uint32_t base, const void* tmap, int col,
                                           int row, int& n, int lane) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; j++) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j] * alpha, v[2 * j + 1] * alpha);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    const uint32_t buf = chunk_buffer(base, n++, lane);
    stage_chunk(w, buf, lane);
    if (lane == 0) {
        tc::tma_store_2d(tmap, col, row, buf);
        tc::bulk_commit();
    }
}
__device__ __forceinline__ void store_acc(const float (&v)[32], uint32_t base, const void* tmap, int col, int row, int split,
                                          bool add, int& n, int lane) {
#pragma unroll
    for (int c = 0; c < 2; c++) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; j++) w[j] = __float_as_uint(v[16 * c + j]);
        const uint32_t buf = chunk_buffer(base, n++, lane);
        stage_chunk(w, buf, lane);
        if (lane == 0) {
            if (add) tma_store_3d<true>(tmap, col + 16 * c, row, split, buf);
            else tma_store_3d<false>(tmap, col + 16 * c, row, split, buf);
            tc::bulk_commit();
        }
    }
}
// store_acc through a staging area of its own (struct Staging)
template <typename S>
__device__ __forceinline__ void store_part(const float (&v)[32], S& st, const void* tmap, int col, int row, int split, int lane) {
#pragma unroll
    for (int c = 0; c < 2; c++) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; j++) w[j] = __float_as_uint(v[16 * c + j]);
        const uint32_t buf = st.next(lane);
        stage_chunk(w, buf, lane);
        if (lane == 0) {
            tma_store_3d<false>(tmap, col + 16 * c, row, split, buf);
            tc::bulk_commit();
        }
    }
}
// 16 more columns of a chunk's accumulator onto a running sum
__device__ __forceinline__ void add_acc(float* sum, uint32_t taddr) {
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
    tc::tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; j++) sum[j] += __uint_as_float(r[j]);
}
// 32 columns of the accumulator at `taddr`
__device__ __forceinline__ void load_acc(float (&v)[32], uint32_t taddr) {
    uint32_t r[32];
    BSQ_TMEM_LD32(r, taddr);
    tc::tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; j++) v[j] = __uint_as_float(r[j]);
}

// A bounded wait that polls for a while (some 2000 cycles) before it suspends the
// thread: waking up again costs more than most of these waits last.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* status,
                                     uint64_t limit_ns) {
#pragma unroll 1
    for (int i = 0; i < 64; i++)
        if (tc::mbar_test(bar, parity)) return true;
    return tc::mbar_wait_slow(bar, parity, abort_flag, status, limit_ns);
}

struct TileAt {
    int mt, nt, split, k0, k1;
};
template <typename P>
__device__ __forceinline__ TileAt tile_at(const P& p, int t) {
    TileAt a;
    const int per = p.m_tiles * p.n_tiles;
    a.split = p.splits > 1 ? t / per : 0;
    t -= a.split * per;
    const int MT = p.raster_n ? p.n_tiles : p.m_tiles, NT = p.raster_n ? p.m_tiles : p.n_tiles;
    const int g = t / (p.raster * NT);
    const int first = g * p.raster;
    const int gm = min(p.raster, MT - first);
    const int local = t - g * p.raster * NT;
    const int x = first + local % gm, y = local / gm;
    a.mt = p.raster_n ? y : x;
    a.nt = p.raster_n ? x : y;
    a.k0 = a.split * p.split_stages;
    a.k1 = min(p.k_stages, a.k0 + p.split_stages);
    return a;
}

// After an abort: every stage load in flight lands before the pair exits.
// Load k goes to stage k % stages, phase (k / stages) & 1, on the even CTA,
// which arms each load with both CTAs' bytes; a load that only one CTA issued
// gets the missing half of that accounting here.
static __device__ __noinline__ void drain_loads(uint32_t full0, int stages, int n_own, int n_peer, uint32_t tx) {
    const int n = max(n_own, n_peer);
    for (int k = max(0, n - stages); k < n; k++) {
        const uint32_t bar = full0 + 8 * (uint32_t)(k % stages);
        if (k < n_own && k >= n_peer) tc::mbar_complete_tx(bar, tx);
        if (k < n_peer && k >= n_own) tc::mbar_expect_tx(bar, tx);
        volatile int no_abort = 0;
        tc::mbar_wait(bar, (uint32_t)((k / stages) & 1), &no_abort, nullptr, 100000000ull);
    }
}

// BF16 matrix [rows, cols] with pitch ld, box 64 columns x box_rows, 128-byte
// swizzle; elements outside read as zero.
inline bool map_operand(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows) {
    tmap::EncodeTiledFn enc = tmap::encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(ld * 2)};
    cuuint32_t box[2] = {64u, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// FP32 accumulator [splits][rows][cols], box 16 columns x 32 rows, 64-byte swizzle
inline bool map_acc(CUtensorMap* m, float* p, int64_t splits, int64_t rows, int64_t cols) {
    tmap::EncodeTiledFn enc = tmap::encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)splits};
    cuuint64_t strides[2] = {(cuuint64_t)(cols * 4), (cuuint64_t)(rows * cols * 4)};
    cuuint32_t box[3] = {16u, 32u, 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}


// Order of the tiles: groups of `raster` tiles along m (or n), swept along the
// other dimension.  A group's strips (a strip: 256 rows of an operand, all of
// K) that fit in L2 are read from memory once, the other operand once per
// group; where they do not, each wave of tiles reads the strips it touches.
// The order with the fewest bytes is taken.  Measured (8192 x 65536 x 4096):
// 16 row tiles 2.451 ms, 12 2.481, 24 2.458, and 8 or 32 (67 MB, which do not
// stay) 4 to 6% slower.
template <typename P>
void choose_raster(P& p, int64_t K, int pairs) {
    const double strip_a = 512.0 * K, strip_b = 2.0 * p.tile_n * K;
    const double a_bytes = strip_a * p.m_tiles, b_bytes = strip_b * p.n_tiles;
    const double waves = (double)p.m_tiles * p.n_tiles / pairs;
    double best = 0.0;
    for (int along_n = 0; along_n < 2; along_n++) {
        const int tiles = along_n ? p.n_tiles : p.m_tiles, others = along_n ? p.m_tiles : p.n_tiles;
        const double own = along_n ? strip_b : strip_a, other = along_n ? strip_a : strip_b;
        for (int most = 1; most <= std::min(tiles, 2 * pairs); most++) {
            const int groups = (tiles + most - 1) / most, g = (tiles + groups - 1) / groups;
            const double across = std::min<double>(others, std::max(1.0, (double)pairs / g));
            const double bytes = g * own <= (double)kL2Resident
                                     ? (along_n ? b_bytes : a_bytes) + groups * (along_n ? a_bytes : b_bytes)
                                     : waves * (std::min(g, pairs) * own + across * other);
            if (best == 0.0 || bytes < best) {
                best = bytes;
                p.raster = g;
                p.raster_n = along_n;
            }
        }
    }
}

// Rows of w that a pair takes at a time when the time goes to streaming w (few
// tokens): the pairs should get equally many, so the size that gives the
// busiest pair the fewest.  (50021 rows: 196 tiles of 256 leave 76 pairs 2 or 3
// each, 224 of 224 nearly always 3.)
inline int stream_rows(int64_t vocab, int num_sms) {
    const int64_t pairs = std::max(1, num_sms / 2);
    int best = kTile;
    int64_t least = INT64_MAX;
    for (int t = kTile; t >= 96; t -= 16) {
        const int64_t load = ((vocab + t - 1) / t + pairs - 1) / pairs * t;
        if (load < least) {
            least = load;
            best = t;
        }
    }
    return best;
}

}  // namespace pair
}  // namespace bsq
