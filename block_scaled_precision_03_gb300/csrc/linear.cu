// Linear layers on BF16 operands with their epilogue, and the gated half of a
// feed-forward block, forward and backward:
//   linear   z = x w^T + bias, y = act(z) + residual
//   gated    a = x wg^T, u = x wu^T, h = act(a) * u
//   backward dz = dy act'(z); dx = dz w, dw = dz^T x, dbias = sum of dz's rows
//            da = dh u act'(a), du = dh act(a); dx = da wg + du wu, dwg = da^T x,
//            dwu = du^T x
//
// The products run on CTA pairs (tcgen05 cta_group::2, M = N = 256, K = 16 per
// MMA): each CTA stages its own 128 rows of A and of B by TMA (128-byte
// swizzle), the even CTA issues the MMAs, and two accumulators of 256
// tensor-memory columns let the epilogue of one tile run under the MMAs of the
// next.  An operand is read in the layout it has in memory, K-major or MN-major.
//
// Gated: a pair's tile is 128 columns of both projections.  The even CTA's 128
// rows of B are wg's, the odd one's wu's, so that one MMA makes both, and each
// CTA has gate and up of its own rows in its own tensor memory, 128 columns
// apart: the activation and the product need nothing from anywhere else.
//
// Of up to 192 tokens a tile has 64, 128 or 192 rows, half of them in either CTA: the MMA is the same, but the operand
// takes less of a stage, more stages are in flight, and a box mostly outside the matrix costs the copy engine more than
// its bytes (4096 -> 14336 of 8 tokens, gated, 41 us; 74 with boxes of 128 rows).  (The other way round, z^T = w x^T with
// w's rows as the tile's and the tokens its columns, was as fast at 8 tokens and slower from 32 on: 128 tokens of 4096 ->
// 4096 29 us, 21 now.)
//
// dx of a gated layer is one product over K = 2 F: first da wg, then du wu.
// Where there are too few tiles for the pairs the sum over K is split; a second
// kernel adds the parts in their order and does the epilogue.
//
// The tensor cores' FP32 sums are not rounded to nearest: a sum over K = 4096
// loses some 6e-6, over K = 16384 some 1e-4.  An accumulator is read out every
// kSumChunk stages (K = 16384) where a BF16 result hides that, every kChunk (K =
// 512) for FP32 results, and added up in registers.  (Read out every K = 4096 the
// batch of 8192 x 14336 -> 4096 took 3% longer.)
#include <algorithm>
#include <cuda.h>
#include "common.cuh"
#include "fused.cuh"
#include "internal.h"
#include "launch.cuh"
#include "pair_gemm.cuh"
#include "per_device.h"
#include "tcgen05.cuh"
#include "tmap.h"

namespace bsq {
namespace {

using namespace pair;

enum { kFwd, kDx, kDw, kGrad };                     // kGrad: dx and dw

constexpr int kStages = 3;
constexpr int kMaxStages = 12;                      // of smaller tiles: as many as fit
constexpr int kChunk = 4, kSumChunk = 128;          // stages of K = 128
constexpr int kSubBytes = 128 * kSubK * 2;          // one CTA's 128 rows of an operand, one sub-step
constexpr int kOpBytes = kSub * kSubBytes;
constexpr int kMmas = 4 * kSub;                     // per stage
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr uint32_t kTmemCols = 512;
constexpr int kBarBytes = 320;
constexpr int kStageBytes = 4096;                   // a warp's staging: two chunks of 32 rows x 64 bytes
constexpr int kSmem = 1024 + kStages * 2 * kOpBytes + kEpiWarps * kStageBytes + kBarBytes;
static_assert(kSmem <= 232448, "shared memory per block");

struct Params {
    int64_t M, N;                  // output
    int32_t k_stages, chunk;       // K stages in all; stages per accumulator
    int32_t m_tiles, n_tiles, splits, split_stages, total;
    int32_t raster, raster_n;
    int32_t tile_m, tile_n;
    int32_t sub_a, sub_b;          // one CTA's bytes of A and B per sub-step
    int32_t half;                  // gated: dx's stages of the first pair of operands; dw's tiles along M
    Fused f;
};
struct Job {
    CUtensorMap a[2], b[2], out[3];
    Params p;
};
// dbias from the column sums of the row blocks [blocks][cols], added in their order: 32 columns a round of a CTA, eight
// warps that take every eighth block each.  `all`: their sums in shared memory; sync: of the eight.
constexpr int kSumWarps = 8;
struct BlockSums {
    const float* from;
    int64_t blocks, cols;
    float* out;                    // or nullptr
};
template <typename SYNC>
__device__ __forceinline__ void add_blocks(const BlockSums& b, int warp, int lane, float (*all)[32], SYNC sync) {
    for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < b.cols; c0 += (int64_t)gridDim.x * 32) {
        const int64_t c = c0 + lane;
        float s = 0.0f;
        if (c < b.cols)
#pragma unroll 4
            for (int64_t i = warp; i < b.blocks; i += kSumWarps) s += b.from[i * b.cols + c];
        all[warp][lane] = s;
        sync();
        if (warp == 0 && c < b.cols) {
            s = 0.0f;
#pragma unroll
            for (int w = 0; w < kSumWarps; w++) s += all[w][lane];
            b.out[c] = s;
        }
        sync();
    }
}
// A product, or dx and dw in one launch, whose tiles follow one another: small gradients gain by it (294 x 80 -> 576
// 5.8 us, two launches 8.3; 2048 x 4096 -> 4096 97, 109); of many tiles each has its own launch and program (8192 x 4096 ->
// 14336 with gelu_tanh 1.16 ms, 1.18 in one).  The first launch's epilogue warps add up dbias while they would wait for their first tile.
template <int MODE>
struct Jobs {
    Job job[MODE == kGrad ? 2 : 1];
    int32_t stages, a_bytes, b_bytes;  // stages of the ring, and its room for one CTA's A and B per stage
    int32_t extra;                 // dw's tiles that a pair with one of dx's fewer takes in its place
    BlockSums dbias;
    unsigned* status;
    uint64_t timeout_ns;
};
// A pair's i-th tile, dx's first, each dealt in turn.  Where dx's last round does not reach every pair, the others take
// `extra` tiles of dw in its place, and the rest goes round from the first of them.
template <int MODE>
__device__ __forceinline__ bool nth_tile(const Jobs<MODE>& j, int cid, int ncl, int i, bool& dw, int& t) {
    const int n = j.job[0].p.total;
    t = cid + i * ncl;
    dw = MODE == kDw;
    if (MODE != kGrad || t < n) return t < n;
    dw = true;
    const int all = j.job[MODE == kGrad].p.total, rest = n % ncl, light = ncl - rest;
    int k = i - (cid < n ? (n - cid + ncl - 1) / ncl : 0);
    if (cid >= rest) {
        t = cid - rest + k * light;
        if (k < j.extra) return t < all;
        k -= j.extra;
    }
    t = j.extra * light + (cid >= rest ? cid - rest : cid - rest + ncl) + k * ncl;
    return t < all;
}
// After an abort, as pair::drain_loads: loads of a stage, of the same size or of sizes that the CTA which issued them noted
// per slot
__device__ __noinline__ void drain_ring(uint32_t full0, int stages, int n_own, int n_peer, const volatile uint32_t* tx, uint32_t peer_tx,
                                        uint32_t same) {
    const int n = max(n_own, n_peer);
    for (int k = max(0, n - stages); k < n; k++) {
        const int s = k % stages;
        const uint32_t bar = full0 + 8 * (uint32_t)s;
        const uint32_t bytes = same ? same : k < n_own ? tx[s] : (uint32_t)tc::ld_cluster_s32(peer_tx + 4 * (uint32_t)s);
        if (k < n_own && k >= n_peer) tc::mbar_complete_tx(bar, bytes);
        if (k < n_peer && k >= n_own) tc::mbar_expect_tx(bar, bytes);
        volatile int no_abort = 0;
        tc::mbar_wait(bar, (uint32_t)((k / stages) & 1), &no_abort, nullptr, 100000000ull);
    }
}

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t div_up(int64_t v, int64_t m) { return (v + m - 1) / m; }

// Reads a line of each part of a job, so that its parameters are there when the wait for the kernel before is over
__device__ __forceinline__ void read_ahead(const Params& p) {
    asm volatile("" :: "l"(p.M), "r"(p.k_stages), "r"(p.raster), "r"(p.tile_n), "r"(p.sub_b), "r"(p.f.act), "l"(p.f.bias), "l"(p.f.y),
                 "l"(p.f.u));
}
template <uint32_t V>
struct Constant {
    static constexpr uint32_t value = V;
};

// LONG: a tile's sum over K takes several accumulators.
template <int MODE, bool GATED, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
linear_gemm_kernel(const __grid_constant__ Jobs<MODE> j) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // [stages] of A, [stages] of B, the epilogue's staging; the barriers come last
    constexpr bool GRAD = MODE != kFwd, BOTH = MODE == kGrad;
    const int S = j.stages, a_bytes = j.a_bytes, b_bytes = j.b_bytes;
    uint8_t* smA = base;
    uint8_t* smB = smA + S * a_bytes;
    uint8_t* smOut = base + kStages * 2 * kOpBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + (kSmem - 1024 - kBarBytes));
    // full[S], empty[S], tfull[2], tempty[2], drain, and the bytes of a load per stage
    const uint32_t full0 = tc::smem_u32(bars), empty0 = tc::smem_u32(bars + kMaxStages);
    const uint32_t tfull0 = tc::smem_u32(bars + 2 * kMaxStages), tempty0 = tc::smem_u32(bars + 2 * kMaxStages + 2);
    const uint32_t drain = tc::smem_u32(bars + 2 * kMaxStages + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* issued_slot = reinterpret_cast<volatile int*>(tmem_slot + 2);
    volatile int* peer_abort = reinterpret_cast<volatile int*>(tmem_slot + 3);
    volatile uint32_t* load_tx = tmem_slot + 4;
    static_assert(8 * (2 * kMaxStages + 5) + 16 + 4 * kMaxStages <= kBarBytes, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const bool leader = rank == 0;
    const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    const Job& ahead = j.job[BOTH && cid >= j.job[0].p.total];
    read_ahead(ahead.p);
    if (warp == 0 && lane == 0) {
        for (int s = 0; s < S; s++) {
            tc::mbar_init(full0 + 8 * s, 1);
            tc::mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; b++) {
            tc::mbar_init(tfull0 + 8 * b, 1);
            tc::mbar_init(tempty0 + 8 * b, 2 * kEpiWarps);
        }
        tc::mbar_init(drain, 1);
        *abort_flag = 0;
        *issued_slot = 0;
        *peer_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tc::prefetch_tmap(&ahead.a[0]);
        tc::prefetch_tmap(&ahead.b[0]);
    }
    if (warp == 1) tc::tmem_alloc<2>(tc::smem_u32(tmem_slot), kTmemCols);
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs)
        if (lane == 0) {
            const uint32_t full_c0 = tc::mapa(full0, 0);
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            // (its set-up runs beside the kernel before it on the stream)
            pdl_wait();
            bool dw;
            for (int i = 0, t; ok && nth_tile(j, cid, ncl, i, dw, t); i++) {
                const Job& job = j.job[BOTH && dw];
                const Params& p = job.p;
                const TileAt ti = tile_at(p, t);
                // which of the two operand pairs of a gated layer's dw
                const int which = GATED && dw && ti.mt >= p.half ? 1 : 0;
                const int am = (ti.mt - which * p.half) * p.tile_m + (int)rank * (p.tile_m / 2);
                // a gated layer's tile is half as many columns of either projection
                const int bn = !GRAD && GATED ? ti.nt * (p.tile_n / 2) : ti.nt * p.tile_n + (int)rank * (p.tile_n / 2);
                const int half = GATED && GRAD && !dw ? p.half : ti.k1, sub_a = p.sub_a, sub_b = p.sub_b;
                const uint32_t tx = (uint32_t)(kSub * (sub_a + sub_b));
                const bool wide = p.tile_n > 128;
                for (int kb = ti.k0; kb < ti.k1; kb++) {
                    if (!wait(empty0 + 8 * stage, phase ^ 1, abort_flag, j.status, j.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full_c0 + 8 * stage;
                    if (BOTH) load_tx[stage] = tx;
                    if (leader) tc::mbar_expect_tx(full0 + 8 * stage, 2 * tx);
                    const int second = GRAD && GATED && kb >= half ? 1 : 0;        // dx of a gated layer
                    const CUtensorMap* ma = &job.a[GRAD ? (dw ? which : second) : 0];
                    const CUtensorMap* mb = &job.b[GRAD ? second : GATED ? (int)rank : 0];
#pragma unroll
                    for (int u = 0; u < kSub; u++) {
                        const int k = ((kb - second * half) * kSub + u) * kSubK;
                        const uint32_t da = tc::smem_u32(smA + stage * a_bytes + u * sub_a);
                        const uint32_t db = tc::smem_u32(smB + stage * b_bytes + u * sub_b);
                        if (dw) {
                            tc::tma_load_2d_pair(da, ma, am, k, fb);
                            tc::tma_load_2d_pair(da + 8192, ma, am + 64, k, fb);
                        } else {
                            tc::tma_load_2d_pair(da, ma, k, am, fb);
                        }
                        if (GRAD) {
                            tc::tma_load_2d_pair(db, mb, bn, k, fb);
                            if (wide) tc::tma_load_2d_pair(db + 8192, mb, bn + 64, k, fb);
                        } else {
                            tc::tma_load_2d_pair(db, mb, k, bn, fb);
                        }
                    }
                    ++issued;
                    if (++stage == S) { stage = 0; phase ^= 1; }
                }
            }
            // What comes next on the stream starts when every CTA has its last loads under way.  (From the wait on, its CTAs
            // crowded into the first SMs that were free: the gradient of 1021 x 2040 -> 1531 with gelu 34.3 us in a row, 30.4 now.)
            pdl_launch_dependents();
            *issued_slot = issued;
            if (!ok) *abort_flag = 1;
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (even CTA)
        if (lane == 0 && leader) {
            // K-major and MN-major operands; 16 k further: 32 bytes of a K-major row, 16 rows of an MN-major tile
            constexpr uint32_t k_step = 2, mn_step = 2048 >> 4, b_step = GRAD ? mn_step : k_step;
            const uint64_t bd0 = GRAD ? desc_mn_sw128(tc::smem_u32(smB)) : tc::desc_sw128(tc::smem_u32(smB));
            int stage = 0, iter = 0;
            uint32_t phase = 0;
            bool ok = true, any = false, ready = false;
            pdl_wait();                                    // the limit of its waits counts from there
            bool dw;
            for (int i = 0, t; ok && nth_tile(j, cid, ncl, i, dw, t); i++) {
                const Params& p = j.job[BOTH && dw].p;
                const TileAt ti = tile_at(p, t);
                const uint32_t idesc = idesc_bf16(dw, GRAD) | ((uint32_t)(p.tile_n >> 3) << 17);
                const uint64_t ad0 = dw ? desc_mn_sw128(tc::smem_u32(smA)) : tc::desc_sw128(tc::smem_u32(smA));
                const uint32_t sub_a = (uint32_t)p.sub_a >> 4, sub_b = (uint32_t)p.sub_b >> 4;
                const int chunk = p.chunk;
                const auto run = [&](auto a_step) {
                    for (int c0 = ti.k0; c0 < ti.k1 && ok; c0 += chunk, ++iter) {
                        const int c1 = min(ti.k1, c0 + chunk), buf = iter & 1;
                        if (!wait(tempty0 + 8 * buf, ((iter >> 1) & 1) ^ 1, abort_flag, j.status, j.timeout_ns)) {
                            ok = false;
                            break;
                        }
                        const uint32_t d = tmem + (uint32_t)buf * kTile;
                        for (int kb = c0; kb < c1; kb++) {
                            if (!ready && !wait(full0 + 8 * stage, phase, abort_flag, j.status, j.timeout_ns)) {
                                ok = false;
                                break;
                            }
                            tc::fence_after();
                            const Desc ad = Desc(ad0) + (uint32_t)(stage * (a_bytes >> 4));
                            const Desc bd = Desc(bd0) + (uint32_t)(stage * (b_bytes >> 4));
                            const int next = stage + 1 == S ? 0 : stage + 1;
                            const uint32_t next_phase = next == 0 ? phase ^ 1 : phase;
                            // the next stage's barrier is tested while this stage's MMAs run
#pragma unroll
                            for (int m = 0; m < kMmas; m++) {
                                if (m == kMmas - 1) ready = tc::mbar_test(full0 + 8 * next, next_phase);
                                const Desc am = ad + (m >> 2) * sub_a + (m & 3) * a_step.value;
                                const Desc bm = bd + (m >> 2) * sub_b + (m & 3) * b_step;
                                if (m == 0) mma_bf16<false>(d, am, bm, idesc, kb != c0);
                                else mma_bf16<true>(d, am, bm, idesc, 1);
                            }
                            any = true;
                            tc::commit<2>(empty0 + 8 * stage, 3);
                            if (kb == c1 - 1) tc::commit<2>(tfull0 + 8 * buf, 3);
                            stage = next;
                            phase = next_phase;
                        }
                    }
                };
                if (dw) run(Constant<mn_step>());
                else run(Constant<k_step>());
            }
            if (!ok) *abort_flag = 1;
            if (any) {
                // every MMA issued finishes before tensor memory is released
                tc::commit<2>(drain, 1);
                volatile int no_abort = 0;
                tc::mbar_wait(drain, 0, &no_abort, nullptr, 100000000ull);
            }
        }
    } else {
        // ------------------------------------------------ epilogue (both CTAs)
        const int q = warp & 3, half = (warp - 2) >> 2;
        const uint32_t tempty_c0 = tc::mapa(tempty0, 0);
        Staging<2> st{tc::smem_u32(smOut + (warp - 2) * kStageBytes), 0};
        pdl_wait();
        if (GRAD && j.dbias.out)
            add_blocks(j.dbias, warp - 2, lane, reinterpret_cast<float (*)[32]>(smOut),
                       [] { asm volatile("bar.sync 1, %0;" :: "n"(32 * kEpiWarps) : "memory"); });
        int iter = 0;
        // A thread owns one row and half of the tile's columns in chunks of 32, at most 128 (gated: of each
        // projection's, at most 64); of an odd number of chunks the first half has one more
        constexpr bool PROJ = !GRAD && GATED;
        bool dw;
        for (int i = 0, t; nth_tile(j, cid, ncl, i, dw, t); i++) {
            const Job& job = j.job[BOTH && dw];
            const Params& p = job.p;
            const TileAt ti = tile_at(p, t);
            const int cols = PROJ ? p.tile_n / 2 : p.tile_n, first = (cols / 32 + 1) / 2 * 32;
            const int own = half == 0 ? first : cols - first;
            const uint32_t second = PROJ ? (uint32_t)cols : 0;
            const int which = GATED && dw && ti.mt >= p.half ? 1 : 0;
            const int64_t row0 = (int64_t)(ti.mt - which * p.half) * p.tile_m + rank * (p.tile_m / 2) + q * 32;
            const int64_t col0 = (int64_t)ti.nt * cols + half * first;
            const bool live = q * 32 < p.tile_m / 2 && row0 < p.M && col0 < p.N;
            const uint32_t ta0 = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * first);
            // 32 columns of the sums, from the thread's column c on, leave
            const auto leave = [&](float (&v)[32], const float (&u)[32], int c) {
                if (p.splits > 1) {
                    const int64_t at = PROJ ? gate_col(col0 + c) : col0 + c;
                    const int64_t r = row0 + (int64_t)which * p.half * kTile;
                    store_part(v, st, &job.out[0], (int)at, (int)r, ti.split, lane);
                    if (PROJ) store_part(u, st, &job.out[0], (int)at + 128, (int)r, ti.split, lane);
                } else if (GRAD) {
                    if (col0 + c < p.N) store_bf16(v, 1.0f, st.base, &job.out[which], (int)col0 + c, (int)row0, st.n, lane);
                } else if (col0 + c < p.N) {
                    if (PROJ) finish_gated(v, u, p.f, &job.out[0], &job.out[1], &job.out[2], row0, col0 + c, p.M, p.N, st, lane);
                    else finish_linear(v, p.f, &job.out[0], &job.out[1], row0, col0 + c, p.M, p.N, st, lane);
                }
            };
            if constexpr (!LONG) {
                const int buf = iter & 1;
                if (!wait(tfull0 + 8 * buf, (iter >> 1) & 1, abort_flag, j.status, j.timeout_ns)) break;
                tc::fence_after();
                ++iter;
                if (live)
#pragma unroll 1
                    for (int c = 0; c < own; c += 32) {
                        float v[32], u[32];
                        load_acc(v, ta0 + (uint32_t)(buf * kTile + c));
                        if (PROJ) load_acc(u, ta0 + second + (uint32_t)(buf * kTile + c));
                        leave(v, u, c);
                    }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(tempty_c0 + 8 * buf);
            } else {
                float z[128] = {};
                bool ok = true;
                for (int c0 = ti.k0; c0 < ti.k1; c0 += p.chunk, ++iter) {
                    ok = wait(tfull0 + 8 * (iter & 1), (iter >> 1) & 1, abort_flag, j.status, j.timeout_ns);
                    if (!ok) break;
                    tc::fence_after();
                    if (live)
#pragma unroll
                        for (int c = 0; c < 128; c += 16)
                            if ((PROJ ? c & 63 : c) < own)
                                add_acc(z + c, ta0 + (PROJ && c >= 64 ? second : 0u) + (uint32_t)((iter & 1) * kTile + (PROJ ? c & 63 : c)));
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive_cluster(tempty_c0 + 8 * (iter & 1));
                }
                if (!ok) break;
                if (!live) continue;
                // the loop stays one, and z moves on: the epilogue's code is long
#pragma unroll 1
                for (int c = 0; c < own; c += 32) {
                    float v[32], u[32];
#pragma unroll
                    for (int j = 0; j < 32; j++) {
                        v[j] = z[j];
                        if (PROJ) u[j] = z[64 + j];
                    }
                    leave(v, u, c);
#pragma unroll
                    for (int j = 0; j < 96; j++) z[j] = z[j + 32];
                }
            }
        }
        if (lane == 0) tc::bulk_wait_all();
    }

    // Both CTAs have stopped issuing.  If either gave up, both know after the barrier, and the even CTA
    // waits (bounded) for the loads still in flight before either may exit.
    tc::fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) st_cluster(tc::mapa(tc::smem_u32((const void*)peer_abort), rank ^ 1), 1);
    tc::cluster_sync();
    if (*abort_flag || *peer_abort) {
        if (leader && warp == 0 && lane == 0)
            drain_ring(full0, S, *issued_slot, tc::ld_cluster_s32(tc::mapa(tc::smem_u32((const void*)issued_slot), 1)), load_tx,
                       tc::mapa(tc::smem_u32((const void*)load_tx), 1), BOTH ? 0 : (uint32_t)(kSub * (j.job[0].p.sub_a + j.job[0].p.sub_b)));
        tc::cluster_sync();
    }
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_dealloc<2>(tmem, kTmemCols);
    }
}

// ------------------------------------------------------- up to four tokens
// Rows of w by up to TOK tokens on the CUDA cores: a warp takes kRows rows of w (gated: of both, for half as many
// features), 16 bytes a lane and row at a time, and the tokens' same columns from L1; `parts` warps of a CTA share a
// row's columns.  Bound by streaming w: there is no set-up before its first loads, where the tensor cores' kernel has
// barriers, tensor memory and descriptors to prepare, and enough of them are in flight (16 warps per SM with 4 KB
// each).  More tokens cost more than the stream: 13 instructions an element of w for eight of them.
constexpr int kGemvThreads = 256;
constexpr int kRows = 4, kAhead = 2;               // a warp's rows, and their loads in flight
struct Gemv {
    const __nv_bfloat16* x;
    int64_t ldx;
    const __nv_bfloat16* w[2];
    int64_t ldw[2];
    int64_t N;
    int64_t vectors, part;         // 8 columns each: of a row, and of one of its parts
    int32_t T, parts;
    Fused f;
};
// (not .nc, for data that does not change while the kernel runs: it runs already while the kernel before it writes w)
__device__ __forceinline__ uint4 stream16(const __nv_bfloat16* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
template <int TOK, bool GATED>
__global__ void __launch_bounds__(kGemvThreads) linear_gemv_kernel(const __grid_constant__ Gemv p) {
    constexpr int WARPS = kGemvThreads / 32, FEATURES = GATED ? kRows / 2 : kRows;
    __shared__ float sums[WARPS][kRows * TOK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / p.parts, part = warp - group * p.parts, groups = WARPS / p.parts;
    const int64_t feature0 = (int64_t)blockIdx.x * groups * FEATURES;
    const __nv_bfloat16* row[kRows];
#pragma unroll
    for (int r = 0; r < kRows; r++) {
        // features past the last read the last one's row and are not written
        const int64_t f = min(p.N - 1, feature0 + group * FEATURES + (GATED ? r >> 1 : r));
        const int which = GATED ? r & 1 : 0;
        row[r] = p.w[which] + f * p.ldw[which];
    }
    float acc[kRows][TOK] = {};
    pdl_launch_dependents();
    pdl_wait();
    const int64_t end = min(p.vectors, (part + 1) * p.part);
    for (int64_t k = part * p.part + lane; k < end; k += 32 * kAhead) {
        Pack<__nv_bfloat16, 8> w[kAhead][kRows], x[kAhead][TOK];
#pragma unroll
        for (int a = 0; a < kAhead; a++) {
            const bool in = k + 32 * a < end;
#pragma unroll
            for (int r = 0; r < kRows; r++) {
                w[a][r].zero();
                if (in) w[a][r].v = stream16(row[r] + (k + 32 * a) * 8);
            }
#pragma unroll
            for (int t = 0; t < TOK; t++) {
                x[a][t].zero();
                if (in && t < p.T) x[a][t].load(p.x + t * p.ldx + (k + 32 * a) * 8);
            }
        }
#pragma unroll
        for (int a = 0; a < kAhead; a++) {
            float v[TOK][8];
#pragma unroll
            for (int t = 0; t < TOK; t++) x[a][t].unpack(v[t]);
#pragma unroll
            for (int r = 0; r < kRows; r++) {
                float u[8];
                w[a][r].unpack(u);
#pragma unroll
                for (int t = 0; t < TOK; t++)
#pragma unroll
                    for (int e = 0; e < 8; e++) acc[r][t] = fmaf(u[e], v[t][e], acc[r][t]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; r++)
#pragma unroll
        for (int t = 0; t < TOK; t++) {
            float s = acc[r][t];
#pragma unroll
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (lane == 0) sums[warp][r * TOK + t] = s;
        }
    __syncthreads();
    // one output a thread, the parts of a row in their order
    const int i = threadIdx.x;
    if (i >= groups * FEATURES * TOK) return;
    const int t = i / (groups * FEATURES), g = i - t * groups * FEATURES, mine = g / FEATURES, at = g - mine * FEATURES;
    const int64_t feature = feature0 + g;
    if (t >= p.T || feature >= p.N) return;
    const auto sum = [&](int r) {
        float s = 0.0f;
        for (int k = 0; k < p.parts; k++) s += sums[mine * p.parts + k][r * TOK + t];
        return s;
    };
    finish_one<GATED>(sum(GATED ? 2 * at : at), GATED ? sum(2 * at + 1) : 1.0f, p.f, t, feature);
}

// ------------------------------------------------------- gradients of few tokens
// Up to kGemvTokens tokens the gradients come from the CUDA cores in FP32, with dz unrounded: a CTA takes 1024 columns
// of `rows` rows of w, makes those rows' dz, reads w once, leaves dw and its part of dx.  Bound by reading w and writing dw.
constexpr int kFewThreads = 128;
struct FewGrad {
    const __nv_bfloat16* dy;
    int64_t ld_dy;
    const __nv_bfloat16* z;        // gated: the gate's
    int64_t ldz;
    const __nv_bfloat16* u;
    int64_t ldu;
    const __nv_bfloat16* x;
    int64_t ldx;
    const __nv_bfloat16* w[2];
    int64_t ldw[2];
    __nv_bfloat16* dw[2];          // or nullptr
    int64_t ld_dw[2];
    __nv_bfloat16* dx;             // the only part of dx, or nullptr
    int64_t ld_dx;
    float* acc;                    // parts of dx [gridDim.x][T][D], or nullptr
    float* dbias;
    int64_t T, N, D;
    int32_t rows, act;
};
template <int ACT, bool GATED>
__device__ __forceinline__ float2 dz_of(const FewGrad& p, int64_t t, int64_t n) {
    const float d = __bfloat162float(p.dy[t * p.ld_dy + n]);
    const float z = ACT != kActIdentity || GATED ? __bfloat162float(p.z[t * p.ldz + n]) : 0.0f;
    F2 value;
    const float slope = act_slope<ACT>(F2(z), value).get().x;
    if (!GATED) return make_float2(ACT == kActIdentity ? d : d * slope, 0.0f);
    return make_float2(d * __bfloat162float(p.u[t * p.ldu + n]) * slope, d * value.get().x);
}
__device__ __forceinline__ void fma8(F2 (&s)[4], float f, const F2 (&v)[4]) {
    const F2 k(f);
#pragma unroll
    for (int e = 0; e < 4; e++) s[e] = fma2(k, v[e], s[e]);
}
// 8 columns of a token's dx, or of its part
__device__ __forceinline__ void put_dx(const FewGrad& p, int64_t part, int64_t t, int64_t c, const F2 (&s)[4]) {
    if (p.acc) {
        float4* to = reinterpret_cast<float4*>(p.acc + (part * p.T + t) * p.D + c);
        const float2 a = s[0].get(), b = s[1].get(), d = s[2].get(), e = s[3].get();
        to[0] = make_float4(a.x, a.y, b.x, b.y);
        to[1] = make_float4(d.x, d.y, e.x, e.y);
    } else {
        Pack<__nv_bfloat16, 8> k;
        pack2(k, s);
        k.store(p.dx + t * p.ld_dx + c);
    }
}
// TOK: 1, 2 or 4 tokens
template <bool GATED, int TOK>
__global__ void __launch_bounds__(kFewThreads) linear_few_grad_kernel(const __grid_constant__ FewGrad p) {
    extern __shared__ float dz[];                  // [row][part][token]
    constexpr int P = GATED ? 2 : 1;
    const int64_t n0 = (int64_t)blockIdx.x * p.rows;
    const int rows = (int)min((int64_t)p.rows, p.N - n0), T = (int)p.T;
    pdl_launch_dependents();
    pdl_wait();
    for (int i = threadIdx.x; i < rows * T; i += kFewThreads) {
        const int t = i / rows, r = i - t * rows;
        float2 d;
#define F(A) d = dz_of<A, GATED>(p, t, n0 + r)
        BSQ_WITH_ACT(p.act, F)
#undef F
        dz[(r * P) * T + t] = d.x;
        if (GATED) dz[(r * P + 1) * T + t] = d.y;
    }
    __syncthreads();
    if (!GATED && p.dbias && blockIdx.y == 0)
        for (int r = threadIdx.x; r < rows; r += kFewThreads) {
            float s = 0.0f;
            for (int t = 0; t < T; t++) s += dz[r * T + t];
            p.dbias[n0 + r] = s;
        }
    const int64_t c = ((int64_t)blockIdx.y * kFewThreads + threadIdx.x) * 8;
    if (c >= p.D || (!p.dw[0] && !p.dx && !p.acc)) return;
    const bool want_dx = p.dx || p.acc;
    F2 x[TOK][4], sum[TOK][4];
#pragma unroll
    for (int t = 0; t < TOK; t++) {
        Pack<__nv_bfloat16, 8> k;
        k.zero();
        if (p.dw[0] && t < T) k.load(p.x + t * p.ldx + c);
        unpack2(k, x[t]);
#pragma unroll
        for (int e = 0; e < 4; e++) sum[t][e] = F2(0.0f);
    }
    constexpr int AHEAD = 4 / P;
    for (int r0 = 0; r0 < rows; r0 += AHEAD) {
        Pack<__nv_bfloat16, 8> w[AHEAD][P];
#pragma unroll
        for (int a = 0; a < AHEAD; a++)
#pragma unroll
            for (int i = 0; i < P; i++) {
                w[a][i].zero();
                if (want_dx && r0 + a < rows) w[a][i].v = stream16(p.w[i] + (n0 + r0 + a) * p.ldw[i] + c);
            }
#pragma unroll
        for (int a = 0; a < AHEAD; a++) {
            if (r0 + a >= rows) break;
#pragma unroll
            for (int i = 0; i < P; i++) {
                F2 v[4], g[4] = {F2(0.0f), F2(0.0f), F2(0.0f), F2(0.0f)};
                unpack2(w[a][i], v);
                const float* d = dz + ((r0 + a) * P + i) * T;
#pragma unroll
                for (int t = 0; t < TOK; t++) {
                    const float f = t < T ? d[t] : 0.0f;
                    if (t < T) fma8(sum[t], f, v);
                    fma8(g, f, x[t]);
                }
                if (p.dw[i]) {
                    Pack<__nv_bfloat16, 8> k;
                    pack2(k, g);
                    k.store(p.dw[i] + (n0 + r0 + a) * p.ld_dw[i] + c);
                }
            }
        }
    }
    if (want_dx)
#pragma unroll
        for (int t = 0; t < TOK; t++)
            if (t < T) put_dx(p, blockIdx.x, t, c, sum[t]);
}
// Up to kSmallTokens tokens: a CTA has either 8 rows of dw and all the tokens, or 8 tokens of dx and kDxRows rows of w
// (grid.x: first those, then these), the eight in registers while the others pass by.
constexpr int kSmallTokens = 128, kEight = 8, kDxRows = 32;
template <bool GATED>
__global__ void __launch_bounds__(kFewThreads) linear_small_grad_kernel(const __grid_constant__ FewGrad p, int dw_ctas) {
    constexpr int P = GATED ? 2 : 1;
    __shared__ float dz[kEight * kSmallTokens * P];
    static_assert(kEight * kSmallTokens >= kDxRows * kEight, "dz");
    const bool dw = (int)blockIdx.x < dw_ctas;
    const int T = (int)p.T, groups = (T + kEight - 1) / kEight, b = (int)blockIdx.x - dw_ctas;
    const int t0 = dw ? 0 : b % groups * kEight, tokens = dw ? T : min(kEight, T - t0);
    const int64_t n0 = dw ? (int64_t)blockIdx.x * kEight : (int64_t)(b / groups) * kDxRows;
    const int rows = (int)min((int64_t)(dw ? kEight : kDxRows), p.N - n0);
    pdl_launch_dependents();
    pdl_wait();
    // [part][token][8 rows], or [part][row][8 tokens]: the eight next to each other, 0 where there are fewer
    for (int i = threadIdx.x; i < (dw ? tokens : rows) * kEight; i += kFewThreads) {
        const int k = i / kEight, j = i - k * kEight, r = dw ? j : k, t = dw ? k : j;
        float2 d = make_float2(0.0f, 0.0f);
        if (r < rows && t < tokens) {
#define F(A) d = dz_of<A, GATED>(p, t0 + t, n0 + r)
            BSQ_WITH_ACT(p.act, F)
#undef F
        }
        dz[i] = d.x;
        if (GATED) dz[kEight * kSmallTokens + i] = d.y;
    }
    __syncthreads();
    if (!GATED && p.dbias && dw && blockIdx.y == 0 && (int)threadIdx.x < rows) {
        float s = 0.0f;
        for (int t = 0; t < T; t++) s += dz[t * kEight + threadIdx.x];
        p.dbias[n0 + threadIdx.x] = s;
    }
    const int64_t c = ((int64_t)blockIdx.y * kFewThreads + threadIdx.x) * 8;
    if (c >= p.D || (dw && !p.dw[0])) return;
    F2 sum[kEight][4];
    const auto clear = [&] {
#pragma unroll
        for (int j = 0; j < kEight; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) sum[j][e] = F2(0.0f);
    };
    // n rows pass by, eight loads at a time
    const auto pass = [&](int n, auto row, const float* f) {
        for (int k0 = 0; k0 < n; k0 += kEight) {
            Pack<__nv_bfloat16, 8> k[kEight];
#pragma unroll
            for (int j = 0; j < kEight; j++) {
                k[j].zero();
                if (k0 + j < n) k[j].load(row(k0 + j) + c);
            }
#pragma unroll
            for (int j = 0; j < kEight; j++) {
                if (k0 + j >= n) break;
                F2 v[4];
                unpack2(k[j], v);
                const float4 a = *reinterpret_cast<const float4*>(f + (k0 + j) * kEight), g = *reinterpret_cast<const float4*>(f + (k0 + j) * kEight + 4);
                const float q[kEight] = {a.x, a.y, a.z, a.w, g.x, g.y, g.z, g.w};
#pragma unroll
                for (int e = 0; e < kEight; e++) fma8(sum[e], q[e], v);
            }
        }
    };
    if (dw) {
#pragma unroll
        for (int i = 0; i < P; i++) {
            clear();
            pass(T, [&](int t) { return p.x + t * p.ldx; }, dz + i * kSmallTokens * kEight);
#pragma unroll
            for (int r = 0; r < kEight; r++)
                if (r < rows) {
                    Pack<__nv_bfloat16, 8> k;
                    pack2(k, sum[r]);
                    k.store(p.dw[i] + (n0 + r) * p.ld_dw[i] + c);
                }
        }
        return;
    }
    clear();
#pragma unroll
    for (int i = 0; i < P; i++)
        pass(rows, [&](int r) { return p.w[i] + (n0 + r) * p.ldw[i]; }, dz + i * kSmallTokens * kEight);
#pragma unroll
    for (int t = 0; t < kEight; t++)
        if (t < tokens) put_dx(p, b / groups, t0 + t, c, sum[t]);
}

// ------------------------------------------------------- around the products
// The parts of a split sum [splits][M][ld], added in their order, and the forward epilogue: 4 columns a thread.
template <bool GATED>
__global__ void __launch_bounds__(256) linear_join_kernel(const float* acc, int splits, int64_t M, int64_t N, int64_t ld,
                                                         const __grid_constant__ Fused f) {
    const int64_t per = (N + 3) / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (i >= M * per) return;
    const int64_t row = i / per, col = (i - row * per) * 4;
    const int n = (int)min((int64_t)4, N - col);
    const auto sum = [&](int64_t at) {
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = 0; k < splits; k++) {
            const float4 x = *reinterpret_cast<const float4*>(acc + (k * M + row) * ld + at);
            s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
        }
        return s;
    };
    const float4 s = sum(GATED ? gate_col(col) : col), t = GATED ? sum(gate_col(col) + 128) : s;
    float v[4] = {s.x, s.y, s.z, s.w};
    const float u[4] = {t.x, t.y, t.z, t.w};
    if (!GATED && f.bias)
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (j < n) v[j] += load_as_float(f.bias, col + j, f.bias_bf16);
    if (f.z)
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (j < n) {
                f.z[row * f.ldz + col + j] = __float2bfloat16_rn(v[j]);
                if (GATED) f.u[row * f.ldu + col + j] = __float2bfloat16_rn(u[j]);
            }
    activate(f.act, v);
    // (all of the residual before the first store, which may be to its place)
#pragma unroll
    for (int j = 0; j < 4; j++) {
        if (GATED) v[j] *= u[j];
        else if (f.residual && j < n) v[j] += load_as_float(f.residual, row * f.ld_res + col + j, f.y_bf16);
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (j < n) {
            const int64_t at = row * f.ldy + col + j;
            if (f.y_bf16) static_cast<__nv_bfloat16*>(f.y)[at] = __float2bfloat16_rn(v[j]);
            else static_cast<float*>(f.y)[at] = v[j];
        }
}

// out = the sum of the parts [splits][rows_all][D] from row `row0` on; 8 columns a thread
__global__ void __launch_bounds__(256) linear_sum_kernel(const float* acc, int splits, int64_t rows_all, int64_t row0,
                                                        int64_t rows, int64_t D, __nv_bfloat16* out, int64_t ld) {
    const int64_t per = D / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (i >= rows * per) return;
    const int64_t r = i / per, c = (i - r * per) * 8;
    float v[8] = {};
    for (int s = 0; s < splits; s++) {
        const float4* a = reinterpret_cast<const float4*>(acc + (s * rows_all + row0 + r) * D + c);
        const float4 x = a[0], y = a[1];
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
    Pack<__nv_bfloat16, 8> k;
    k.pack(v);
    k.store(out + r * ld + c);
}

// dx = the sum of many parts [parts][T][D]: 16 threads share 4 columns, each sums every sixteenth part
__global__ void __launch_bounds__(256) linear_few_sum_kernel(const float* acc, int64_t parts, int64_t T, int64_t D, __nv_bfloat16* out,
                                                            int64_t ld) {
    __shared__ float4 all[16][16];
    const int col = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int64_t per = D / 4, i = (int64_t)blockIdx.x * 16 + col;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    pdl_wait();
    if (i < T * per)
#pragma unroll 8
        for (int64_t k = group; k < parts; k += 16) {
            const float4 x = reinterpret_cast<const float4*>(acc)[k * T * per + i];
            s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
        }
    all[group][col] = s;
    __syncthreads();
    if (group != 0 || i >= T * per) return;
#pragma unroll
    for (int g = 1; g < 16; g++) {
        const float4 x = all[g][col];
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    const int64_t t = i / per;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
    *reinterpret_cast<uint2*>(out + t * ld + (i - t * per) * 4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// The epilogue's gradient, 8 columns of kRows rows a thread:
//   linear  dz = dy act'(z) (z nullptr: dz = dy), and the column sums of a CTA's rows for dbias
//   gated   da = dh u act'(a), du = dh act(a)
// BF16 in, FP32 in between, BF16 out (nullptr: the sums only).  Bound by memory.
constexpr int kGradRows = 64;                       // of a CTA: 8 threads' rows of 8
struct SlopeArgs {
    const __nv_bfloat16* dy;
    int64_t ld_dy;
    const __nv_bfloat16* z;        // gated: the gate's
    int64_t ldz;
    const __nv_bfloat16* u;
    int64_t ldu;
    __nv_bfloat16* dz;             // [rows][ld]; gated: da, and du behind it
    __nv_bfloat16* du;
    int64_t ld;
    float* sums;                   // [row blocks][cols]
    int64_t rows, cols;
};
template <int ACT, bool GATED, bool VEC>
__global__ void __launch_bounds__(256) linear_slope_kernel(const SlopeArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t col = ((int64_t)blockIdx.y * 32 + (threadIdx.x & 31)) * 8;
    const int64_t row0 = (int64_t)blockIdx.x * kGradRows;
    const int n = (int)max((int64_t)0, min((int64_t)8, a.cols - col));
    float sum[8] = {};
    if (n > 0)
#pragma unroll 2
        for (int k = threadIdx.x >> 5; k < kGradRows; k += 8) {
            const int64_t row = row0 + k;
            if (row >= a.rows) break;
            const auto get = [&](const __nv_bfloat16* p, int64_t ld, float (&f)[8]) {
                if (VEC) {
                    Pack<__nv_bfloat16, 8> v;
                    v.load(p + row * ld + col);
                    v.unpack(f);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j++) f[j] = j < n ? __bfloat162float(p[row * ld + col + j]) : 0.0f;
                }
            };
            float d[8], z[8] = {}, u[8] = {};
            get(a.dy, a.ld_dy, d);
            if (ACT != kActIdentity || GATED) get(a.z, a.ldz, z);
            if (GATED) get(a.u, a.ldu, u);
            float o[8], w[8];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                F2 value;
                const F2 dd(d[j], d[j + 1]), slope = act_slope<ACT>(F2(z[j], z[j + 1]), value);
                const float2 a2 = (GATED ? dd * F2(u[j], u[j + 1]) * slope : ACT == kActIdentity ? dd : dd * slope).get();
                const float2 b2 = (dd * value).get();
                o[j] = a2.x;
                o[j + 1] = a2.y;
                w[j] = b2.x;
                w[j + 1] = b2.y;
                // (single additions: not contracted with the product, dbias alone comes out as it does beside the products)
                if (!GATED) {
                    sum[j] = __fadd_rn(sum[j], a2.x);
                    sum[j + 1] = __fadd_rn(sum[j + 1], a2.y);
                }
            }
            // the workspace's rows hold whole vectors
            if (a.dz) {
                Pack<__nv_bfloat16, 8> v;
                v.pack(o);
                v.store(a.dz + row * a.ld + col);
                if (GATED) {
                    v.pack(w);
                    v.store(a.du + row * a.ld + col);
                }
            }
        }
    if (GATED || !a.sums) return;
    __shared__ float all[8][256 + 8];
#pragma unroll
    for (int j = 0; j < 8; j++) all[threadIdx.x >> 5][(threadIdx.x & 31) * 8 + j] = sum[j];
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.y * 256 + threadIdx.x;
    if (c >= a.cols) return;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; w++) s += all[w][threadIdx.x];
    a.sums[(int64_t)blockIdx.x * a.cols + c] = s;
}
// dbias without a product behind it
__global__ void __launch_bounds__(32 * kSumWarps) linear_bias_kernel(const BlockSums b) {
    __shared__ float all[kSumWarps][32];
    pdl_launch_dependents();
    pdl_wait();
    add_blocks(b, threadIdx.x >> 5, threadIdx.x & 31, all, [] { __syncthreads(); });
}

constexpr double kPartUs = 4.0;                     // the epilogue of a part's tile, behind which the next tile's stages may hide
struct Cut {
    int tile_m, tile_n, splits;
};
// How a product is cut: rows and columns of a pair's tile, and parts of the sum over K.  The estimate: what the
// busiest pair computes, and the last tile's epilogue.  A narrower tile's stage is not shorter in proportion (the MMAs
// of few columns wait for A's rows, and cost the issuing thread the same), but the tiles fill the pairs better: 4096 x
// 4096 -> 4096 in 84 us with 224 columns, 88 with 256, 96 with 192; 512 x 4096 -> 14336 in 53 with 192, 58 with 256.
// With one row of tiles a stage takes as long as its share of the memory's rate for w.  `per`: columns of the result
// for a column of a tile; `step`: widths that the kernel takes (32 columns are a chunk of the epilogue; gated, of either
// projection; an MN-major operand is read in boxes of 64 columns for either CTA); part_bytes: a part's, written and read.
Cut wide_cut(int64_t rows, int64_t cols, double per, int64_t stages, double part_bytes, int step, int num_sms) {
    static constexpr struct { int n; double stage_us, end_us; } kWidths[] = {
        {256, 0.60, 4.0}, {224, 0.57, 4.0}, {192, 0.54, 3.5}, {160, 0.50, 3.0}, {128, 0.435, 2.0}, {96, 0.43, 1.5}, {64, 0.42, 1.0}};
    const int pairs = std::max(1, num_sms / 2), tile_m = rows > kTile - 64 ? kTile : (int)up(rows, 64);
    const int64_t m_tiles = div_up(rows, kTile);
    Cut best{};
    double fewest = 0.0;
    for (const auto& w : kWidths) {
        if (w.n % step) continue;
        const int64_t tiles = m_tiles * div_up(cols, (int64_t)(w.n * per));
        const double stage_us = m_tiles == 1 ? std::max(w.stage_us, w.n * 256 / 88e3) : w.stage_us;
        const int splits = fused_splits(tiles, stages, stage_us, 0.0, kPartUs, part_bytes, pairs);
        const double us = split_us(tiles, stages, splits, stage_us, 0.0, kPartUs, part_bytes, pairs) + w.end_us;
        if (fewest == 0.0 || us < fewest) {
            fewest = us;
            best = {tile_m, w.n, splits};
        }
    }
    return best;
}
Cut forward_cut(int64_t T, int64_t N, int64_t K, bool gated, int num_sms) {
    return wide_cut(T, N, gated ? 0.5 : 1.0, div_up(K, kSub * kSubK), (double)T * fused_acc_cols(N, gated) * 8,
                    gated ? 64 : 32, num_sms);
}

struct Operand {
    const void* p;
    int64_t rows, cols, ld;
};

template <int MODE, bool GATED, bool LONG>
cudaError_t launch_gemm(const Jobs<MODE>& j, int pairs, cudaStream_t st) {
    static SharedMemory smem;
    const cudaError_t e = smem.allow(reinterpret_cast<const void*>(linear_gemm_kernel<MODE, GATED, LONG>), kSmem);
    if (e != cudaSuccess) return e;
    return launch_k(true, linear_gemm_kernel<MODE, GATED, LONG>, dim3(2 * pairs), kThreads, kSmem, st, j);
}
// A job but for its outputs; K: the depth of each operand pair
template <int KIND, bool GATED>
bool set_up(Job& job, const Operand (&a)[2], const Operand (&b)[2], int64_t M, int64_t N, int64_t K, const Cut& cut, bool fine, int num_sms) {
    constexpr bool A_MN = KIND == kDw, B_MN = KIND != kFwd;
    const int tile_n = cut.tile_n;
    // the second operands where there are any
    constexpr bool TWO_A = GATED && KIND != kFwd, TWO_B = GATED && KIND != kDw;
    for (int i = 0; i < 2; i++) {
        if ((i == 0 || TWO_A) && !map_operand(&job.a[i], a[i].p, a[i].rows, a[i].cols, a[i].ld, A_MN ? kSubK : cut.tile_m / 2)) return false;
        if ((i == 0 || TWO_B) && !map_operand(&job.b[i], b[i].p, b[i].rows, b[i].cols, b[i].ld, B_MN ? kSubK : tile_n / 2)) return false;
    }
    Params& p = job.p;
    p.M = M;
    p.N = N;
    const int64_t stages = div_up(K, kSub * kSubK);
    p.half = KIND == kDx ? (int32_t)stages : (int32_t)div_up(M, cut.tile_m);
    p.k_stages = (int32_t)(KIND == kDx && GATED ? 2 * stages : stages);
    p.tile_m = cut.tile_m;
    p.tile_n = tile_n;
    // (of an MN-major operand whole boxes of 64 columns)
    p.sub_a = cut.tile_m / 2 * kSubK * 2;
    p.sub_b = (int)(B_MN ? up(tile_n / 2, 64) : tile_n / 2) * kSubK * 2;
    p.m_tiles = (int32_t)div_up(M, cut.tile_m) * (KIND == kDw && GATED ? 2 : 1);
    p.n_tiles = (int32_t)div_up(N, KIND == kFwd && GATED ? tile_n / 2 : tile_n);
    p.split_stages = (int32_t)div_up(p.k_stages, cut.splits);
    p.splits = (int32_t)div_up(p.k_stages, p.split_stages);
    p.chunk = fine ? kChunk : kSumChunk;
    const int64_t total = (int64_t)p.m_tiles * p.n_tiles * p.splits;
    if (total > 0x3FFFFFFF) return false;
    p.total = (int32_t)total;
    choose_raster(p, K, (int)std::max<int64_t>(1, std::min<int64_t>(num_sms / 2, total)));
    return true;
}
template <int MODE, bool GATED>
cudaError_t gemm(Jobs<MODE>& j, const LinearArgs& args, cudaStream_t st) {
    int total = 0;
    bool is_long = false;
    for (const Job& job : j.job) {
        const Params& p = job.p;
        total += p.total;
        if (!p.total) continue;
        is_long |= p.split_stages > p.chunk;
        j.a_bytes = std::max(j.a_bytes, kSub * p.sub_a);
        j.b_bytes = std::max(j.b_bytes, kSub * p.sub_b);
    }
    j.stages = std::min(kMaxStages, kStages * 2 * kOpBytes / (j.a_bytes + j.b_bytes));
    j.status = args.status;
    j.timeout_ns = args.timeout_ns;
    // (a pair without a tile may still have columns of dbias)
    const int64_t work = std::max<int64_t>(total, j.dbias.out ? div_up(j.dbias.cols, 64) : 0);
    const int pairs = (int)std::max<int64_t>(1, std::min<int64_t>(args.num_sms / 2, work));
    if (MODE == kGrad) {
        const Params &dx = j.job[0].p, &dw = j.job[MODE == kGrad].p;
        // (of few stages the epilogue is what a tile takes)
        const auto us = [](const Params& p) { return std::max(p.split_stages * 0.6, 4.0); };
        j.extra = dx.total % pairs && dw.total ? (int)(us(dx) / us(dw)) : 0;
    }
    return is_long ? launch_gemm<MODE, GATED, true>(j, pairs, st) : launch_gemm<MODE, GATED, false>(j, pairs, st);
}

template <bool GATED>
cudaError_t gemv(const LinearArgs& a, cudaStream_t st) {
    Gemv p{};
    p.x = static_cast<const __nv_bfloat16*>(a.x);
    p.ldx = a.ldx;
    p.w[0] = static_cast<const __nv_bfloat16*>(a.w);
    p.ldw[0] = a.ldw;
    p.w[1] = static_cast<const __nv_bfloat16*>(a.w2);
    p.ldw[1] = a.ldw2;
    p.N = a.out;
    p.T = (int32_t)a.tokens;
    p.vectors = a.cols / 8;
    fused_args(p.f, a);
    // a row's columns are shared by several warps where the rows alone would not fill the SMs a few times over, and every
    // lane has some (288 -> 8625 with each of eight warps on 36 vectors 6.2 us, 3.0 with one)
    // (gated, 1 token of 4096 -> 14336: 36.3 us with two, 38.0 with one; 4 tokens 45.8 with one, 49.8 with two)
    constexpr int WARPS = kGemvThreads / 32;
    const int64_t tasks = div_up(a.out, GATED ? kRows / 2 : kRows);
    p.parts = 1;
    while (p.parts < WARPS && tasks * p.parts * p.T < (int64_t)a.num_sms * 64 && p.vectors > 32 * p.parts) p.parts *= 2;
    p.part = up(div_up(p.vectors, p.parts), 32);
    const dim3 grid((unsigned)div_up(tasks, WARPS / p.parts));
    if (p.T == 1) return launch_k(true, linear_gemv_kernel<1, GATED>, grid, kGemvThreads, 0, st, p);
    if (p.T == 2) return launch_k(true, linear_gemv_kernel<2, GATED>, grid, kGemvThreads, 0, st, p);
    return launch_k(true, linear_gemv_kernel<4, GATED>, grid, kGemvThreads, 0, st, p);
}

template <bool GATED>
cudaError_t forward(const LinearArgs& a, cudaStream_t st) {
    const int64_t T = a.tokens, N = a.out, K = a.cols;
    if (T <= kGemvTokens) return gemv<GATED>(a, st);
    const Cut cut = forward_cut(T, N, K, GATED, a.num_sms);
    Jobs<kFwd> j{};
    Job& job = j.job[0];
    Fused& f = job.p.f;
    fused_args(f, a);
    float* acc = static_cast<float*>(a.ws);
    const Operand x{a.x, T, K, a.ldx}, w0{a.w, N, K, a.ldw}, w1{GATED ? a.w2 : a.w, N, K, GATED ? a.ldw2 : a.ldw};
    if (!set_up<kFwd, GATED>(job, {x, x}, {w0, w1}, T, N, K, cut, !a.y_bf16, a.num_sms)) return cudaErrorInvalidValue;
    if (cut.splits > 1) {
        if (!map_acc(&job.out[0], acc, cut.splits, T, fused_acc_cols(N, GATED))) return cudaErrorInvalidValue;
    } else {
        f.y_tma = fused_map(&job.out[0], a.y, T, N, a.ldy, a.y_bf16);
        f.z_tma = fused_map(&job.out[1], a.z, T, N, a.ldz, true);
        f.u_tma = GATED ? fused_map(&job.out[2], a.u, T, N, a.ldu, true) : kNone;
    }
    const cudaError_t err = gemm<kFwd, GATED>(j, a, st);
    return err != cudaSuccess || cut.splits == 1 ? err : run_linear_join(acc, cut.splits, T, N, GATED, a, st);
}

// ------------------------------------------------------------- backward
struct GradPlan {
    int64_t ld, blocks;
    Cut dx, dw;
    size_t dz_bytes, sums_bytes, dx_bytes, dw_bytes;
};
GradPlan grad_plan(int64_t T, int64_t N, int64_t D, bool gated, int num_sms) {
    GradPlan g{};
    g.ld = up(N, 8);
    g.blocks = div_up(T, kGradRows);
    g.dx = wide_cut(T, D, 1.0, div_up(N, kSub * kSubK) * (gated ? 2 : 1), (double)T * D * 8, 128, num_sms);
    const int64_t rows = up(N, kTile) * (gated ? 2 : 1);
    g.dw = wide_cut(rows, D, 1.0, div_up(T, kSub * kSubK), (double)rows * D * 8, 128, num_sms);
    g.dz_bytes = (size_t)(T * g.ld * 2 * (gated ? 2 : 1));
    g.sums_bytes = gated ? 0 : (size_t)up(g.blocks * N * 4, 16);
    g.dx_bytes = g.dx.splits > 1 ? (size_t)(g.dx.splits * T * D * 4) : 0;
    g.dw_bytes = g.dw.splits > 1 ? (size_t)(g.dw.splits * rows * D * 4) : 0;
    return g;
}

template <bool GATED>
cudaError_t slope(const LinearArgs& a, const SlopeArgs& s, cudaStream_t st) {
    const auto whole = [&](const void* p, int64_t ld) { return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0); };
    const bool vec = s.cols % 8 == 0 && whole(s.dy, s.ld_dy) && whole(s.z, s.ldz) && whole(s.u, s.ldu);
    const dim3 grid((unsigned)div_up(s.rows, kGradRows), (unsigned)div_up(s.cols, 256));
    cudaError_t e = cudaErrorInvalidValue;
#define F(A)                                                                                             \
    e = vec ? launch_k(true, linear_slope_kernel<A, GATED, true>, grid, 256, 0, st, s)                  \
            : launch_k(true, linear_slope_kernel<A, GATED, false>, grid, 256, 0, st, s)
    BSQ_WITH_ACT(a.act, F)
#undef F
    return e;
}

// In FP32 and with dz unrounded: up to kGemvTokens tokens, and, where dz is not dy itself, small products, where the
// rounding of few elements of dz to BF16, or of few results, does not average out.  Measured against the tensor cores' way
// (silu): 5 tokens of 4096 -> 1000 19.2 us (19.5), 60 of 512 -> 64 16.4 (19.3), 100 of 4096 -> 40 29 (20); 16 of 4096 ->
// 1000 would take 22.5 (20.4).
bool few_grad(int64_t tokens, int64_t out, int64_t cols, bool exact) {
    if (tokens <= kGemvTokens || exact) return tokens <= kGemvTokens;
    return tokens <= kSmallTokens && (tokens * out <= 4096 || tokens * cols <= 4096) && (double)tokens * out * cols <= 0x1p28;
}
// Rows of w for a part of dx.  Up to kGemvTokens tokens: some four CTAs for every SM.
int few_rows(int64_t tokens, int64_t out, int64_t cols, int num_sms) {
    if (tokens > kGemvTokens) return kDxRows;
    const int64_t wide = div_up(cols, 8 * kFewThreads), ctas = std::max<int64_t>(1, 4 * (int64_t)num_sms / wide);
    return (int)std::min({std::max<int64_t>(8, div_up(out, ctas)), (int64_t)1024, out});
}
template <bool GATED>
cudaError_t backward_few(const LinearArgs& a, cudaStream_t st) {
    const auto bf = [](const void* p) { return static_cast<const __nv_bfloat16*>(p); };
    const auto to = [](void* p) { return static_cast<__nv_bfloat16*>(p); };
    const int64_t T = a.tokens, N = a.out, D = a.cols;
    const int rows = few_rows(T, N, D, a.num_sms);
    const int64_t parts = div_up(N, rows);
    const bool direct = parts == 1;
    FewGrad p{bf(a.dy), a.ld_dy, bf(a.z), a.ldz, bf(a.u), a.ldu, bf(a.x), a.ldx, {bf(a.w), bf(a.w2)}, {a.ldw, a.ldw2},
              {to(a.dw), to(a.dw2)}, {a.ld_dw, a.ld_dw2}, direct ? to(a.dx) : nullptr, a.ld_dx,
              a.dx && !direct ? static_cast<float*>(a.ws) : nullptr, a.dbias, T, N, D, rows, a.act};
    const unsigned wide = (unsigned)(a.dx || a.dw ? div_up(D, 8 * kFewThreads) : 1);
    cudaError_t e;
    if (T <= kGemvTokens) {
        const auto k = T == 1 ? linear_few_grad_kernel<GATED, 1> : T == 2 ? linear_few_grad_kernel<GATED, 2> : linear_few_grad_kernel<GATED, 4>;
        e = launch_k(true, k, dim3((unsigned)parts, wide), kFewThreads, (size_t)rows * (GATED ? 2 : 1) * T * 4, st, p);
    } else {
        const int dw_ctas = a.dw || a.dbias ? (int)div_up(N, kEight) : 0, dx_ctas = a.dx ? (int)(parts * div_up(T, kEight)) : 0;
        e = launch_k(true, linear_small_grad_kernel<GATED>, dim3((unsigned)(dw_ctas + dx_ctas), wide), kFewThreads, 0, st, p, dw_ctas);
    }
    if (e == cudaSuccess && p.acc)
        e = launch_k(true, linear_few_sum_kernel, dim3((unsigned)div_up(T * (D / 4), 16)), 256, 0, st, p.acc, parts, T, D, to(a.dx), a.ld_dx);
    return e;
}

template <bool GATED>
cudaError_t backward(const LinearArgs& a, cudaStream_t st) {
    const int64_t T = a.tokens, N = a.out, D = a.cols;
    // (the identity's dz is dy)
    if (few_grad(T, N, D, !GATED && a.act == kActIdentity)) return backward_few<GATED>(a, st);
    const GradPlan g = grad_plan(T, N, D, GATED, a.num_sms);
    // dz is made in the workspace, or copied there for its address or pitch
    const bool copy = GATED || a.act != kActIdentity || reinterpret_cast<uintptr_t>(a.dy) % 16 || (a.ld_dy % 8 && T > 1);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    __nv_bfloat16* dz = reinterpret_cast<__nv_bfloat16*>(ws);
    __nv_bfloat16* du = dz + T * g.ld;
    float* sums = reinterpret_cast<float*>(ws + g.dz_bytes);
    float* dx_acc = reinterpret_cast<float*>(ws + g.dz_bytes + g.sums_bytes);
    float* dw_acc = reinterpret_cast<float*>(ws + g.dz_bytes + g.sums_bytes + g.dx_bytes);
    cudaError_t e = cudaSuccess;
    const bool products = a.dx || a.dw;
    if ((copy && products) || a.dbias) {
        SlopeArgs s{static_cast<const __nv_bfloat16*>(a.dy), a.ld_dy, static_cast<const __nv_bfloat16*>(a.z), a.ldz,
                    static_cast<const __nv_bfloat16*>(a.u), a.ldu, copy && products ? dz : nullptr, du, g.ld,
                    a.dbias ? sums : nullptr, T, N};
        e = slope<GATED>(a, s, st);
    }
    const BlockSums dbias{sums, g.blocks, N, a.dbias};
    const Operand d0 = copy ? Operand{dz, T, N, g.ld} : Operand{a.dy, T, N, T > 1 ? a.ld_dy : up(N, 8)};
    const Operand d1 = GATED ? Operand{du, T, N, g.ld} : d0;
    const Operand w0{a.w, N, D, a.ldw}, w1{GATED ? a.w2 : a.w, N, D, GATED ? a.ldw2 : a.ldw}, x{a.x, T, D, a.ldx};
    const auto sum = [&](const float* acc, int splits, int64_t all, int64_t row0, int64_t rows, void* to, int64_t ld) {
        return launch_k(true, linear_sum_kernel, dim3((unsigned)div_up(rows * (D / 8), 256)), 256, 0, st, acc, splits, all, row0, rows,
                        D, static_cast<__nv_bfloat16*>(to), ld);
    };
    if (e == cudaSuccess && products) {
        Jobs<kGrad> j{};
        Job &dx = j.job[0], &dw = j.job[1];
        const int64_t half = up(N, kTile), all = GATED ? 2 * half : half;
        if (a.dx && (!set_up<kDx, GATED>(dx, {d0, d1}, {w0, w1}, T, D, N, g.dx, false, a.num_sms) ||
                     !(g.dx.splits > 1 ? map_acc(&dx.out[0], dx_acc, g.dx.splits, T, D) : tmap::out_2d(&dx.out[0], a.dx, T, D, a.ld_dx, true))))
            return cudaErrorInvalidValue;
        if (a.dw && (!set_up<kDw, GATED>(dw, {d0, d1}, {x, x}, N, D, T, g.dw, false, a.num_sms) ||
                     !(g.dw.splits > 1 ? map_acc(&dw.out[0], dw_acc, g.dw.splits, all, D)
                                       : tmap::out_2d(&dw.out[0], a.dw, N, D, a.ld_dw, true) &&
                                             (!GATED || tmap::out_2d(&dw.out[1], a.dw2, N, D, a.ld_dw2, true)))))
            return cudaErrorInvalidValue;
        if (a.dx && a.dw && dx.p.total + dw.p.total <= 8 * (a.num_sms / 2)) {
            j.dbias = dbias;
            e = gemm<kGrad, GATED>(j, a, st);
        } else {
            if (a.dx) {
                Jobs<kDx> one{};
                one.job[0] = dx;
                one.dbias = dbias;
                e = gemm<kDx, GATED>(one, a, st);
            }
            if (a.dw && e == cudaSuccess) {
                Jobs<kDw> one{};
                one.job[0] = dw;
                if (!a.dx) one.dbias = dbias;
                e = gemm<kDw, GATED>(one, a, st);
            }
        }
    }
    if (e == cudaSuccess && a.dbias && !products)
        e = launch_k(true, linear_bias_kernel, dim3((unsigned)div_up(N, 32)), 32 * kSumWarps, 0, st, dbias);
    if (e == cudaSuccess && a.dx && g.dx.splits > 1) e = sum(dx_acc, g.dx.splits, T, 0, T, a.dx, a.ld_dx);
    if (a.dw && g.dw.splits > 1) {
        const int64_t half = up(N, kTile), all = GATED ? 2 * half : half;
        if (e == cudaSuccess) e = sum(dw_acc, g.dw.splits, all, 0, N, a.dw, a.ld_dw);
        if (e == cudaSuccess && GATED) e = sum(dw_acc, g.dw.splits, all, half, N, a.dw2, a.ld_dw2);
    }
    return e;
}

}  // namespace

void fused_args(Fused& f, const LinearArgs& a) {
    f.act = a.act;
    f.y_bf16 = a.y_bf16;
    f.bias = a.bias;
    f.bias_bf16 = a.bias_bf16;
    f.bias_vec = reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    f.residual = a.residual;
    f.ld_res = a.ld_res;
    f.res_vec = reinterpret_cast<uintptr_t>(a.residual) % 16 == 0 && a.ld_res * (a.y_bf16 ? 2 : 4) % 16 == 0;
    f.y = a.y;
    f.ldy = a.ldy;
    f.z = static_cast<__nv_bfloat16*>(a.z);
    f.ldz = a.ldz;
    f.u = static_cast<__nv_bfloat16*>(a.u);
    f.ldu = a.ldu;
}
int64_t fused_acc_cols(int64_t N, bool gated) { return gated ? div_up(N, 128) * 256 : up(N, 4); }
int fused_parts(int64_t stages, int64_t n) {
    const int64_t per = div_up(stages, n);
    return (int)div_up(stages, per);
}
double split_us(int64_t tiles, int64_t stages, int64_t n, double stage_us, double tile_us, double part_us, double part_bytes, int pairs) {
    const double tile = div_up(stages, n) * stage_us + tile_us;
    if (n == 1) return div_up(tiles, pairs) * tile;
    return tile + (div_up(tiles * n, pairs) - 1) * std::max(tile, part_us) + 2.0 + n * part_bytes / 6.7e6;
}
int fused_splits(int64_t tiles, int64_t stages, double stage_us, double tile_us, double part_us, double part_bytes, int pairs) {
    int64_t best = 1;
    double least = 0.0;
    pairs = std::max(1, pairs);
    for (int64_t n = 1; n == 1 || (n * 4 <= stages && n * tiles <= 8 * pairs); n++) {
        const double us = split_us(tiles, stages, n, stage_us, tile_us, part_us, part_bytes, pairs);
        if (n == 1 || us < least) {
            least = us;
            best = n;
        }
    }
    return fused_parts(stages, best);
}
cudaError_t run_linear_join(const float* acc, int splits, int64_t M, int64_t N, bool gated, const LinearArgs& a, cudaStream_t st) {
    Fused f{};
    fused_args(f, a);
    return launch_k(true, gated ? linear_join_kernel<true> : linear_join_kernel<false>, dim3((unsigned)div_up(M * div_up(N, 4), 256)),
                    256, 0, st, acc, splits, M, N, fused_acc_cols(N, gated), f);
}

size_t linear_workspace(int64_t tokens, int64_t out, int64_t cols, bool gated, int num_sms) {
    if (tokens <= kGemvTokens) return 0;
    const Cut c = forward_cut(tokens, out, cols, gated, num_sms);
    return c.splits > 1 ? (size_t)c.splits * tokens * fused_acc_cols(out, gated) * 4 : 0;
}
size_t linear_backward_workspace(int64_t tokens, int64_t out, int64_t cols, bool gated, int num_sms) {
    // whichever way the activation takes
    size_t most = 0;
    if (few_grad(tokens, out, cols, false)) {
        const int64_t parts = div_up(out, few_rows(tokens, out, cols, num_sms));
        most = parts > 1 ? (size_t)(parts * tokens * cols * 4) : 0;
        if (gated || tokens <= kGemvTokens) return most;
    }
    const GradPlan g = grad_plan(tokens, out, cols, gated, num_sms);
    return std::max(most, g.dz_bytes + g.sums_bytes + g.dx_bytes + g.dw_bytes);
}
cudaError_t run_linear(const LinearArgs& a, bool gated, cudaStream_t st) {
    return gated ? forward<true>(a, st) : forward<false>(a, st);
}
cudaError_t run_linear_backward(const LinearArgs& a, bool gated, cudaStream_t st) {
    return gated ? backward<true>(a, st) : backward<false>(a, st);
}

}  // namespace bsq
