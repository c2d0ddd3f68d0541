// Softmax cross entropy of a linear head, without keeping the logits.
//
// z = h w^T (BF16 operands, FP32 accumulation).  Forward: each output tile
// leaves, per row and 128 columns, the maximum m and s = sum exp(z - m) (the
// target's logit beside it); a second kernel joins a row's parts,
//   lse = M + log sum_i s_i exp(m_i - M),  M = max_i m_i,
// and loss = lse - z[target].  Backward, a piece of the vocabulary at a time:
// the logits' tile again, g = ratio (exp(z - lse) - [v = target]) in BF16 with
// ratio = dloss / max |dloss| (of the finite ones), then dh += g w (FP32 between
// pieces) and dw = g^T h, both times max |dloss| in FP32, so that no dloss, however
// small, leaves BF16's range.  The target's entry of g, p - 1, is by far the largest
// of its row and shares its rounding with every token of that target (p = 1 / V rounds
// to -1 for all of them), so it enters in full: what BF16 loses of it, lo, is added as
// lo w[target] to dh and lo h to dw.  (Without that dh and dw were 1.0e-3 off before
// their own rounding, 1.66e-3, and elements of a common target's row of dw up to 10%.)
//
// All four products run in one kernel on CTA pairs (tcgen05 cta_group::2,
// M = N = 256, K = 16 per MMA): each CTA stages its own 128 rows of A and of
// B by TMA (128-byte swizzle), the even CTA issues the MMAs, and two
// accumulators of 256 tensor-memory columns let the epilogue of one tile run
// under the MMAs of the next.  An operand is read in the layout it has in
// memory: K-major (h and w for the logits, g for dh) or MN-major (w for dh; g
// and h for dw), so nothing is transposed on the way.
//
// Up to kFewTokens tokens the logits' product is bound by streaming w, and runs
// the other way round, z^T = w h^T: w's rows are the tile's 256 rows and the
// tokens its 16 to 128 columns, so that a stage is nearly all w and four to six
// of them (192 KB per SM) are in flight instead of three half-filled ones.
//
// The tensor cores' FP32 sums are not rounded to nearest: over K = 4096 the
// logits came out up to 3e-6 to 6e-6 (relative) too small in magnitude, ten
// times an FP32 product's error.  For the loss and for the gradient's logits the
// accumulators are therefore read out every kChunk of K and added up in
// registers, rounded to nearest (3e-6 -> 4e-7).  The gradient needs it as much as
// the loss: at the target g = exp(z - lse) - 1 cancels, so an error of 1e-4 in z
// (a logit of 20) made the entry of a target with 1 - p = 1e-5 ten times too large.
// dh and dw read theirs out every kSumChunk.
//
// Measured, BF16: the loss of 8192 tokens, 65536 x 4096, in 2.46 to 2.59 ms (up to 1790 TFLOP/s,
// what a library product holds under the power cap, 0.92 of its burst; boxes differ),
// its gradient in 7.7 to 8.0 ms (1650 to 1720 TFLOP/s: bound by the power cap, and dh reads w
// and dw h again); 64 tokens' gradient, 50021 x 4096, in 226 us (w read twice, dw written); 7 tokens, 50021 x 4096, in 70 us (5.9 TB/s, 0.88 of a copy's
// rate), the rest the start of the stream, the last tile and the join.  Calls
// below a few microseconds of work take 10 us (loss) to 20 us (gradient): two to
// five launches in a chain, each with some 3000 cycles of set-up and first loads
// and as many at the end.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cuda.h>
#include "common.cuh"
#include "epilogue.cuh"
#include "internal.h"
#include "launch.cuh"
#include "per_device.h"
#include "tcgen05.cuh"
#include "tmap.h"

namespace bsq {
namespace {

constexpr int64_t kPieceBytes = 256ll << 20;       // of g
constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.44269504088896340736f;

enum { kStats, kGrad, kDh, kDw, kFewStats, kFewGrad, kDwFull };
// When a product waits for the kernel before it on the stream: that kernel is done
// when it is launched; before it reads or writes anything (its set-up runs
// earlier); before its epilogue (only the epilogue needs that kernel); at its end
// (it needs nothing of that kernel, and runs beside it).
enum { kWaitLaunch, kWaitStart, kWaitEpilogue, kWaitEnd };

// ------------------------------------------------------------ the products
constexpr int kTile = 256;                          // output rows and columns of a pair
constexpr int kSubK = 64;                           // K of one 128-byte sub-step
constexpr int kSub = 2;                             // sub-steps per stage
constexpr int kStages = 3;
constexpr int kMaxStages = 6;                       // few tokens: as many as fit
constexpr int kFewTokens = 128;
constexpr int kFewTable = kFewTokens * 12;          // their lse, ratio and target
constexpr int kFewOut = kFewTable + 8 * 2048;       // and 32 rows by 16 tokens for each warp of the epilogue
// Stages (K = 512) that one accumulator sums for the logits.  Against 64 bits, 1024
// x 20000 x 4096: 3.2e-7 (2 stages 1.6e-7, 8 6.7e-7; a plain FP32 product
// 6.8e-7); the batch takes 2.46 ms with 4 or 8, 2.59 with 2.
constexpr int kChunk = 4;
// and for dh and dw (K = 4096), whose results are rounded to BF16: a sum loses some 6e-6,
// whatever the number of tokens or columns.  (In one accumulator dw over 200003 tokens
// came out 1.2e-3 too small, dh over 131072 columns 5.8e-4.)  The gradient of the batch
// took 7.6 to 7.7 ms with 16 or 32, 8.0 with 4.
constexpr int kSumChunk = 32;
constexpr int kSubBytes = 128 * kSubK * 2;          // one CTA's 128 rows of an operand, one sub-step
constexpr int kOpBytes = kSub * kSubBytes;
constexpr int kMmas = 4 * kSub;                     // per stage
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = 32 * (2 + kEpiWarps);
constexpr uint32_t kTmemCols = 512;
constexpr int kStage = 4096;                        // a warp's staging: two chunks of 32 rows x 64 bytes
constexpr int kSmem = 1024 + kStages * 2 * kOpBytes + kEpiWarps * kStage + 256;
static_assert(kSmem <= 232448, "shared memory per block");
__host__ __device__ constexpr bool is_few(int mode) { return mode == kFewStats || mode == kFewGrad; }
constexpr int64_t kL2Resident = 40ll << 20;         // operand bytes that stay in L2 while others stream past

// MODE's operand layouts: K-major (false) or MN-major (true)
__host__ __device__ constexpr bool is_dw(int mode) { return mode == kDw || mode == kDwFull; }
__host__ __device__ constexpr bool a_mn(int mode) { return is_dw(mode); }
__host__ __device__ constexpr bool b_mn(int mode) { return mode == kDh || is_dw(mode); }
// whose rows get what the targets' entries of g lost to BF16 in the epilogue
__host__ __device__ constexpr bool takes_extra(int mode) { return mode == kDh || mode == kDw; }

// The tokens with a vocabulary row as their target: the first of them, and their number
struct Owner {
    int32_t first, count;
};
// What the targets' entries of g lost to BF16, summed for the vocabulary rows that several tokens have as their
// target: in fixed point, so that the sums do not depend on the order of the additions.  A sum of `count` terms
// lo h, |lo| < 2^-8 and |h| at most hmax, is held in units of 2^unit, below 2^30 of them.
struct Sums {
    int32_t* rows;                 // [rows][cols], of a vocabulary row, or of its first token
    int64_t cols;
    int32_t by_row;
    const float* hmax;             // [hmaxes]: partial maxima; *hmaxes: all of them
    int32_t hmaxes;
};
__device__ __forceinline__ int sum_unit(float hmax, int count) {
    return hmax > 0.0f ? ilogbf(hmax) + 1 - 8 + (32 - __clz(count)) - 30 : 0;
}

struct GemmParams {
    int64_t M, N;                  // output
    int32_t k_stages, mma_last;    // K stages in all; MMAs of the last one
    int32_t chunk;                 // stages per accumulator
    int32_t m_tiles, n_tiles, splits, split_stages, total;
    int32_t raster, raster_n;
    int32_t tile_n;                // output columns of a pair: 256; few tokens: the tokens in sixteens
    int32_t tile_m;                // rows of a pair: 256, or fewer (few tokens) for balance
    int32_t stages, b_bytes;       // few tokens: stages, and one CTA's bytes of B per stage
    uint32_t tx;                   // bytes one CTA loads per stage
    int32_t wait;                  // kWait...: when it waits for the kernel before it
    const int64_t* targets;
    int64_t vocab;
    int64_t col0;                  // first vocabulary column of the piece
    float2* part;                  // kStats: [part][M] (max, sum), a part per tile and 128 columns
    float* hit;                    // kStats: the target's logit
    __nv_bfloat16* g;              // kFewGrad: g [tokens][ld_g]; g_lo has the same pitch
    int64_t ld_g;
    const float* lse;
    const float* dloss;
    float* smax;
    int32_t put_smax;              // kFewGrad: leave max |dloss| there
    float* lo;                     // [tokens] what the target's entry of g lost to BF16 (kGrad, kFewGrad leave it)
    __nv_bfloat16* g_lo;           // kGrad, kFewGrad: the same as a matrix like g, for kDwFull
    Owner* owner;                  // kGrad fills, kDw reads: [the piece's columns]
    const __nv_bfloat16* w;        // kDh: the piece
    int64_t ldw;
    int64_t piece_cols;            // kDh: columns of the piece
    Sums sums;                     // kDw
    const __nv_bfloat16* h;        // kDw
    int64_t ldh;
    int32_t half_subs, sub_mmas;   // kDwFull: sub-steps of g (as many of g_lo follow), and the MMAs of each
    int32_t add;                   // kDh: add to what is there
    int32_t direct;                // kDh, kDw: the only piece and split, so dh or dw itself leaves
    unsigned* status;
    uint64_t timeout_ns;
};

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
// The maximum as it is taken out of the exponentials.  An infinite one is not: exp(-inf) is 0 and
// exp(inf) is inf as they are, while inf - inf would be NaN.
__device__ __forceinline__ float finite_or_zero(float m) { return fabsf(m) == INFINITY ? 0.0f : m; }
// An element of g; ratio 0 (a token that does not count) gives 0 whatever its logits
__device__ __forceinline__ float few_g(float z, float lse, float ratio, bool target) {
    const float g = exp2_fast((z - lse) * kLog2e) - (target ? 1.0f : 0.0f);
    return ratio == 0.0f ? 0.0f : g * ratio;
}
// What an entry of g loses to BF16 (nothing where it is not finite)
__device__ __forceinline__ float left_over(float g) {
    return fabsf(g) <= FLT_MAX ? g - __bfloat162float(__float2bfloat16_rn(g)) : 0.0f;
}
// Where lane l's i-th group of four rows starts: its 16 rows, begun at another
// place for each of four neighbouring tokens
__device__ __forceinline__ int turn(int lane, int i) { return 16 * (lane & 1) + ((i + 2 * (lane & ~1)) & 15); }
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
__device__ __forceinline__ void stage_chunk(const uint32_t (&w)[16], uint32_t buf, int lane) {
    const uint32_t row = buf + (uint32_t)lane * 64u, sw = (uint32_t)((lane >> 1) & 3);
#pragma unroll
    for (int u = 0; u < 4; u++)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                     :: "r"(row + ((u ^ sw) << 4)), "r"(w[4 * u]), "r"(w[4 * u + 1]), "r"(w[4 * u + 2]), "r"(w[4 * u + 3])
                     : "memory");
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
__device__ __forceinline__ TileAt tile_at(const GemmParams& p, int t) {
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
__device__ __noinline__ void drain_loads(uint32_t full0, int stages, int n_own, int n_peer, uint32_t tx) {
    const int n = max(n_own, n_peer);
    for (int k = max(0, n - stages); k < n; k++) {
        const uint32_t bar = full0 + 8 * (uint32_t)(k % stages);
        if (k < n_own && k >= n_peer) tc::mbar_complete_tx(bar, tx);
        if (k < n_peer && k >= n_own) tc::mbar_expect_tx(bar, tx);
        volatile int no_abort = 0;
        tc::mbar_wait(bar, (uint32_t)((k / stages) & 1), &no_abort, nullptr, 100000000ull);
    }
}

// The largest finite |dloss| over the tokens that count, of this warp's lanes' tokens lane, lane + step, ...
// (A NaN or an infinity must not scale the other tokens' rows: it stays in its own, as ratio.)
__device__ __forceinline__ float largest_dloss(const float* dloss, const int64_t* targets, int64_t T, int64_t V, int64_t first,
                                               int step) {
    float m = 0.0f;
#pragma unroll 4
    for (int64_t t = first; t < T; t += step) {
        const int64_t id = targets[t];
        const float d = fabsf(dloss[t]);
        if (id >= 0 && id < V && d <= FLT_MAX) m = fmaxf(m, d);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
}

// what is taken out of dloss: 1 where there is nothing to take out, so that dloss / it is dloss
__device__ __forceinline__ float dloss_scale(float largest) { return largest > 0.0f ? largest : 1.0f; }

// The tokens' table of the few-token kernels, filled by the epilogue's warps
template <int MODE>
__device__ __forceinline__ void few_tokens(const GemmParams& p, float* lse, float* ratio, int* target) {
    const int t = threadIdx.x - 64;
    float smax = 0.0f;
    if (MODE == kFewGrad) {
        smax = dloss_scale(largest_dloss(p.dloss, p.targets, p.N, p.vocab, t & 31, 32));
        if (p.put_smax && blockIdx.x == 0 && t == 0) *p.smax = smax;
    }
    if (t < kFewTokens) {
        const int64_t id = t < p.N ? p.targets[t] : -1;
        const bool counts = id >= 0 && id < p.vocab;
        target[t] = counts && id >= p.col0 && id - p.col0 < p.M ? (int)(id - p.col0) : -1;
        lse[t] = MODE == kFewGrad && counts ? p.lse[t] : 0.0f;
        ratio[t] = MODE == kFewGrad && counts ? p.dloss[t] / smax : 0.0f;
    }
    asm volatile("bar.sync 1, %0;" :: "n"(32 * kEpiWarps) : "memory");
}

// Bound by the tensor cores: of 2048 tokens and 16384 x 4096 every product takes
// 149 to 162 us, tensor pipes 75 to 81% busy (few tokens: by reading w, 6.1 TB/s).
// One thread issues all MMAs, about 88 cycles each; with 256 columns an MMA
// takes longer than that.
// LONG: a tile's sum over K takes several accumulators, which the epilogue adds up in
// registers.  Without it a thread keeps 32 columns at a time: a shorter program with
// half the registers, which short calls run once.
template <int MODE, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
head_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ GemmParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // [stages] of A, [stages] of B, then the epilogue's staging (few tokens: their
    // table, then the warps' turned rows); the barriers come last
    constexpr bool FEW = is_few(MODE);
    const int S = FEW ? p.stages : kStages, b_bytes = FEW ? p.b_bytes : kOpBytes, sub_b = b_bytes / kSub;
    uint8_t* smA = base;
    uint8_t* smB = smA + S * kOpBytes;
    uint8_t* smOut = smB + S * b_bytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + (kSmem - 1024 - 256));
    // full[S], empty[S], tfull[2], tempty[2], drain
    const uint32_t full0 = tc::smem_u32(bars), empty0 = tc::smem_u32(bars + kMaxStages);
    const uint32_t tfull0 = tc::smem_u32(bars + 2 * kMaxStages), tempty0 = tc::smem_u32(bars + 2 * kMaxStages + 2);
    const uint32_t drain = tc::smem_u32(bars + 2 * kMaxStages + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* issued_slot = reinterpret_cast<volatile int*>(tmem_slot + 2);
    volatile int* peer_abort = reinterpret_cast<volatile int*>(tmem_slot + 3);
    static_assert(8 * (2 * kMaxStages + 5) + 16 <= 256, "barrier area");

    // a kernel that may run beside this one starts as soon as SMs are free, but not before what
    // this one waits for is done
    if (p.wait != kWaitStart) pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const bool leader = rank == 0;
    const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;

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
        tc::prefetch_tmap(&tmA);
        tc::prefetch_tmap(&tmB);
    }
    if (warp == 1) tc::tmem_alloc<2>(tc::smem_u32(tmem_slot), kTmemCols);
    float* few_lse = reinterpret_cast<float*>(smOut);
    float* few_ratio = few_lse + kFewTokens;
    int* few_target = reinterpret_cast<int*>(few_ratio + kFewTokens);
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
            if (p.wait == kWaitStart) {
                pdl_wait();
                pdl_launch_dependents();
            }
            for (int t = cid; t < p.total && ok; t += ncl) {
                const TileAt ti = tile_at(p, t);
                const int am = ti.mt * p.tile_m + (int)rank * (p.tile_m / 2), bn = ti.nt * p.tile_n + (int)rank * (p.tile_n / 2);
                for (int kb = ti.k0; kb < ti.k1; kb++) {
                    if (!wait(empty0 + 8 * stage, phase ^ 1, abort_flag, p.status, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full_c0 + 8 * stage;
                    if (leader) tc::mbar_expect_tx(full0 + 8 * stage, 2 * p.tx);
#pragma unroll
                    for (int j = 0; j < kSub; j++) {
                        const int sub = kb * kSub + j, half = MODE == kDwFull && sub >= p.half_subs ? 1 : 0;
                        const int k = (sub - half * p.half_subs) * kSubK;
                        const uint32_t da = tc::smem_u32(smA + stage * kOpBytes + j * kSubBytes);
                        const uint32_t db = tc::smem_u32(smB + stage * b_bytes + j * sub_b);
                        if (MODE == kDwFull) {              // g, then g_lo, against the same rows of h
                            tc::tma_load_3d_pair(da, &tmA, am, k, half, fb);
                            tc::tma_load_3d_pair(da + 8192, &tmA, am + 64, k, half, fb);
                        } else if (a_mn(MODE)) {
                            tc::tma_load_2d_pair(da, &tmA, am, k, fb);
                            tc::tma_load_2d_pair(da + 8192, &tmA, am + 64, k, fb);
                        } else {
                            tc::tma_load_2d_pair(da, &tmA, k, am, fb);
                        }
                        if (b_mn(MODE)) {
                            tc::tma_load_2d_pair(db, &tmB, bn, k, fb);
                            tc::tma_load_2d_pair(db + 8192, &tmB, bn + 64, k, fb);
                        } else {
                            tc::tma_load_2d_pair(db, &tmB, k, bn, fb);
                        }
                    }
                    ++issued;
                    if (++stage == S) { stage = 0; phase ^= 1; }
                }
            }
            *issued_slot = issued;
            if (!ok) *abort_flag = 1;
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (even CTA)
        if (lane == 0 && leader) {
            const uint32_t idesc = idesc_bf16(a_mn(MODE), b_mn(MODE)) | ((uint32_t)(p.tile_n >> 3) << 17);
            // 16 k further: 32 bytes of a K-major row, 16 rows of an MN-major tile
            constexpr uint32_t a_step = a_mn(MODE) ? 2048 >> 4 : 2, b_step = b_mn(MODE) ? 2048 >> 4 : 2;
            const uint64_t ad0 = a_mn(MODE) ? desc_mn_sw128(tc::smem_u32(smA)) : tc::desc_sw128(tc::smem_u32(smA));
            const uint64_t bd0 = b_mn(MODE) ? desc_mn_sw128(tc::smem_u32(smB)) : tc::desc_sw128(tc::smem_u32(smB));
            int stage = 0, iter = 0;
            uint32_t phase = 0;
            bool ok = true, any = false, ready = false;
            if (p.wait == kWaitStart) pdl_wait();          // the limit of its waits counts from there
            for (int t = cid; t < p.total && ok; t += ncl) {
                const TileAt ti = tile_at(p, t);
                for (int c0 = ti.k0; c0 < ti.k1 && ok; c0 += p.chunk, ++iter) {
                    const int c1 = min(ti.k1, c0 + p.chunk), buf = iter & 1;
                    if (!wait(tempty0 + 8 * buf, ((iter >> 1) & 1) ^ 1, abort_flag, p.status, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t d = tmem + (uint32_t)buf * kTile;
                    for (int kb = c0; kb < c1; kb++) {
                        if (!ready && !wait(full0 + 8 * stage, phase, abort_flag, p.status, p.timeout_ns)) {
                            ok = false;
                            break;
                        }
                        tc::fence_after();
                        const Desc ad = Desc(ad0) + (uint32_t)(stage * (kOpBytes >> 4));
                        const Desc bd = Desc(bd0) + (uint32_t)(stage * (b_bytes >> 4));
                        const int next = stage + 1 == S ? 0 : stage + 1;
                        const uint32_t next_phase = next == 0 ? phase ^ 1 : phase;
                        if (MODE == kDwFull && p.sub_mmas < 4) {
                            for (int m = 0; m < kMmas; m++)
                                if ((m & 3) < p.sub_mmas)
                                    mma_bf16<false>(d, ad + (m >> 2) * (kSubBytes >> 4) + (m & 3) * a_step,
                                                    bd + (m >> 2) * (sub_b >> 4) + (m & 3) * b_step, idesc, (kb != c0) | (m != 0));
                            ready = false;
                        } else if (kb != p.k_stages - 1 || p.mma_last == kMmas) {
                            // the next stage's barrier is tested while this stage's MMAs run
                            mma_bf16<false>(d, ad, bd, idesc, kb != c0);
#pragma unroll
                            for (int m = 1; m < kMmas; m++) {
                                if (m == kMmas - 1) ready = tc::mbar_test(full0 + 8 * next, next_phase);
                                mma_bf16<true>(d, ad + (m >> 2) * (kSubBytes >> 4) + (m & 3) * a_step,
                                               bd + (m >> 2) * (sub_b >> 4) + (m & 3) * b_step, idesc, 1);
                            }
                        } else {
                            for (int m = 0; m < p.mma_last; m++)
                                mma_bf16<false>(d, ad + (m >> 2) * (kSubBytes >> 4) + (m & 3) * a_step,
                                         bd + (m >> 2) * (sub_b >> 4) + (m & 3) * b_step, idesc, (kb != c0) | (m != 0));
                            ready = false;
                        }
                        any = true;
                        tc::commit<2>(empty0 + 8 * stage, 3);
                        if (kb == c1 - 1) tc::commit<2>(tfull0 + 8 * buf, 3);
                        stage = next;
                        phase = next_phase;
                    }
                }
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
        // A thread owns one row and 128 of the tile's columns.
        const int q = warp & 3, half = (warp - 2) >> 2;
        const uint32_t tempty_c0 = tc::mapa(tempty0, 0);
        const uint32_t stage_buf = tc::smem_u32(smOut + (warp - 2) * kStage);
        if (p.wait == kWaitStart || p.wait == kWaitEpilogue) pdl_wait();
        const float smax = MODE == kGrad || is_dw(MODE) || MODE == kDh ? __ldcg(p.smax) : 1.0f;
        int iter = 0, n = 0;
        if (FEW) {
            few_tokens<MODE>(p, few_lse, few_ratio, few_target);
            // A thread owns one row of w (rows past the tile's are whatever shared memory held: they
            // stay in their rows) and half of the tokens, in sixteens.
            const int share = ((int)p.N + 31) / 32 * 16, own = half * share;
            float* turned = reinterpret_cast<float*>(smOut + kFewTable) + (warp - 2) * 512;
            for (int t = cid; t < p.total; t += ncl) {
                const int mt = tile_at(p, t).mt;
                const int row = mt * p.tile_m + (int)rank * (p.tile_m / 2) + q * 32 + lane;     // of the piece
                const bool in = q * 32 + lane < p.tile_m / 2 && row < p.M;
                const int64_t part = ((int64_t)mt * 2 + rank) * 4 + q;
                const int tokens = min(share, (int)p.N - own);         // of this warp, at most 64; 0 or less: none
                float z[64] = {};
                bool ok = true;
                for (int c0 = 0; c0 < p.k_stages && ok; c0 += p.chunk, ++iter) {
                    const int buf = iter & 1;
                    ok = wait(tfull0 + 8 * buf, (iter >> 1) & 1, abort_flag, p.status, p.timeout_ns);
                    if (!ok) break;
                    tc::fence_after();
                    const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * kTile + own);
#pragma unroll
                    for (int c = 0; c < 64; c += 16)
                        if (c < tokens) add_acc(z + c, ta + c);
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive_cluster(tempty_c0 + 8 * buf);
                }
                if (!ok) break;
                // sixteen tokens at a time; the loop stays one, and z moves on: this code is mostly run
                // once per call, and fetching it four times over took longer than running it
#pragma unroll 1
                for (int c = 0; c < tokens; c += 16) {
                    // the 32 rows by 16 tokens turn in shared memory: two lanes a token, 16 rows each.  (Sums
                    // across the lanes and stores of single elements took three times the instructions, and
                    // with one or two warps a scheduler an instruction costs its latency.)
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 16; j++) turned[32 * j + lane] = MODE == kFewGrad || in ? z[j] : kNegInf;
                    __syncwarp();
                    const int j = lane >> 1, token = own + c + j, row0 = row - lane;
                    const bool live = c + j < tokens;
                    const float* mine = turned + 32 * j;
                    const int at = few_target[token] - row0;       // the target's row, if it is one of these 32
                    if (MODE == kFewStats) {
                        float x[16], m4[4] = {kNegInf, kNegInf, kNegInf, kNegInf}, s4[4] = {};
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {          // four tokens read four different sets of banks
                            *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(mine + turn(lane, i));
#pragma unroll
                            for (int k = 0; k < 4; k++) m4[k] = fmaxf(m4[k], x[i + k]);
                        }
                        float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                        const float m0 = finite_or_zero(m);
#pragma unroll
                        for (int i = 0; i < 16; i++) s4[i & 3] += exp2_fast((x[i] - m0) * kLog2e);
                        float sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
                        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                        if ((lane & 1) == 0 && live) {
                            p.part[part * p.N + token] = make_float2(m, sum);
                            if (at >= 0 && at < 32 && row0 + at < p.M && q * 32 + at < p.tile_m / 2) p.hit[token] = mine[at];
                        }
                    } else if (live) {
                        const float ratio = few_ratio[token], lse = few_lse[token];
                        __nv_bfloat16* g = p.g + (int64_t)token * p.ld_g + row0;
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            // (tile_m / 2 is a multiple of 8, and a row of g has room for whole tiles of 256)
                            const int r = turn(lane, i);
                            if (q * 32 + r >= p.tile_m / 2 || row0 + r >= p.M) continue;
                            const float4 x = *reinterpret_cast<const float4*>(mine + r);
                            const float v[4] = {few_g(x.x, lse, ratio, at == r), few_g(x.y, lse, ratio, at == r + 1),
                                                few_g(x.z, lse, ratio, at == r + 2), few_g(x.w, lse, ratio, at == r + 3)};
                            const auto put = [](__nv_bfloat16* to, float a, float b, float c, float d) {
                                const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
                                *reinterpret_cast<uint2*>(to) =
                                    make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                            };
                            put(g + r, v[0], v[1], v[2], v[3]);
                            float lost = 0.0f;
                            if (at >= r && at < r + 4) {
                                lost = left_over(at < r + 2 ? (at == r ? v[0] : v[1]) : (at == r + 2 ? v[2] : v[3]));
                                p.lo[token] = lost;
                            }
                            if (p.g_lo)
                                put(p.g_lo + (g - p.g) + r, at == r ? lost : 0.0f, at == r + 1 ? lost : 0.0f,
                                    at == r + 2 ? lost : 0.0f, at == r + 3 ? lost : 0.0f);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 48; j++) z[j] = z[j + 16];
                }
            }
        } else {
        // kDw: first and count of this thread's row of tile t, read a tile ahead
        const auto owner_of = [&](int t) {
            const TileAt at = tile_at(p, min(t, p.total - 1));
            const int64_t r = (int64_t)at.mt * kTile + rank * 128 + q * 32 + lane;
            return r < p.M && at.split == 0 ? *reinterpret_cast<const int2*>(p.owner + r) : make_int2(0, 0);
        };
        int2 next_owner = MODE == kDw ? owner_of(cid) : make_int2(0, 0);
        for (int t = cid; t < p.total; t += ncl) {
            const TileAt ti = tile_at(p, t);
            const int64_t row0 = (int64_t)ti.mt * kTile + rank * 128 + q * 32, row = row0 + lane;       // tile_m is 256
            const int64_t col0 = (int64_t)ti.nt * kTile + half * 128;
            // what the row needs, read while the tile is computed
            int target = -1;                       // the target's column among this thread's 128
            float lse = 0.0f, ratio = 0.0f;
            if ((MODE == kStats || MODE == kGrad) && row < p.M) {
                const int64_t id = p.targets[row];
                if (id >= 0 && id < p.vocab) {
                    if (MODE == kGrad) {
                        lse = p.lse[row];
                        ratio = p.dloss[row] / smax;
                    }
                    const int64_t at = id - p.col0 - col0;
                    if (at >= 0 && at < 128) target = (int)at;
                }
            }
            // what the targets' entries lost adds to this row: `factor` times a row, or a row of sums
            const __nv_bfloat16* extra = nullptr;
            const int32_t* sums = nullptr;
            float factor = 1.0f, factor2 = 1.0f;
            if (MODE == kDh && row < p.M && ti.split == 0) {
                const int64_t id = p.targets[row] - p.col0;
                if (id >= 0 && id < p.piece_cols) {
                    factor = p.lo[row];
                    if (factor != 0.0f) extra = p.w + id * p.ldw;
                }
            }
            if (MODE == kDw) {
                const int2 o = next_owner;
                next_owner = owner_of(t + ncl);
                if (o.y == 1) {
                    extra = p.h + o.x * p.ldh;
                    factor = p.lo[o.x];
                } else if (o.y > 1) {
                    sums = p.sums.rows + (p.sums.by_row ? p.col0 + row : o.x) * p.sums.cols;
                    const int unit = sum_unit(p.sums.hmax[p.sums.hmaxes], o.y);
                    factor = scalbnf(1.0f, unit / 2);      // (2^unit may not be a float)
                    factor2 = scalbnf(1.0f, unit - unit / 2);
                }
            }
            const int own_cols = (int)min((int64_t)128, p.N - col0);        // a multiple of 8 where it is used
            const auto add_extra = [&](float* v, int u0) {         // to 32 columns, the tile's from 8 u0 on
                if (extra) {
                    Pack<__nv_bfloat16, 8> from[4];
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        from[u].zero();
                        if (8 * (u0 + u) < own_cols) from[u].load(extra + col0 + 8 * (u0 + u));
                    }
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        float f[8];
                        from[u].unpack(f);
#pragma unroll
                        for (int e = 0; e < 8; e++) v[8 * u + e] = fmaf(factor, f[e], v[8 * u + e]);
                    }
                } else if (MODE == kDw && sums) {
                    int4 q[8];
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        q[e] = make_int4(0, 0, 0, 0);
                        if (8 * u0 + 4 * e < own_cols) q[e] = *reinterpret_cast<const int4*>(sums + col0 + 8 * u0 + 4 * e);
                    }
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        v[4 * e] = fmaf((float)q[e].x * factor, factor2, v[4 * e]);
                        v[4 * e + 1] = fmaf((float)q[e].y * factor, factor2, v[4 * e + 1]);
                        v[4 * e + 2] = fmaf((float)q[e].z * factor, factor2, v[4 * e + 2]);
                        v[4 * e + 3] = fmaf((float)q[e].w * factor, factor2, v[4 * e + 3]);
                    }
                }
            };
            const bool live = row0 < p.M && (MODE == kStats || col0 < p.N);
            const uint32_t ta0 = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * 128);
            // 32 columns of the product, from the tile's column c on, leave
            const auto leave = [&](float (&v)[32], int c) {
                const int col = (int)col0 + c;
                if ((MODE == kDh || is_dw(MODE)) && !p.direct) {
                    store_acc(v, stage_buf, &tmOut, col, (int)row0, ti.split, p.add != 0, n, lane);
                    return;
                }
                if (MODE == kGrad) {
                    // ratio 0 (a token that does not count) gives 0 whatever its logits
#pragma unroll
                    for (int j = 0; j < 32; j++) {
                        const float g = exp2_fast((v[j] - lse) * kLog2e) - (target == c + j ? 1.0f : 0.0f);
                        v[j] = ratio == 0.0f ? 0.0f : g;
                    }
                    const bool here = target >= c && target < c + 32;
                    if (__any_sync(0xffffffffu, here)) {
                        float at = 0.0f;
#pragma unroll
                        for (int j = 0; j < 32; j++) at = target == c + j ? v[j] : at;
                        if (here) {
                            const float lost = left_over(at * ratio);
                            p.lo[row] = lost;
                            if (p.g_lo) p.g_lo[row * p.ld_g + col0 + target] = __float2bfloat16_rn(lost);
                            if (p.owner) {                 // the smallest and the number: in whatever order
                                Owner* o = p.owner + col0 + target;
                                atomicMin(&o->first, (int)row);
                                atomicAdd(&o->count, 1);
                            }
                        }
                    }
                }
                store_bf16(v, MODE == kGrad ? ratio : smax, stage_buf, &tmOut, col, (int)row0, n, lane);
            };
            if constexpr (!LONG) {
                const int buf = iter & 1;
                // on its way while the tile is computed (held in registers it cost 64 tokens' dh 8 of 148 us)
                if (takes_extra(MODE) && extra)
                    for (int u = 0; 8 * u < own_cols; u += 8)
                        asm volatile("prefetch.global.L1 [%0];" :: "l"(extra + col0 + 8 * u));
                if (!wait(tfull0 + 8 * buf, (iter >> 1) & 1, abort_flag, p.status, p.timeout_ns)) break;
                tc::fence_after();
                ++iter;
                if (live)
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        float v[32];
                        load_acc(v, ta0 + (uint32_t)(buf * kTile + c));
                        if (takes_extra(MODE)) add_extra(v, c / 8);
                        leave(v, c);
                    }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(tempty_c0 + 8 * buf);
                continue;
            }
            float z[128] = {};
            if (takes_extra(MODE))
#pragma unroll
                for (int u = 0; u < 16; u += 4) add_extra(z + 8 * u, u);
            bool ok = true;
            for (int c0 = ti.k0; c0 < ti.k1; c0 += p.chunk, ++iter) {
                ok = wait(tfull0 + 8 * (iter & 1), (iter >> 1) & 1, abort_flag, p.status, p.timeout_ns);
                if (!ok) break;
                tc::fence_after();
                if (MODE == kStats || live)
#pragma unroll
                    for (int c = 0; c < 128; c += 16) add_acc(z + c, ta0 + (uint32_t)((iter & 1) * kTile + c));
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(tempty_c0 + 8 * (iter & 1));
            }
            if (!ok) break;
            if (!live) continue;
            if constexpr (MODE == kStats) {
                const int cols = (int)min((int64_t)128, p.N - col0);       // 0 or less: an empty part
                if (cols < 128)
#pragma unroll
                    for (int j = 0; j < 128; j++) z[j] = j < cols ? z[j] : kNegInf;
                if (__any_sync(0xffffffffu, target >= 0)) {
                    float hit = 0.0f;
#pragma unroll
                    for (int j = 0; j < 128; j++) hit = target == j ? z[j] : hit;
                    if (target >= 0) p.hit[row] = hit;         // a target is below the vocabulary's end
                }
                float m4[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
                for (int j = 4; j < 128; j++) m4[j & 3] = fmaxf(m4[j & 3], z[j]);
                const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                // z - m is formed first: a product with log2(e) before it would round away the
                // difference of large logits
                const float m0 = finite_or_zero(m);
                float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < 128; j++) s[j & 3] += exp2_fast((z[j] - m0) * kLog2e);
                if (row < p.M) p.part[((int64_t)2 * ti.nt + half) * p.M + row] = make_float2(m, (s[0] + s[1]) + (s[2] + s[3]));
            } else {
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; j++) v[j] = z[c + j];
                    leave(v, c);
                }
            }
        }
        }
        if (lane == 0) tc::bulk_wait_all();
    }

    // what was launched before this kernel is done when this kernel is
    if (p.wait == kWaitEnd) pdl_wait();
    // Both CTAs have stopped issuing.  If either gave up, both know after the barrier, and the even CTA
    // waits (bounded) for the loads still in flight before either may exit.
    tc::fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) st_cluster(tc::mapa(tc::smem_u32((const void*)peer_abort), rank ^ 1), 1);
    tc::cluster_sync();
    if (*abort_flag || *peer_abort) {
        if (leader && warp == 0 && lane == 0)
            drain_loads(full0, S, *issued_slot, tc::ld_cluster_s32(tc::mapa(tc::smem_u32((const void*)issued_slot), 1)), p.tx);
        tc::cluster_sync();
    }
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_dealloc<2>(tmem, kTmemCols);
    }
}

// BF16 matrix [rows, cols] with pitch ld, box 64 columns x box_rows, 128-byte
// swizzle; elements outside read as zero.
bool map_operand(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows) {
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
// g and g_lo [2][tokens][ld], box 64 columns x 64 tokens x 1: tokens past the last read as zero
bool map_halves(CUtensorMap* m, const void* p, int64_t tokens, int64_t cols, int64_t ld) {
    tmap::EncodeTiledFn enc = tmap::encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)tokens, 2};
    cuuint64_t strides[2] = {(cuuint64_t)(ld * 2), (cuuint64_t)(tokens * ld * 2)};
    cuuint32_t box[3] = {64u, (cuuint32_t)kSubK, 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// FP32 accumulator [splits][rows][cols], box 16 columns x 32 rows, 64-byte swizzle
bool map_acc(CUtensorMap* m, float* p, int64_t splits, int64_t rows, int64_t cols) {
    tmap::EncodeTiledFn enc = tmap::encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)splits};
    cuuint64_t strides[2] = {(cuuint64_t)(cols * 4), (cuuint64_t)(rows * cols * 4)};
    cuuint32_t box[3] = {16u, 32u, 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One operand of a product: its matrix in memory ([rows, cols], pitch ld)
struct Operand {
    const void* p;
    int64_t rows, cols, ld;
};

// Order of the tiles: groups of `raster` tiles along m (or n), swept along the
// other dimension.  A group's strips (a strip: 256 rows of an operand, all of
// K) that fit in L2 are read from memory once, the other operand once per
// group; where they do not, each wave of tiles reads the strips it touches.
// The order with the fewest bytes is taken.  Measured (8192 x 65536 x 4096):
// 16 row tiles 2.451 ms, 12 2.481, 24 2.458, and 8 or 32 (67 MB, which do not
// stay) 4 to 6% slower.
void choose_raster(GemmParams& p, int64_t K, int pairs) {
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
int stream_rows(int64_t vocab, int num_sms) {
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
template <int MODE, bool LONG>
cudaError_t launch_gemm(const GemmParams& p, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& out, int pairs,
                        cudaStream_t st) {
    static SharedMemory smem;
    const cudaError_t e = smem.allow(reinterpret_cast<const void*>(head_gemm_kernel<MODE, LONG>), kSmem);
    if (e != cudaSuccess) return e;
    return launch_k(p.wait != kWaitLaunch, head_gemm_kernel<MODE, LONG>, dim3(2 * pairs), kGemmThreads, kSmem, st, ta, tb, out, p);
}
template <int MODE>
cudaError_t gemm(GemmParams p, const Operand& a, const Operand& b, const CUtensorMap* out, int64_t K, int splits,
                 int tile_m, int tile_n, int wait, const HeadArgs& args, cudaStream_t st) {
    CUtensorMap ta, tb;
    if (!(MODE == kDwFull ? map_halves(&ta, a.p, a.rows, a.cols, a.ld)
                         : map_operand(&ta, a.p, a.rows, a.cols, a.ld, a_mn(MODE) ? kSubK : tile_m / 2)) ||
        !map_operand(&tb, b.p, b.rows, b.cols, b.ld, b_mn(MODE) ? kSubK : tile_n / 2))
        return cudaErrorInvalidValue;
    p.tile_n = tile_n;
    p.k_stages = (int32_t)((K + kSub * kSubK - 1) / (kSub * kSubK));
    p.chunk = MODE == kDh || is_dw(MODE) ? kSumChunk : kChunk;
    p.mma_last = (int32_t)((K - (int64_t)(p.k_stages - 1) * kSub * kSubK + 15) / 16);
    p.tile_m = tile_m;
    p.b_bytes = kSub * (tile_n / 2) * kSubK * 2;
    p.stages = std::min(kMaxStages, (kSmem - 1024 - 256 - kFewOut) / (kOpBytes + p.b_bytes));
    p.tx = (uint32_t)(kSub * (tile_m / 2) * kSubK * 2 + p.b_bytes);
    p.m_tiles = (int32_t)((p.M + tile_m - 1) / tile_m);
    p.n_tiles = (int32_t)((p.N + tile_n - 1) / tile_n);
    p.split_stages = (p.k_stages + splits - 1) / splits;
    p.splits = (p.k_stages + p.split_stages - 1) / p.split_stages;
    const int64_t total = (int64_t)p.m_tiles * p.n_tiles * p.splits;
    if (total > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.total = (int32_t)total;
    p.wait = wait;
    p.status = args.status;
    p.timeout_ns = args.timeout_ns;
    const int pairs = (int)std::max<int64_t>(1, std::min<int64_t>(args.num_sms / 2, total));
    choose_raster(p, K, pairs);
    if constexpr (MODE == kGrad || MODE == kDh || is_dw(MODE))
        if (p.split_stages <= p.chunk) return launch_gemm<MODE, false>(p, ta, tb, out ? *out : ta, pairs, st);
    return launch_gemm<MODE, true>(p, ta, tb, out ? *out : ta, pairs, st);
}

// ------------------------------------------------------- around the products
// A part of a row's statistics: the maximum m and sum exp(z - m).  NaN sums stay
// NaN, also beside parts without a number (m = -inf).
struct Stat {
    float m, s;
};
__device__ __forceinline__ Stat join(Stat a, Stat b) {
    const float m = fmaxf(a.m, b.m), m0 = finite_or_zero(m);
    return {m, a.s * exp2_fast((a.m - m0) * kLog2e) + b.s * exp2_fast((b.m - m0) * kLog2e)};
}

// Joins a row's parts: TT tokens a CTA, the parts dealt to 512 / TT threads
// each, eight at a time (one rescaling for the eight), whose results one warp
// joins.  Bound by latency: what 7 tokens of 50021 columns (1792 parts) wait for.
template <int TT>
__global__ void __launch_bounds__(512) head_join_kernel(const float2* part, int64_t parts, int64_t T, int64_t V,
                                                        const float* hit, const int64_t* targets, float* loss,
                                                        float* lse) {
    constexpr int G = 512 / TT;
    __shared__ Stat joined[TT][G + 1];
    const int tt = threadIdx.x % TT, g = threadIdx.x / TT;
    const int64_t first = (int64_t)blockIdx.x * TT;
    pdl_wait();
    Stat own = {kNegInf, 0.0f};
    if (first + tt < T) {
        for (int64_t i = g; i < parts; i += 8 * G) {
            float2 v[8];
            float m = own.m;
#pragma unroll
            for (int u = 0; u < 8; u++)
                v[u] = i + u * G < parts ? part[(i + u * G) * T + first + tt] : make_float2(kNegInf, 0.0f);
#pragma unroll
            for (int u = 0; u < 8; u++) m = fmaxf(m, v[u].x);
            const float m0 = finite_or_zero(m);
            float s = own.s * exp2_fast((own.m - m0) * kLog2e);
#pragma unroll
            for (int u = 0; u < 8; u++) s += v[u].y * exp2_fast((v[u].x - m0) * kLog2e);
            own = {m, s};
        }
    }
    joined[tt][g] = own;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (int k = threadIdx.x >> 5; k < TT && first + k < T; k += 16) {
        Stat a = {kNegInf, 0.0f};
        for (int i = lane; i < G; i += 32) a = join(a, joined[k][i]);
#pragma unroll
        for (int d = 16; d; d >>= 1)
            a = join(a, {__shfl_xor_sync(0xffffffffu, a.m, d), __shfl_xor_sync(0xffffffffu, a.s, d)});
        if (lane == 0) {
            const float l = a.m + logf(a.s);
            const int64_t t = first + k, target = targets[t];
            lse[t] = l;
            loss[t] = target >= 0 && target < V ? l - hit[t] : 0.0f;
        }
    }
}

// What is taken out of dloss: its largest finite magnitude over the tokens that count (the first CTA).  And what
// g's epilogue and head_target_kernel start from: g_lo or the sums are 0 (`zeros` 16-byte vectors at `zero`), and, with
// `owner`, no token has any vocabulary row as its target, and each CTA's largest finite |h|.
__global__ void __launch_bounds__(1024) head_scale_kernel(const float* dloss, const int64_t* targets, int64_t T, int64_t V,
                                                          float* smax, uint4* zero, int64_t zeros, Owner* owner, float* hmax,
                                                          const __nv_bfloat16* h, int64_t ldh, int64_t D) {
    __shared__ float part[32];
    pdl_launch_dependents();
    const int64_t at = (int64_t)blockIdx.x * 1024 + threadIdx.x, step = (int64_t)gridDim.x * 1024;
    const auto largest = [&](float m) {            // of the CTA, known to the first thread
        __syncthreads();
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
        if (threadIdx.x == 0)
            for (int w = 1; w < 32; w++) m = fmaxf(m, part[w]);
        return m;
    };
    if (blockIdx.x == 0) {
        const float m = largest(largest_dloss(dloss, targets, T, V, threadIdx.x, 1024));
        if (threadIdx.x == 0) *smax = dloss_scale(m);
    }
    for (int64_t i = at; i < zeros; i += step) zero[i] = make_uint4(0, 0, 0, 0);
    if (!owner) return;
    for (int64_t v = at; v < V; v += step) owner[v] = {INT_MAX, 0};
    float m = 0.0f;
    const int64_t per = D / 8;
#pragma unroll 4
    for (int64_t i = at; i < T * per; i += step) {
        const int64_t t = i / per;
        Pack<__nv_bfloat16, 8> p;
        float f[8];
        p.load(h + t * ldh + (i - t * per) * 8);
        p.unpack(f);
#pragma unroll
        for (int e = 0; e < 8; e++)
            if (fabsf(f[e]) <= FLT_MAX) m = fmaxf(m, fabsf(f[e]));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    m = largest(m);
    if (threadIdx.x == 0) hmax[blockIdx.x] = m;
}

// Adds lo[t] h[t, :] to its target's sums where several tokens have that target (kDw adds a single token's itself):
// `wpt` warps a token, a column a lane.  Bound by the atomics: 200000 tokens of 257 x 256 in some 170 us (all of one target
// 1.4 ms).
// Right behind g (`after_g`), or beside dh, which leaves an SM 700 bytes of shared memory and 11000 registers.
constexpr int kTargetThreads = 256;
__global__ void __launch_bounds__(kTargetThreads, 5)
head_target_kernel(const __nv_bfloat16* h, int64_t ldh, const int64_t* targets, const float* lo, int64_t T, int64_t v0,
                   int64_t n, const Owner* owner, int after_g, Sums sums, float* all_hmax, int wpt) {
    if (after_g) pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * (kTargetThreads / 32 / wpt) + warp / wpt, v = t < T ? targets[t] - v0 : -1;
    Owner o = {0, 0};
    if (v >= 0 && v < n) o = owner[v];
    if (o.count > 1 || blockIdx.x == 0) {
        float hmax = 0.0f;
        for (int i = lane; i < sums.hmaxes; i += 32) hmax = fmaxf(hmax, sums.hmax[i]);
#pragma unroll
        for (int d = 16; d; d >>= 1) hmax = fmaxf(hmax, __shfl_xor_sync(0xffffffffu, hmax, d));
        if (blockIdx.x == 0 && threadIdx.x == 0) *all_hmax = hmax;
        if (o.count > 1) {
            const int unit = sum_unit(hmax, o.count);
            const float f = lo[t], up = scalbnf(1.0f, -unit / 2), up2 = scalbnf(1.0f, -unit - (-unit / 2));
            int32_t* row = sums.rows + (sums.by_row ? v0 + v : o.first) * sums.cols;
            const __nv_bfloat16* from = h + t * ldh;
#pragma unroll 8
            for (int64_t c = warp % wpt * 32 + lane; c < sums.cols; c += 32 * wpt) {
                const float x = __bfloat162float(from[c]);
                if (fabsf(x) <= FLT_MAX) atomicAdd(row + c, __float2int_rn(f * x * up * up2));
            }
        }
    }
    // what was launched before this kernel is done when this kernel is
    if (!after_g && blockIdx.x == 0) pdl_wait();
}

// dh (or dw) = smax * the sum of the splits' accumulators [splits][T][D], 8 columns a
// thread.  Bound by memory; of the batch of 8192 x 4096 it is about 40 of 7800 us.
__global__ void __launch_bounds__(256) head_sum_kernel(const float* acc, int splits, int64_t T, int64_t D,
                                                      const float* smax, __nv_bfloat16* out, int64_t ld) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = D / 8;
    if (i >= T * per) return;
    pdl_wait();
    const int64_t t = i / per, c = (i - t * per) * 8;
    float v[8] = {};
    for (int s = 0; s < splits; s++) {
        const float4* a = reinterpret_cast<const float4*>(acc + ((int64_t)s * T + t) * D + c);
        const float4 x = a[0], y = a[1];
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
    const float f = *smax;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++)
        w[j] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * j] * f)) |
               ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * j + 1] * f)) << 16);
    *reinterpret_cast<uint4*>(out + t * ld + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// columns of one piece of the vocabulary
int64_t piece_cols(int64_t tokens, int64_t vocab) {
    const int64_t most = std::max<int64_t>(2048, kPieceBytes / (2 * tokens) / kTile * kTile);
    return std::min(round_up(vocab, kTile), most);
}
// dh has few tiles when there are few tokens, and dw when the vocabulary is
// small: the sum over K is then split, so that the pairs get equally much.  The
// estimate: a stage takes 0.55 us, and a split's FP32 tile is written and read.
// (526 tokens, 35368 x 3656: 45 tiles of dh on 76 pairs, 458 us for the gradient
// in one split, 418 in 5; 5180 tokens, 596 x 72: dw in one split kept 3 pairs
// busy for 24 us.)
int splits_of(int64_t rows, int64_t cols, int64_t k, int num_sms) {
    const int64_t tiles = (rows + kTile - 1) / kTile * ((cols + kTile - 1) / kTile), pairs = std::max(1, num_sms / 2);
    const int64_t stages = (k + kSub * kSubK - 1) / (kSub * kSubK);
    const double split_us = (double)rows * cols * 8 / 6.7e6;
    int64_t best = 1;
    double least = 0.0;
    for (int64_t n = 1; n == 1 || (n * 8 <= stages && n * tiles <= 8 * pairs); n++) {
        const double us = (double)((tiles * n + pairs - 1) / pairs) * ((stages + n - 1) / n) * 0.55 + (n > 1 ? n * split_us : 0.0);
        if (n == 1 || us < least) {
            least = us;
            best = n;
        }
    }
    const int64_t per = (stages + best - 1) / best;
    return (int)((stages + per - 1) / per);        // those that get any
}
// The targets' entries of g, which are by far its largest, enter dw in full.  Either what each lost to BF16 is a
// second matrix g_lo, zero elsewhere, whose product with h is summed behind g's; or it is added by row, in kDw's
// epilogue, from h or from the sums of head_target_kernel.  The matrix costs a third of the gradient's operations and
// the bytes of g twice, the rows a launch beside dh and loads in the epilogue.  So the matrix is for few tokens, whose
// dw is bound by its writes, for small products, and for vocabularies of whose rows each has several tokens.
// (Matrix and rows: 64 tokens of 50021 x 4096 226 and 254 us, 129 of 300 x 64 23 and 27, 1909 of 409 x 1448 44 and 54,
// 200 of 50021 x 4096 332 and 288.)
bool full_matrix(int64_t tokens, int64_t vocab, int64_t cols, int64_t piece) {
    const int64_t entries = tokens * piece;
    return tokens <= kFewTokens || (piece >= vocab && (entries <= 1 << 20 || (tokens >= vocab && entries <= 1 << 24 &&
                                                                              (double)tokens * vocab * cols <= 8e9)));
}
int half_subs(int64_t tokens) { return (int)((tokens + kSubK - 1) / kSubK); }
// of dw: only where the vocabulary is one piece
int dw_splits(int64_t tokens, int64_t vocab, int64_t cols, int64_t piece, int num_sms) {
    if (piece < vocab) return 1;
    return splits_of(vocab, cols, full_matrix(tokens, vocab, cols, piece) ? (int64_t)half_subs(tokens) * kSub * kSubK : tokens, num_sms);
}
// dh comes out of one product as it is
bool dh_direct(int splits, int64_t piece, int64_t vocab) { return splits == 1 && piece >= vocab; }

// parts of a row's statistics
int64_t head_parts(int64_t tokens, int64_t vocab, int num_sms) {
    if (tokens <= kFewTokens) {
        const int tm = stream_rows(vocab, num_sms);
        return (vocab + tm - 1) / tm * 8;
    }
    return (vocab + kTile - 1) / kTile * 2;
}

}  // namespace

size_t head_workspace(int64_t tokens, int64_t vocab, int64_t cols, bool backward, int num_sms) {
    if (!backward) return (size_t)(head_parts(tokens, vocab, num_sms) * tokens * 8 + round_up(tokens * 4, 16));
    const int64_t piece = piece_cols(tokens, vocab);
    const int splits = splits_of(tokens, cols, std::min(piece, vocab), num_sms), dw = dw_splits(tokens, vocab, cols, piece, num_sms);
    // g and g_lo; or g, the targets' owners, the sums of several tokens and the maxima of h
    const bool full = full_matrix(tokens, vocab, cols, piece);
    return (size_t)(256 + (piece < vocab ? 2 : 1) * (full ? 2 : 1) * tokens * piece * 2 + round_up(tokens * 4, 16) +
                    (full ? 0 : round_up(vocab * (int64_t)sizeof(Owner), 16) + std::min(tokens, vocab) * cols * 4 +
                                   round_up((num_sms + 1) * 4, 16)) +
                    (dh_direct(splits, piece, vocab) ? 0 : splits * tokens * cols * 4) + (dw > 1 ? dw * vocab * cols * 4 : 0));
}

cudaError_t run_head(const HeadArgs& a, cudaStream_t st) {
    const int64_t T = a.tokens, parts = head_parts(T, a.vocab, a.num_sms);
    GemmParams p{};
    p.M = T;
    p.N = a.vocab;
    p.targets = a.targets;
    p.vocab = a.vocab;
    p.part = static_cast<float2*>(a.ws);
    p.hit = reinterpret_cast<float*>(p.part + parts * T);
    const Operand h{a.h, T, a.cols, a.ldh}, w{a.w, a.vocab, a.cols, a.ldw};
    cudaError_t e;
    if (T <= kFewTokens) {
        std::swap(p.M, p.N);
        e = gemm<kFewStats>(p, w, h, nullptr, a.cols, 1, stream_rows(a.vocab, a.num_sms), (int)round_up(T, 16), kWaitLaunch, a, st);
    } else {
        e = gemm<kStats>(p, h, w, nullptr, a.cols, 1, kTile, kTile, kWaitLaunch, a, st);
    }
    if (e != cudaSuccess) return e;
    // tokens a CTA: few where there are few, so that more threads share a token's parts
    const auto k = T >= 4096 ? head_join_kernel<32> : T > kFewTokens ? head_join_kernel<8> : head_join_kernel<2>;
    const int tt = T >= 4096 ? 32 : T > kFewTokens ? 8 : 2;
    return launch_k(true, k, dim3((unsigned)((T + tt - 1) / tt)), 512, 0, st, p.part, parts, T, a.vocab, p.hit, a.targets,
                    a.loss, a.lse);
}

// Per piece: g, then dh and dw from it.  dw (or the sums for its epilogue, and then dw) runs beside dh's last tiles, and
// the next piece's g (in the other of two buffers) beside dw's: each kernel is
// launched while the one before it drains, so that no SM waits for the end of
// a wave.  dh waits until everything before it is done: it needs g, and its
// accumulator takes the pieces in order; dw and the next g start after dh has
// waited.  max |dloss| is needed by the first g's epilogue only; few tokens
// find it themselves.
cudaError_t run_head_backward(const HeadArgs& a, cudaStream_t st) {
    const int64_t T = a.tokens, V = a.vocab, D = a.cols, piece = piece_cols(T, V);
    const int splits = splits_of(T, D, std::min(piece, V), a.num_sms), dw_split = dw_splits(T, V, D, piece, a.num_sms);
    const bool few = T <= kFewTokens, full = full_matrix(T, V, D, piece), direct = dh_direct(splits, piece, V);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    float* smax = reinterpret_cast<float*>(ws);
    uint8_t* g0 = ws + 256;
    const int64_t g_bytes = (full ? 2 : 1) * T * piece * 2;
    float* lo = reinterpret_cast<float*>(g0 + (piece < V ? 2 : 1) * g_bytes);
    uint8_t* rest = reinterpret_cast<uint8_t*>(lo) + round_up(T * 4, 16);
    Owner* owner = full || !a.dw ? nullptr : reinterpret_cast<Owner*>(rest);
    // what head_scale_kernel clears: g_lo (one piece: behind the only g), or the sums
    const int64_t zeros = !a.dw ? 0 : full ? T * piece / 8 : std::min(T, V) * D / 4;
    const int ctas = (int)std::max<int64_t>(1, std::min<int64_t>(a.num_sms, owner ? std::max(V / 2048, T * D / 8192) : zeros / 2048));
    Sums sums{};
    float* hmax = nullptr;
    if (!full) {
        rest += round_up(V * (int64_t)sizeof(Owner), 16);
        sums.rows = reinterpret_cast<int32_t*>(rest);
        sums.cols = D;
        sums.by_row = V <= T;
        rest += std::min(T, V) * D * 4;
        sums.hmax = hmax = reinterpret_cast<float*>(rest);
        sums.hmaxes = ctas;
        rest += round_up((a.num_sms + 1) * 4, 16);
    }
    float* acc = reinterpret_cast<float*>(rest);
    float* dw_acc = acc + (direct ? 0 : splits * T * D);
    cudaError_t e = cudaSuccess;
    if (!few) {
        head_scale_kernel<<<ctas, 1024, 0, st>>>(a.dloss, a.targets, T, V, smax,
                                                 reinterpret_cast<uint4*>(full ? g0 + T * piece * 2 : reinterpret_cast<uint8_t*>(sums.rows)),
                                                 zeros, owner, hmax, static_cast<const __nv_bfloat16*>(a.h), a.ldh, D);
        e = cudaGetLastError();
    }
    for (int64_t v0 = 0, i = 0; v0 < V && e == cudaSuccess; v0 += piece, i++) {
        const int64_t n = std::min(piece, V - v0);
        const uint8_t* w = static_cast<const uint8_t*>(a.w) + v0 * a.ldw * 2;
        uint8_t* g = g0 + (i & 1) * g_bytes;
        GemmParams p{};
        p.targets = a.targets;
        p.vocab = V;
        p.col0 = v0;
        p.lse = a.lse;
        p.dloss = a.dloss;
        p.smax = smax;
        p.lo = lo;
        p.owner = owner ? owner + v0 : nullptr;
        p.put_smax = i == 0;
        p.M = T;
        p.N = n;
        CUtensorMap out;
        const Operand h{a.h, T, D, a.ldh}, wp{w, n, D, a.ldw}, gp{g, T, n, piece};
        // without dw in between, the kernel before may be the dh of the piece that this buffer held
        const int wait = i == 0 ? (few ? kWaitLaunch : kWaitEpilogue) : a.dh && a.dw ? kWaitEnd : kWaitStart;
        p.g = reinterpret_cast<__nv_bfloat16*>(g);
        p.g_lo = full && a.dw ? p.g + T * piece : nullptr;
        p.ld_g = piece;
        if (few) {
            p.M = n;
            p.N = T;
            e = gemm<kFewGrad>(p, wp, h, nullptr, D, 1, stream_rows(n, a.num_sms), (int)round_up(T, 16), wait, a, st);
        } else {
            if (!tmap::out_2d(&out, g, T, n, piece, true)) return cudaErrorInvalidValue;
            e = gemm<kGrad>(p, h, wp, &out, D, 1, kTile, kTile, wait, a, st);
        }
        if (e == cudaSuccess && a.dh) {
            p.M = T;
            p.N = D;
            p.add = v0 > 0;
            p.direct = direct;
            p.w = reinterpret_cast<const __nv_bfloat16*>(w);
            p.ldw = a.ldw;
            p.piece_cols = n;
            if (!(direct ? tmap::out_2d(&out, a.dh, T, D, a.ld_dh, true) : map_acc(&out, acc, splits, T, D)))
                return cudaErrorInvalidValue;
            e = gemm<kDh>(p, gp, wp, &out, n, splits, kTile, kTile, kWaitStart, a, st);
        }
        if (e == cudaSuccess && a.dw) {
            p.M = n;
            p.N = D;
            p.add = 0;
            p.direct = dw_split == 1;
            if (!(p.direct ? tmap::out_2d(&out, static_cast<uint8_t*>(a.dw) + v0 * a.ld_dw * 2, n, D, a.ld_dw, true)
                           : map_acc(&out, dw_acc, dw_split, V, D)))
                return cudaErrorInvalidValue;
            if (full) {
                p.half_subs = half_subs(T);
                p.sub_mmas = (int32_t)((std::min<int64_t>(T, kSubK) + 15) / 16);
                e = gemm<kDwFull>(p, gp, h, &out, (int64_t)p.half_subs * kSub * kSubK, dw_split, kTile, kTile,
                                  a.dh ? kWaitEnd : kWaitStart, a, st);
            } else {
                int wpt = 1;                       // about 512 columns each
                while (wpt < kTargetThreads / 32 && D > 512 * wpt) wpt *= 2;
                const int tokens = kTargetThreads / 32 / wpt;
                p.h = static_cast<const __nv_bfloat16*>(a.h);
                p.ldh = a.ldh;
                p.sums = sums;
                e = launch_k(true, head_target_kernel, dim3((unsigned)((T + tokens - 1) / tokens)), kTargetThreads, 0, st, p.h, a.ldh,
                             a.targets, lo, T, v0, n, p.owner, a.dh ? 0 : 1, sums, hmax + ctas, wpt);
                if (e == cudaSuccess) e = gemm<kDw>(p, gp, h, &out, T, dw_split, kTile, kTile, kWaitEpilogue, a, st);
            }
        }
    }
    const auto sum = [&](const float* from, int n, int64_t rows, void* to, int64_t ld) {
        return launch_k(true, head_sum_kernel, dim3((unsigned)((rows * (D / 8) + 255) / 256)), 256, 0, st, from, n, rows, D, smax,
                        static_cast<__nv_bfloat16*>(to), ld);
    };
    if (e == cudaSuccess && a.dh && !direct) e = sum(acc, splits, T, a.dh, a.ld_dh);
    if (e == cudaSuccess && a.dw && dw_split > 1) e = sum(dw_acc, dw_split, V, a.dw, a.ld_dw);
    return e;
}

}  // namespace bsq
