// Softmax cross entropy of a linear head, without keeping the logits.
//
// z = h w^T (BF16 operands, FP32 accumulation).  Forward: each output tile
// leaves, per row, its maximum m and s = sum exp(z - m) over its columns (the
// target's logit beside it); a second kernel joins the tiles of a row,
//   lse = M + log sum_i s_i exp(m_i - M),  M = max_i m_i,
// and loss = lse - z[target].  Backward, a piece of the vocabulary at a time:
// the logits' tile again, g = ratio (exp(z - lse) - [v = target]) in BF16 with
// ratio = dloss / max |dloss|, then dh += g w (FP32 between pieces) and
// dw = g^T h, both times max |dloss| in FP32.
#include <algorithm>
#include "common.cuh"
#include "internal.h"

namespace bsq {
namespace {

constexpr int BM = 128, BN = 128, BK = 16, kThreads = 256;
constexpr int64_t kPieceBytes = 256ll << 20;       // of g
constexpr float kNegInf = -INFINITY;

enum { kStats, kGrad, kDh, kDw };

// C(m, n) = sum_k A(m, k) B(n, k): an operand is K-major (k contiguous, ld
// between rows) or MN-major (m or n contiguous, ld between k).
struct TileArgs {
    const __nv_bfloat16 *a, *b;
    int64_t lda, ldb;
    int64_t M, N, K;
    const int64_t* targets;
    int64_t vocab;
    int64_t col0;                  // first vocabulary column of the piece
    float2* part;                  // kStats: [n tile][M] (max, sum)
    float* hit;                    // kStats: target's logit
    const float* lse;
    const float* dloss;
    const float* smax;
    __nv_bfloat16* out;            // kGrad: g; kDw: dw
    int64_t ldo;
    float* acc;                    // kDh: [M][N]
    int first;
};

template <int MODE, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kThreads) head_tile_kernel(const TileArgs p) {
    __shared__ float sa[BK][BM + 4], sb[BK][BN + 4];
    const int64_t m0 = (int64_t)blockIdx.y * BM, n0 = (int64_t)blockIdx.x * BN;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    float c[8][8] = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += BK) {
        for (int i = tid; i < BM * BK; i += kThreads) {
            const int k = A_MN ? i / BM : i % BK, m = A_MN ? i % BM : i / BK;
            const bool in = m0 + m < p.M && k0 + k < p.K;
            sa[k][m] = in ? __bfloat162float(A_MN ? p.a[(k0 + k) * p.lda + m0 + m] : p.a[(m0 + m) * p.lda + k0 + k]) : 0.0f;
        }
        for (int i = tid; i < BN * BK; i += kThreads) {
            const int k = B_MN ? i / BN : i % BK, n = B_MN ? i % BN : i / BK;
            const bool in = n0 + n < p.N && k0 + k < p.K;
            sb[k][n] = in ? __bfloat162float(B_MN ? p.b[(k0 + k) * p.ldb + n0 + n] : p.b[(n0 + n) * p.ldb + k0 + k]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < BK; k++) {
            float x[8], y[8];
#pragma unroll
            for (int i = 0; i < 8; i++) x[i] = sa[k][ty * 8 + i];
#pragma unroll
            for (int j = 0; j < 8; j++) y[j] = sb[k][tx * 8 + j];
#pragma unroll
            for (int i = 0; i < 8; i++)
#pragma unroll
                for (int j = 0; j < 8; j++) c[i][j] = fmaf(x[i], y[j], c[i][j]);
        }
        __syncthreads();
    }
    const float smax = MODE == kStats ? 0.0f : *p.smax;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int64_t m = m0 + ty * 8 + i;
        if (MODE == kStats) {
            const int64_t target = m < p.M ? p.targets[m] : -1;
            float mx = kNegInf;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int64_t n = n0 + tx * 8 + j;
                if (n >= p.N) c[i][j] = kNegInf;
                else if (n == target) p.hit[m] = c[i][j];
                mx = fmaxf(mx, c[i][j]);
            }
#pragma unroll
            for (int d = 8; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; j++) s += mx == kNegInf ? 0.0f : expf(c[i][j] - mx);
#pragma unroll
            for (int d = 8; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (tx == 0 && m < p.M) p.part[(int64_t)blockIdx.x * p.M + m] = make_float2(mx, s);
        } else if (m < p.M) {
            float ratio = 0.0f, lse = 0.0f;
            int64_t target = -1;
            if (MODE == kGrad) {
                target = p.targets[m];
                lse = p.lse[m];
                ratio = target >= 0 && target < p.vocab && smax > 0.0f ? p.dloss[m] / smax : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int64_t n = n0 + tx * 8 + j;
                if (n >= p.N) continue;
                if (MODE == kGrad) {
                    const float g = expf(c[i][j] - lse) - (p.col0 + n == target ? 1.0f : 0.0f);
                    p.out[m * p.ldo + n] = __float2bfloat16_rn(ratio == 0.0f ? 0.0f : ratio * g);
                } else if (MODE == kDh) {
                    float* a = p.acc + m * p.N + n;
                    *a = p.first ? c[i][j] : *a + c[i][j];
                } else {
                    p.out[m * p.ldo + n] = __float2bfloat16_rn(c[i][j] * smax);
                }
            }
        }
    }
}

__global__ void __launch_bounds__(256) head_join_kernel(const float2* part, int64_t parts, int64_t T, int64_t V,
                                                        const float* hit, const int64_t* targets, float* loss,
                                                        float* lse) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= T) return;
    float m = kNegInf, s = 0.0f;
    for (int64_t i = 0; i < parts; i++) {
        const float2 v = part[i * T + t];
        const float n = fmaxf(m, v.x);
        if (n != kNegInf) s = s * expf(m - n) + v.y * expf(v.x - n);
        m = n;
    }
    const float l = m + logf(s);
    lse[t] = l;
    const int64_t target = targets[t];
    loss[t] = target >= 0 && target < V ? l - hit[t] : 0.0f;
}

// max |dloss| over the tokens that count
__global__ void __launch_bounds__(1024) head_scale_kernel(const float* dloss, const int64_t* targets, int64_t T, int64_t V,
                                                          float* smax) {
    __shared__ float part[32];
    float m = 0.0f;
    for (int64_t t = threadIdx.x; t < T; t += 1024)
        if (targets[t] >= 0 && targets[t] < V) m = fmaxf(m, fabsf(dloss[t]));
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 32; w++) m = fmaxf(m, part[w]);
        *smax = m;
    }
}

__global__ void __launch_bounds__(256) head_dh_kernel(const float* acc, int64_t T, int64_t D, const float* smax,
                                                      __nv_bfloat16* dh, int64_t ld) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < T * D) dh[i / D * ld + i % D] = __float2bfloat16_rn(acc[i] * *smax);
}

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// columns of one piece of the vocabulary
int64_t piece_cols(int64_t tokens, int64_t vocab) {
    const int64_t most = std::max<int64_t>(2048, kPieceBytes / (2 * tokens) / 256 * 256);
    return std::min(round_up(vocab, 256), most);
}

}  // namespace

size_t head_workspace(int64_t tokens, int64_t vocab, int64_t cols, bool backward, int) {
    if (!backward) return (size_t)(round_up(vocab, BN) / BN * tokens * 8 + round_up(tokens * 4, 16));
    return (size_t)(16 + round_up(tokens * piece_cols(tokens, vocab) * 2, 16) + tokens * cols * 4);
}

cudaError_t run_head(const HeadArgs& a, cudaStream_t st) {
    const int64_t parts = round_up(a.vocab, BN) / BN;
    TileArgs p{};
    p.a = static_cast<const __nv_bfloat16*>(a.h);
    p.b = static_cast<const __nv_bfloat16*>(a.w);
    p.lda = a.ldh;
    p.ldb = a.ldw;
    p.M = a.tokens;
    p.N = a.vocab;
    p.K = a.cols;
    p.targets = a.targets;
    p.part = static_cast<float2*>(a.ws);
    p.hit = reinterpret_cast<float*>(p.part + parts * a.tokens);
    const dim3 grid((unsigned)parts, (unsigned)((a.tokens + BM - 1) / BM));
    head_tile_kernel<kStats, false, false><<<grid, kThreads, 0, st>>>(p);
    head_join_kernel<<<(unsigned)((a.tokens + 255) / 256), 256, 0, st>>>(p.part, parts, a.tokens, a.vocab, p.hit,
                                                                         a.targets, a.loss, a.lse);
    return cudaGetLastError();
}

cudaError_t run_head_backward(const HeadArgs& a, cudaStream_t st) {
    const int64_t T = a.tokens, V = a.vocab, D = a.cols, piece = piece_cols(T, V);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    float* smax = reinterpret_cast<float*>(ws);
    __nv_bfloat16* g = reinterpret_cast<__nv_bfloat16*>(ws + 16);
    float* acc = reinterpret_cast<float*>(ws + 16 + round_up(T * piece * 2, 16));
    head_scale_kernel<<<1, 1024, 0, st>>>(a.dloss, a.targets, T, V, smax);
    const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(a.h);
    const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(a.w);
    const unsigned mt = (unsigned)((T + BM - 1) / BM), dt = (unsigned)((D + BN - 1) / BN);
    for (int64_t v0 = 0; v0 < V; v0 += piece) {
        const int64_t n = std::min(piece, V - v0);
        TileArgs p{};
        p.targets = a.targets;
        p.vocab = V;
        p.lse = a.lse;
        p.dloss = a.dloss;
        p.smax = smax;
        p.col0 = v0;
        p.a = h;
        p.lda = a.ldh;
        p.b = w + v0 * a.ldw;
        p.ldb = a.ldw;
        p.M = T;
        p.N = n;
        p.K = D;
        p.out = g;
        p.ldo = piece;
        head_tile_kernel<kGrad, false, false><<<dim3((unsigned)((n + BN - 1) / BN), mt), kThreads, 0, st>>>(p);
        if (a.dh) {
            TileArgs q = p;
            q.a = g;
            q.lda = piece;
            q.N = D;
            q.K = n;
            q.acc = acc;
            q.first = v0 == 0;
            head_tile_kernel<kDh, false, true><<<dim3(dt, mt), kThreads, 0, st>>>(q);
        }
        if (a.dw) {
            TileArgs q = p;
            q.a = g;
            q.lda = piece;
            q.b = h;
            q.ldb = a.ldh;
            q.M = n;
            q.N = D;
            q.K = T;
            q.out = static_cast<__nv_bfloat16*>(a.dw) + v0 * a.ld_dw;
            q.ldo = a.ld_dw;
            head_tile_kernel<kDw, true, true><<<dim3(dt, (unsigned)((n + BM - 1) / BM)), kThreads, 0, st>>>(q);
        }
    }
    if (a.dh)
        head_dh_kernel<<<(unsigned)((T * D + 255) / 256), 256, 0, st>>>(acc, T, D, smax,
                                                                         static_cast<__nv_bfloat16*>(a.dh), a.ld_dh);
    return cudaGetLastError();
}

}  // namespace bsq
