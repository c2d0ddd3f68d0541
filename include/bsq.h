/*
 * bsq.h -- C ABI of libbsq.so: block-scaled low-precision linear layer on
 * NVIDIA GB300 (sm_103a).
 *
 * What the library computes (the pages give the method in prose only):
 *  - Quantize BF16 tensors to MXFP8 (E4M3 for forward activations and
 *    weights, E5M2 for gradients), to MXFP4 and to NVFP4, row-wise and
 *    column-wise ("FP8 Training Infrastructure", sections "O panorama da
 *    precisao numerica" and "Estrategias de escalonamento"; "Practical FP4
 *    Training for Large-Scale MoE Models on Hopper GPUs", section 2,
 *    kernel BF16ToFP4Row and the transposed FP4RowToFP8Col layout).
 *  - A block-scaled GEMM with FP32 accumulation that consumes codes and
 *    scales directly on the tensor cores (MoE FP4 page, section 2, heavy
 *    GEMMs stay on native FP8 tensor cores), dense and grouped over ragged
 *    expert batches (same section, "tensores ragged").
 *  - The direct integer-domain MXFP4 -> MXFP8 re-encode (same section,
 *    "Algoritmo de Conversao Direta"; kernel FP4RowToFP8Row), also writing
 *    per-expert padded scales for the grouped GEMM.
 *  - Around that path: FP4RowToFP8Col (MXFP4 rows to MXFP8 columns in one
 *    pass, same section, "Kernels"), MXFP4 -> FP8 with 1 x 128 blocks (the
 *    Hopper FP8 block of the same section), NVFP4 with delayed scaling
 *    from an amax history (FP8 page, "Estrategias de escalonamento"), and
 *    the GEMM on MXFP4 x MXFP4 operands natively.
 *  - What a mixture-of-experts step runs next to it: tokens sorted by expert
 *    and back, layer norm, the softmax cross entropy of a linear head and
 *    the global gradient norm with clipping, each with its gradient.
 *  - The dense feed-forward block and its update: linear layers with bias,
 *    activation and residual in the product's epilogue, the gated half with
 *    both projections in one kernel (BF16 with gradients, and on block-scaled
 *    operands), and AdamW over many tensors with moments in 32 or 8 bits.
 *
 * Conventions shared by every entry point
 *  - Matrices are row-major.  A GEMM computes C[M,N] = A[M,K] * B[N,K]^T:
 *    both operands are stored K-major (K is the contiguous last axis).
 *  - "Row-wise" quantization puts blocks along the last (contiguous) axis.
 *    "Column-wise" puts blocks along axis 0 and stores the TRANSPOSE: the
 *    column-wise output of a [R, C] input is a [C, R] tensor whose blocks
 *    run along its last axis, so every GEMM operand is K-major.
 *  - Codes: FP8 formats one byte per element; FP4 formats two elements per
 *    byte, the even-index element in the low nibble.
 *  - Scales: one byte per block (E8M0 for the MX formats, UE4M3 for NVFP4),
 *    stored in 512-byte tiles of 128 rows x 4 scale columns: the byte of
 *    scale (r, c) of a [rows, S] scale matrix is at
 *        ((r/128) * ceil(S/4) + c/4) * 512 + (r%32)*16 + ((r/32)%4)*4 + c%4.
 *    Rows are padded to a multiple of 128, scale columns to a multiple of
 *    4, and padding bytes are zero.  This is the scale-operand layout the
 *    tcgen05 block-scaled MMA reads.
 *  - MX block scale: e = floor(log2(block amax)) - emax, emax = 8 (E4M3),
 *    15 (E5M2), 2 (E2M1), clamped to [-127, 127]; an all-zero block gets
 *    e = -127; a block holding NaN/Inf gets scale 0xFF and NaN codes
 *    (E2M1: zero codes).  Codes are round-to-nearest-even of x * 2^-e with
 *    saturation to +-448 / +-57344 / +-6; the sign of zero is kept.
 *  - NVFP4: s_t = amax(finite |x|) / 2688 in FP32 (1 when the amax is 0);
 *    per 16-block s_b = UE4M3(RNE((amax_b / 6) / s_t)); codes are
 *    E2M1(RNE(x / (s_b * s_t))) with each step an IEEE FP32 operation; a
 *    zero s_b gives zero codes; a block holding NaN/Inf gets s_b = 0x7F and
 *    zero codes.
 *
 * Ownership: the caller allocates and frees every buffer (sizes from
 * bsq_codes_bytes / bsq_scales_bytes / bsq_grouped_scales_bytes).  Pointers passed to the compute
 * calls are DEVICE pointers.  The library keeps no allocation between calls;
 * its only state is a device status word in static device memory.
 *
 * Streams: `stream` is a cudaStream_t (NULL = legacy default stream).  All
 * compute calls are asynchronous on that stream.
 *
 * Errors: arguments are checked on the host before any launch; on failure
 * the call returns a status, launches nothing and writes nothing.  An empty
 * tensor (0 rows or 0 columns) is BSQ_ERR_INVALID_ARG; empty experts inside
 * a grouped batch (equal consecutive offsets) are valid.  The GEMMs and the
 * grouped re-encode take row counts up to 2^31 - 256 (their kernels index
 * rows in 32 bits; the grouped GEMM also bounds num_groups x B.rows);
 * larger ones are BSQ_ERR_UNSUPPORTED.  No C++
 * exception crosses this boundary.  Faults detected on the device (a wait
 * that exceeded its limit) set the device status word, which
 * bsq_sync_status() returns and clears.
 */
#ifndef BSQ_H
#define BSQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    BSQ_OK = 0,
    BSQ_ERR_INVALID_ARG = 1,   /* null pointer, bad enum, shape mismatch        */
    BSQ_ERR_UNSUPPORTED = 2,   /* valid request this library does not handle    */
    BSQ_ERR_ALIGNMENT = 3,     /* a pointer or a row pitch is not 16-byte aligned */
    BSQ_ERR_CUDA = 4,          /* a CUDA runtime call failed                    */
    BSQ_ERR_TIMEOUT = 5        /* a device-side wait ran past its limit         */
} bsq_status;

typedef enum {
    BSQ_MXFP8_E4M3 = 0,        /* E4M3 codes, 32-element blocks, E8M0 scales    */
    BSQ_MXFP8_E5M2 = 1,        /* E5M2 codes, 32-element blocks, E8M0 scales    */
    BSQ_MXFP4_E2M1 = 2,        /* E2M1 codes, 32-element blocks, E8M0 scales    */
    BSQ_NVFP4_E2M1 = 3         /* E2M1 codes, 16-element blocks, UE4M3 scales,
                                  plus one FP32 tensor scale                    */
} bsq_format;

typedef enum { BSQ_ROWWISE = 1, BSQ_COLWISE = 2, BSQ_BOTH = 3 } bsq_axis;

typedef enum { BSQ_OUT_F32 = 0, BSQ_OUT_BF16 = 1 } bsq_out;

/* A quantized tensor as stored: `rows` x `cols` logical elements with blocks
 * along `cols`.  codes / scales / tensor_scale are device pointers;
 * tensor_scale (one float) is used by NVFP4 only and may be NULL otherwise. */
typedef struct {
    int32_t fmt;               /* bsq_format */
    int32_t reserved;          /* must be 0  */
    int64_t rows;
    int64_t cols;
    void* codes;
    uint8_t* scales;
    float* tensor_scale;
} bsq_tensor;

/* Bytes of the code buffer of a rows x cols tensor (0 on a bad format). */
size_t bsq_codes_bytes(int32_t fmt, int64_t rows, int64_t cols);

/* Bytes of the tiled scale buffer: ceil(rows/128)*128 * ceil(S/4)*4 with
 * S = cols / block (0 on a bad format or when cols is not a block multiple). */
size_t bsq_scales_bytes(int32_t fmt, int64_t rows, int64_t cols);

/* Quantize a row-major BF16 matrix src[rows, cols] (device).
 *   axis BSQ_ROWWISE: out_row gets a [rows, cols] tensor (cols % block == 0).
 *   axis BSQ_COLWISE: out_col gets the transposed [cols, rows] tensor
 *                     (rows % block == 0).
 *   axis BSQ_BOTH:    both, from one read of src.
 * The caller fills the out tensors' fmt / rows / cols / pointers; they must
 * match the request.  For NVFP4 each written tensor's tensor_scale must be a
 * device float; the call computes the tensor amax first (two passes).
 * Citations: FP8 page "Estrategias de escalonamento" (block scaling); MoE
 * FP4 page section 2, BF16ToFP4Row (row quantize and pack) and the
 * transposed operand of FP4RowToFP8Col. */
bsq_status bsq_quantize(const void* src_bf16, int64_t rows, int64_t cols, int32_t fmt, int32_t axis,
                        bsq_tensor* out_row, bsq_tensor* out_col, void* stream);

/* NVFP4 quantize with delayed scaling: one pass instead of two.  The tensor
 * scale is taken from the amax of previous steps instead of this tensor:
 *   s_t = max(amax_history) / 2688 (FP32; positive finite entries only;
 *         1 when there is none),
 * the blocks are then encoded as by bsq_quantize with that s_t (values
 * beyond its range saturate to the largest block scale and code), each
 * written tensor_scale receives s_t, and last this tensor's amax (largest
 * finite |x|) is pushed to the front of amax_history and its oldest entry
 * dropped.  amax_history: DEVICE float[history_len], 4-byte aligned, owned
 * by the caller, read and updated in stream order (zero-filled before the
 * first step); 1 <= history_len <= 4096.  Arguments and outputs otherwise
 * as bsq_quantize with fmt = BSQ_NVFP4_E2M1; on an argument error nothing
 * is launched and the history is unchanged.  Citation: FP8 page,
 * "Transformer Engine: a fundacao de software" (DelayedScaling recipe:
 * amax_history_len = 16, amax_compute_algo = "max", margin = 0) and
 * "Estrategias de escalonamento e estabilidade" (scale factors from the
 * statistics of previous iterations). */
bsq_status bsq_quantize_nvfp4_delayed(const void* src_bf16, int64_t rows, int64_t cols, int32_t axis,
                                      bsq_tensor* out_row, bsq_tensor* out_col, float* amax_history,
                                      int32_t history_len, void* stream);

/* Exact dequantization dst[rows, cols] = code * scale (* tensor scale),
 * rounded once to FP32 or BF16 (nearest-even).  dst is device memory,
 * 16-byte aligned.  Citation: MoE FP4 page section 2 (the dequantization
 * step that FP4RowToFP8Row replaces). */
bsq_status bsq_dequantize(const bsq_tensor* in, void* dst, int32_t dst_type, void* stream);

/* C[M,N] = A[M,K] * B[N,K]^T with FP32 accumulation on tcgen05 block-scaled
 * tensor-core MMAs; C row-major with leading dimension N, FP32 or BF16.
 * Supported pairs: any of MXFP8 E4M3 / E5M2 with each other; NVFP4 with
 * NVFP4 (the result is multiplied by both tensor scales); MXFP4 with MXFP4
 * (native FP4 MMA with UE8M0 scales, no re-encode).  K = A.cols =
 * B.cols; K % 32 == 0.  M, N >= 1 of any size.  Citation: MoE FP4 page
 * section 2 ("Calculo Intenso": GEMMs stay on native FP8 tensor cores);
 * FP8 page "MXFP8 e NVFP4 do Blackwell" (hardware block scaling). */
bsq_status bsq_gemm(const bsq_tensor* A, const bsq_tensor* B, void* C, int32_t out_type, void* stream);

/* Grouped GEMM over ragged expert batches: for g in [0, num_groups)
 *   C[o_g:o_{g+1}, :] = A[o_g:o_{g+1}, :] * B_g^T
 * where o = group_offsets_dev (DEVICE int64[num_groups+1], o_0 = 0,
 * non-decreasing, o_G = A.rows).  B_groups is a HOST array of num_groups
 * tensors of identical shape [N, K] and format; their code buffers must be
 * consecutive slices of one allocation (B_g.codes = B_0.codes + g * codes
 * bytes); scale buffers may be anywhere.  A's scales use the plain tiled
 * layout of the whole [A.rows, K] matrix.  num_groups <= 256; MXFP8
 * (any mix of E4M3 / E5M2) or MXFP4 x MXFP4; for MXFP4 the experts' scale
 * buffers must also be evenly spaced (BSQ_ERR_UNSUPPORTED otherwise).
 * Citation: MoE FP4 page section 2, ragged tensors whose per-expert token
 * counts vary. */
bsq_status bsq_grouped_gemm(const bsq_tensor* A, const int64_t* group_offsets_dev, int32_t num_groups,
                            const bsq_tensor* B_groups, void* C, int32_t out_type, void* stream);

/* Per-expert padded scale layout of a grouped activation tensor A[rows, cols]
 * with expert row offsets o (o_0 = 0, non-decreasing, o_G = rows): the scales
 * of expert g's rows start at scale row P_g = sum over earlier experts of
 * their row counts rounded up to 128, so no 128x4 scale tile holds two
 * experts (the tile layout itself is the plain one, over P_G rows; bytes
 * between experts are zero).  Codes keep their plain row-major layout.
 * This returns the buffer size that holds it for any offsets:
 * (ceil(rows/128)*128 + 128*num_groups) * ceil(S/4)*4, S = cols / block;
 * 0 on a bad format, shape or group count (1..256). */
size_t bsq_grouped_scales_bytes(int32_t fmt, int64_t rows, int64_t cols, int32_t num_groups);

/* MXFP4 -> MXFP8 re-encode (as bsq_mxfp4_to_mxfp8) whose output scales are
 * written in the per-expert padded layout for the given DEVICE offsets
 * (int64[num_groups+1]); out->scales must hold
 * bsq_grouped_scales_bytes(BSQ_MXFP8_E4M3, rows, cols, num_groups) bytes
 * (zero-filled by the call).  Offsets are clamped to [0, rows] and made
 * non-decreasing on the device.  Citation: MoE FP4 page section 2
 * (FP4RowToFP8Row feeding the per-expert FP8 GEMM). */
bsq_status bsq_mxfp4_to_mxfp8_grouped(const bsq_tensor* in_mxfp4, bsq_tensor* out_e4m3,
                                      const int64_t* group_offsets_dev, int32_t num_groups, void* stream);

/* Grouped GEMM as bsq_grouped_gemm, with A's scales in the per-expert padded
 * layout (as written by bsq_mxfp4_to_mxfp8_grouped).  Output tiles then start
 * at each expert's first row, so only the last tile of an expert is partly
 * idle (with the plain layout a 128-row scale tile shared by two experts is
 * computed for both).  Same formats, limits and errors as
 * bsq_grouped_gemm. */
bsq_status bsq_grouped_gemm_padded(const bsq_tensor* A, const int64_t* group_offsets_dev, int32_t num_groups,
                                   const bsq_tensor* B_groups, void* C, int32_t out_type, void* stream);

/* Direct MXFP4 -> MXFP8 (E4M3) re-encode in the integer domain, same shape
 * and block grid.  Per 32-block with scale exponent e and largest code
 * magnitude exponent e_c: new scale e + e_c - 8 (clamped at -127), every
 * code moved to the E4M3 code of the same value.  The result equals the
 * E4M3 MX quantization of the exactly dequantized MXFP4 block.  Citation:
 * MoE FP4 page section 2, "Algoritmo de Conversao Direta" and kernel
 * FP4RowToFP8Row. */
bsq_status bsq_mxfp4_to_mxfp8(const bsq_tensor* in_mxfp4, bsq_tensor* out_e4m3, void* stream);

/* FP4RowToFP8Col: dequantize a row-wise MXFP4 tensor in[R, C], transpose and
 * re-quantize column-wise to MXFP8 E4M3: out[C, R] holds the K-major codes
 * of the transpose with E8M0 scales over 32-row blocks of each column.  The
 * result equals the column-wise E4M3 MX quantization of the exactly
 * dequantized input (computed in the integer domain, no BF16 or FP32
 * intermediate that could round); a NaN row scale makes its blocks NaN.
 * R % 32 == 0 and C % 32 == 0; out->rows == C, out->cols == R; buffers as
 * for bsq_mxfp4_to_mxfp8 (device, caller-owned, 16-byte aligned).
 * Citation: MoE FP4 page section 2, "Kernels" (FP4RowToFP8Col: fused
 * dequantization, transposition and requantization for the weight
 * gradient). */
bsq_status bsq_mxfp4_to_mxfp8_col(const bsq_tensor* in_mxfp4, bsq_tensor* out_e4m3, void* stream);

/* MXFP4 -> FP8 E4M3 with 1 x 128 blocks, the FP8 block of the pages'
 * Hopper path.  Per row, each group of four 32-blocks (128 elements; the
 * last group of a row may hold fewer) takes the largest of their E8M0 scale
 * bytes S as its scale, and every element becomes the E4M3 code (RNE) of
 * its exact value code * 2^(s - 127) over 2^(S - 127), s its own block's
 * scale.  Exact while s >= S - 5; blocks further below round into E4M3's
 * subnormals and then to zero.  A NaN scale byte (0xFF) in a group makes
 * its scale 0xFF and all its codes NaN (0x7F).
 *   in_mxfp4:   row-wise MXFP4 tensor [rows, cols], cols % 32 == 0 (device)
 *   out_codes:  DEVICE [rows, cols] E4M3 bytes, row-major, 16-byte aligned
 *               (BSQ_ERR_ALIGNMENT otherwise), caller-owned
 *   out_scales: DEVICE [rows, ceil(cols / 128)] E8M0 bytes, row-major,
 *               caller-owned
 * Asynchronous on `stream`.  Citation: MoE FP4 page section 2, "Algoritmo
 * de Conversao Direta" (FP8 blocks of 128, the largest of four FP4 block
 * scales, exponents adjusted locally). */
bsq_status bsq_mxfp4_to_fp8_1x128(const bsq_tensor* in_mxfp4, void* out_codes, void* out_scales, void* stream);

/* ======================================================================
 * Operators around the layer: what a mixture-of-experts training or serving
 * step runs next to the GEMMs.  Conventions as above, and:
 *  - A matrix is given by its first element, its type (bsq_out: FP32 or
 *    BF16), its shape and `ld`, the distance between two rows in ELEMENTS
 *    (ld >= cols; the last axis is contiguous).  Any ld and any address that
 *    is a multiple of the element size is valid; rows that start on 16-byte
 *    boundaries are faster.  The linear cross entropy and the operands of the
 *    linear layers ask for 16-byte rows.
 *  - Inputs and outputs may not overlap unless a call says so.
 *  - Sums, statistics and softmax terms are held in FP32 (the global norm in
 *    FP64); a BF16 result is rounded once, at its store.  No result depends
 *    on the order in which thread blocks run: the same inputs give the same
 *    bits.
 *  - A workspace is device memory, 16-byte aligned, of at least the size the
 *    *_workspace_bytes function gives (0: none needed, NULL is valid).  Its
 *    contents need no preparation and mean nothing after the call; two calls
 *    that may run at the same time need one each.
 * ====================================================================== */

/* -- tokens sorted by expert and back --------------------------------- */

typedef enum { BSQ_ID_I32 = 0, BSQ_ID_I64 = 1 } bsq_id_type;

/* Where the k slots of each token go.  Slot i = t * k + j is token t's j-th
 * expert; a slot whose id lies outside [0, num_experts) is left out (a
 * padding token, or a token over its expert's capacity).  The others are
 * sorted by expert, slots of one expert in slot order:
 *   offsets[e]  = number of slots with an expert before e (DEVICE
 *                 int64[num_experts + 1]; what bsq_grouped_gemm takes)
 *   slot_row[i] = slot i's row in that order, -1 for a slot left out
 *                 (DEVICE int32[tokens * k])
 *   row_slot[r] = the slot in row r, -1 from row offsets[num_experts] on
 *                 (DEVICE int32[tokens * k])
 * All three arrays are the caller's.  1 <= k <= 256, 1 <= num_experts <=
 * 1024, tokens * k < 2^31 - 256; rows of up to 2^30 columns. */
typedef struct {
    int64_t tokens;
    int32_t k;
    int32_t num_experts;
    int64_t* offsets;
    int32_t* slot_row;
    int32_t* row_slot;
} bsq_moe_plan;

/* Workspace of bsq_moe_sort and bsq_moe_dispatch (0 on bad sizes too). */
size_t bsq_moe_workspace_bytes(int64_t tokens, int32_t k, int32_t num_experts);

/* Fill `plan` from the expert ids [tokens, k] (DEVICE, contiguous). */
bsq_status bsq_moe_sort(const void* expert_ids, int32_t id_type, const bsq_moe_plan* plan, void* workspace,
                        size_t workspace_bytes, void* stream);

/* bsq_moe_sort, then rows[r, :] = x[row_slot[r] / k, :] for every row of
 * rows[tokens * k, cols]; rows that hold no slot are written as zeros. */
bsq_status bsq_moe_dispatch(const void* x, int64_t ldx, int32_t type, int64_t cols, const void* expert_ids,
                            int32_t id_type, const bsq_moe_plan* plan, void* rows, int64_t ld_rows, void* workspace,
                            size_t workspace_bytes, void* stream);

/* The gather of bsq_moe_dispatch with a plan that is already filled. */
bsq_status bsq_moe_gather(const void* x, int64_t ldx, int32_t type, int64_t cols, const bsq_moe_plan* plan,
                          void* rows, int64_t ld_rows, void* stream);

/* out[t, :] = sum_j weights[t, j] * rows[slot_row[t, j], :], the sum over the
 * slots that are not left out, in the order of j; 0 for a token that has
 * none.  weights: DEVICE float[tokens, k], contiguous; NULL takes 1, which is
 * the gradient of bsq_moe_dispatch and bsq_moe_gather.  A slot left out
 * contributes nothing, whatever its weight. */
bsq_status bsq_moe_combine(const void* rows, int64_t ld_rows, int32_t type, int64_t cols, const float* weights,
                           const bsq_moe_plan* plan, void* out, int64_t ldo, void* stream);

/* Gradient of bsq_moe_combine for dout[tokens, cols]:
 *   drows[r, :]   = weights[slot] * dout[slot / k, :] with slot = row_slot[r]
 *                   (0 in rows that hold no slot)
 *   dweights[t,j] = dout[t, :] . rows[slot_row[t, j], :] (0 for a slot left
 *                   out)
 * dweights may be NULL (then rows is not read and may be NULL too). */
bsq_status bsq_moe_combine_backward(const void* dout, int64_t ldd, const void* rows, int64_t ld_rows, int32_t type,
                                    int64_t cols, const float* weights, const bsq_moe_plan* plan, void* drows,
                                    int64_t ld_drows, float* dweights, void* stream);

/* -- layer norm --------------------------------------------------------- */

/* Per row of x[rows, cols]: mean = sum x / cols, var = sum (x - mean)^2 /
 * cols, rstd = 1 / sqrt(var + eps), y = (x - mean) * rstd * weight + bias.
 * weight, bias: DEVICE [cols] of `param_type` (bsq_out), either may be NULL
 * (1, 0).  mean, rstd: DEVICE float[rows] for the backward pass, either may
 * be NULL.  y has x's type and may be x itself (same pointer and ld).
 * eps >= 0. */
bsq_status bsq_layer_norm(const void* x, int64_t ldx, int32_t type, int64_t rows, int64_t cols, const void* weight,
                          const void* bias, int32_t param_type, float eps, void* y, int64_t ldy, float* mean,
                          float* rstd, void* stream);

/* Workspace of bsq_layer_norm_backward (0 on bad sizes too). */
size_t bsq_layer_norm_workspace_bytes(int64_t rows, int64_t cols);

/* Gradient of bsq_layer_norm for dy[rows, cols] (dy, x and dx of one type),
 * with xh = (x - mean) * rstd and g = dy * weight:
 *   dx      = rstd * (g - sum(g) / cols - xh * sum(g * xh) / cols)
 *   dweight = sum over the rows of dy * xh   (DEVICE float[cols])
 *   dbias   = sum over the rows of dy        (DEVICE float[cols])
 * dweight and dbias may each be NULL.  dx may be dy itself. */
bsq_status bsq_layer_norm_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ldx, int32_t type,
                                   int64_t rows, int64_t cols, const void* weight, int32_t param_type,
                                   const float* mean, const float* rstd, void* dx, int64_t ld_dx, float* dweight,
                                   float* dbias, void* workspace, size_t workspace_bytes, void* stream);

/* -- softmax cross entropy of a linear head ----------------------------- */

/* Workspace of bsq_linear_cross_entropy (backward = 0) and of
 * bsq_linear_cross_entropy_backward (backward = 1); 0 on bad sizes. */
size_t bsq_linear_cross_entropy_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols, int32_t backward);

/* With logits z[t, v] = h[t, :] . w[v, :], which are never stored:
 *   lse[t]  = log(sum_v exp(z[t, v]))
 *   loss[t] = lse[t] - z[t, targets[t]], 0 where targets[t] lies outside
 *             [0, vocab) (a token that does not count)
 * h: BF16 [tokens, cols], w: BF16 [vocab, cols], both on 16-byte boundaries
 * with cols, ldh and ldw multiples of 8 (BSQ_ERR_ALIGNMENT otherwise);
 * targets: DEVICE int64[tokens]; loss, lse: DEVICE float[tokens].
 * FP32 accumulation on the tensor cores.  tokens, vocab, cols up to
 * 2^31 - 256. */
bsq_status bsq_linear_cross_entropy(const void* h, int64_t ldh, const void* w, int64_t ldw, const int64_t* targets,
                                    int64_t tokens, int64_t vocab, int64_t cols, float* loss, float* lse,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of sum_t dloss[t] * loss[t], with lse from the forward call and
 * g[t, v] = dloss[t] * (exp(z[t, v] - lse[t]) - [v == targets[t]]), 0 for a
 * token that does not count:
 *   dh = g w  (BF16 [tokens, cols]),  dw = g^T h  (BF16 [vocab, cols])
 * Either of dh, dw may be NULL (a frozen head, or frozen states).  The logits
 * are computed again, a piece of the vocabulary at a time.  g enters the two
 * products in BF16, with the largest |dloss| taken out of it and put back in
 * FP32; what the target's entry, by far the largest of its row, loses to BF16
 * is added to dh and dw beside the products.  dh, dw on 16-byte boundaries, ld_dh and ld_dw multiples of 8;
 * dloss: DEVICE float[tokens].  A NaN or infinite dloss[t] of a token that
 * counts makes dh[t] and dw NaN or infinite, as the formula says, and leaves
 * the other rows of dh as they are.  A token that does not count enters dw
 * with g = 0, so its h has to be finite. */
bsq_status bsq_linear_cross_entropy_backward(const void* h, int64_t ldh, const void* w, int64_t ldw,
                                             const int64_t* targets, int64_t tokens, int64_t vocab, int64_t cols,
                                             const float* lse, const float* dloss, void* dh, int64_t ld_dh, void* dw,
                                             int64_t ld_dw, void* workspace, size_t workspace_bytes, void* stream);

/* -- linear layers with their epilogue, and the gated feed-forward -------- */

/* act(z), and act'(z) in the gradients:
 *   IDENTITY z;  RELU max(z, 0);  SILU z / (1 + exp(-z));
 *   GELU z (1 + erf(z / sqrt(2))) / 2;
 *   GELU_TANH z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
typedef enum {
    BSQ_ACT_IDENTITY = 0,
    BSQ_ACT_RELU = 1,
    BSQ_ACT_SILU = 2,
    BSQ_ACT_GELU = 3,
    BSQ_ACT_GELU_TANH = 4
} bsq_activation;

/* Workspaces of the four BF16 calls below (0 on bad sizes too).  `out` is w's
 * rows, for a gated layer its width. */
size_t bsq_linear_workspace_bytes(int64_t tokens, int64_t out, int64_t cols);
size_t bsq_linear_backward_workspace_bytes(int64_t tokens, int64_t out, int64_t cols);
size_t bsq_gated_linear_workspace_bytes(int64_t tokens, int64_t out, int64_t cols);
size_t bsq_gated_linear_backward_workspace_bytes(int64_t tokens, int64_t out, int64_t cols);

/* z = x w^T + bias, y = act(z) + residual, in the product's epilogue.
 * x: BF16 [tokens, cols], w: BF16 [out, cols], both on 16-byte boundaries
 * with cols, ldx and ldw multiples of 8 (BSQ_ERR_ALIGNMENT otherwise; the
 * pitch of a single row says nothing); tokens up to 2^31 - 256, out and cols up to
 * 2^23, no matrix of more than 2^44 elements.  bias: DEVICE [out] of `bias_type` (bsq_out) or NULL.  residual:
 * [tokens, out] of y's type or NULL; y may be residual itself (same pointer and
 * pitch).  y: [tokens, out] of `type` (bsq_out).  z: BF16 [tokens, out] for the
 * backward pass, or NULL.  FP32 sums on the tensor cores, whose additions are
 * truncated: a sum is read out every K = 16384 where y is BF16 (off by some 1e-4
 * of the sum of its magnitudes at most), every K = 512 where it is FP32 (1e-6);
 * z, act and the residual in FP32, each output rounded once. */
bsq_status bsq_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t tokens, int64_t out, int64_t cols,
                      const void* bias, int32_t bias_type, int32_t activation, const void* residual,
                      int64_t ld_residual, void* y, int64_t ldy, int32_t type, void* z, int64_t ldz, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Gradient of bsq_linear for dy: BF16 [tokens, out] (the residual's gradient is
 * dy itself), with z as the forward call left it (BF16; not read, and may be
 * NULL, with BSQ_ACT_IDENTITY):
 *   dz = dy act'(z), rounded to BF16 for the two products (not where there are
 *        up to 4 tokens, or little to sum)
 *   dx = dz w      BF16 [tokens, cols]
 *   dw = dz^T x    BF16 [out, cols]
 *   dbias = the sum of dz's rows, before that rounding   DEVICE float[out]
 * Each of dx, dw, dbias may be NULL, but not all; w is read for dx only and x
 * for dw only (else each may be NULL).  dx, dw on 16-byte boundaries with
 * pitches that are multiples of 8; dy and z of any address and pitch. */
bsq_status bsq_linear_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                               int64_t tokens, int64_t out, int64_t cols, int32_t activation, const void* z, int64_t ldz,
                               void* dx, int64_t ld_dx, void* dw, int64_t ld_dw, float* dbias, void* workspace,
                               size_t workspace_bytes, void* stream);

/* The gated half of a feed-forward block, both projections in one kernel:
 *   gate = x w_gate^T, up = x w_up^T, h = act(gate) * up
 * x, w_gate, w_up: BF16 as x and w of bsq_linear, w_gate and w_up [out, cols].
 * h: [tokens, out] of `type` (bsq_out).  gate, up: BF16 [tokens, out] for the
 * backward pass, both or neither. */
bsq_status bsq_gated_linear(const void* x, int64_t ldx, const void* w_gate, int64_t ld_gate_w, const void* w_up,
                            int64_t ld_up_w, int64_t tokens, int64_t out, int64_t cols, int32_t activation, void* h,
                            int64_t ldh, int32_t type, void* gate, int64_t ld_gate, void* up, int64_t ld_up,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of bsq_gated_linear for dh: BF16 [tokens, out], with gate and up as
 * the forward call left them:
 *   dgate = dh up act'(gate), dup = dh act(gate), rounded as dz there
 *   dx = dgate w_gate + dup w_up, dw_gate = dgate^T x, dw_up = dup^T x (BF16)
 * dx may be NULL (then w_gate and w_up may be), and so may dw_gate and dw_up
 * together (then x may be); alignments as for bsq_linear_backward. */
bsq_status bsq_gated_linear_backward(const void* dh, int64_t ld_dh, const void* x, int64_t ldx, const void* w_gate,
                                     int64_t ld_gate_w, const void* w_up, int64_t ld_up_w, int64_t tokens, int64_t out,
                                     int64_t cols, int32_t activation, const void* gate, int64_t ld_gate, const void* up,
                                     int64_t ld_up, void* dx, int64_t ld_dx, void* dw_gate, int64_t ld_dw_gate,
                                     void* dw_up, int64_t ld_dw_up, void* workspace, size_t workspace_bytes,
                                     void* stream);

/* Workspaces of the two calls below for operands of A's format (0 on bad sizes too). */
size_t bsq_gemm_linear_workspace_bytes(int32_t fmt, int64_t tokens, int64_t out, int64_t cols);
size_t bsq_gemm_gated_workspace_bytes(int32_t fmt, int64_t tokens, int64_t out, int64_t cols);

/* bsq_gemm with the epilogue of bsq_linear: z = A B^T + bias, y = act(z) +
 * residual.  Operands and formats as for bsq_gemm, B.rows up to 2^23; bias, residual, y
 * and z as for bsq_linear (A.rows tokens, B.rows out).  A sum is read out every K =
 * 65536 where y is BF16 (off by 5e-5 of its magnitudes at most), every K = 4096 of
 * MXFP8 and 8192 of MXFP4 and NVFP4 where it is FP32 (1e-6); bsq_gemm takes any K in one. */
bsq_status bsq_gemm_linear(const bsq_tensor* A, const bsq_tensor* B, const void* bias, int32_t bias_type,
                           int32_t activation, const void* residual, int64_t ld_residual, void* y, int64_t ldy,
                           int32_t type, void* z, int64_t ldz, void* workspace, size_t workspace_bytes, void* stream);

/* bsq_gated_linear on block-scaled operands: gate = A B_gate^T, up = A B_up^T,
 * h = act(gate) * up.  B_gate and B_up have one format and one shape; operands
 * and limits as for bsq_gemm_linear. */
bsq_status bsq_gemm_gated(const bsq_tensor* A, const bsq_tensor* B_gate, const bsq_tensor* B_up, int32_t activation,
                          void* h, int64_t ldh, int32_t type, void* gate, int64_t ld_gate, void* up, int64_t ld_up,
                          void* workspace, size_t workspace_bytes, void* stream);

/* -- global norm and clipping ------------------------------------------- */

/* One gradient: n contiguous elements (0 is valid) of `type` (bsq_out) at
 * `grad`, and where its clipped copy goes (`out`: same type and length; may
 * be `grad` itself; ignored by bsq_grad_norm). */
typedef struct {
    const void* grad;
    void* out;
    int64_t n;
    int32_t type;
    int32_t reserved;          /* must be 0 */
} bsq_grad;

/* Workspace of the two calls below for `count` gradients. */
size_t bsq_grad_workspace_bytes(int32_t count);

/* norm[0] = sqrt(sum of the squares of all elements) (DEVICE float): squares
 * and runs of at most 128 of them in FP32, the sum of the runs in FP64 (an
 * element beyond 1.8e19 makes the norm infinite).  `grads` is a HOST array,
 * read before the call returns; count <= 2^20, and at most 2^40 elements. */
bsq_status bsq_grad_norm(const bsq_grad* grads, int32_t count, float* norm, void* workspace, size_t workspace_bytes,
                         void* stream);

/* bsq_grad_norm, then out = grad * min(1, max_norm / (norm + eps)) for every
 * element, the factor and the product in FP32.  An infinite norm gives the
 * factor 0 and a NaN norm makes every output NaN, as the formula says.
 * max_norm >= 0, eps >= 0. */
bsq_status bsq_clip_grad_norm(const bsq_grad* grads, int32_t count, float max_norm, float eps, float* norm,
                              void* workspace, size_t workspace_bytes, void* stream);

/* -- AdamW ---------------------------------------------------------------- */

typedef enum { BSQ_MOMENTS_F32 = 0, BSQ_MOMENTS_8BIT = 1 } bsq_moments;

/* One parameter tensor of n contiguous elements (0 is valid) and its moments.
 *   BSQ_MOMENTS_F32   m, v: float[n]; m_scales, v_scales unused
 *   BSQ_MOMENTS_8BIT  m, v: n E4M3 codes, m_scales, v_scales: ceil(n / 32) E8M0
 *                     bytes, one for 32 elements; v's codes hold its square root
 * A tensor of zeros is the start of either (codes and scales).  `copy`: BF16[n],
 * the new parameters, before their own rounding, rounded to nearest, or NULL.  No two
 * tensors overlap.
 * Elements of any address that is a multiple of their size; 16-byte boundaries
 * (codes: 8) are faster. */
typedef struct {
    void* param;
    const void* grad;
    void* m;
    void* v;
    uint8_t* m_scales;
    uint8_t* v_scales;
    void* copy;
    int64_t n;
    int32_t param_type;        /* bsq_out */
    int32_t grad_type;         /* bsq_out */
    int32_t state;             /* bsq_moments */
    int32_t reserved;          /* must be 0 */
} bsq_adamw_tensor;

typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;              /* of this update, from 1 on */
    const int64_t* step_device;/* DEVICE int64[1] instead of `step`, or NULL */
    const float* lr_device;    /* DEVICE float[1] instead of `lr`, or NULL */
    const float* norm;         /* DEVICE float[1], or NULL: gradients as they are */
    double max_norm, clip_eps; /* with norm */
    uint64_t seed;             /* with stochastic */
    int32_t stochastic;
    int32_t reserved;          /* must be 0 */
} bsq_adamw_options;

/* One AdamW step of every tensor, in FP32, each operation rounded to nearest in
 * this order:
 *   g = grad * min(1, max_norm / (norm + clip_eps))      (norm: of bsq_grad_norm)
 *   m = beta1 m + (1 - beta1) g
 *   v = beta2 v + ((1 - beta2) g) g
 *   param = (1 - lr weight_decay) param
 *           - lr / (1 - beta1^step) * (m / (sqrt(v) / sqrt(1 - beta2^step) + eps))
 * where the factors of lr, the betas and the step are computed in FP64 and
 * rounded (with step_device or lr_device in FP32 on the device, so that a
 * captured call takes the step's number and learning rate of each replay).
 *
 * Moments in 8 bits: with x a block's largest magnitude, its scale is 2^e with e =
 * floor(log2(x * 8/7)) - 8 (the product in FP32; e >= -127), which keeps |x| 2^-e at
 * 448 or below; a code is x 2^-e rounded to E4M3; a v that is not 0 keeps a code that
 * is not; a block with a NaN or an infinity gets scale 0xFF and NaN codes, and its 32
 * parameters are NaN from the next step on: a gradient that may not be finite is to
 * be looked at (its norm is enough) before it comes here.  The update takes the moments
 * before that rounding.
 *
 * stochastic = 0: codes and BF16 parameters are rounded to nearest.  Else they
 * are rounded up in magnitude with the probability of what is cut off, from 16
 * random bits each.  With mix(x) = lowbias32 (xor x >> 16, times 0x7FEB352D, xor
 * x >> 15, times 0x846CA68B, xor x >> 16; 32 bits), element j of tensor i has
 *   key  = mix(mix(mix(i ^ low(seed)) ^ high(seed)) ^ low(step))
 *          + high(j) * 0x9E3779B9
 *   bits = mix(low(j) ^ key)
 * (low and high: 32 bits); its lower half rounds m's code, its upper half v's,
 * and bits 16 .. 31 of bits * 0x9E3779B1 the parameter.  A seed may stay the same
 * from step to step.
 *
 * `tensors` is a HOST array, read before the call returns, and so are the
 * options; count <= 2^20, at most 2^40 elements.  lr, eps, weight_decay,
 * max_norm, clip_eps >= 0 and finite (max_norm may be infinite), 0 <= beta < 1, step >= 1. */
bsq_status bsq_adamw(const bsq_adamw_tensor* tensors, int32_t count, const bsq_adamw_options* options, void* stream);

/* Take and clear the device status word (one atomic exchange on the
 * device, ordered after the work already on `stream`), synchronize
 * `stream`, and return BSQ_ERR_TIMEOUT if any kernel recorded a timed-out
 * wait since the word was last taken, BSQ_ERR_CUDA if the stream reported an
 * error, else BSQ_OK.  The word is shared by every stream of the device: a
 * timeout recorded by a kernel on another stream is reported by whichever
 * call takes the word first. */
bsq_status bsq_sync_status(void* stream);

/* Test hook for the failure path: launches one kernel that waits on a
 * barrier nothing ever arrives on, gives up after `limit_ns` nanoseconds
 * (capped at 1e9) and records BSQ_ERR_TIMEOUT in the status word.  It
 * touches no memory besides the status word. */
bsq_status bsq_debug_timeout_probe(uint64_t limit_ns, void* stream);

/* Test hook for the GEMM kernels' failure path: bsq_gemm with every wait of
 * the kernel limited to `timeout_ns` nanoseconds (1 .. 4e9; bsq_gemm uses
 * 4e9) instead of the default.  With a limit shorter than the GEMM takes,
 * the kernel gives up part-way: it records BSQ_ERR_TIMEOUT in the status
 * word, lets every stage load, scale copy and MMA it issued land, releases
 * tensor memory and exits; C is then partly written.  `kernel` 0 runs the
 * kernel bsq_gemm would choose, 1 the single-CTA kernel (not for MXFP4,
 * BSQ_ERR_UNSUPPORTED).  Argument rules and errors as for bsq_gemm. */
bsq_status bsq_debug_gemm_timeout(const bsq_tensor* A, const bsq_tensor* B, void* C, int32_t out_type,
                                  uint64_t timeout_ns, int32_t kernel, void* stream);

/* Static description of a status code. */
const char* bsq_status_string(int32_t status);

/* Library version string. */
const char* bsq_version(void);

#ifdef __cplusplus
}
#endif
#endif /* BSQ_H */
