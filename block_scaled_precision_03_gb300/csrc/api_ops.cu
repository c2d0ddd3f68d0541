// C ABI of the operators around the layer (expert sort, layer norm, linear
// cross entropy, linear layers and the gated feed-forward, gradient clipping,
// AdamW): argument checks on the host, then dispatch to the kernels.  A rejected call launches nothing.
#include <cmath>
#include <initializer_list>
#include "../../include/bsq.h"
#include "internal.h"

namespace {

constexpr int64_t kMaxRows = 0x7FFFFF00LL;
// of expert rows: their kernels count a row's elements in 32 bits, up to 622592 past its end
constexpr int64_t kMaxMoeCols = 1LL << 30;
constexpr int32_t kMaxGrads = 1 << 20;
constexpr int64_t kMaxElements = 1ll << 40;       // of all gradients of a call
const uint64_t kWaitNs = 4000000000ull;            // 4 s per device-side wait, as the GEMMs

bool valid_type(int32_t t) { return t == BSQ_OUT_F32 || t == BSQ_OUT_BF16; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
uintptr_t elem(int32_t t) { return t == BSQ_OUT_BF16 ? 2 : 4; }
bsq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? BSQ_OK : BSQ_ERR_CUDA; }

// a matrix of `cols` columns: pointer, pitch and element alignment
bsq_status check_matrix(const void* p, int64_t ld, int32_t type, int64_t cols) {
    if (!p || ld < cols) return BSQ_ERR_INVALID_ARG;
    return aligned(p, elem(type)) ? BSQ_OK : BSQ_ERR_ALIGNMENT;
}

bsq_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return BSQ_OK;
    if (!ws || have < need) return BSQ_ERR_INVALID_ARG;
    return aligned(ws, 16) ? BSQ_OK : BSQ_ERR_ALIGNMENT;
}

bool moe_sizes_ok(int64_t tokens, int32_t k, int32_t experts) {
    return tokens >= 1 && k >= 1 && experts >= 1;
}
bool moe_sizes_supported(int64_t tokens, int32_t k, int32_t experts) {
    return k <= bsq::kMoeMaxK && experts <= bsq::kMoeMaxExperts && tokens <= kMaxRows / k;
}

bsq_status check_plan(const bsq_moe_plan* p, bsq::MoePlanArgs& a) {
    if (!p || !moe_sizes_ok(p->tokens, p->k, p->num_experts) || !p->offsets || !p->slot_row || !p->row_slot)
        return BSQ_ERR_INVALID_ARG;
    if (!moe_sizes_supported(p->tokens, p->k, p->num_experts)) return BSQ_ERR_UNSUPPORTED;
    if (!aligned(p->offsets, 8) || !aligned(p->slot_row, 4) || !aligned(p->row_slot, 4)) return BSQ_ERR_ALIGNMENT;
    a.tokens = p->tokens;
    a.k = p->k;
    a.num_experts = p->num_experts;
    a.offsets = p->offsets;
    a.slot_row = p->slot_row;
    a.row_slot = p->row_slot;
    a.num_sms = bsq::device_sms();
    return BSQ_OK;
}

bsq_status check_ids(const void* ids, int32_t id_type) {
    if (!ids || (id_type != BSQ_ID_I32 && id_type != BSQ_ID_I64)) return BSQ_ERR_INVALID_ARG;
    return aligned(ids, id_type == BSQ_ID_I64 ? 8 : 4) ? BSQ_OK : BSQ_ERR_ALIGNMENT;
}

// source and destination rows of a gather or a combine
bsq_status check_rows(const void* src, int64_t ld_src, int32_t type, int64_t cols, void* dst, int64_t ld_dst,
                      bsq::MoeRowsArgs& r) {
    if (!valid_type(type) || cols < 1) return BSQ_ERR_INVALID_ARG;
    bsq_status s = check_matrix(src, ld_src, type, cols);
    if (s != BSQ_OK) return s;
    if ((s = check_matrix(dst, ld_dst, type, cols)) != BSQ_OK) return s;
    if (cols > kMaxMoeCols) return BSQ_ERR_UNSUPPORTED;
    r.src = src;
    r.ld_src = ld_src;
    r.dst = dst;
    r.ld_dst = ld_dst;
    r.cols = cols;
    r.bf16 = type == BSQ_OUT_BF16;
    return BSQ_OK;
}

bool norm_sizes_ok(int64_t rows, int64_t cols) { return rows >= 1 && cols >= 1; }

// h, w and the sizes of the two linear cross entropy calls
bsq_status check_head(const void* h, int64_t ldh, const void* w, int64_t ldw, const int64_t* targets, int64_t tokens,
                      int64_t vocab, int64_t cols, bsq::HeadArgs& a) {
    if (!h || !w || !targets || tokens < 1 || vocab < 1 || cols < 1 || ldh < cols || ldw < cols)
        return BSQ_ERR_INVALID_ARG;
    if (tokens > kMaxRows || vocab > kMaxRows || cols > kMaxRows) return BSQ_ERR_UNSUPPORTED;
    if (!aligned(h, 16) || !aligned(w, 16) || !aligned(targets, 8) || cols % 8 || ldh % 8 || ldw % 8)
        return BSQ_ERR_ALIGNMENT;
    a.h = h;
    a.ldh = ldh;
    a.w = w;
    a.ldw = ldw;
    a.targets = targets;
    a.tokens = tokens;
    a.vocab = vocab;
    a.cols = cols;
    a.num_sms = bsq::device_sms();
    a.status = bsq::device_status();
    a.timeout_ns = kWaitNs;
    return a.status ? BSQ_OK : BSQ_ERR_CUDA;
}

bsq_status clip_common(const bsq_grad* grads, int32_t count, bool scale, float max_norm, float eps, float* norm,
                       void* workspace, size_t workspace_bytes, void* stream) {
    if (!grads || count < 1 || !norm) return BSQ_ERR_INVALID_ARG;
    if (count > kMaxGrads) return BSQ_ERR_UNSUPPORTED;
    if (!aligned(norm, 4)) return BSQ_ERR_ALIGNMENT;
    int64_t total = 0;
    for (int32_t i = 0; i < count; i++) {
        const bsq_grad& g = grads[i];
        if (!valid_type(g.type) || g.reserved != 0 || g.n < 0) return BSQ_ERR_INVALID_ARG;
        if (g.n > kMaxElements || (total += g.n) > kMaxElements) return BSQ_ERR_UNSUPPORTED;
        if (g.n == 0) continue;
        if (!g.grad || (scale && !g.out)) return BSQ_ERR_INVALID_ARG;
        if (!aligned(g.grad, elem(g.type)) || (scale && !aligned(g.out, elem(g.type)))) return BSQ_ERR_ALIGNMENT;
    }
    bsq_status s = check_workspace(workspace, workspace_bytes, bsq::clip_workspace(count, bsq::device_sms()));
    if (s != BSQ_OK) return s;
    bsq::ClipArgs a{};
    a.grads = grads;
    a.count = count;
    a.scale = scale;
    a.max_norm = max_norm;
    a.eps = eps;
    a.norm = norm;
    a.ws = static_cast<double*>(workspace);
    a.num_sms = bsq::device_sms();
    return from_cuda(bsq::run_clip(a, static_cast<cudaStream_t>(stream)));
}

// ---- linear layers
bool valid_act(int32_t a) { return a >= BSQ_ACT_IDENTITY && a <= BSQ_ACT_GELU_TANH; }
bool linear_sizes_ok(int64_t tokens, int64_t out, int64_t cols) { return tokens >= 1 && out >= 1 && cols >= 1; }
bool linear_sizes_supported(int64_t tokens, int64_t out, int64_t cols) {
    return tokens <= kMaxRows && out <= bsq::kLinearMax && cols <= bsq::kLinearMax && tokens * out <= bsq::kLinearMaxElements &&
           tokens * cols <= bsq::kLinearMaxElements && out * cols <= bsq::kLinearMaxElements;
}
// a matrix that TMA reads or writes, or null
bsq_status check_tiled(const void* p, int64_t ld, int64_t rows, int64_t cols) {
    if (!p) return BSQ_OK;
    if (ld < cols) return BSQ_ERR_INVALID_ARG;
    return aligned(p, 16) && (rows == 1 || ld % 8 == 0) ? BSQ_OK : BSQ_ERR_ALIGNMENT;
}
bsq_status check_optional(const void* p, int64_t ld, int32_t type, int64_t cols) {
    return p ? check_matrix(p, ld, type, cols) : BSQ_OK;
}
bsq_status first_bad(std::initializer_list<bsq_status> all) {
    for (bsq_status s : all)
        if (s == BSQ_ERR_INVALID_ARG) return s;
    for (bsq_status s : all)
        if (s != BSQ_OK) return s;
    return BSQ_OK;
}
// a row's pitch where there is one row only: TMA wants a multiple of 16 bytes
int64_t pitch(int64_t ld, int64_t rows, int64_t cols) { return rows == 1 ? cols : ld; }

bsq_status linear_common(bsq::LinearArgs& a, int64_t tokens, int64_t out, int64_t cols, int32_t activation) {
    if (!linear_sizes_ok(tokens, out, cols) || !valid_act(activation)) return BSQ_ERR_INVALID_ARG;
    if (!linear_sizes_supported(tokens, out, cols)) return BSQ_ERR_UNSUPPORTED;
    if (cols % 8) return BSQ_ERR_ALIGNMENT;
    a.tokens = tokens;
    a.out = out;
    a.cols = cols;
    a.act = activation;
    return BSQ_OK;
}
// the last check: of the workspace; and what a launch needs of the device
bsq_status linear_ready(bsq::LinearArgs& a, void* ws, size_t have, size_t need) {
    const bsq_status s = check_workspace(ws, have, need);
    if (s != BSQ_OK) return s;
    a.ws = ws;
    a.num_sms = bsq::device_sms();
    a.status = bsq::device_status();
    a.timeout_ns = kWaitNs;
    return a.status ? BSQ_OK : BSQ_ERR_CUDA;
}
size_t linear_bytes(int64_t tokens, int64_t out, int64_t cols, bool gated, bool backward) {
    if (!linear_sizes_ok(tokens, out, cols) || !linear_sizes_supported(tokens, out, cols)) return 0;
    return backward ? bsq::linear_backward_workspace(tokens, out, cols, gated, bsq::device_sms())
                    : bsq::linear_workspace(tokens, out, cols, gated, bsq::device_sms());
}
bool finite_and_not_negative(double x) { return x >= 0.0 && !std::isinf(x); }

}  // namespace

extern "C" {

size_t bsq_moe_workspace_bytes(int64_t tokens, int32_t k, int32_t num_experts) {
    if (!moe_sizes_ok(tokens, k, num_experts) || !moe_sizes_supported(tokens, k, num_experts)) return 0;
    return bsq::moe_sort_workspace(tokens, k, num_experts);
}

bsq_status bsq_moe_sort(const void* expert_ids, int32_t id_type, const bsq_moe_plan* plan, void* workspace,
                        size_t workspace_bytes, void* stream) {
    bsq::MoePlanArgs p{};
    bsq_status s = check_ids(expert_ids, id_type);
    if (s != BSQ_OK) return s;
    if ((s = check_plan(plan, p)) != BSQ_OK) return s;
    s = check_workspace(workspace, workspace_bytes, bsq::moe_sort_workspace(p.tokens, p.k, p.num_experts));
    if (s != BSQ_OK) return s;
    return from_cuda(bsq::run_moe_sort(p, expert_ids, id_type == BSQ_ID_I64, workspace,
                                       static_cast<cudaStream_t>(stream)));
}

bsq_status bsq_moe_dispatch(const void* x, int64_t ldx, int32_t type, int64_t cols, const void* expert_ids,
                            int32_t id_type, const bsq_moe_plan* plan, void* rows, int64_t ld_rows, void* workspace,
                            size_t workspace_bytes, void* stream) {
    bsq::MoePlanArgs p{};
    bsq::MoeRowsArgs r{};
    bsq_status s = check_rows(x, ldx, type, cols, rows, ld_rows, r);
    if (s != BSQ_OK) return s;
    if ((s = check_ids(expert_ids, id_type)) != BSQ_OK) return s;
    if ((s = check_plan(plan, p)) != BSQ_OK) return s;
    s = check_workspace(workspace, workspace_bytes, bsq::moe_sort_workspace(p.tokens, p.k, p.num_experts));
    if (s != BSQ_OK) return s;
    return from_cuda(bsq::run_moe_dispatch(p, r, expert_ids, id_type == BSQ_ID_I64, workspace,
                                           static_cast<cudaStream_t>(stream)));
}

bsq_status bsq_moe_gather(const void* x, int64_t ldx, int32_t type, int64_t cols, const bsq_moe_plan* plan,
                          void* rows, int64_t ld_rows, void* stream) {
    bsq::MoePlanArgs p{};
    bsq::MoeRowsArgs r{};
    bsq_status s = check_rows(x, ldx, type, cols, rows, ld_rows, r);
    if (s != BSQ_OK) return s;
    if ((s = check_plan(plan, p)) != BSQ_OK) return s;
    return from_cuda(bsq::run_moe_gather(p, r, static_cast<cudaStream_t>(stream)));
}

bsq_status bsq_moe_combine(const void* rows, int64_t ld_rows, int32_t type, int64_t cols, const float* weights,
                           const bsq_moe_plan* plan, void* out, int64_t ldo, void* stream) {
    bsq::MoePlanArgs p{};
    bsq::MoeRowsArgs r{};
    bsq_status s = check_rows(rows, ld_rows, type, cols, out, ldo, r);
    if (s != BSQ_OK) return s;
    if ((s = check_plan(plan, p)) != BSQ_OK) return s;
    if (!aligned(weights, 4)) return BSQ_ERR_ALIGNMENT;
    r.weights = weights;
    return from_cuda(bsq::run_moe_combine(p, r, static_cast<cudaStream_t>(stream)));
}

bsq_status bsq_moe_combine_backward(const void* dout, int64_t ldd, const void* rows, int64_t ld_rows, int32_t type,
                                    int64_t cols, const float* weights, const bsq_moe_plan* plan, void* drows,
                                    int64_t ld_drows, float* dweights, void* stream) {
    bsq::MoePlanArgs p{};
    bsq::MoeRowsArgs r{};
    bsq_status s = check_rows(dout, ldd, type, cols, drows, ld_drows, r);
    if (s != BSQ_OK) return s;
    if (dweights && (s = check_matrix(rows, ld_rows, type, cols)) != BSQ_OK) return s;
    if ((s = check_plan(plan, p)) != BSQ_OK) return s;
    if (!weights) return BSQ_ERR_INVALID_ARG;
    if (!aligned(weights, 4) || !aligned(dweights, 4)) return BSQ_ERR_ALIGNMENT;
    r.weights = weights;
    r.rows = dweights ? rows : nullptr;
    r.ld_rows = ld_rows;
    r.dweights = dweights;
    return from_cuda(bsq::run_moe_combine_backward(p, r, static_cast<cudaStream_t>(stream)));
}

bsq_status bsq_layer_norm(const void* x, int64_t ldx, int32_t type, int64_t rows, int64_t cols, const void* weight,
                          const void* bias, int32_t param_type, float eps, void* y, int64_t ldy, float* mean,
                          float* rstd, void* stream) {
    if (!valid_type(type) || !valid_type(param_type) || !norm_sizes_ok(rows, cols)) return BSQ_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || std::isinf(eps)) return BSQ_ERR_INVALID_ARG;
    bsq_status s = check_matrix(x, ldx, type, cols);
    if (s != BSQ_OK) return s;
    if ((s = check_matrix(y, ldy, type, cols)) != BSQ_OK) return s;
    if (!aligned(weight, elem(param_type)) || !aligned(bias, elem(param_type)) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return BSQ_ERR_ALIGNMENT;
    if (rows > kMaxRows || cols > kMaxRows) return BSQ_ERR_UNSUPPORTED;
    bsq::NormArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.bf16 = type == BSQ_OUT_BF16;
    a.rows = rows;
    a.cols = cols;
    a.weight = weight;
    a.bias = bias;
    a.param_bf16 = param_type == BSQ_OUT_BF16;
    a.eps = eps;
    a.y = y;
    a.ldy = ldy;
    a.mean = mean;
    a.rstd = rstd;
    a.num_sms = bsq::device_sms();
    return from_cuda(bsq::run_layer_norm(a, static_cast<cudaStream_t>(stream)));
}

size_t bsq_layer_norm_workspace_bytes(int64_t rows, int64_t cols) {
    if (!norm_sizes_ok(rows, cols) || rows > kMaxRows || cols > kMaxRows) return 0;
    return bsq::norm_workspace(rows, cols, bsq::device_sms());
}

bsq_status bsq_layer_norm_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ldx, int32_t type,
                                   int64_t rows, int64_t cols, const void* weight, int32_t param_type,
                                   const float* mean, const float* rstd, void* dx, int64_t ld_dx, float* dweight,
                                   float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_type(type) || !valid_type(param_type) || !norm_sizes_ok(rows, cols) || !mean || !rstd)
        return BSQ_ERR_INVALID_ARG;
    bsq_status s = check_matrix(dy, ld_dy, type, cols);
    if (s != BSQ_OK) return s;
    if ((s = check_matrix(x, ldx, type, cols)) != BSQ_OK) return s;
    if ((s = check_matrix(dx, ld_dx, type, cols)) != BSQ_OK) return s;
    if (!aligned(weight, elem(param_type)) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) ||
        !aligned(dbias, 4))
        return BSQ_ERR_ALIGNMENT;
    if (rows > kMaxRows || cols > kMaxRows) return BSQ_ERR_UNSUPPORTED;
    const size_t need = dweight || dbias ? bsq::norm_workspace(rows, cols, bsq::device_sms()) : 0;
    if ((s = check_workspace(workspace, workspace_bytes, need)) != BSQ_OK) return s;
    bsq::NormArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.bf16 = type == BSQ_OUT_BF16;
    a.rows = rows;
    a.cols = cols;
    a.weight = weight;
    a.param_bf16 = param_type == BSQ_OUT_BF16;
    a.y = dx;
    a.ldy = ld_dx;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.ld_dy = ld_dy;
    a.dweight = dweight;
    a.dbias = dbias;
    a.ws = static_cast<float*>(workspace);
    a.num_sms = bsq::device_sms();
    return from_cuda(bsq::run_layer_norm_backward(a, static_cast<cudaStream_t>(stream)));
}

size_t bsq_linear_cross_entropy_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols, int32_t backward) {
    if (tokens < 1 || vocab < 1 || cols < 1 || tokens > kMaxRows || vocab > kMaxRows || cols > kMaxRows) return 0;
    return bsq::head_workspace(tokens, vocab, cols, backward != 0, bsq::device_sms());
}

bsq_status bsq_linear_cross_entropy(const void* h, int64_t ldh, const void* w, int64_t ldw, const int64_t* targets,
                                    int64_t tokens, int64_t vocab, int64_t cols, float* loss, float* lse,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    bsq::HeadArgs a{};
    if (!loss || !lse) return BSQ_ERR_INVALID_ARG;
    bsq_status s = check_head(h, ldh, w, ldw, targets, tokens, vocab, cols, a);
    if (s != BSQ_OK) return s;
    if (!aligned(loss, 4) || !aligned(lse, 4)) return BSQ_ERR_ALIGNMENT;
    s = check_workspace(workspace, workspace_bytes, bsq::head_workspace(tokens, vocab, cols, false, a.num_sms));
    if (s != BSQ_OK) return s;
    a.loss = loss;
    a.lse = lse;
    a.ws = workspace;
    return from_cuda(bsq::run_head(a, static_cast<cudaStream_t>(stream)));
}

bsq_status bsq_linear_cross_entropy_backward(const void* h, int64_t ldh, const void* w, int64_t ldw,
                                             const int64_t* targets, int64_t tokens, int64_t vocab, int64_t cols,
                                             const float* lse, const float* dloss, void* dh, int64_t ld_dh, void* dw,
                                             int64_t ld_dw, void* workspace, size_t workspace_bytes, void* stream) {
    bsq::HeadArgs a{};
    if (!lse || !dloss || (!dh && !dw)) return BSQ_ERR_INVALID_ARG;
    if ((dh && ld_dh < cols) || (dw && ld_dw < cols)) return BSQ_ERR_INVALID_ARG;
    bsq_status s = check_head(h, ldh, w, ldw, targets, tokens, vocab, cols, a);
    if (s != BSQ_OK) return s;
    if (!aligned(lse, 4) || !aligned(dloss, 4) || !aligned(dh, 16) || !aligned(dw, 16)) return BSQ_ERR_ALIGNMENT;
    if ((dh && ld_dh % 8) || (dw && ld_dw % 8)) return BSQ_ERR_ALIGNMENT;
    s = check_workspace(workspace, workspace_bytes, bsq::head_workspace(tokens, vocab, cols, true, a.num_sms));
    if (s != BSQ_OK) return s;
    a.lse = const_cast<float*>(lse);
    a.dloss = dloss;
    a.dh = dh;
    a.ld_dh = ld_dh;
    a.dw = dw;
    a.ld_dw = ld_dw;
    a.ws = workspace;
    return from_cuda(bsq::run_head_backward(a, static_cast<cudaStream_t>(stream)));
}

size_t bsq_grad_workspace_bytes(int32_t count) {
    return count < 1 || count > kMaxGrads ? 0 : bsq::clip_workspace(count, bsq::device_sms());
}

bsq_status bsq_grad_norm(const bsq_grad* grads, int32_t count, float* norm, void* workspace, size_t workspace_bytes,
                         void* stream) {
    return clip_common(grads, count, false, 0.0f, 0.0f, norm, workspace, workspace_bytes, stream);
}

bsq_status bsq_clip_grad_norm(const bsq_grad* grads, int32_t count, float max_norm, float eps, float* norm,
                              void* workspace, size_t workspace_bytes, void* stream) {
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f)) return BSQ_ERR_INVALID_ARG;
    return clip_common(grads, count, true, max_norm, eps, norm, workspace, workspace_bytes, stream);
}

size_t bsq_linear_workspace_bytes(int64_t tokens, int64_t out, int64_t cols) {
    return linear_bytes(tokens, out, cols, false, false);
}
size_t bsq_linear_backward_workspace_bytes(int64_t tokens, int64_t out, int64_t cols) {
    return linear_bytes(tokens, out, cols, false, true);
}
size_t bsq_gated_linear_workspace_bytes(int64_t tokens, int64_t out, int64_t cols) {
    return linear_bytes(tokens, out, cols, true, false);
}
size_t bsq_gated_linear_backward_workspace_bytes(int64_t tokens, int64_t out, int64_t cols) {
    return linear_bytes(tokens, out, cols, true, true);
}

bsq_status bsq_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t tokens, int64_t out, int64_t cols,
                      const void* bias, int32_t bias_type, int32_t activation, const void* residual,
                      int64_t ld_residual, void* y, int64_t ldy, int32_t type, void* z, int64_t ldz, void* workspace,
                      size_t workspace_bytes, void* stream) {
    bsq::LinearArgs a{};
    if (!x || !w || !valid_type(type) || (bias && !valid_type(bias_type))) return BSQ_ERR_INVALID_ARG;
    bsq_status s = linear_common(a, tokens, out, cols, activation);
    if (s != BSQ_OK) return s;
    s = first_bad({check_tiled(x, ldx, tokens, cols), check_tiled(w, ldw, out, cols), check_matrix(y, ldy, type, out),
                   check_optional(residual, ld_residual, type, out), check_optional(z, ldz, BSQ_OUT_BF16, out),
                   bias && !aligned(bias, elem(bias_type)) ? BSQ_ERR_ALIGNMENT : BSQ_OK});
    if (s != BSQ_OK) return s;
    s = linear_ready(a, workspace, workspace_bytes, linear_bytes(tokens, out, cols, false, false));
    if (s != BSQ_OK) return s;
    a.x = x;
    a.ldx = pitch(ldx, tokens, cols);
    a.w = w;
    a.ldw = pitch(ldw, out, cols);
    a.bias = bias;
    a.bias_bf16 = bias_type == BSQ_OUT_BF16;
    a.residual = residual;
    a.ld_res = ld_residual;
    a.y = y;
    a.ldy = ldy;
    a.y_bf16 = type == BSQ_OUT_BF16;
    a.z = z;
    a.ldz = ldz;
    return from_cuda(bsq::run_linear(a, false, static_cast<cudaStream_t>(stream)));
}

bsq_status bsq_linear_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                               int64_t tokens, int64_t out, int64_t cols, int32_t activation, const void* z, int64_t ldz,
                               void* dx, int64_t ld_dx, void* dw, int64_t ld_dw, float* dbias, void* workspace,
                               size_t workspace_bytes, void* stream) {
    bsq::LinearArgs a{};
    if ((!dx && !dw && !dbias) || (dx && !w) || (dw && !x)) return BSQ_ERR_INVALID_ARG;
    bsq_status s = linear_common(a, tokens, out, cols, activation);
    if (s != BSQ_OK) return s;
    const bool reads_z = activation != BSQ_ACT_IDENTITY;
    if (reads_z && !z) return BSQ_ERR_INVALID_ARG;
    s = first_bad({check_matrix(dy, ld_dy, BSQ_OUT_BF16, out), check_optional(reads_z ? z : nullptr, ldz, BSQ_OUT_BF16, out),
                   check_tiled(dw ? x : nullptr, ldx, tokens, cols), check_tiled(dx ? w : nullptr, ldw, out, cols),
                   check_tiled(dx, ld_dx, tokens, cols), check_tiled(dw, ld_dw, out, cols),
                   aligned(dbias, 4) ? BSQ_OK : BSQ_ERR_ALIGNMENT});
    if (s != BSQ_OK) return s;
    s = linear_ready(a, workspace, workspace_bytes, linear_bytes(tokens, out, cols, false, true));
    if (s != BSQ_OK) return s;
    a.x = x;
    a.ldx = pitch(ldx, tokens, cols);
    a.w = w;
    a.ldw = pitch(ldw, out, cols);
    a.dy = dy;
    a.ld_dy = ld_dy;
    a.z = reads_z ? const_cast<void*>(z) : nullptr;
    a.ldz = ldz;
    a.dx = dx;
    a.ld_dx = pitch(ld_dx, tokens, cols);
    a.dw = dw;
    a.ld_dw = pitch(ld_dw, out, cols);
    a.dbias = dbias;
    return from_cuda(bsq::run_linear_backward(a, false, static_cast<cudaStream_t>(stream)));
}

bsq_status bsq_gated_linear(const void* x, int64_t ldx, const void* w_gate, int64_t ld_gate_w, const void* w_up,
                            int64_t ld_up_w, int64_t tokens, int64_t out, int64_t cols, int32_t activation, void* h,
                            int64_t ldh, int32_t type, void* gate, int64_t ld_gate, void* up, int64_t ld_up,
                            void* workspace, size_t workspace_bytes, void* stream) {
    bsq::LinearArgs a{};
    if (!x || !w_gate || !w_up || !valid_type(type) || (gate == nullptr) != (up == nullptr)) return BSQ_ERR_INVALID_ARG;
    bsq_status s = linear_common(a, tokens, out, cols, activation);
    if (s != BSQ_OK) return s;
    s = first_bad({check_tiled(x, ldx, tokens, cols), check_tiled(w_gate, ld_gate_w, out, cols),
                   check_tiled(w_up, ld_up_w, out, cols), check_matrix(h, ldh, type, out),
                   check_optional(gate, ld_gate, BSQ_OUT_BF16, out), check_optional(up, ld_up, BSQ_OUT_BF16, out)});
    if (s != BSQ_OK) return s;
    s = linear_ready(a, workspace, workspace_bytes, linear_bytes(tokens, out, cols, true, false));
    if (s != BSQ_OK) return s;
    a.x = x;
    a.ldx = pitch(ldx, tokens, cols);
    a.w = w_gate;
    a.ldw = pitch(ld_gate_w, out, cols);
    a.w2 = w_up;
    a.ldw2 = pitch(ld_up_w, out, cols);
    a.y = h;
    a.ldy = ldh;
    a.y_bf16 = type == BSQ_OUT_BF16;
    a.z = gate;
    a.ldz = ld_gate;
    a.u = up;
    a.ldu = ld_up;
    return from_cuda(bsq::run_linear(a, true, static_cast<cudaStream_t>(stream)));
}

bsq_status bsq_gated_linear_backward(const void* dh, int64_t ld_dh, const void* x, int64_t ldx, const void* w_gate,
                                     int64_t ld_gate_w, const void* w_up, int64_t ld_up_w, int64_t tokens, int64_t out,
                                     int64_t cols, int32_t activation, const void* gate, int64_t ld_gate, const void* up,
                                     int64_t ld_up, void* dx, int64_t ld_dx, void* dw_gate, int64_t ld_dw_gate,
                                     void* dw_up, int64_t ld_dw_up, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    bsq::LinearArgs a{};
    if ((!dx && !dw_gate) || (dw_gate == nullptr) != (dw_up == nullptr) || (dx && (!w_gate || !w_up)) || (dw_gate && !x) ||
        !gate || !up)
        return BSQ_ERR_INVALID_ARG;
    bsq_status s = linear_common(a, tokens, out, cols, activation);
    if (s != BSQ_OK) return s;
    s = first_bad({check_matrix(dh, ld_dh, BSQ_OUT_BF16, out), check_matrix(gate, ld_gate, BSQ_OUT_BF16, out),
                   check_matrix(up, ld_up, BSQ_OUT_BF16, out), check_tiled(dw_gate ? x : nullptr, ldx, tokens, cols),
                   check_tiled(dx ? w_gate : nullptr, ld_gate_w, out, cols), check_tiled(dx ? w_up : nullptr, ld_up_w, out, cols),
                   check_tiled(dx, ld_dx, tokens, cols), check_tiled(dw_gate, ld_dw_gate, out, cols),
                   check_tiled(dw_up, ld_dw_up, out, cols)});
    if (s != BSQ_OK) return s;
    s = linear_ready(a, workspace, workspace_bytes, linear_bytes(tokens, out, cols, true, true));
    if (s != BSQ_OK) return s;
    a.x = x;
    a.ldx = pitch(ldx, tokens, cols);
    a.w = w_gate;
    a.ldw = pitch(ld_gate_w, out, cols);
    a.w2 = w_up;
    a.ldw2 = pitch(ld_up_w, out, cols);
    a.dy = dh;
    a.ld_dy = ld_dh;
    a.z = const_cast<void*>(gate);
    a.ldz = ld_gate;
    a.u = const_cast<void*>(up);
    a.ldu = ld_up;
    a.dx = dx;
    a.ld_dx = pitch(ld_dx, tokens, cols);
    a.dw = dw_gate;
    a.ld_dw = pitch(ld_dw_gate, out, cols);
    a.dw2 = dw_up;
    a.ld_dw2 = pitch(ld_dw_up, out, cols);
    return from_cuda(bsq::run_linear_backward(a, true, static_cast<cudaStream_t>(stream)));
}

bsq_status bsq_adamw(const bsq_adamw_tensor* tensors, int32_t count, const bsq_adamw_options* options, void* stream) {
    if (!tensors || count < 1 || !options || options->reserved != 0) return BSQ_ERR_INVALID_ARG;
    const bsq_adamw_options& o = *options;
    if (!finite_and_not_negative(o.lr) || !finite_and_not_negative(o.eps) || !finite_and_not_negative(o.weight_decay) ||
        !(o.beta1 >= 0.0 && o.beta1 < 1.0) || !(o.beta2 >= 0.0 && o.beta2 < 1.0) || (!o.step_device && o.step < 1) ||
        (o.norm && (!(o.max_norm >= 0.0) || !finite_and_not_negative(o.clip_eps))))
        return BSQ_ERR_INVALID_ARG;
    if (count > kMaxGrads) return BSQ_ERR_UNSUPPORTED;
    if (!aligned(o.step_device, 8) || !aligned(o.lr_device, 4) || !aligned(o.norm, 4)) return BSQ_ERR_ALIGNMENT;
    int64_t total = 0;
    for (int32_t i = 0; i < count; i++) {
        const bsq_adamw_tensor& t = tensors[i];
        if (!valid_type(t.param_type) || !valid_type(t.grad_type) || t.reserved != 0 || t.n < 0 ||
            (t.state != BSQ_MOMENTS_F32 && t.state != BSQ_MOMENTS_8BIT))
            return BSQ_ERR_INVALID_ARG;
        if (t.n > kMaxElements || (total += t.n) > kMaxElements) return BSQ_ERR_UNSUPPORTED;
        if (t.n == 0) continue;
        const bool codes = t.state == BSQ_MOMENTS_8BIT;
        if (!t.param || !t.grad || !t.m || !t.v || (codes && (!t.m_scales || !t.v_scales))) return BSQ_ERR_INVALID_ARG;
        if (!aligned(t.param, elem(t.param_type)) || !aligned(t.grad, elem(t.grad_type)) || !aligned(t.copy, 2) ||
            (!codes && (!aligned(t.m, 4) || !aligned(t.v, 4))))
            return BSQ_ERR_ALIGNMENT;
    }
    bsq::AdamwArgs a{tensors, count, options, bsq::device_sms()};
    return from_cuda(bsq::run_adamw(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
