// Python binding of the operators around the layer, as a native module: the
// argument checks and the marshalling of a call in a few hundred nanoseconds
// (the same in Python took 4 to 7 us, more than the smallest kernels).  The
// entry points of libbsq.so come in by address (bind), so that the module and
// ctypes use one loaded library.  Every function raises BsqError(status, what).
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAException.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <optional>
#include <utility>
#include "../../include/bsq.h"

namespace {

#define BSQ_FUNCTIONS(F)                                                                              \
    F(bsq_moe_workspace_bytes) F(bsq_moe_sort) F(bsq_moe_dispatch) F(bsq_moe_gather) F(bsq_moe_combine) \
    F(bsq_moe_combine_backward) F(bsq_layer_norm) F(bsq_layer_norm_workspace_bytes)                    \
    F(bsq_layer_norm_backward) F(bsq_linear_cross_entropy_workspace_bytes) F(bsq_linear_cross_entropy) \
    F(bsq_linear_cross_entropy_backward) F(bsq_grad_norm) F(bsq_clip_grad_norm)                        \
    F(bsq_codes_bytes) F(bsq_scales_bytes) F(bsq_linear_workspace_bytes) F(bsq_linear)                 \
    F(bsq_linear_backward_workspace_bytes) F(bsq_linear_backward) F(bsq_gated_linear_workspace_bytes)  \
    F(bsq_gated_linear) F(bsq_gated_linear_backward_workspace_bytes) F(bsq_gated_linear_backward)      \
    F(bsq_gemm_linear_workspace_bytes) F(bsq_gemm_linear) F(bsq_gemm_gated_workspace_bytes)            \
    F(bsq_gemm_gated) F(bsq_adamw)

struct Api {
#define F(name) decltype(&::name) name;
    BSQ_FUNCTIONS(F)
#undef F
} api;

PyObject* error_class;             // BsqError
PyObject *s_num_experts, *s_offsets, *s_slot_row, *s_row_slot, *s_cuda_stream;
PyObject *s_fmt, *s_rows, *s_cols, *s_codes, *s_scales, *s_tensor_scale;

// A refused call: the Python error is set.
struct Refused {};

[[noreturn]] void refuse(int status, const char* format, ...) {
    char text[256];
    va_list args;
    va_start(args, format);
    vsnprintf(text, sizeof text, format, args);
    va_end(args);
    if (PyObject* e = PyObject_CallFunction(error_class, "is", status, text)) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    throw Refused{};
}

void check(bsq_status status, const char* what) {
    if (status != BSQ_OK) refuse(status, "%s", what);
}

bool none(PyObject* o) { return !o || o == Py_None; }

// The device of a call's tensors: that of the first one it looks at (-1 before).  Set by guarded();
// under Python's lock, like every call here.
int call_device = -1;

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!o || !THPVariable_Check(o)) refuse(BSQ_ERR_INVALID_ARG, "%s must be a CUDA tensor", name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(BSQ_ERR_INVALID_ARG, "%s must be a CUDA tensor", name);
    if (call_device < 0) call_device = t.get_device();
    if (t.get_device() != call_device)
        refuse(BSQ_ERR_INVALID_ARG, "%s is on cuda:%d, other arguments of the call on cuda:%d", name, (int)t.get_device(),
               call_device);
    return t;
}

int32_t type_of(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kBFloat16) return BSQ_OUT_BF16;
    if (t.scalar_type() == at::kFloat) return BSQ_OUT_F32;
    refuse(BSQ_ERR_UNSUPPORTED, "%s: %s (BFloat16 and Float are supported)", name, c10::toString(t.scalar_type()));
}

// A matrix with unit stride along its columns
struct Matrix {
    const at::Tensor* t = nullptr;
    void* p = nullptr;
    int64_t ld = 0, rows = 0, cols = 0;
};
Matrix matrix(PyObject* o, const char* name, int64_t rows = -1, int64_t cols = -1, const Matrix* like = nullptr) {
    Matrix m;
    m.t = &tensor(o, name);
    if (m.t->dim() != 2) refuse(BSQ_ERR_INVALID_ARG, "%s must be a CUDA matrix", name);
    m.rows = m.t->size(0);
    m.cols = m.t->size(1);
    if ((rows >= 0 && m.rows != rows) || (cols >= 0 && m.cols != cols))
        refuse(BSQ_ERR_INVALID_ARG, "%s is %lld x %lld, not %lld x %lld", name, (long long)m.rows, (long long)m.cols,
               (long long)(rows >= 0 ? rows : m.rows), (long long)(cols >= 0 ? cols : m.cols));
    if (like && m.t->scalar_type() != like->t->scalar_type())
        refuse(BSQ_ERR_INVALID_ARG, "%s is %s, not %s", name, c10::toString(m.t->scalar_type()),
               c10::toString(like->t->scalar_type()));
    if (m.cols > 1 && m.t->stride(1) != 1)
        refuse(BSQ_ERR_INVALID_ARG, "%s must have unit stride along its columns", name);
    m.ld = m.rows > 1 ? m.t->stride(0) : std::max(m.t->stride(0), m.cols);
    m.p = m.t->data_ptr();
    return m;
}

// Pointer of a contiguous tensor of n elements; null for None
void* vector(PyObject* o, const char* name, int64_t n, at::ScalarType type) {
    if (none(o)) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || t.numel() != n || !t.is_contiguous())
        refuse(BSQ_ERR_INVALID_ARG, "%s must be a contiguous %s tensor of %lld elements", name, c10::toString(type),
               (long long)n);
    return t.data_ptr();
}

// The stream to launch on (given, or the current one of the tensor's device)
// and scratch that belongs to it: the allocator hands the scratch out again
// only to work behind this call on that stream.  That device is the current
// one as long as this lives: the library launches on the current device.
struct Launch {
    c10::cuda::CUDAGuard device;
    cudaStream_t stream = nullptr;
    at::Tensor scratch;
    const at::Tensor& like;
    bool given;
    Launch(PyObject* s, const at::Tensor& t) : device(t.get_device()), like(t), given(!none(s)) {
        if (!given) {
            stream = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
            return;
        }
        PyObject* raw = PyObject_GetAttr(s, s_cuda_stream);
        if (!raw) throw Refused{};
        stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(raw));
        Py_DECREF(raw);
        if (PyErr_Occurred()) throw Refused{};
    }
    void* workspace(size_t bytes) {
        if (bytes == 0) return nullptr;
        std::optional<c10::cuda::CUDAStreamGuard> guard;
        if (given) guard.emplace(c10::cuda::getStreamFromExternal(stream, like.get_device()));
        scratch = at::empty({(int64_t)bytes}, like.options().dtype(at::kByte));
        return scratch.data_ptr();
    }
};

// Arguments by position or name; `required` of them must be there.
template <int N>
struct Args {
    PyObject* v[N] = {};
    Args(const char* function, const char* const (&names)[N], int required, PyObject* const* args, Py_ssize_t n,
         PyObject* kwnames) {
        if (n > N) fail(function, "too many arguments", "");
        for (Py_ssize_t i = 0; i < n; i++) v[i] = args[i];
        const Py_ssize_t k = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
        for (Py_ssize_t i = 0; i < k; i++) {
            PyObject* name = PyTuple_GET_ITEM(kwnames, i);
            int at = 0;
            while (at < N && PyUnicode_CompareWithASCIIString(name, names[at]) != 0) at++;
            if (at == N) fail(function, "unexpected argument ", PyUnicode_AsUTF8(name));
            if (v[at]) fail(function, "two values for ", names[at]);
            v[at] = args[n + i];
        }
        for (int i = 0; i < required; i++)
            if (!v[i]) fail(function, "missing argument ", names[i]);
    }
    [[noreturn]] static void fail(const char* function, const char* what, const char* name) {
        PyErr_Format(PyExc_TypeError, "%s(): %s%s", function, what, name ? name : "");
        throw Refused{};
    }
    PyObject* operator[](int i) const { return v[i]; }
};

double number(PyObject* o) {
    const double d = PyFloat_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) throw Refused{};
    return d;
}

PyObject* returned(PyObject* o) {
    if (!o) o = Py_None;
    Py_INCREF(o);
    return o;
}
PyObject* returned(PyObject* a, PyObject* b) { return PyTuple_Pack(2, a ? a : Py_None, b ? b : Py_None); }
PyObject* returned(PyObject* a, PyObject* b, PyObject* c) {
    return PyTuple_Pack(3, a ? a : Py_None, b ? b : Py_None, c ? c : Py_None);
}

// Runs a call; C++ exceptions end here.  (Reading a plan's attributes may run Python, and so another call.)
template <typename F>
PyObject* guarded(F f) {
    struct Device {
        int before = std::exchange(call_device, -1);
        ~Device() { call_device = before; }
    } own;
    try {
        return f();
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

struct Ref {
    PyObject* o;
    Ref(PyObject* from, PyObject* name) : o(PyObject_GetAttr(from, name)) {
        if (!o) throw Refused{};
    }
    ~Ref() { Py_DECREF(o); }
};

bsq_moe_plan plan_of(PyObject* plan) {
    const Ref experts(plan, s_num_experts), offsets(plan, s_offsets), slots(plan, s_slot_row), rows(plan, s_row_slot);
    const at::Tensor& s = tensor(slots.o, "slot_row");
    if (s.dim() != 2) refuse(BSQ_ERR_INVALID_ARG, "slot_row must be [tokens, k]");
    const long e = PyLong_AsLong(experts.o);
    if (e == -1 && PyErr_Occurred()) throw Refused{};
    if (e < 0 || e > INT32_MAX || s.size(1) > INT32_MAX) refuse(BSQ_ERR_INVALID_ARG, "num_experts or k out of range");
    bsq_moe_plan p;
    p.tokens = s.size(0);
    p.k = (int32_t)s.size(1);
    p.num_experts = (int32_t)e;
    p.offsets = static_cast<int64_t*>(vector(offsets.o, "offsets", e + 1, at::kLong));
    p.slot_row = static_cast<int32_t*>(vector(slots.o, "slot_row", p.tokens * p.k, at::kInt));
    p.row_slot = static_cast<int32_t*>(vector(rows.o, "row_slot", p.tokens * p.k, at::kInt));
    return p;
}

const void* ids_of(PyObject* o, const bsq_moe_plan& p, int32_t& id_type) {
    const at::Tensor& t = tensor(o, "expert_ids");
    const bool wide = t.scalar_type() == at::kLong;
    if ((!wide && t.scalar_type() != at::kInt) || t.dim() != 2 || t.size(0) != p.tokens || t.size(1) != p.k ||
        !t.is_contiguous())
        refuse(BSQ_ERR_INVALID_ARG, "expert_ids must be a contiguous int32 or int64 matrix of %lld x %d",
               (long long)p.tokens, (int)p.k);
    id_type = wide ? BSQ_ID_I64 : BSQ_ID_I32;
    return t.data_ptr();
}

#define ENTRY(name) PyObject* name(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames)

ENTRY(moe_sort_into) {
    return guarded([&] {
        static const char* const names[] = {"expert_ids", "plan", "stream"};
        const Args a("moe_sort_into", names, 2, args, n, kwnames);
        const bsq_moe_plan p = plan_of(a[1]);
        int32_t id_type;
        const void* ids = ids_of(a[0], p, id_type);
        Launch l(a[2], tensor(a[0], "expert_ids"));
        const size_t bytes = api.bsq_moe_workspace_bytes(p.tokens, p.k, p.num_experts);
        check(api.bsq_moe_sort(ids, id_type, &p, l.workspace(bytes), bytes, l.stream), "bsq_moe_sort");
        return returned(a[1]);
    });
}

ENTRY(moe_dispatch_into) {
    return guarded([&] {
        static const char* const names[] = {"x", "expert_ids", "plan", "rows", "stream"};
        const Args a("moe_dispatch_into", names, 4, args, n, kwnames);
        const bsq_moe_plan p = plan_of(a[2]);
        int32_t id_type;
        const void* ids = ids_of(a[1], p, id_type);
        const Matrix x = matrix(a[0], "x", p.tokens), r = matrix(a[3], "rows", p.tokens * p.k, x.cols, &x);
        Launch l(a[4], *x.t);
        const size_t bytes = api.bsq_moe_workspace_bytes(p.tokens, p.k, p.num_experts);
        check(api.bsq_moe_dispatch(x.p, x.ld, type_of(*x.t, "x"), x.cols, ids, id_type, &p, r.p, r.ld, l.workspace(bytes),
                                   bytes, l.stream),
              "bsq_moe_dispatch");
        return returned(a[3]);
    });
}

ENTRY(moe_gather_into) {
    return guarded([&] {
        static const char* const names[] = {"x", "plan", "rows", "stream"};
        const Args a("moe_gather_into", names, 3, args, n, kwnames);
        const bsq_moe_plan p = plan_of(a[1]);
        const Matrix x = matrix(a[0], "x", p.tokens), r = matrix(a[2], "rows", p.tokens * p.k, x.cols, &x);
        Launch l(a[3], *x.t);
        check(api.bsq_moe_gather(x.p, x.ld, type_of(*x.t, "x"), x.cols, &p, r.p, r.ld, l.stream), "bsq_moe_gather");
        return returned(a[2]);
    });
}

ENTRY(moe_combine_into) {
    return guarded([&] {
        static const char* const names[] = {"rows", "weights", "plan", "out", "stream"};
        const Args a("moe_combine_into", names, 4, args, n, kwnames);
        const bsq_moe_plan p = plan_of(a[2]);
        const Matrix r = matrix(a[0], "rows", p.tokens * p.k), o = matrix(a[3], "out", p.tokens, r.cols, &r);
        const float* w = static_cast<float*>(vector(a[1], "weights", p.tokens * p.k, at::kFloat));
        Launch l(a[4], *r.t);
        check(api.bsq_moe_combine(r.p, r.ld, type_of(*r.t, "rows"), r.cols, w, &p, o.p, o.ld, l.stream), "bsq_moe_combine");
        return returned(a[3]);
    });
}

ENTRY(moe_combine_backward_into) {
    return guarded([&] {
        static const char* const names[] = {"dout", "rows", "weights", "plan", "drows", "dweights", "stream"};
        const Args a("moe_combine_backward_into", names, 6, args, n, kwnames);
        const bsq_moe_plan p = plan_of(a[3]);
        const int64_t slots = p.tokens * p.k;
        const Matrix d = matrix(a[0], "dout", p.tokens);
        Matrix r;
        if (!none(a[1])) r = matrix(a[1], "rows", slots, d.cols, &d);
        const Matrix g = matrix(a[4], "drows", slots, d.cols, &d);
        const float* w = static_cast<float*>(vector(a[2], "weights", slots, at::kFloat));
        float* dw = static_cast<float*>(vector(a[5], "dweights", slots, at::kFloat));
        Launch l(a[6], *d.t);
        check(api.bsq_moe_combine_backward(d.p, d.ld, r.p, r.ld, type_of(*d.t, "dout"), d.cols, w, &p, g.p, g.ld, dw, l.stream),
              "bsq_moe_combine_backward");
        return returned(a[4], a[5]);
    });
}

// weight and bias, both of one type, each may be None
void params_of(PyObject* weight, PyObject* bias, int64_t cols, const void*& w, const void*& b, int32_t& type) {
    w = b = nullptr;
    type = BSQ_OUT_F32;
    PyObject* first = none(weight) ? bias : weight;
    if (none(first)) return;
    const at::Tensor& t = tensor(first, "weight or bias");
    type = type_of(t, "weight or bias");
    w = vector(weight, "weight", cols, t.scalar_type());
    b = vector(bias, "bias", cols, t.scalar_type());
}

ENTRY(layer_norm_into) {
    return guarded([&] {
        static const char* const names[] = {"x", "weight", "bias", "eps", "y", "mean", "rstd", "stream"};
        const Args a("layer_norm_into", names, 5, args, n, kwnames);
        const Matrix x = matrix(a[0], "x"), y = matrix(a[4], "y", x.rows, x.cols, &x);
        const void *w, *b;
        int32_t type;
        params_of(a[1], a[2], x.cols, w, b, type);
        float* mean = static_cast<float*>(vector(a[5], "mean", x.rows, at::kFloat));
        float* rstd = static_cast<float*>(vector(a[6], "rstd", x.rows, at::kFloat));
        Launch l(a[7], *x.t);
        check(api.bsq_layer_norm(x.p, x.ld, type_of(*x.t, "x"), x.rows, x.cols, w, b, type, (float)number(a[3]), y.p, y.ld,
                                 mean, rstd, l.stream),
              "bsq_layer_norm");
        return returned(a[4], a[5], a[6]);
    });
}

ENTRY(layer_norm_backward_into) {
    return guarded([&] {
        static const char* const names[] = {"dy", "x", "weight", "mean", "rstd", "dx", "dweight", "dbias", "stream"};
        const Args a("layer_norm_backward_into", names, 6, args, n, kwnames);
        const Matrix x = matrix(a[1], "x"), dy = matrix(a[0], "dy", x.rows, x.cols, &x),
                     dx = matrix(a[5], "dx", x.rows, x.cols, &x);
        const void *w, *b;
        int32_t type;
        params_of(a[2], nullptr, x.cols, w, b, type);
        const float* mean = static_cast<float*>(vector(a[3], "mean", x.rows, at::kFloat));
        const float* rstd = static_cast<float*>(vector(a[4], "rstd", x.rows, at::kFloat));
        float* dw = static_cast<float*>(vector(a[6], "dweight", x.cols, at::kFloat));
        float* db = static_cast<float*>(vector(a[7], "dbias", x.cols, at::kFloat));
        Launch l(a[8], *x.t);
        const size_t bytes = dw || db ? api.bsq_layer_norm_workspace_bytes(x.rows, x.cols) : 0;
        check(api.bsq_layer_norm_backward(dy.p, dy.ld, x.p, x.ld, type_of(*x.t, "x"), x.rows, x.cols, w, type, mean, rstd,
                                          dx.p, dx.ld, dw, db, l.workspace(bytes), bytes, l.stream),
              "bsq_layer_norm_backward");
        return returned(a[5], a[6], a[7]);
    });
}

// A matrix of the head, whose pitches have to be whole vectors; that of a single row says nothing.
Matrix head_matrix(PyObject* o, const char* name, int64_t rows = -1, int64_t cols = -1, const Matrix* like = nullptr) {
    Matrix m = matrix(o, name, rows, cols, like);
    if (m.rows == 1) m.ld = m.cols;
    return m;
}

struct Head {
    Matrix h, w;
    const int64_t* targets;
    Head(PyObject* ph, PyObject* pw, PyObject* pt) {
        h = head_matrix(ph, "h");
        for (const char* name : {"h", "w"}) {
            const at::Tensor& t = tensor(name[0] == 'h' ? ph : pw, name);
            if (t.scalar_type() != at::kBFloat16)
                refuse(BSQ_ERR_UNSUPPORTED, "%s: %s (BFloat16 is supported)", name, c10::toString(t.scalar_type()));
        }
        w = head_matrix(pw, "w", -1, h.cols);
        targets = static_cast<int64_t*>(vector(pt, "targets", h.rows, at::kLong));
    }
};

ENTRY(linear_cross_entropy_into) {
    return guarded([&] {
        static const char* const names[] = {"h", "w", "targets", "loss", "lse", "stream"};
        const Args a("linear_cross_entropy_into", names, 5, args, n, kwnames);
        const Head d(a[0], a[1], a[2]);
        float* loss = static_cast<float*>(vector(a[3], "loss", d.h.rows, at::kFloat));
        float* lse = static_cast<float*>(vector(a[4], "lse", d.h.rows, at::kFloat));
        Launch l(a[5], *d.h.t);
        const size_t bytes = api.bsq_linear_cross_entropy_workspace_bytes(d.h.rows, d.w.rows, d.h.cols, 0);
        check(api.bsq_linear_cross_entropy(d.h.p, d.h.ld, d.w.p, d.w.ld, d.targets, d.h.rows, d.w.rows, d.h.cols, loss, lse,
                                           l.workspace(bytes), bytes, l.stream),
              "bsq_linear_cross_entropy");
        return returned(a[3], a[4]);
    });
}

ENTRY(linear_cross_entropy_backward_into) {
    return guarded([&] {
        static const char* const names[] = {"h", "w", "targets", "lse", "dloss", "dh", "dw", "stream"};
        const Args a("linear_cross_entropy_backward_into", names, 7, args, n, kwnames);
        const Head d(a[0], a[1], a[2]);
        Matrix dh, dw;
        if (!none(a[5])) dh = head_matrix(a[5], "dh", d.h.rows, d.h.cols, &d.h);
        if (!none(a[6])) dw = head_matrix(a[6], "dw", d.w.rows, d.w.cols, &d.w);
        const float* lse = static_cast<float*>(vector(a[3], "lse", d.h.rows, at::kFloat));
        const float* dloss = static_cast<float*>(vector(a[4], "dloss", d.h.rows, at::kFloat));
        Launch l(a[7], *d.h.t);
        const size_t bytes = api.bsq_linear_cross_entropy_workspace_bytes(d.h.rows, d.w.rows, d.h.cols, 1);
        check(api.bsq_linear_cross_entropy_backward(d.h.p, d.h.ld, d.w.p, d.w.ld, d.targets, d.h.rows, d.w.rows, d.h.cols,
                                                    lse, dloss, dh.p, dh.ld, dw.p, dw.ld, l.workspace(bytes), bytes,
                                                    l.stream),
              "bsq_linear_cross_entropy_backward");
        return returned(a[5], a[6]);
    });
}

// ---- linear layers
int32_t activation(PyObject* o, int32_t standard) {
    if (none(o)) return standard;
    static const char* const names[] = {"identity", "relu", "silu", "gelu", "gelu_tanh"};
    if (PyUnicode_Check(o)) {
        for (int32_t i = 0; i < 5; i++)
            if (PyUnicode_CompareWithASCIIString(o, names[i]) == 0) return i;
        refuse(BSQ_ERR_INVALID_ARG, "activation must be identity, relu, silu, gelu or gelu_tanh");
    }
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    if (v < 0 || v > 4) refuse(BSQ_ERR_INVALID_ARG, "activation %ld", v);
    return (int32_t)v;
}
// BF16 matrices, or none
Matrix bf16_matrix(PyObject* o, const char* name, int64_t rows = -1, int64_t cols = -1) {
    const Matrix m = head_matrix(o, name, rows, cols);
    if (m.t->scalar_type() != at::kBFloat16)
        refuse(BSQ_ERR_UNSUPPORTED, "%s: %s (BFloat16 is supported)", name, c10::toString(m.t->scalar_type()));
    return m;
}
Matrix maybe_bf16(PyObject* o, const char* name, int64_t rows, int64_t cols) {
    return none(o) ? Matrix{} : bf16_matrix(o, name, rows, cols);
}
// bias, of either type, or none
const void* bias_of(PyObject* o, int64_t n, int32_t& type) {
    type = BSQ_OUT_F32;
    if (none(o)) return nullptr;
    const at::Tensor& t = tensor(o, "bias");
    type = type_of(t, "bias");
    return vector(o, "bias", n, t.scalar_type());
}

ENTRY(linear_into) {
    return guarded([&] {
        static const char* const names[] = {"x", "w", "y", "bias", "residual", "activation", "z", "stream"};
        const Args a("linear_into", names, 3, args, n, kwnames);
        const Matrix x = bf16_matrix(a[0], "x"), w = bf16_matrix(a[1], "w", -1, x.cols), y = matrix(a[2], "y", x.rows, w.rows);
        Matrix r;
        if (!none(a[4])) r = matrix(a[4], "residual", x.rows, w.rows, &y);
        const Matrix z = maybe_bf16(a[6], "z", x.rows, w.rows);
        int32_t type;
        const void* bias = bias_of(a[3], w.rows, type);
        const int32_t act = activation(a[5], BSQ_ACT_IDENTITY), out = type_of(*y.t, "y");
        Launch l(a[7], *x.t);
        const size_t bytes = api.bsq_linear_workspace_bytes(x.rows, w.rows, x.cols);
        check(api.bsq_linear(x.p, x.ld, w.p, w.ld, x.rows, w.rows, x.cols, bias, type, act, r.p, r.ld, y.p, y.ld,
                             out, z.p, z.ld, l.workspace(bytes), bytes, l.stream),
              "bsq_linear");
        return returned(a[2], a[6]);
    });
}

ENTRY(linear_backward_into) {
    return guarded([&] {
        static const char* const names[] = {"dy", "x", "w", "dx", "dw", "dbias", "z", "activation", "stream"};
        const Args a("linear_backward_into", names, 3, args, n, kwnames);
        const Matrix dy = bf16_matrix(a[0], "dy");
        const Matrix x = maybe_bf16(a[1], "x", dy.rows, -1), w = maybe_bf16(a[2], "w", dy.cols, x.t ? x.cols : -1);
        const int64_t cols = x.t ? x.cols : w.t ? w.cols : 0;
        if (!x.t && !w.t) refuse(BSQ_ERR_INVALID_ARG, "x or w must be given");
        const Matrix dx = maybe_bf16(a[3], "dx", dy.rows, cols), dw = maybe_bf16(a[4], "dw", dy.cols, cols);
        float* dbias = static_cast<float*>(vector(a[5], "dbias", dy.cols, at::kFloat));
        const Matrix z = maybe_bf16(a[6], "z", dy.rows, dy.cols);
        const int32_t act = activation(a[7], BSQ_ACT_IDENTITY);
        Launch l(a[8], *dy.t);
        const size_t bytes = api.bsq_linear_backward_workspace_bytes(dy.rows, dy.cols, cols);
        check(api.bsq_linear_backward(dy.p, dy.ld, x.p, x.ld, w.p, w.ld, dy.rows, dy.cols, cols, act, z.p, z.ld, dx.p, dx.ld,
                                      dw.p, dw.ld, dbias, l.workspace(bytes), bytes, l.stream),
              "bsq_linear_backward");
        return returned(a[3], a[4], a[5]);
    });
}

ENTRY(gated_linear_into) {
    return guarded([&] {
        static const char* const names[] = {"x", "w_gate", "w_up", "h", "activation", "gate", "up", "stream"};
        const Args a("gated_linear_into", names, 4, args, n, kwnames);
        const Matrix x = bf16_matrix(a[0], "x"), g = bf16_matrix(a[1], "w_gate", -1, x.cols),
                     u = bf16_matrix(a[2], "w_up", g.rows, x.cols), h = matrix(a[3], "h", x.rows, g.rows);
        const Matrix gate = maybe_bf16(a[5], "gate", x.rows, g.rows), up = maybe_bf16(a[6], "up", x.rows, g.rows);
        const int32_t act = activation(a[4], BSQ_ACT_SILU), out = type_of(*h.t, "h");
        Launch l(a[7], *x.t);
        const size_t bytes = api.bsq_gated_linear_workspace_bytes(x.rows, g.rows, x.cols);
        check(api.bsq_gated_linear(x.p, x.ld, g.p, g.ld, u.p, u.ld, x.rows, g.rows, x.cols, act, h.p, h.ld,
                                   out, gate.p, gate.ld, up.p, up.ld, l.workspace(bytes), bytes, l.stream),
              "bsq_gated_linear");
        return returned(a[3], a[5], a[6]);
    });
}

ENTRY(gated_linear_backward_into) {
    return guarded([&] {
        static const char* const names[] = {"dh", "x",  "w_gate",  "w_up",  "gate",       "up",
                                            "dx", "dw_gate", "dw_up", "activation", "stream"};
        const Args a("gated_linear_backward_into", names, 6, args, n, kwnames);
        const Matrix dh = bf16_matrix(a[0], "dh");
        const int64_t T = dh.rows, F = dh.cols;
        const Matrix x = maybe_bf16(a[1], "x", T, -1), g = maybe_bf16(a[2], "w_gate", F, x.t ? x.cols : -1);
        const int64_t cols = x.t ? x.cols : g.t ? g.cols : 0;
        if (!x.t && !g.t) refuse(BSQ_ERR_INVALID_ARG, "x or w_gate must be given");
        const Matrix u = maybe_bf16(a[3], "w_up", F, cols), gate = bf16_matrix(a[4], "gate", T, F), up = bf16_matrix(a[5], "up", T, F);
        const Matrix dx = maybe_bf16(a[6], "dx", T, cols), dg = maybe_bf16(a[7], "dw_gate", F, cols),
                     du = maybe_bf16(a[8], "dw_up", F, cols);
        const int32_t act = activation(a[9], BSQ_ACT_SILU);
        Launch l(a[10], *dh.t);
        const size_t bytes = api.bsq_gated_linear_backward_workspace_bytes(T, F, cols);
        check(api.bsq_gated_linear_backward(dh.p, dh.ld, x.p, x.ld, g.p, g.ld, u.p, u.ld, T, F, cols, act, gate.p, gate.ld, up.p,
                                            up.ld, dx.p, dx.ld, dg.p, dg.ld, du.p, du.ld, l.workspace(bytes), bytes, l.stream),
              "bsq_gated_linear_backward");
        return returned(a[6], a[7], a[8]);
    });
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}

// A quantized tensor (QTensor): its buffers have to be there in full, and live as long as this, whatever made them
struct Quantized {
    const Ref pc, ps, pt;
    bsq_tensor c{};
    const at::Tensor* codes;
    Quantized(PyObject* o, const char* name) : pc(o, s_codes), ps(o, s_scales), pt(o, s_tensor_scale) {
        const Ref fmt(o, s_fmt), rows(o, s_rows), cols(o, s_cols);
        c.fmt = (int32_t)integer(fmt.o);
        c.rows = integer(rows.o);
        c.cols = integer(cols.o);
        codes = &tensor(pc.o, name);
        const at::Tensor& scales = tensor(ps.o, name);
        for (const at::Tensor* t : {codes, &scales})
            if (t->element_size() != 1 || !t->is_contiguous())
                refuse(BSQ_ERR_INVALID_ARG, "%s: codes and scales must be contiguous bytes", name);
        if (c.rows < 1 || c.cols < 1 || c.rows > INT32_MAX || c.cols > INT32_MAX ||
            (size_t)codes->numel() < api.bsq_codes_bytes(c.fmt, c.rows, c.cols) ||
            (size_t)scales.numel() < api.bsq_scales_bytes(c.fmt, c.rows, c.cols))
            refuse(BSQ_ERR_INVALID_ARG, "%s: codes or scales are shorter than its shape", name);
        c.codes = codes->data_ptr();
        c.scales = static_cast<uint8_t*>(scales.data_ptr());
        c.tensor_scale = static_cast<float*>(vector(pt.o, name, 1, at::kFloat));
    }
};

ENTRY(gemm_linear_into) {
    return guarded([&] {
        static const char* const names[] = {"A", "B", "y", "bias", "residual", "activation", "z", "stream"};
        const Args a("gemm_linear_into", names, 3, args, n, kwnames);
        const Quantized qa(a[0], "A"), qb(a[1], "B");
        const int64_t T = qa.c.rows, N = qb.c.rows;
        const Matrix y = matrix(a[2], "y", T, N);
        Matrix r;
        if (!none(a[4])) r = matrix(a[4], "residual", T, N, &y);
        const Matrix z = maybe_bf16(a[6], "z", T, N);
        int32_t type;
        const void* bias = bias_of(a[3], N, type);
        const int32_t act = activation(a[5], BSQ_ACT_IDENTITY), out = type_of(*y.t, "y");
        Launch l(a[7], *qa.codes);
        const size_t bytes = api.bsq_gemm_linear_workspace_bytes(qa.c.fmt, T, N, qa.c.cols);
        check(api.bsq_gemm_linear(&qa.c, &qb.c, bias, type, act, r.p, r.ld, y.p, y.ld, out, z.p, z.ld,
                                  l.workspace(bytes), bytes, l.stream),
              "bsq_gemm_linear");
        return returned(a[2], a[6]);
    });
}

ENTRY(gemm_gated_into) {
    return guarded([&] {
        static const char* const names[] = {"A", "B_gate", "B_up", "h", "activation", "gate", "up", "stream"};
        const Args a("gemm_gated_into", names, 4, args, n, kwnames);
        const Quantized qa(a[0], "A"), qg(a[1], "B_gate"), qu(a[2], "B_up");
        const int64_t T = qa.c.rows, F = qg.c.rows;
        const Matrix h = matrix(a[3], "h", T, F), gate = maybe_bf16(a[5], "gate", T, F), up = maybe_bf16(a[6], "up", T, F);
        const int32_t act = activation(a[4], BSQ_ACT_SILU), out = type_of(*h.t, "h");
        Launch l(a[7], *qa.codes);
        const size_t bytes = api.bsq_gemm_gated_workspace_bytes(qa.c.fmt, T, F, qa.c.cols);
        check(api.bsq_gemm_gated(&qa.c, &qg.c, &qu.c, act, h.p, h.ld, out, gate.p, gate.ld, up.p, up.ld,
                                 l.workspace(bytes), bytes, l.stream),
              "bsq_gemm_gated");
        return returned(a[3], a[5], a[6]);
    });
}

// The address of a bsq_adamw_tensor array and its length (an AdamWList keeps both); `like`: one of its tensors.
// lr and step may be numbers, or tensors on the device; norm and seed may be None.
ENTRY(adamw_into) {
    return guarded([&] {
        static const char* const names[] = {"array", "count", "like", "lr", "step", "beta1", "beta2", "eps", "weight_decay",
                                            "norm", "max_norm", "clip_eps", "seed", "stream"};
        const Args a("adamw_into", names, 13, args, n, kwnames);
        const auto* tensors = static_cast<const bsq_adamw_tensor*>(PyLong_AsVoidPtr(a[0]));
        const int32_t count = (int32_t)integer(a[1]);
        if (PyErr_Occurred()) throw Refused{};
        const at::Tensor& like = tensor(a[2], "like");
        bsq_adamw_options o{};
        if (THPVariable_Check(a[3])) o.lr_device = static_cast<float*>(vector(a[3], "lr", 1, at::kFloat));
        else o.lr = number(a[3]);
        if (THPVariable_Check(a[4])) o.step_device = static_cast<int64_t*>(vector(a[4], "step", 1, at::kLong));
        else o.step = integer(a[4]);
        o.beta1 = number(a[5]);
        o.beta2 = number(a[6]);
        o.eps = number(a[7]);
        o.weight_decay = number(a[8]);
        o.norm = static_cast<float*>(vector(a[9], "norm", 1, at::kFloat));
        if (o.norm) {
            o.max_norm = number(a[10]);
            o.clip_eps = number(a[11]);
        }
        o.stochastic = !none(a[12]);
        if (o.stochastic) {
            o.seed = PyLong_AsUnsignedLongLongMask(a[12]);
            if (PyErr_Occurred()) throw Refused{};
        }
        Launch l(a[13], like);
        check(api.bsq_adamw(tensors, count, &o, l.stream), "bsq_adamw");
        Py_RETURN_NONE;
    });
}

// grads: the address of a bsq_grad array and its length (a GradList keeps both
// and a workspace); max_norm None: the norm only.
ENTRY(grads_into) {
    return guarded([&] {
        static const char* const names[] = {"array", "count", "max_norm", "eps", "norm", "workspace", "stream"};
        const Args a("grads_into", names, 7, args, n, kwnames);
        const auto* grads = static_cast<const bsq_grad*>(PyLong_AsVoidPtr(a[0]));
        const int32_t count = (int32_t)PyLong_AsLong(a[1]);
        if (PyErr_Occurred()) throw Refused{};
        float* norm = static_cast<float*>(vector(a[4], "norm", 1, at::kFloat));
        const at::Tensor& ws = tensor(a[5], "workspace");
        Launch l(a[6], ws);
        if (none(a[2]))
            check(api.bsq_grad_norm(grads, count, norm, ws.data_ptr(), (size_t)ws.numel(), l.stream), "bsq_grad_norm");
        else
            check(api.bsq_clip_grad_norm(grads, count, (float)number(a[2]), (float)number(a[3]), norm, ws.data_ptr(),
                                         (size_t)ws.numel(), l.stream),
                  "bsq_clip_grad_norm");
        return returned(a[4]);
    });
}

// stream_state(tensor, stream) -> (handle, whether it captures a graph) of the stream a call with it launches on
ENTRY(stream_state) {
    return guarded([&] {
        static const char* const names[] = {"tensor", "stream"};
        const Args a("stream_state", names, 1, args, n, kwnames);
        const Launch l(a[1], tensor(a[0], "tensor"));
        cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
        C10_CUDA_CHECK(cudaStreamIsCapturing(l.stream, &status));
        return Py_BuildValue("NN", PyLong_FromVoidPtr(l.stream),
                             PyBool_FromLong(status != cudaStreamCaptureStatusNone));
    });
}

extern PyMethodDef methods[];

// bind(addresses by name, BsqError, documentation by name)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 3 || !PyDict_Check(args[0]) || !PyDict_Check(args[2])) {
        PyErr_SetString(PyExc_TypeError, "bind(addresses, BsqError, documentation)");
        return nullptr;
    }
#define F(name)                                                                    \
    {                                                                              \
        PyObject* o = PyDict_GetItemString(args[0], #name);                        \
        if (!o) {                                                                  \
            PyErr_SetString(PyExc_KeyError, #name);                                \
            return nullptr;                                                        \
        }                                                                          \
        void* p = PyLong_AsVoidPtr(o);                                             \
        if (PyErr_Occurred()) return nullptr;                                      \
        std::memcpy(&api.name, &p, sizeof p);                                      \
    }
    BSQ_FUNCTIONS(F)
#undef F
    for (PyMethodDef* m = methods; m->ml_name; m++)
        if (PyObject* doc = PyDict_GetItemString(args[2], m->ml_name)) {
            const char* text = PyUnicode_AsUTF8(doc);
            if (!text) return nullptr;
            m->ml_doc = strdup(text);              // kept, like the table
        }
    Py_INCREF(args[1]);
    error_class = args[1];
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL | METH_KEYWORDS, nullptr}
PyMethodDef methods[] = {
    METHOD(moe_sort_into), METHOD(moe_dispatch_into), METHOD(moe_gather_into), METHOD(moe_combine_into),
    METHOD(moe_combine_backward_into), METHOD(layer_norm_into), METHOD(layer_norm_backward_into),
    METHOD(linear_cross_entropy_into), METHOD(linear_cross_entropy_backward_into), METHOD(grads_into),
    METHOD(stream_state), METHOD(linear_into), METHOD(linear_backward_into), METHOD(gated_linear_into),
    METHOD(gated_linear_backward_into), METHOD(gemm_linear_into), METHOD(gemm_gated_into), METHOD(adamw_into),
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef definition = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    s_num_experts = PyUnicode_InternFromString("num_experts");
    s_offsets = PyUnicode_InternFromString("offsets");
    s_slot_row = PyUnicode_InternFromString("slot_row");
    s_row_slot = PyUnicode_InternFromString("row_slot");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    s_fmt = PyUnicode_InternFromString("fmt");
    s_rows = PyUnicode_InternFromString("rows");
    s_cols = PyUnicode_InternFromString("cols");
    s_codes = PyUnicode_InternFromString("codes");
    s_scales = PyUnicode_InternFromString("scales");
    s_tensor_scale = PyUnicode_InternFromString("tensor_scale");
    return PyModule_Create(&definition);
}
