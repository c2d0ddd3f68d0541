"""Binding of the operators around the layer: tokens sorted by expert and
back, layer norm, the softmax cross entropy of a linear head, linear layers with
their epilogue and the gated feed-forward, the global gradient norm with
clipping, and AdamW.  Like the rest of the binding it marshals
arguments only, here mostly in a native module, since the smallest calls take
no longer on the GPU than their marshalling in Python; include/bsq.h has the
formulas, limits and errors.

    moe_dispatch(x, expert_ids, num_experts)      -> (rows, MoePlan)
    moe_sort(expert_ids, num_experts)             -> MoePlan
    moe_gather(x, plan)                           -> rows
    moe_combine(rows, weights, plan)              -> out
    moe_combine_backward(dout, rows, weights, plan) -> (drows, dweights)
    moe_dispatch_backward(drows, plan)            -> dx
    layer_norm(x, weight, bias, eps)              -> (y, mean, rstd)
    layer_norm_backward(dy, x, weight, mean, rstd)  -> (dx, dweight, dbias)
    linear_cross_entropy(h, w, targets)           -> (loss, lse)
    linear_cross_entropy_backward(h, w, targets, lse, dloss) -> (dh, dw)
    linear(x, w, bias, residual, activation)      -> y
    linear_backward(dy, x, w, z, activation)      -> (dx, dw, dbias)
    gated_linear(x, w_gate, w_up, activation)     -> h
    gated_linear_backward(dh, x, w_gate, w_up, gate, up, activation) -> (dx, dw_gate, dw_up)
    gemm_linear(A, B, ...), gemm_gated(A, B_gate, B_up, ...): the two forward calls on QTensors
    grad_norm(grads), clip_grad_norm(grads, max_norm) -> norm
    adamw_step(AdamWList(params, grads), lr, step, ...)

Matrices are CUDA tensors [rows, cols] with unit stride along cols and any
row stride; each *_into form writes given tensors and allocates nothing but a
workspace on the launching stream.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import inspect
import os
import sys
from dataclasses import dataclass

from . import OUT_BF16, OUT_F32, BsqError, lib

ID_I32, ID_I64 = 0, 1
BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")


class BsqMoePlanC(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("k", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("offsets", ctypes.c_void_p), ("slot_row", ctypes.c_void_p), ("row_slot", ctypes.c_void_p)]


class BsqGradC(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class BsqAdamwTensorC(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("param_type", ctypes.c_int32), ("grad_type", ctypes.c_int32),
                ("state", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class BsqAdamwOptionsC(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64), ("step_device", ctypes.c_void_p),
                ("lr_device", ctypes.c_void_p), ("norm", ctypes.c_void_p), ("max_norm", ctypes.c_double),
                ("clip_eps", ctypes.c_double), ("seed", ctypes.c_uint64), ("stochastic", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def _signatures():
    i32, i64, vp, sz, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    PP, PG = ctypes.POINTER(BsqMoePlanC), ctypes.POINTER(BsqGradC)
    PA, PO = ctypes.POINTER(BsqAdamwTensorC), ctypes.POINTER(BsqAdamwOptionsC)
    return {
        "bsq_moe_workspace_bytes": (sz, [i64, i32, i32]),
        "bsq_moe_sort": (i32, [vp, i32, PP, vp, sz, vp]),
        "bsq_moe_dispatch": (i32, [vp, i64, i32, i64, vp, i32, PP, vp, i64, vp, sz, vp]),
        "bsq_moe_gather": (i32, [vp, i64, i32, i64, PP, vp, i64, vp]),
        "bsq_moe_combine": (i32, [vp, i64, i32, i64, vp, PP, vp, i64, vp]),
        "bsq_moe_combine_backward": (i32, [vp, i64, vp, i64, i32, i64, vp, PP, vp, i64, vp, vp]),
        "bsq_layer_norm": (i32, [vp, i64, i32, i64, i64, vp, vp, i32, f32, vp, i64, vp, vp, vp]),
        "bsq_layer_norm_workspace_bytes": (sz, [i64, i64]),
        "bsq_layer_norm_backward": (i32, [vp, i64, vp, i64, i32, i64, i64, vp, i32, vp, vp, vp, i64, vp, vp, vp, sz,
                                          vp]),
        "bsq_linear_cross_entropy_workspace_bytes": (sz, [i64, i64, i64, i32]),
        "bsq_linear_cross_entropy": (i32, [vp, i64, vp, i64, vp, i64, i64, i64, vp, vp, vp, sz, vp]),
        "bsq_linear_cross_entropy_backward": (i32, [vp, i64, vp, i64, vp, i64, i64, i64, vp, vp, vp, i64, vp, i64, vp,
                                                    sz, vp]),
        "bsq_linear_workspace_bytes": (sz, [i64, i64, i64]),
        "bsq_linear": (i32, [vp, i64, vp, i64, i64, i64, i64, vp, i32, i32, vp, i64, vp, i64, i32, vp, i64, vp, sz, vp]),
        "bsq_linear_backward_workspace_bytes": (sz, [i64, i64, i64]),
        "bsq_linear_backward": (i32, [vp, i64, vp, i64, vp, i64, i64, i64, i64, i32, vp, i64, vp, i64, vp, i64, vp, vp, sz,
                                      vp]),
        "bsq_gated_linear_workspace_bytes": (sz, [i64, i64, i64]),
        "bsq_gated_linear": (i32, [vp, i64, vp, i64, vp, i64, i64, i64, i64, i32, vp, i64, i32, vp, i64, vp, i64, vp, sz,
                                   vp]),
        "bsq_gated_linear_backward_workspace_bytes": (sz, [i64, i64, i64]),
        "bsq_gated_linear_backward": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64, i32, vp, i64, vp, i64, vp,
                                            i64, vp, i64, vp, i64, vp, sz, vp]),
        "bsq_gemm_linear_workspace_bytes": (sz, [i32, i64, i64, i64]),
        "bsq_gemm_linear": (i32, [vp, vp, vp, i32, i32, vp, i64, vp, i64, i32, vp, i64, vp, sz, vp]),
        "bsq_gemm_gated_workspace_bytes": (sz, [i32, i64, i64, i64]),
        "bsq_gemm_gated": (i32, [vp, vp, vp, i32, vp, i64, i32, vp, i64, vp, i64, vp, sz, vp]),
        "bsq_adamw": (i32, [PA, i32, PO, vp]),
        "bsq_grad_workspace_bytes": (sz, [i32]),
        "bsq_grad_norm": (i32, [PG, i32, vp, vp, sz, vp]),
        "bsq_clip_grad_norm": (i32, [PG, i32, f32, f32, vp, vp, sz, vp]),
    }


# The calls below marked @_bound are made by the native module (csrc/
# binding.cpp), which checks and marshals their arguments.  It is loaded at the
# first of them and then stands in the place of the functions here; like the
# library it has no fallback.
_native_module = None
_BOUND = {}


def _native():
    global _native_module
    if _native_module is None:
        if not os.path.exists(BINDING_PATH):
            raise ImportError(f"native binding not built ({BINDING_PATH}); run {__package__}._build.build()")
        import torch  # noqa: F401  (its libraries have to be loaded)
        library = lib()
        loader = importlib.machinery.ExtensionFileLoader("_binding", BINDING_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_binding", loader))
        loader.exec_module(module)
        names = [*_signatures(), "bsq_codes_bytes", "bsq_scales_bytes"]
        module.bind({name: ctypes.cast(getattr(library, name), ctypes.c_void_p).value for name in names},
                    BsqError, {name: _documentation(f) for name, f in _BOUND.items()})
        for name in _BOUND:
            native = getattr(module, name)
            setattr(sys.modules[__name__], name, native)
            setattr(sys.modules[__package__], name, native)
        _native_module = module
    return _native_module


def _documentation(f) -> str:
    """A native function's documentation: its signature in the form inspect reads, then the text."""
    signature = inspect.signature(f)
    bare = [p.replace(annotation=p.empty) for p in signature.parameters.values()]
    return f"{f.__name__}{inspect.Signature(bare)}\n--\n\n{inspect.getdoc(f)}"


def _bound(f):
    _BOUND[f.__name__] = f

    def call(*args, **kwargs):
        return getattr(_native(), f.__name__)(*args, **kwargs)
    call.__name__, call.__doc__, call.__wrapped__ = f.__name__, f.__doc__, f
    return call


# ------------------------------------------------------------- argument checks
def _refuse(what: str):
    raise BsqError(1, what)


def _type(t, name: str) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return OUT_BF16
    if t.dtype == torch.float32:
        return OUT_F32
    raise BsqError(2, f"{name}: {t.dtype} (bfloat16 and float32 are supported)")


def _elements(t, name: str, n: int, dtype):
    """Pointer of a contiguous CUDA tensor of n elements of `dtype`."""
    if not t.is_cuda or t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous {dtype} CUDA tensor of {n} elements")
    return t.data_ptr()


def _new(shape, dtype, stream, like):
    """A tensor that belongs to the launching stream."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


# ------------------------------------------- tokens sorted by expert and back
@dataclass
class MoePlan:
    """Where the slots of tokens go (see bsq_moe_plan): offsets int64 [experts
    + 1] (what grouped_gemm takes), slot_row int32 [tokens, k], row_slot int32
    [tokens * k]."""
    num_experts: int
    offsets: "object"
    slot_row: "object"
    row_slot: "object"


def moe_plan(tokens: int, k: int, num_experts: int, device="cuda") -> MoePlan:
    """An uninitialized plan, for the *_into forms."""
    import torch
    return MoePlan(num_experts, torch.empty(num_experts + 1, dtype=torch.int64, device=device),
                   torch.empty((tokens, k), dtype=torch.int32, device=device),
                   torch.empty(tokens * k, dtype=torch.int32, device=device))


def _new_plan(expert_ids, num_experts, stream):
    import torch
    if expert_ids.dim() != 2:
        _refuse("expert_ids must be [tokens, k]")
    T, k = expert_ids.shape
    return MoePlan(num_experts, _new(num_experts + 1, torch.int64, stream, expert_ids),
                   _new((T, k), torch.int32, stream, expert_ids), _new(T * k, torch.int32, stream, expert_ids))


@_bound
def moe_sort_into(expert_ids, plan: MoePlan, stream=None):
    """Fill `plan`; returns it."""


def moe_sort(expert_ids, num_experts: int, stream=None) -> MoePlan:
    """Sort the slots of expert_ids [tokens, k] by expert; ids outside [0, num_experts) are left out."""
    return moe_sort_into(expert_ids, _new_plan(expert_ids, num_experts, stream), stream)


@_bound
def moe_dispatch_into(x, expert_ids, plan: MoePlan, rows, stream=None):
    """Fill `plan` and `rows`; returns rows."""


def moe_dispatch(x, expert_ids, num_experts: int, stream=None):
    """Sort the slots and gather their tokens' rows: returns (rows [tokens * k, cols], plan)."""
    plan = _new_plan(expert_ids, num_experts, stream)
    rows = _new((expert_ids.numel(), x.shape[1]), x.dtype, stream, x)
    return moe_dispatch_into(x, expert_ids, plan, rows, stream), plan


@_bound
def moe_gather_into(x, plan: MoePlan, rows, stream=None):
    """Gather by a plan that is already filled; returns rows."""


def moe_gather(x, plan: MoePlan, stream=None):
    return moe_gather_into(x, plan, _new((plan.row_slot.numel(), x.shape[1]), x.dtype, stream, x), stream)


@_bound
def moe_combine_into(rows, weights, plan: MoePlan, out, stream=None):
    """weights None takes 1; returns out."""


def moe_combine(rows, weights, plan: MoePlan, stream=None):
    """out[t] = sum_j weights[t, j] * rows[slot_row[t, j]]; weights None takes 1."""
    out = _new((plan.slot_row.shape[0], rows.shape[1]), rows.dtype, stream, rows)
    return moe_combine_into(rows, weights, plan, out, stream)


def moe_dispatch_backward(drows, plan: MoePlan, stream=None):
    """Gradient of moe_dispatch and moe_gather with respect to x."""
    return moe_combine(drows, None, plan, stream)


@_bound
def moe_combine_backward_into(dout, rows, weights, plan: MoePlan, drows, dweights, stream=None):
    """dweights None: only drows (rows is then not read and may be None)."""


def moe_combine_backward(dout, rows, weights, plan: MoePlan, stream=None):
    import torch
    drows = _new(tuple(rows.shape), dout.dtype, stream, dout)
    dweights = _new(tuple(plan.slot_row.shape), torch.float32, stream, dout)
    return moe_combine_backward_into(dout, rows, weights, plan, drows, dweights, stream)


# ------------------------------------------------------------------ layer norm
@_bound
def layer_norm_into(x, weight, bias, eps: float, y, mean=None, rstd=None, stream=None):
    """weight, bias, mean and rstd may each be None, and y may be x; returns (y, mean, rstd)."""


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, stream=None):
    """Layer norm of the rows of x; returns (y, mean, rstd)."""
    import torch
    y = _new(tuple(x.shape), x.dtype, stream, x)
    mean, rstd = (_new(x.shape[0], torch.float32, stream, x) for _ in range(2))
    return layer_norm_into(x, weight, bias, eps, y, mean, rstd, stream)


@_bound
def layer_norm_backward_into(dy, x, weight, mean, rstd, dx, dweight=None, dbias=None, stream=None):
    """dweight and dbias may each be None, and dx may be dy; returns (dx, dweight, dbias)."""


def layer_norm_backward(dy, x, weight, mean, rstd, stream=None):
    """Gradient of layer_norm; returns (dx, dweight, dbias), the last two float32."""
    import torch
    dx = _new(tuple(x.shape), x.dtype, stream, x)
    dweight, dbias = (_new(x.shape[1], torch.float32, stream, x) for _ in range(2))
    return layer_norm_backward_into(dy, x, weight, mean, rstd, dx, dweight, dbias, stream)


# ----------------------------------------- softmax cross entropy of a linear head
@_bound
def linear_cross_entropy_into(h, w, targets, loss, lse, stream=None):
    """Returns (loss, lse)."""


def linear_cross_entropy(h, w, targets, stream=None):
    """Softmax cross entropy of the logits h @ w.T, which are never stored:
    returns (loss, lse), float32 [tokens]; a target outside [0, vocab) does
    not count (loss 0, no gradient)."""
    import torch
    loss, lse = (_new(h.shape[0], torch.float32, stream, h) for _ in range(2))
    return linear_cross_entropy_into(h, w, targets, loss, lse, stream)


@_bound
def linear_cross_entropy_backward_into(h, w, targets, lse, dloss, dh, dw, stream=None):
    """Either of dh, dw may be None; returns (dh, dw)."""


def linear_cross_entropy_backward(h, w, targets, lse, dloss, stream=None):
    """Gradient of sum(dloss * loss); returns (dh, dw)."""
    dh = _new(tuple(h.shape), h.dtype, stream, h)
    dw = _new(tuple(w.shape), w.dtype, stream, w)
    return linear_cross_entropy_backward_into(h, w, targets, lse, dloss, dh, dw, stream)


# ------------------------------------- linear layers and the gated feed-forward
ACTIVATIONS = ("identity", "relu", "silu", "gelu", "gelu_tanh")


@_bound
def linear_into(x, w, y, bias=None, residual=None, activation="identity", z=None, stream=None):
    """y = act(z) + residual with z = x @ w.T + bias; bias, residual and z (the
    pre-activation, for the backward pass) may each be None, and residual may be
    y; returns (y, z)."""


def linear(x, w, bias=None, residual=None, activation="identity", out_dtype=None, stream=None):
    """act(x @ w.T + bias) + residual, of type `out_dtype` (x's)."""
    y = _new((x.shape[0], w.shape[0]), out_dtype or x.dtype, stream, x)
    return linear_into(x, w, y, bias, residual, activation, None, stream)[0]


@_bound
def linear_backward_into(dy, x, w, dx=None, dw=None, dbias=None, z=None, activation="identity", stream=None):
    """Gradient of linear_into; dx, dw and dbias may each be None (x and w where dw and dx are),
    z where the activation is the identity; returns (dx, dw, dbias)."""


def linear_backward(dy, x, w, z=None, activation="identity", bias=True, stream=None):
    """Gradient of linear: returns (dx, dw, dbias), dbias float32 (None without `bias`)."""
    import torch
    dx, dw = _new(tuple(x.shape), x.dtype, stream, x), _new(tuple(w.shape), w.dtype, stream, w)
    dbias = _new(w.shape[0], torch.float32, stream, w) if bias else None
    return linear_backward_into(dy, x, w, dx, dw, dbias, z, activation, stream)


@_bound
def gated_linear_into(x, w_gate, w_up, h, activation="silu", gate=None, up=None, stream=None):
    """h = act(x @ w_gate.T) * (x @ w_up.T); gate and up, the two factors before the activation, are for
    the backward pass and may both be None; returns (h, gate, up)."""


def gated_linear(x, w_gate, w_up, activation="silu", out_dtype=None, stream=None):
    """act(x @ w_gate.T) * (x @ w_up.T), of type `out_dtype` (x's)."""
    h = _new((x.shape[0], w_gate.shape[0]), out_dtype or x.dtype, stream, x)
    return gated_linear_into(x, w_gate, w_up, h, activation, None, None, stream)[0]


@_bound
def gated_linear_backward_into(dh, x, w_gate, w_up, gate, up, dx=None, dw_gate=None, dw_up=None, activation="silu",
                               stream=None):
    """Gradient of gated_linear_into; dx may be None (then the weights may be), and dw_gate and dw_up
    together (then x may be); returns (dx, dw_gate, dw_up)."""


def gated_linear_backward(dh, x, w_gate, w_up, gate, up, activation="silu", stream=None):
    """Gradient of gated_linear: returns (dx, dw_gate, dw_up)."""
    dx, dg, du = (_new(tuple(t.shape), t.dtype, stream, t) for t in (x, w_gate, w_up))
    return gated_linear_backward_into(dh, x, w_gate, w_up, gate, up, dx, dg, du, activation, stream)


@_bound
def gemm_linear_into(A, B, y, bias=None, residual=None, activation="identity", z=None, stream=None):
    """linear_into on the QTensors A and B; returns (y, z)."""


def gemm_linear(A, B, bias=None, residual=None, activation="identity", out_dtype=None, stream=None):
    """act(A @ B.T + bias) + residual of QTensors, bfloat16 or `out_dtype`."""
    import torch
    y = _new((A.rows, B.rows), out_dtype or torch.bfloat16, stream, A.codes)
    return gemm_linear_into(A, B, y, bias, residual, activation, None, stream)[0]


@_bound
def gemm_gated_into(A, B_gate, B_up, h, activation="silu", gate=None, up=None, stream=None):
    """gated_linear_into on the QTensors A, B_gate and B_up; returns (h, gate, up)."""


def gemm_gated(A, B_gate, B_up, activation="silu", out_dtype=None, stream=None):
    """act(A @ B_gate.T) * (A @ B_up.T) of QTensors, bfloat16 or `out_dtype`."""
    import torch
    h = _new((A.rows, B_gate.rows), out_dtype or torch.bfloat16, stream, A.codes)
    return gemm_gated_into(A, B_gate, B_up, h, activation, None, None, stream)[0]


# ------------------------------------------------------ global norm and clipping
class GradList:
    """The gradients of a step and where their clipped copies go (`outs`; in
    place without it): contiguous tensors of one GPU, bfloat16 or float32.
    Built once for buffers that stay (some 2 us of host time a tensor); it
    keeps them alive, and with them a workspace for each stream it is used on
    and each call that a graph captured."""

    def __init__(self, grads, outs=None):
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        if not grads or len(outs) != len(grads):
            _refuse("a gradient list needs at least one gradient, and one output for each")
        arr = (BsqGradC * len(grads))()
        where = grads[0].get_device()
        for i, (g, o) in enumerate(zip(grads, outs)):
            n = g.numel()
            t = _type(g, f"gradient {i}")
            if g.get_device() != where or o.get_device() != where:
                name, x = (f"gradient {i}", g) if g.get_device() != where else (f"output {i}", o)
                _refuse(f"{name} is on {x.device}, gradient 0 on {grads[0].device}")
            at = _elements(g, f"gradient {i}", n, g.dtype)
            to = at if o is g else _elements(o, f"output {i}", n, g.dtype)
            arr[i] = BsqGradC(at, to, n, t, 0)
        self.grads, self.outs, self.array = grads, outs, arr
        self.address, self.count = ctypes.addressof(arr), len(grads)
        self.workspace_bytes = int(lib().bsq_grad_workspace_bytes(len(grads)))
        self._workspaces, self._captured = {}, []

    def workspace(self, stream):
        """Scratch kept for the launching stream: calls on one stream run in
        order, calls on two get one each.  A call captured in a graph gets its
        own: the graph may replay beside later calls."""
        import torch
        raw, capturing = _native().stream_state(self.grads[0], stream)
        if capturing:
            self._captured.append(_new(self.workspace_bytes, torch.uint8, stream, self.grads[0]))
            return self._captured[-1]
        ws = self._workspaces.get(raw)
        if ws is None:
            ws = self._workspaces[raw] = _new(self.workspace_bytes, torch.uint8, stream, self.grads[0])
        return ws


def _grad_list(grads) -> GradList:
    return grads if isinstance(grads, GradList) else GradList(grads)


def _needs_bound(max_norm):
    if max_norm is None:                               # the native call takes it for the norm only
        _refuse("max_norm must be a number")


def grad_norm(grads, stream=None):
    """The global 2-norm of a GradList or of tensors: float32 [1] on the device."""
    import torch
    g = _grad_list(grads)
    norm = _new(1, torch.float32, stream, g.grads[0])
    return _native().grads_into(g.address, g.count, None, 0.0, norm, g.workspace(stream), stream)


def clip_grad_norm_into(grads, max_norm: float, norm, eps: float = 1e-6, stream=None):
    _needs_bound(max_norm)
    g = _grad_list(grads)
    return _native().grads_into(g.address, g.count, max_norm, eps, norm, g.workspace(stream), stream)


def clip_grad_norm(grads, max_norm: float, eps: float = 1e-6, stream=None):
    """Write every gradient times min(1, max_norm / (norm + eps)) to its
    output (a list of tensors: in place); returns the norm, float32 [1].  A
    list of tensors costs what building its GradList costs, at every call."""
    import torch
    _needs_bound(max_norm)
    g = _grad_list(grads)
    return clip_grad_norm_into(g, max_norm, _new(1, torch.float32, stream, g.grads[0]), eps, stream)


# -------------------------------------------------------------------- AdamW
MOMENTS_F32, MOMENTS_8BIT = 0, 1


def adamw_states(params, bits: int = 32):
    """Moments to start with, zeros: for each parameter (m, v) float32, or with
    bits = 8 (m, m_scales, v, v_scales) uint8, E4M3 codes and an E8M0 byte for 32."""
    import torch
    if bits not in (8, 32):
        _refuse(f"moments of {bits} bits (8 and 32 are supported)")

    def zeros(n, dtype, p):
        return torch.zeros(n, dtype=dtype, device=p.device)

    if bits == 32:
        return [(zeros(p.numel(), torch.float32, p), zeros(p.numel(), torch.float32, p)) for p in params]
    return [tuple(zeros(n, torch.uint8, p) for n in (p.numel(), -(-p.numel() // 32)) * 2) for p in params]


class AdamWList:
    """The parameters of a step, their gradients and moments: contiguous tensors
    of one GPU.  params, grads: bfloat16 or float32 each; states: 32 or 8 (bits of
    moments that start at 0), or what adamw_states returns; copies: None, or for
    each parameter a bfloat16 tensor for its rounded copy (or None).  No two of all
    these overlap.  Built once for buffers that stay, at 3 to 5 us of host time a
    parameter, which new gradient tensors cost at every step; keeps them alive."""

    def __init__(self, params, grads, states=32, copies=None):
        import torch
        params, grads = list(params), list(grads)
        states = adamw_states(params, states) if isinstance(states, int) else [tuple(s) for s in states]
        copies = [None] * len(params) if copies is None else list(copies)
        if not params or not len(params) == len(grads) == len(states) == len(copies):
            _refuse("an AdamW list needs at least one parameter, and a gradient and moments for each")
        where = params[0].device
        arr = (BsqAdamwTensorC * len(params))()
        for i, (p, g, state, c) in enumerate(zip(params, grads, states, copies)):
            n, blocks = p.numel(), -(-p.numel() // 32)
            if len(state) not in (2, 4):
                _refuse(f"moments {i} must be (m, v) or (m, m_scales, v, v_scales)")
            for t in (p, g, *state, *(() if c is None else (c,))):
                if t.device != where:
                    _refuse(f"a tensor of parameter {i} is on {t.device}, parameter 0 on {where}")
            a = arr[i]
            a.param_type, a.grad_type = _type(p, f"parameter {i}"), _type(g, f"gradient {i}")
            a.param, a.grad = _elements(p, f"parameter {i}", n, p.dtype), _elements(g, f"gradient {i}", n, g.dtype)
            if len(state) == 2:
                a.state = MOMENTS_F32
                a.m, a.v = (_elements(t, f"moments {i}", n, torch.float32) for t in state)
            else:
                a.state = MOMENTS_8BIT
                a.m, a.m_scales, a.v, a.v_scales = (
                    _elements(t, f"moments {i}", k, torch.uint8) for t, k in zip(state, (n, blocks, n, blocks)))
            a.copy = None if c is None else _elements(c, f"copy {i}", n, torch.bfloat16)
            a.n = n
        self.params, self.grads, self.states, self.copies, self.array = params, grads, states, copies, arr
        self.address, self.count = ctypes.addressof(arr), len(params)


def adamw_step(tensors: AdamWList, lr, step, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01, norm=None,
               max_norm=None, clip_eps: float = 1e-6, seed=None, stream=None):
    """One AdamW step of an AdamWList, in place.  step: its number, from 1 on; lr
    and step may be float32 and int64 tensors [1] on the device, which a captured
    step reads at each replay.  norm (of grad_norm) and max_norm clip the gradients in
    the same pass, as clip_grad_norm would, without writing them.  seed: codes of
    8-bit moments and bfloat16 parameters are rounded stochastically (None: to
    nearest); it may stay the same from step to step."""
    if (norm is None) != (max_norm is None):
        _refuse("norm and max_norm go together")
    _native().adamw_into(tensors.address, tensors.count, tensors.params[0], lr, step, betas[0], betas[1], eps, weight_decay,
                         norm, max_norm, clip_eps, seed, stream)
