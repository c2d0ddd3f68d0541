"""Binding of the operators around the layer: tokens sorted by expert and
back, layer norm, the softmax cross entropy of a linear head, and the global
gradient norm with clipping.  Like the rest of the binding it marshals
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
    grad_norm(grads), clip_grad_norm(grads, max_norm) -> norm

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


def _signatures():
    i32, i64, vp, sz, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    PP, PG = ctypes.POINTER(BsqMoePlanC), ctypes.POINTER(BsqGradC)
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
        module.bind({name: ctypes.cast(getattr(library, name), ctypes.c_void_p).value for name in _signatures()},
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
