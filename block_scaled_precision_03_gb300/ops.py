"""Binding of the operators around the layer: tokens sorted by expert and
back, layer norm, the softmax cross entropy of a linear head, and the global
gradient norm with clipping.  Like the rest of the binding it marshals
arguments only; include/bsq.h has the formulas, limits and errors.

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
from dataclasses import dataclass

from . import OUT_BF16, OUT_F32, BsqError, _check, lib

ID_I32, ID_I64 = 0, 1


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


_raw_stream = None


def _stream(stream, like) -> int:
    """Handle of the stream to launch on: the given one, or the current one of
    the tensor's device (by the call behind torch.cuda.current_stream, which
    costs more than a small kernel here)."""
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _raw_stream(like.get_device())


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


def _matrix(t, name: str, rows=None, cols=None, dtype=None):
    """(pointer, row pitch in elements) of a CUDA matrix with unit stride along its columns."""
    if not t.is_cuda or t.dim() != 2:
        _refuse(f"{name} must be a CUDA matrix")
    r, c = t.shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        _refuse(f"{name} is {r} x {c}, not {rows if rows is not None else r} x {cols if cols is not None else c}")
    if dtype is not None and t.dtype != dtype:
        _refuse(f"{name} is {t.dtype}, not {dtype}")
    s0, s1 = t.stride()
    if c > 1 and s1 != 1:
        _refuse(f"{name} must have unit stride along its columns")
    return t.data_ptr(), (s0 if r > 1 else max(s0, c))


def _vector(t, name: str, n: int, dtype):
    """Pointer of a contiguous CUDA tensor of n elements of `dtype`; None for None."""
    if t is None:
        return None
    if not t.is_cuda or t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous {dtype} CUDA tensor of {n} elements")
    return t.data_ptr()


def _workspace(nbytes: int, stream, like):
    """Device scratch that belongs to the launching stream: the allocator hands
    it out again only to work behind this call on that stream."""
    import torch
    if nbytes == 0:
        return None, None
    if stream is None:
        w = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    else:
        with torch.cuda.stream(stream):
            w = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    return w, w.data_ptr()


def _new(shape, dtype, stream, like):
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

    def c(self) -> BsqMoePlanC:
        import torch
        if self.slot_row.dim() != 2:
            _refuse("slot_row must be [tokens, k]")
        T, k = self.slot_row.shape
        return BsqMoePlanC(T, k, self.num_experts,
                           _vector(self.offsets, "offsets", self.num_experts + 1, torch.int64),
                           _vector(self.slot_row, "slot_row", T * k, torch.int32),
                           _vector(self.row_slot, "row_slot", T * k, torch.int32))


def moe_plan(tokens: int, k: int, num_experts: int, device="cuda") -> MoePlan:
    """An uninitialized plan, for the *_into forms."""
    import torch
    return MoePlan(num_experts, torch.empty(num_experts + 1, dtype=torch.int64, device=device),
                   torch.empty((tokens, k), dtype=torch.int32, device=device),
                   torch.empty(tokens * k, dtype=torch.int32, device=device))


def _ids(expert_ids, plan: BsqMoePlanC):
    import torch
    if expert_ids.dtype not in (torch.int32, torch.int64) or expert_ids.dim() != 2 or \
            expert_ids.shape != (plan.tokens, plan.k):
        _refuse(f"expert_ids must be an int32 or int64 matrix of {plan.tokens} x {plan.k}")
    return (_vector(expert_ids, "expert_ids", plan.tokens * plan.k, expert_ids.dtype),
            ID_I64 if expert_ids.dtype == torch.int64 else ID_I32)


def _new_plan(expert_ids, num_experts, stream):
    import torch
    if expert_ids.dim() != 2:
        _refuse("expert_ids must be [tokens, k]")
    T, k = expert_ids.shape
    return MoePlan(num_experts, _new(num_experts + 1, torch.int64, stream, expert_ids),
                   _new((T, k), torch.int32, stream, expert_ids), _new(T * k, torch.int32, stream, expert_ids))


def moe_sort_into(expert_ids, plan: MoePlan, stream=None) -> MoePlan:
    p = plan.c()
    ids, id_type = _ids(expert_ids, p)
    n = lib().bsq_moe_workspace_bytes(p.tokens, p.k, p.num_experts)
    keep, ws = _workspace(n, stream, expert_ids)
    _check(lib().bsq_moe_sort(ids, id_type, ctypes.byref(p), ws, n, _stream(stream, expert_ids)), "bsq_moe_sort")
    return plan


def moe_sort(expert_ids, num_experts: int, stream=None) -> MoePlan:
    """Sort the slots of expert_ids [tokens, k] by expert; ids outside [0, num_experts) are left out."""
    return moe_sort_into(expert_ids, _new_plan(expert_ids, num_experts, stream), stream)


def moe_dispatch_into(x, expert_ids, plan: MoePlan, rows, stream=None):
    p = plan.c()
    ids, id_type = _ids(expert_ids, p)
    px, ldx = _matrix(x, "x", p.tokens)
    pr, ldr = _matrix(rows, "rows", p.tokens * p.k, x.shape[1], x.dtype)
    n = lib().bsq_moe_workspace_bytes(p.tokens, p.k, p.num_experts)
    keep, ws = _workspace(n, stream, x)
    _check(lib().bsq_moe_dispatch(px, ldx, _type(x, "x"), x.shape[1], ids, id_type, ctypes.byref(p), pr, ldr, ws, n,
                                  _stream(stream, x)), "bsq_moe_dispatch")
    return rows


def moe_dispatch(x, expert_ids, num_experts: int, stream=None):
    """Sort the slots and gather their tokens' rows: returns (rows [tokens * k, cols], plan)."""
    plan = _new_plan(expert_ids, num_experts, stream)
    rows = _new((expert_ids.numel(), x.shape[1]), x.dtype, stream, x)
    return moe_dispatch_into(x, expert_ids, plan, rows, stream), plan


def moe_gather_into(x, plan: MoePlan, rows, stream=None):
    p = plan.c()
    px, ldx = _matrix(x, "x", p.tokens)
    pr, ldr = _matrix(rows, "rows", p.tokens * p.k, x.shape[1], x.dtype)
    _check(lib().bsq_moe_gather(px, ldx, _type(x, "x"), x.shape[1], ctypes.byref(p), pr, ldr, _stream(stream, x)),
           "bsq_moe_gather")
    return rows


def moe_gather(x, plan: MoePlan, stream=None):
    return moe_gather_into(x, plan, _new((plan.row_slot.numel(), x.shape[1]), x.dtype, stream, x), stream)


def moe_combine_into(rows, weights, plan: MoePlan, out, stream=None):
    import torch
    p = plan.c()
    pr, ldr = _matrix(rows, "rows", p.tokens * p.k)
    po, ldo = _matrix(out, "out", p.tokens, rows.shape[1], rows.dtype)
    pw = _vector(weights, "weights", p.tokens * p.k, torch.float32)
    _check(lib().bsq_moe_combine(pr, ldr, _type(rows, "rows"), rows.shape[1], pw, ctypes.byref(p), po, ldo,
                                 _stream(stream, rows)), "bsq_moe_combine")
    return out


def moe_combine(rows, weights, plan: MoePlan, stream=None):
    """out[t] = sum_j weights[t, j] * rows[slot_row[t, j]]; weights None takes 1."""
    out = _new((plan.slot_row.shape[0], rows.shape[1]), rows.dtype, stream, rows)
    return moe_combine_into(rows, weights, plan, out, stream)


def moe_dispatch_backward(drows, plan: MoePlan, stream=None):
    """Gradient of moe_dispatch and moe_gather with respect to x."""
    return moe_combine(drows, None, plan, stream)


def moe_combine_backward_into(dout, rows, weights, plan: MoePlan, drows, dweights, stream=None):
    """dweights None: only drows (rows is then not read and may be None)."""
    import torch
    p = plan.c()
    pd, ldd = _matrix(dout, "dout", p.tokens)
    C = dout.shape[1]
    pr, ldr = _matrix(rows, "rows", p.tokens * p.k, C, dout.dtype) if rows is not None else (None, 0)
    pg, ldg = _matrix(drows, "drows", p.tokens * p.k, C, dout.dtype)
    pw = _vector(weights, "weights", p.tokens * p.k, torch.float32)
    pdw = _vector(dweights, "dweights", p.tokens * p.k, torch.float32)
    _check(lib().bsq_moe_combine_backward(pd, ldd, pr, ldr, _type(dout, "dout"), C, pw, ctypes.byref(p), pg, ldg, pdw,
                                          _stream(stream, dout)), "bsq_moe_combine_backward")
    return drows, dweights


def moe_combine_backward(dout, rows, weights, plan: MoePlan, stream=None):
    import torch
    drows = _new(tuple(rows.shape), dout.dtype, stream, dout)
    dweights = _new(tuple(plan.slot_row.shape), torch.float32, stream, dout)
    return moe_combine_backward_into(dout, rows, weights, plan, drows, dweights, stream)


# ------------------------------------------------------------------ layer norm
def _params(weight, bias, cols: int):
    """Pointers and type of the (optional) weight and bias."""
    first = weight if weight is not None else bias
    if first is None:
        return None, None, OUT_F32
    t = _type(first, "weight" if weight is not None else "bias")
    return _vector(weight, "weight", cols, first.dtype), _vector(bias, "bias", cols, first.dtype), t


def layer_norm_into(x, weight, bias, eps: float, y, mean=None, rstd=None, stream=None):
    import torch
    px, ldx = _matrix(x, "x")
    R, C = x.shape
    py, ldy = _matrix(y, "y", R, C, x.dtype)
    pw, pb, pt = _params(weight, bias, C)
    _check(lib().bsq_layer_norm(px, ldx, _type(x, "x"), R, C, pw, pb, pt, eps, py, ldy,
                                _vector(mean, "mean", R, torch.float32), _vector(rstd, "rstd", R, torch.float32),
                                _stream(stream, x)), "bsq_layer_norm")
    return y, mean, rstd


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, stream=None):
    """Layer norm of the rows of x; returns (y, mean, rstd)."""
    import torch
    y = _new(tuple(x.shape), x.dtype, stream, x)
    mean, rstd = (_new(x.shape[0], torch.float32, stream, x) for _ in range(2))
    return layer_norm_into(x, weight, bias, eps, y, mean, rstd, stream)


def layer_norm_backward_into(dy, x, weight, mean, rstd, dx, dweight=None, dbias=None, stream=None):
    import torch
    px, ldx = _matrix(x, "x")
    R, C = x.shape
    pdy, ld_dy = _matrix(dy, "dy", R, C, x.dtype)
    pdx, ld_dx = _matrix(dx, "dx", R, C, x.dtype)
    pw, _, pt = _params(weight, None, C)
    f32 = torch.float32
    n = lib().bsq_layer_norm_workspace_bytes(R, C) if dweight is not None or dbias is not None else 0
    keep, ws = _workspace(n, stream, x)
    _check(lib().bsq_layer_norm_backward(pdy, ld_dy, px, ldx, _type(x, "x"), R, C, pw, pt,
                                         _vector(mean, "mean", R, f32), _vector(rstd, "rstd", R, f32), pdx, ld_dx,
                                         _vector(dweight, "dweight", C, f32), _vector(dbias, "dbias", C, f32), ws, n,
                                         _stream(stream, x)), "bsq_layer_norm_backward")
    return dx, dweight, dbias


def layer_norm_backward(dy, x, weight, mean, rstd, stream=None):
    """Gradient of layer_norm; returns (dx, dweight, dbias), the last two float32."""
    import torch
    dx = _new(tuple(x.shape), x.dtype, stream, x)
    dweight, dbias = (_new(x.shape[1], torch.float32, stream, x) for _ in range(2))
    return layer_norm_backward_into(dy, x, weight, mean, rstd, dx, dweight, dbias, stream)


# ----------------------------------------- softmax cross entropy of a linear head
def _head(h, w, targets):
    import torch
    bf16 = torch.bfloat16
    for t, name in ((h, "h"), (w, "w")):
        if t.dtype != bf16:
            raise BsqError(2, f"{name}: {t.dtype} (bfloat16 is supported)")
    ph, ldh = _matrix(h, "h")
    pw, ldw = _matrix(w, "w", None, h.shape[1])
    T = h.shape[0]
    return ph, ldh, pw, ldw, _vector(targets, "targets", T, torch.int64), T, w.shape[0], h.shape[1]


def linear_cross_entropy_into(h, w, targets, loss, lse, stream=None):
    import torch
    ph, ldh, pw, ldw, pt, T, V, D = _head(h, w, targets)
    n = lib().bsq_linear_cross_entropy_workspace_bytes(T, V, D, 0)
    keep, ws = _workspace(n, stream, h)
    _check(lib().bsq_linear_cross_entropy(ph, ldh, pw, ldw, pt, T, V, D, _vector(loss, "loss", T, torch.float32),
                                          _vector(lse, "lse", T, torch.float32), ws, n, _stream(stream, h)),
           "bsq_linear_cross_entropy")
    return loss, lse


def linear_cross_entropy(h, w, targets, stream=None):
    """Softmax cross entropy of the logits h @ w.T, which are never stored:
    returns (loss, lse), float32 [tokens]; a target outside [0, vocab) does
    not count (loss 0, no gradient)."""
    import torch
    loss, lse = (_new(h.shape[0], torch.float32, stream, h) for _ in range(2))
    return linear_cross_entropy_into(h, w, targets, loss, lse, stream)


def linear_cross_entropy_backward_into(h, w, targets, lse, dloss, dh, dw, stream=None):
    """Either of dh, dw may be None."""
    import torch
    ph, ldh, pw, ldw, pt, T, V, D = _head(h, w, targets)
    pdh, ld_dh = _matrix(dh, "dh", T, D, h.dtype) if dh is not None else (None, 0)
    pdw, ld_dw = _matrix(dw, "dw", V, D, w.dtype) if dw is not None else (None, 0)
    n = lib().bsq_linear_cross_entropy_workspace_bytes(T, V, D, 1)
    keep, ws = _workspace(n, stream, h)
    _check(lib().bsq_linear_cross_entropy_backward(ph, ldh, pw, ldw, pt, T, V, D,
                                                   _vector(lse, "lse", T, torch.float32),
                                                   _vector(dloss, "dloss", T, torch.float32), pdh, ld_dh, pdw, ld_dw,
                                                   ws, n, _stream(stream, h)), "bsq_linear_cross_entropy_backward")
    return dh, dw


def linear_cross_entropy_backward(h, w, targets, lse, dloss, stream=None):
    """Gradient of sum(dloss * loss); returns (dh, dw)."""
    dh = _new(tuple(h.shape), h.dtype, stream, h)
    dw = _new(tuple(w.shape), w.dtype, stream, w)
    return linear_cross_entropy_backward_into(h, w, targets, lse, dloss, dh, dw, stream)


# ------------------------------------------------------ global norm and clipping
class GradList:
    """The gradients of a step and where their clipped copies go (`outs`; in
    place without it): contiguous CUDA tensors, bfloat16 or float32.  Built
    once for buffers that stay; it keeps them alive."""

    def __init__(self, grads, outs=None):
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        if not grads or len(outs) != len(grads):
            _refuse("a gradient list needs at least one gradient, and one output for each")
        arr = (BsqGradC * len(grads))()
        for i, (g, o) in enumerate(zip(grads, outs)):
            t = _type(g, f"gradient {i}")
            arr[i] = BsqGradC(_vector(g, f"gradient {i}", g.numel(), g.dtype),
                              _vector(o, f"output {i}", g.numel(), g.dtype), g.numel(), t, 0)
        self.grads, self.outs, self.array = grads, outs, arr
        self.workspace_bytes = int(lib().bsq_grad_workspace_bytes(len(grads)))
        self._workspaces, self._captured = {}, []

    def workspace(self, stream):
        """(handle of the launching stream, scratch kept for it): calls on one
        stream run in order, calls on two get one each.  A call captured in a
        graph gets its own: the graph may replay beside later calls."""
        import torch
        raw = _stream(stream, self.grads[0])
        if torch.cuda.is_current_stream_capturing():
            self._captured.append(_workspace(self.workspace_bytes, stream, self.grads[0]))
            return raw, self._captured[-1][1]
        ws = self._workspaces.get(raw)
        if ws is None:
            ws = self._workspaces[raw] = _workspace(self.workspace_bytes, stream, self.grads[0])
        return raw, ws[1]


def _grad_list(grads) -> GradList:
    return grads if isinstance(grads, GradList) else GradList(grads)


def grad_norm(grads, stream=None):
    """The global 2-norm of a GradList or of tensors: float32 [1] on the device."""
    import torch
    g = _grad_list(grads)
    norm = _new(1, torch.float32, stream, g.grads[0])
    raw, ws = g.workspace(stream)
    _check(lib().bsq_grad_norm(g.array, len(g.grads), norm.data_ptr(), ws, g.workspace_bytes, raw), "bsq_grad_norm")
    return norm


def clip_grad_norm_into(grads, max_norm: float, norm, eps: float = 1e-6, stream=None):
    import torch
    g = _grad_list(grads)
    pn = _vector(norm, "norm", 1, torch.float32)
    raw, ws = g.workspace(stream)
    _check(lib().bsq_clip_grad_norm(g.array, len(g.grads), max_norm, eps, pn, ws, g.workspace_bytes, raw),
           "bsq_clip_grad_norm")
    return norm


def clip_grad_norm(grads, max_norm: float, eps: float = 1e-6, stream=None):
    """Write every gradient times min(1, max_norm / (norm + eps)) to its
    output (a list of tensors: in place); returns the norm, float32 [1]."""
    import torch
    g = _grad_list(grads)
    return clip_grad_norm_into(g, max_norm, _new(1, torch.float32, stream, g.grads[0]), eps, stream)
