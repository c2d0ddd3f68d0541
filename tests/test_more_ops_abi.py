"""Host-side argument checks of the linear layers, the gated feed-forward and
AdamW, of the C ABI and of the binding (no GPU: a rejected call launches
nothing), and their workspace sizes."""
import ctypes

import pytest
import torch

from test_ops_binding import BF, F32, I64, on

NULL = None
U8 = torch.uint8


@pytest.fixture(scope="module")
def bsq():
    from block_scaled_precision_03_gb300 import _build
    import block_scaled_precision_03_gb300 as b
    _build.build()
    b.lib()
    return b


def caller(f, **standard):
    return lambda **k: f(*{**standard, **k}.values())


def test_linear_checks(bsq):
    L = bsq.lib()
    n = L.bsq_linear_workspace_bytes(100, 300, 8192)
    assert n > 0 and L.bsq_linear_workspace_bytes(1, 300, 8192) == 0
    size = [L.bsq_linear_workspace_bytes, L.bsq_linear_backward_workspace_bytes, L.bsq_gated_linear_workspace_bytes,
            L.bsq_gated_linear_backward_workspace_bytes]
    for s in size:
        assert s(0, 8, 8) == 0 and s(8, 0, 8) == 0 and s(8, 8, 0) == 0
        assert s(1 << 31, 8, 8) == 0 and s(8, (1 << 23) + 1, 8) == 0 and s(8, 8, (1 << 23) + 8) == 0 and s(1 << 30, 1 << 20, 8) == 0
    f = caller(L.bsq_linear, x=256, ldx=8192, w=256, ldw=8192, T=100, N=300, D=8192, bias=256, bt=0, act=3, res=256, ldr=300, y=256,
               ldy=300, t=1, z=256, ldz=300, ws=256, n=n, st=NULL)
    assert f(x=NULL) == 1 and f(w=NULL) == 1 and f(y=NULL) == 1 and f(T=0) == 1 and f(N=0) == 1 and f(D=0) == 1
    assert f(act=-1) == 1 and f(act=5) == 1 and f(t=2) == 1 and f(bt=2) == 1 and f(ldx=8184) == 1 and f(ldw=8184) == 1
    assert f(ldy=299) == 1 and f(ldr=299) == 1 and f(ldz=299) == 1 and f(ws=NULL) == 1 and f(n=n - 1) == 1
    assert f(x=264) == 3 and f(w=264) == 3 and f(ldx=8196) == 3 and f(ldw=8196) == 3 and f(D=8188) == 3 and f(y=257) == 3
    assert f(y=258, t=0) == 3 and f(res=257) == 3 and f(z=257) == 3 and f(bias=258) == 3 and f(bias=257, bt=1) == 3 and f(ws=264) == 3
    assert f(T=1 << 31) == 2 and f(N=(1 << 23) + 1) == 2 and f(D=1 << 24) == 2 and f(T=1 << 30, N=1 << 20) == 2
    m = L.bsq_linear_backward_workspace_bytes(100, 300, 64)
    g = caller(L.bsq_linear_backward, dy=256, ldd=300, x=256, ldx=64, w=256, ldw=64, T=100, N=300, D=64, act=2, z=256, ldz=300,
               dx=256, lddx=64, dw=256, lddw=64, db=256, ws=256, n=m, st=NULL)
    assert m > 0
    assert g(dx=NULL, dw=NULL, db=NULL) == 1 and g(dy=NULL) == 1 and g(z=NULL) == 1 and g(x=NULL) == 1 and g(w=NULL) == 1
    assert g(ldd=299) == 1 and g(ldz=299) == 1 and g(lddx=56) == 1 and g(lddw=56) == 1 and g(act=9) == 1 and g(n=m - 1) == 1
    assert g(dx=264) == 3 and g(dw=264) == 3 and g(lddx=68) == 3 and g(lddw=68) == 3 and g(db=258) == 3 and g(dy=257) == 3
    assert g(z=257) == 3 and g(D=60) == 3 and g(T=1 << 31) == 2


def test_gated_checks(bsq):
    L = bsq.lib()
    n = L.bsq_gated_linear_workspace_bytes(100, 300, 8192)
    f = caller(L.bsq_gated_linear, x=256, ldx=8192, g=256, ldg=8192, u=256, ldu=8192, T=100, N=300, D=8192, act=2, h=256, ldh=300,
               t=1, gate=256, ldgate=300, up=256, ldup=300, ws=256, n=n, st=NULL)
    assert n > 0
    assert f(x=NULL) == 1 and f(g=NULL) == 1 and f(u=NULL) == 1 and f(h=NULL) == 1 and f(gate=NULL) == 1 and f(up=NULL) == 1
    assert f(t=7) == 1 and f(ldh=299) == 1 and f(ldgate=299) == 1 and f(ldup=299) == 1 and f(ws=NULL) == 1 and f(act=5) == 1
    assert f(u=264) == 3 and f(ldu=8196) == 3 and f(gate=257) == 3 and f(up=257) == 3 and f(h=257) == 3 and f(N=1 << 30) == 2
    m = L.bsq_gated_linear_backward_workspace_bytes(100, 300, 64)
    g = caller(L.bsq_gated_linear_backward, dh=256, ldd=300, x=256, ldx=64, g=256, ldg=64, u=256, ldu=64, T=100, N=300, D=64, act=2,
               gate=256, ldgate=300, up=256, ldup=300, dx=256, lddx=64, dg=256, lddg=64, du=256, lddu=64, ws=256, n=m, st=NULL)
    assert g(dx=NULL, dg=NULL, du=NULL) == 1 and g(dg=NULL) == 1 and g(du=NULL) == 1 and g(gate=NULL) == 1 and g(up=NULL) == 1
    assert g(x=NULL) == 1 and g(g=NULL) == 1 and g(u=NULL) == 1 and g(dh=NULL) == 1 and g(n=m - 1) == 1 and g(lddu=56) == 1
    assert g(dg=264) == 3 and g(lddg=68) == 3 and g(up=257) == 3


def test_gemm_checks(bsq):
    L = bsq.lib()
    T = bsq.BsqTensorC

    def q(fmt=0, rows=100, cols=8192, codes=256, scales=256, ts=256):
        return ctypes.byref(T(fmt, 0, rows, cols, codes, scales, ts))

    n = L.bsq_gemm_linear_workspace_bytes(0, 100, 300, 8192)
    m = L.bsq_gemm_gated_workspace_bytes(0, 100, 300, 8192)
    assert n > 0 and m > 0 and L.bsq_gemm_linear_workspace_bytes(9, 100, 300, 8192) == 0
    assert L.bsq_gemm_gated_workspace_bytes(0, 100, 0, 8192) == 0 and L.bsq_gemm_linear_workspace_bytes(0, 8, 1 << 24, 64) == 0
    f = caller(L.bsq_gemm_linear, A=q(), B=q(rows=300), bias=256, bt=0, act=1, res=256, ldr=300, y=256, ldy=300, t=1, z=256, ldz=300,
               ws=256, n=n, st=NULL)
    assert f(A=NULL) == 1 and f(B=NULL) == 1 and f(B=q(cols=4096)) == 1 and f(y=NULL) == 1 and f(act=5) == 1 and f(t=3) == 1
    assert f(bt=4) == 1 and f(ldy=299) == 1 and f(ldr=299) == 1 and f(ldz=299) == 1 and f(ws=NULL) == 1 and f(n=n - 1) == 1
    assert f(B=q(fmt=2)) == 2 and f(A=q(fmt=3), B=q(fmt=2)) == 2 and f(B=q(rows=1 << 24)) == 2
    assert f(A=q(codes=264)) == 3 and f(y=257) == 3 and f(res=257) == 3 and f(z=257) == 3 and f(bias=258) == 3 and f(ws=264) == 3
    g = caller(L.bsq_gemm_gated, A=q(), G=q(rows=300), U=q(rows=300), act=2, h=256, ldh=300, t=1, gate=256, ldg=300, up=256, ldu=300,
               ws=256, n=m, st=NULL)
    assert g(G=NULL) == 1 and g(U=NULL) == 1 and g(U=q(rows=301)) == 1 and g(U=q(fmt=1, rows=300)) == 1 and g(gate=NULL) == 1
    assert g(up=NULL) == 1 and g(n=m - 1) == 1 and g(ldg=299) == 1 and g(ldu=299) == 1 and g(U=q(fmt=2, rows=300)) == 2
    assert g(up=257) == 3 and g(U=q(rows=300, scales=260)) == 3
    assert g(A=q(fmt=3, ts=NULL), G=q(fmt=3, rows=300), U=q(fmt=3, rows=300)) == 1


def test_adamw_checks(bsq):
    L = bsq.lib()
    from block_scaled_precision_03_gb300.ops import BsqAdamwOptionsC as O, BsqAdamwTensorC as P

    def t(param=256, grad=256, m=256, v=256, ms=256, vs=256, copy=NULL, n=10, pt=0, gt=0, state=1, reserved=0):
        return P(param, grad, m, v, ms, vs, copy, n, pt, gt, state, reserved)

    def call(tensor=None, count=1, **o):
        options = O(**{**dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=1), **o})
        return L.bsq_adamw((P * 1)(tensor or t()), count, ctypes.byref(options), NULL)

    nan, inf = float("nan"), float("inf")
    assert L.bsq_adamw(NULL, 1, ctypes.byref(O(step=1)), NULL) == 1 and L.bsq_adamw((P * 1)(t()), 1, NULL, NULL) == 1
    assert call(count=0) == 1 and call(count=(1 << 20) + 1) == 2
    for bad in (dict(lr=-1.0), dict(lr=nan), dict(lr=inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=nan), dict(eps=-1.0),
                dict(weight_decay=inf), dict(step=0), dict(step=-3), dict(reserved=1), dict(norm=256, max_norm=-1.0),
                dict(norm=256, max_norm=nan), dict(norm=256, max_norm=1.0, clip_eps=-1.0)):
        assert call(**bad) == 1, bad
    assert call(step_device=260) == 3 and call(lr_device=258) == 3 and call(norm=258, max_norm=1.0) == 3
    for bad in (dict(param=NULL), dict(grad=NULL), dict(m=NULL), dict(v=NULL), dict(ms=NULL), dict(vs=NULL), dict(n=-1), dict(pt=2),
                dict(gt=-1), dict(state=2), dict(reserved=1)):
        assert call(t(**bad)) == 1, bad
    for bad in (dict(param=258), dict(grad=258), dict(param=257, pt=1), dict(copy=257), dict(m=258, state=0), dict(v=258, state=0)):
        assert call(t(**bad)) == 3, bad
    assert call(t(n=1 << 41)) == 2


def quantized(bsq, rows, cols, devices):
    return bsq.QTensor(0, rows, cols, on(devices[0], rows * cols, dtype=U8), on(devices[1], 128 * 4 * -(-rows // 128) * -(-cols // 128),
                                                                              dtype=U8), None)


T, D, N = 4, 32, 24
# name: the call's tensors (shape, type), numbers and texts standing for themselves
CALLS = {
    "linear_into": [((T, D), BF), ((N, D), BF), ((T, N), BF), ((N,), F32), ((T, N), BF), "gelu", ((T, N), BF)],
    "linear_backward_into": [((T, N), BF), ((T, D), BF), ((N, D), BF), ((T, D), BF), ((N, D), BF), ((N,), F32), ((T, N), BF), "silu"],
    "gated_linear_into": [((T, D), BF), ((N, D), BF), ((N, D), BF), ((T, N), BF), "silu", ((T, N), BF), ((T, N), BF)],
    "gated_linear_backward_into": [((T, N), BF), ((T, D), BF), ((N, D), BF), ((N, D), BF), ((T, N), BF), ((T, N), BF), ((T, D), BF),
                                   ((N, D), BF), ((N, D), BF), "silu"],
    "gemm_linear_into": ["A", "B", ((T, N), BF), ((N,), F32), ((T, N), BF), "relu", ((T, N), BF)],
    "gemm_gated_into": ["A", "B", "B", ((T, N), BF), "silu", ((T, N), BF), ((T, N), BF)],
}


def arguments(bsq, spec, other):
    """On cuda:0, but the tensor number `other` on cuda:1 (a QTensor is two); returns (arguments, number of tensors)."""
    n, args = 0, []

    def device():
        nonlocal n
        n += 1
        return 1 if n - 1 == other else 0
    for a in spec:
        if a in ("A", "B"):
            args.append(quantized(bsq, T if a == "A" else N, D, (device(), device())))
        else:
            args.append(on(device(), *a[0], dtype=a[1]) if isinstance(a, tuple) else a)
    return args, n


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_on_two_devices_are_refused(bsq, name):
    _, n = arguments(bsq, CALLS[name], -1)
    for other in range(n):
        args, _ = arguments(bsq, CALLS[name], other)
        with pytest.raises(bsq.BsqError, match="cuda:[01]") as e:
            getattr(bsq, name)(*args)
        assert e.value.status == 1, other


@pytest.mark.parametrize("name", sorted(CALLS))
def test_other_shapes_and_types_are_refused(bsq, name):
    spec = CALLS[name]
    for i, a in enumerate(spec):
        if not isinstance(a, tuple):
            continue
        # (a vector may have any shape of as many elements)
        three = a[0] + (1,) if len(a[0]) == 2 else (2, *a[0])
        for shape, dtype in ((a[0][:-1] + (a[0][-1] + 8,), a[1]), (three, a[1]), (a[0], torch.float16), (a[0], I64)):
            args, _ = arguments(bsq, spec, -1)
            args[i] = on(0, *shape, dtype=dtype)
            with pytest.raises(bsq.BsqError):
                getattr(bsq, name)(*args)
                pytest.fail(f"argument {i}: {shape} {dtype}")
    at = next(i for i, a in enumerate(spec) if isinstance(a, str) and a not in ("A", "B"))
    for bad in ("swish", 5, -1):
        args, _ = arguments(bsq, spec, -1)
        args[at] = bad
        with pytest.raises(bsq.BsqError):
            getattr(bsq, name)(*args)
    with pytest.raises(TypeError):
        getattr(bsq, name)(*arguments(bsq, spec, -1)[0][:1])
    if name.startswith("gemm"):
        args, _ = arguments(bsq, spec, -1)
        args[0] = bsq.QTensor(0, T, D + 32, args[0].codes, args[0].scales, None)     # longer than its buffers
        with pytest.raises(bsq.BsqError, match="shorter"):
            getattr(bsq, name)(*args)


def test_adamw_lists_on_two_devices_are_refused(bsq):
    p, g = on(0, 64), on(0, 64)
    m = (on(0, 64), on(0, 64))
    assert bsq.AdamWList([p], [g], [m]).count == 1
    far = on(1, 64)
    for params, grads, states, copies in (([p], [far], [m], None), ([p], [g], [(m[0], far)], None), ([p, far], [g, g], [m, m], None),
                                          ([p], [g], [m], [on(1, 64, dtype=BF)])):
        with pytest.raises(bsq.BsqError, match="cuda:1"):
            bsq.AdamWList(params, grads, states, copies)
    lists = bsq.AdamWList([p], [g], [m])
    for k in (dict(norm=on(1, 1), max_norm=1.0), dict(step=on(1, 1, dtype=I64)), dict(lr=on(1, 1))):
        with pytest.raises(bsq.BsqError, match="cuda:1"):
            bsq.adamw_step(lists, **{**dict(lr=1e-3, step=1), **k})
