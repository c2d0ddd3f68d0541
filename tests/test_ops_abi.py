"""Host-side argument checks of the operators around the layer (no GPU: a
rejected call launches nothing) and their workspace sizes."""
import ctypes

import pytest

P = ctypes.c_void_p
NULL = None


@pytest.fixture(scope="module")
def bsq():
    from block_scaled_precision_03_gb300 import _build
    import block_scaled_precision_03_gb300 as b
    _build.build()
    b.lib()
    return b


def test_moe_checks(bsq):
    L = bsq.lib()
    from block_scaled_precision_03_gb300.ops import BsqMoePlanC as Plan
    n = L.bsq_moe_workspace_bytes(4096, 8, 64)
    assert n > 0 and L.bsq_moe_workspace_bytes(0, 8, 64) == 0 and L.bsq_moe_workspace_bytes(4, 257, 64) == 0
    assert L.bsq_moe_workspace_bytes(1 << 31, 2, 64) == 0 and L.bsq_moe_workspace_bytes(4, 2, 1025) == 0
    good = Plan(4096, 8, 64, 256, 256, 256)
    ref = ctypes.byref
    assert L.bsq_moe_sort(NULL, 1, ref(good), 256, n, NULL) == 1
    assert L.bsq_moe_sort(256, 2, ref(good), 256, n, NULL) == 1
    assert L.bsq_moe_sort(260, 1, ref(good), 256, n, NULL) == 3
    assert L.bsq_moe_sort(256, 1, NULL, 256, n, NULL) == 1
    assert L.bsq_moe_sort(256, 1, ref(good), NULL, n, NULL) == 1
    assert L.bsq_moe_sort(256, 1, ref(good), 256, n - 1, NULL) == 1
    assert L.bsq_moe_sort(256, 1, ref(good), 264, n, NULL) == 3
    for bad, status in ((Plan(0, 8, 64, 256, 256, 256), 1), (Plan(4, 0, 64, 256, 256, 256), 1),
                        (Plan(4, 8, 0, 256, 256, 256), 1), (Plan(4, 8, 64, NULL, 256, 256), 1),
                        (Plan(4, 8, 64, 260, 256, 256), 3), (Plan(4, 8, 64, 256, 258, 256), 3),
                        (Plan(4, 257, 64, 256, 256, 256), 2), (Plan(4, 8, 1025, 256, 256, 256), 2),
                        (Plan(1 << 30, 8, 64, 256, 256, 256), 2)):
        assert L.bsq_moe_sort(256, 1, ref(bad), 256, 1 << 40, NULL) == status
        assert L.bsq_moe_gather(256, 16, 1, 16, ref(bad), 256, 16, NULL) == status
    assert L.bsq_moe_gather(256, 15, 1, 16, ref(good), 256, 16, NULL) == 1          # pitch below the width
    assert L.bsq_moe_gather(256, 16, 7, 16, ref(good), 256, 16, NULL) == 1
    assert L.bsq_moe_gather(257, 16, 1, 16, ref(good), 256, 16, NULL) == 3
    assert L.bsq_moe_gather(256, 16, 0, 16, ref(good), 258, 16, NULL) == 3
    assert L.bsq_moe_gather(256, 16, 1, 0, ref(good), 256, 16, NULL) == 1
    assert L.bsq_moe_combine(256, 16, 1, 16, 258, ref(good), 256, 16, NULL) == 3
    assert L.bsq_moe_combine_backward(256, 16, NULL, 16, 1, 16, 256, ref(good), 256, 16, 256, NULL) == 1
    assert L.bsq_moe_combine_backward(256, 16, 256, 16, 1, 16, NULL, ref(good), 256, 16, 256, NULL) == 1
    assert L.bsq_moe_dispatch(256, 16, 1, 16, 256, 1, ref(good), 256, 16, 256, 0, NULL) == 1


def test_norm_checks(bsq):
    L = bsq.lib()
    n = L.bsq_layer_norm_workspace_bytes(100, 64)
    assert n > 0 and L.bsq_layer_norm_workspace_bytes(0, 64) == 0 and L.bsq_layer_norm_workspace_bytes(4, 0) == 0
    f = lambda **k: L.bsq_layer_norm(*{**dict(x=256, ldx=64, t=1, r=4, c=64, w=256, b=256, pt=0, eps=1e-5, y=256,  # noqa: E731
                                              ldy=64, m=256, s=256, st=NULL), **k}.values())
    assert f(x=NULL) == 1 and f(y=NULL) == 1 and f(t=2) == 1 and f(pt=-1) == 1 and f(r=0) == 1 and f(c=0) == 1
    assert f(ldx=63) == 1 and f(ldy=63) == 1 and f(eps=-1.0) == 1 and f(eps=float("nan")) == 1
    assert f(eps=float("inf")) == 1 and f(x=257) == 3 and f(y=257) == 3 and f(w=258) == 3 and f(b=258) == 3
    assert f(m=258) == 3 and f(s=258) == 3 and f(r=1 << 31) == 2
    g = lambda **k: L.bsq_layer_norm_backward(*{**dict(dy=256, ldd=64, x=256, ldx=64, t=1, r=100, c=64, w=256, pt=0,  # noqa: E731
                                                       m=256, s=256, dx=256, lddx=64, dw=256, db=256, ws=256, n=n,
                                                       st=NULL), **k}.values())
    assert g(dy=NULL) == 1 and g(m=NULL) == 1 and g(s=NULL) == 1 and g(dx=NULL) == 1 and g(ws=NULL) == 1
    assert g(n=n - 1) == 1 and g(ws=260) == 3 and g(dw=258) == 3 and g(lddx=3) == 1


def test_head_checks(bsq):
    L = bsq.lib()
    size = L.bsq_linear_cross_entropy_workspace_bytes
    n, m = size(100, 1000, 64, 0), size(100, 1000, 64, 1)
    assert n > 0 and m > 0 and size(0, 10, 8, 0) == 0 and size(4, 1 << 31, 8, 1) == 0
    # the backward pass keeps one piece of the vocabulary, not the logits
    assert size(8192, 1 << 20, 4096, 1) < 8192 * (1 << 20) // 8
    f = lambda **k: L.bsq_linear_cross_entropy(*{**dict(h=256, ldh=64, w=256, ldw=64, t=256, T=100, V=1000, D=64,  # noqa: E731
                                                        loss=256, lse=256, ws=256, n=n, st=NULL), **k}.values())
    assert f(h=NULL) == 1 and f(w=NULL) == 1 and f(t=NULL) == 1 and f(loss=NULL) == 1 and f(lse=NULL) == 1
    assert f(T=0) == 1 and f(V=0) == 1 and f(D=0) == 1 and f(ldh=56) == 1 and f(ldw=56) == 1
    assert f(h=264) == 3 and f(w=264) == 3 and f(ldh=68) == 3 and f(ldw=68) == 3 and f(D=60) == 3 and f(t=260) == 3
    assert f(V=1 << 31) == 2


def test_clip_checks(bsq):
    L = bsq.lib()
    from block_scaled_precision_03_gb300.ops import BsqGradC as G
    n = L.bsq_grad_workspace_bytes(2)
    assert n > 0 and L.bsq_grad_workspace_bytes(0) == 0 and L.bsq_grad_workspace_bytes((1 << 20) + 1) == 0
    f = lambda a, b, norm=256, ws=256, n=n, mx=1.0, eps=0.0, count=2: L.bsq_clip_grad_norm(  # noqa: E731
        (G * 2)(a, b), count, mx, eps, norm, ws, n, NULL)
    ok = G(256, 256, 10, 0, 0)
    assert f(ok, ok, norm=NULL) == 1 and f(ok, ok, norm=258) == 3 and f(ok, ok, ws=NULL) == 1
    assert f(ok, ok, ws=264) == 3 and f(ok, ok, n=n - 1) == 1 and f(ok, ok, count=0) == 1
    assert f(ok, ok, mx=-1.0) == 1 and f(ok, ok, mx=float("nan")) == 1 and f(ok, ok, eps=-1.0) == 1
    assert f(ok, G(NULL, 256, 10, 0, 0)) == 1 and f(ok, G(256, NULL, 10, 0, 0)) == 1
    assert f(ok, G(256, 256, -1, 0, 0)) == 1 and f(ok, G(256, 256, 10, 5, 0)) == 1
    assert f(ok, G(256, 256, 10, 0, 1)) == 1 and f(ok, G(258, 256, 10, 0, 0)) == 3
    assert f(ok, G(256, 257, 10, 1, 0)) == 3 and f(ok, G(256, 256, 1 << 41, 0, 0)) == 2
