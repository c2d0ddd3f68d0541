"""Layer norm forward and backward against FP64 with bounds from the formula,
at one row and one column, odd widths, pitches and addresses, rows of one
value, and the gradient also against differences."""
import pytest
import torch

from _ops_ref import Guard, assert_close, norm_grad_ref, norm_ref, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    return b


SHAPES = [(1, 1), (3, 2), (1, 7168), (5, 3), (7, 31), (300, 64), (9, 100), (33, 257), (700, 1000), (2, 1024),
          (1300, 136), (160, 4096), (11, 4104), (3, 8192), (2, 14336), (3, 20000), (2, 40001), (2, 70000), (5000, 24)]


def params(kind, C, g):
    w = 1 + 0.5 * torch.randn(C, generator=g, device="cuda")
    b = torch.randn(C, generator=g, device="cuda")
    if kind == "bf16":
        return w.bfloat16(), b.bfloat16()
    return {"f32": (w, b), "none": (None, None), "weight": (w, None), "bias": (None, b)}[kind]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("pad,offset,kind", [(0, 0, "f32"), (8, 8, "bf16"), (5, 1, "f32"), (0, 0, "none"),
                                             (0, 0, "weight"), (0, 0, "bias")])
def test_forward(bsq, R, C, dtype, pad, offset, kind):
    g = torch.Generator(device="cuda").manual_seed(R + C)
    x, _ = strided((R, C), dtype, pad, offset, gen=g, scale=3.0)
    x += 5.0
    x[R // 2] = 1.0 if C % 2 else 0.1                   # a row of one value: var is 0 or rounding
    w, b = params(kind, C, g)
    eps = 1e-5
    y, buf = strided((R, C), dtype, pad, offset, fill=float("nan"))
    mean = torch.full((R,), float("nan"), device="cuda")
    rstd = torch.full((R,), float("nan"), device="cuda")
    bsq.layer_norm_into(x, w, b, eps, y, mean, rstd)
    ry, rm, rr, tol, tm, tr = norm_ref(x, w, b, eps)
    assert_close(y, ry, tol, "y")
    assert_close(mean, rm, tm, "mean")
    assert_close(rstd, rr, tr, "rstd")
    Guard(y, buf).check()
    y2 = x.clone()
    bsq.layer_norm_into(y2, w, b, eps, y2)              # in place, without the statistics
    assert torch.equal(y2, bsq.layer_norm(x.contiguous(), w, b, eps)[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("pad,offset,kind", [(0, 0, "f32"), (8, 8, "bf16"), (5, 1, "f32"), (0, 0, "none")])
def test_backward(bsq, R, C, dtype, pad, offset, kind):
    g = torch.Generator(device="cuda").manual_seed(R + C + 1)
    x, _ = strided((R, C), dtype, pad, offset, gen=g, scale=2.0)
    dy, _ = strided((R, C), dtype, pad, offset, gen=g)
    w, _ = params(kind, C, g)
    xd = x.double()
    mean = xd.mean(1).float()
    rstd = (1 / (xd.var(1, unbiased=False) + 1e-5).sqrt()).float()
    dx, buf = strided((R, C), dtype, pad, offset, fill=float("nan"))
    dw, db = (torch.full((C,), float("nan"), device="cuda") for _ in range(2))
    bsq.layer_norm_backward_into(dy, x, w, mean, rstd, dx, dw, db)
    rx, tx, rw, tw, rb, tb = norm_grad_ref(dy, x, w, mean, rstd)
    assert_close(dx, rx, tx, "dx")
    assert_close(dw, rw, tw, "dweight")
    assert_close(db, rb, tb, "dbias")
    Guard(dx, buf).check()
    # each column gradient alone, none, and dx in the place of dy: the same bits
    one, two = torch.empty_like(dw), torch.empty_like(db)
    d2 = dy.clone()
    bsq.layer_norm_backward_into(d2, x, w, mean, rstd, d2, one, None)
    assert torch.equal(d2, dx) and torch.equal(one, dw)
    bsq.layer_norm_backward_into(dy, x, w, mean, rstd, d2, None, two)
    assert torch.equal(d2, dx) and torch.equal(two, db)
    bsq.layer_norm_backward_into(dy, x, w, mean, rstd, d2.fill_(0))
    assert torch.equal(d2, dx)


@pytest.mark.parametrize("R,C,kind", [(400, 9000, "f32"), (350, 16384, "bf16"), (2, 8200, "none"), (1, 12288, "f32"),
                                      (311, 14336, "f32")])
def test_backward_of_long_rows(bsq, R, C, kind):
    test_backward(bsq, R, C, torch.bfloat16, 0, 0, kind)
    test_backward(bsq, R, C, torch.bfloat16, 8, 8, kind)


def test_large_mean_keeps_the_variance(bsq):
    # values 1000 +- 2^-9 (exact in FP32): a variance by differences of squares would be lost
    x = torch.full((4, 4096), 1000.0, device="cuda")
    x[:, ::2] += 2.0 ** -9
    x[:, 1::2] -= 2.0 ** -9
    y, mean, rstd = bsq.layer_norm(x, eps=0.0)
    ry, rm, rr, tol, tm, tr = norm_ref(x, None, None, 0.0)
    assert_close(y, ry, tol)
    # the mean is exact here (pairs cancel), so the tighter bound holds too
    assert (mean == 1000.0).all() and ((rstd - 512.0).abs() <= 512 * 2.0 ** -20).all()


def test_nan_and_inf_stay_in_their_rows(bsq):
    x = torch.randn((6, 513), device="cuda")
    x[1, 7], x[3, 500], x[4, 0] = float("nan"), float("inf"), float("-inf")
    y, mean, rstd = bsq.layer_norm(x)
    bad = torch.tensor([1, 3, 4], device="cuda")
    assert torch.isnan(y[bad]).all()
    good = torch.tensor([0, 2, 5], device="cuda")
    ref = norm_ref(x[good], None, None, 1e-5)
    assert_close(y[good], ref[0], ref[3])


def test_gradient_against_differences(bsq):
    g = torch.Generator(device="cuda").manual_seed(3)
    R, C, eps, h = 13, 77, 1e-5, 1e-5
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w, b, dy = rnd(R, C), 1 + 0.3 * rnd(C), rnd(C), rnd(R, C)
    _, mean, rstd = bsq.layer_norm(x, w, b, eps)
    dx, dw, db = bsq.layer_norm_backward(dy, x, w, mean, rstd)

    def f(x, w, b):
        c = x - x.mean(1, keepdim=True)
        return ((c / (c.square().mean(1, keepdim=True) + eps).sqrt() * w + b) * dy.double()).sum()
    X, W, B = x.double(), w.double(), b.double()
    for grad, at in ((dx, 0), (dw, 1), (db, 2)):
        d = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        args = [X, W, B]
        hi, lo = list(args), list(args)
        hi[at], lo[at] = args[at] + h * d, args[at] - h * d
        want = (f(*hi) - f(*lo)) / (2 * h)
        # FP32 gradient: C + R roundings of terms no larger than 10; the difference: h^2 and 1e-16 / h
        tol = (C + R + 10) * 2.0 ** -24 * 10 * d.abs().sum() + 1e-6 * d.abs().sum()
        assert abs(want - (grad.double() * d).sum()) <= tol


def test_refusals(bsq):
    x = torch.zeros((4, 16), device="cuda")
    w = torch.ones(16, device="cuda")
    m = torch.zeros(4, device="cuda")
    bad = [lambda: bsq.layer_norm(x.half()), lambda: bsq.layer_norm(x.t()), lambda: bsq.layer_norm(x.cpu()),
           lambda: bsq.layer_norm(x, w[:8]), lambda: bsq.layer_norm(x, w, w.bfloat16()),
           lambda: bsq.layer_norm(x, w, eps=-1.0), lambda: bsq.layer_norm(x, w, eps=float("nan")),
           lambda: bsq.layer_norm(x[:0]), lambda: bsq.layer_norm(x[:, :0]),
           lambda: bsq.layer_norm(x[:1].expand(4, 16)), lambda: bsq.layer_norm(x.view(4, 4, 4)),
           lambda: bsq.layer_norm_into(x, w, None, 1e-5, torch.zeros((4, 16), dtype=torch.bfloat16, device="cuda")),
           lambda: bsq.layer_norm_backward(x, x, w, m[:3], m), lambda: bsq.layer_norm_backward(x, x.bfloat16(), w, m, m),
           lambda: bsq.layer_norm_backward(x[:3], x, w, m, m), lambda: bsq.layer_norm_backward(x, x, w, None, m)]
    for i, f in enumerate(bad):
        with pytest.raises(bsq.BsqError):
            f()
            pytest.fail(f"case {i} was not refused")
