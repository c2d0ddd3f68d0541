"""Linear layers with their epilogue and the gated feed-forward, BF16 operands,
against FP64: one row to several tiles, sizes off every tile, splits of the sum
over K, pitches and addresses without alignment, FP32 and BF16 results, every
activation, both directions, values that are not finite, and sums of whole
numbers, where one element left out shows."""
import pytest
import torch

from _linear_ref import ACTS, gated_grad_ref, gated_ref, linear_grad_ref, linear_ref
from _ops_ref import Guard, assert_close, strided

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# tokens, out, cols: few tokens and tiles, one and several accumulators, sums in parts
SIZES = [(1, 1, 8), (1, 33, 64), (2, 4096, 4096), (3, 130, 72), (16, 96, 8200), (17, 257, 136), (100, 1000, 1024), (128, 300, 264),
         (129, 256, 128), (130, 72, 16384), (200, 511, 1000), (256, 256, 256), (257, 513, 4104), (700, 1537, 640), (1100, 40, 328)]


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    yield b
    b.sync_status()


def gen(*seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(hash(seed) & 0xFFFFFFFF)
    return g


def randn(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def operands(g, T, N, K, weights=1):
    return [randn(g, T, K)] + [randn(g, N, K, scale=2 * K ** -0.5) for _ in range(weights)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_linear(bsq, T, N, K, dtype):
    for i, name in enumerate(ACTS):
        g = gen(T, N, K, i)
        x, w = operands(g, T, N, K)
        bias = [None, randn(g, N, dtype=F32), randn(g, N)][i % 3]
        res = randn(g, T, N, dtype=dtype) if i % 2 else None
        # rows that suit 16-byte stores where N does, and rows that do not
        y, ybuf = strided((T, N), dtype, pad=(-N) % 8 if i % 2 == 0 else 1, offset=0 if i % 2 == 0 else 1, fill=float("nan"))
        z, zbuf = strided((T, N), BF, pad=(-N) % 8 if i < 3 else 3, offset=0 if i < 3 else 5, fill=float("nan"))
        keep = i != 1
        assert bsq.linear_into(x, w, y, bias, res, name, z if keep else None)[0] is y
        want, tol, zw, zt = linear_ref(x, w, bias, res, name, dtype)
        assert_close(y, want, tol, f"y {name}")
        Guard(y, ybuf).check()
        if keep:
            assert_close(z, zw, zt, f"z {name}")
            Guard(z, zbuf).check()
        if i == 3:                                     # the residual's own place
            r = res.clone()
            bsq.linear_into(x, w, r, bias, r, name)
            assert torch.equal(r, y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_gated(bsq, T, N, K, dtype):
    for i, name in enumerate(ACTS):
        g = gen(T, N, K, 10 + i)
        x, wg, wu = operands(g, T, N, K, 2)
        h, hbuf = strided((T, N), dtype, pad=(-N) % 8 if i % 2 == 0 else 1, offset=0 if i % 2 == 0 else 1, fill=float("nan"))
        a, abuf = strided((T, N), BF, pad=(-N) % 8 if i < 3 else 3, offset=0 if i < 3 else 5, fill=float("nan"))
        u, ubuf = strided((T, N), BF, pad=(-N) % 8 if i > 1 else 1, fill=float("nan"))
        keep = i != 1
        bsq.gated_linear_into(x, wg, wu, h, name, a if keep else None, u if keep else None)
        want, tol, aw, at, uw, ut = gated_ref(x, wg, wu, name, dtype)
        assert_close(h, want, tol, f"h {name}")
        Guard(h, hbuf).check()
        if keep:
            assert_close(a, aw, at, "gate")
            assert_close(u, uw, ut, "up")
            Guard(a, abuf).check()
            Guard(u, ubuf).check()


@pytest.mark.parametrize("T,N,K", SIZES)
def test_linear_gradient(bsq, T, N, K):
    for i, name in enumerate(ACTS):
        g = gen(T, N, K, 20 + i)
        x, w = operands(g, T, N, K)
        pad = 0 if i % 2 else 1 + (-N) % 8
        dy, _ = strided((T, N), BF, pad=pad, offset=0 if i % 2 else 3, gen=g)
        z = None if name == "identity" else strided((T, N), BF, pad=pad, gen=g, scale=2.0)[0]
        dx, xbuf = strided((T, K), BF, pad=8 * (i % 2), fill=float("nan"))
        dw, wbuf = strided((N, K), BF, pad=8 * (i % 2), fill=float("nan"))
        db = torch.full((N,), float("nan"), device="cuda")
        bsq.linear_backward_into(dy, x, w, dx, dw, db, z, name)
        xr, xt, wr, wt, br, bt = linear_grad_ref(dy, x, w, z, name)
        assert_close(dx, xr, xt, f"dx {name}")
        assert_close(dw, wr, wt, f"dw {name}")
        assert_close(db, br, bt, f"dbias {name}")
        Guard(dx, xbuf).check()
        Guard(dw, wbuf).check()
        # each of them alone
        for only in range(3):
            a, b, c = (torch.full_like(t, float("nan")) if k == only else None for k, t in enumerate((dx, dw, db)))
            bsq.linear_backward_into(dy, x if only == 1 else None, w if only != 1 else None, a, b, c, z, name)
            assert torch.equal([a, b, c][only], [dx, dw, db][only])


@pytest.mark.parametrize("T,N,K", SIZES)
def test_gated_gradient(bsq, T, N, K):
    for i, name in enumerate(ACTS):
        g = gen(T, N, K, 30 + i)
        x, wg, wu = operands(g, T, N, K, 2)
        pad = 0 if i % 2 else 1 + (-N) % 8
        dh, _ = strided((T, N), BF, pad=pad, offset=0 if i % 2 else 3, gen=g)
        gate, up = (strided((T, N), BF, pad=pad, gen=g, scale=2.0)[0] for _ in range(2))
        dx, xbuf = strided((T, K), BF, pad=8 * (i % 2), fill=float("nan"))
        dg, gbuf = strided((N, K), BF, pad=8 * (i % 2), fill=float("nan"))
        du, ubuf = strided((N, K), BF, pad=16, fill=float("nan"))
        bsq.gated_linear_backward_into(dh, x, wg, wu, gate, up, dx, dg, du, name)
        xr, xt, gr, gt, ur, ut = gated_grad_ref(dh, x, wg, wu, gate, up, name)
        assert_close(dx, xr, xt, f"dx {name}")
        assert_close(dg, gr, gt, f"dw_gate {name}")
        assert_close(du, ur, ut, f"dw_up {name}")
        for m, b in ((dx, xbuf), (dg, gbuf), (du, ubuf)):
            Guard(m, b).check()
        only = torch.empty_like(dx)
        bsq.gated_linear_backward_into(dh, None, wg, wu, gate, up, only, None, None, name)
        assert torch.equal(only, dx)
        a, b = torch.empty_like(dg), torch.empty_like(du)
        bsq.gated_linear_backward_into(dh, x, None, None, gate, up, None, a, b, name)
        assert torch.equal(a, dg) and torch.equal(b, du)


@pytest.mark.parametrize("T,N,K", [(1, 1000, 4096), (5, 300, 40), (128, 257, 8192), (129, 300, 264), (520, 700, 8456), (300, 80, 20000)])
def test_sums_of_whole_numbers(bsq, T, N, K):
    # -1, 0, 1: every sum below 2^24 is exact in FP32, in whatever order
    g = gen(T, N, K)
    x, w, v = (torch.randint(-1, 2, s, generator=g, device="cuda").to(BF) for s in ((T, K), (N, K), (N, K)))
    z, u = x.double() @ w.double().T, x.double() @ v.double().T
    bias = torch.randint(-9, 10, (N,), generator=g, device="cuda").float()
    res = torch.randint(-99, 100, (T, N), generator=g, device="cuda").float()
    y = bsq.linear(x, w, bias, res, "relu", F32)
    assert torch.equal(y.double(), (z + bias.double()).clamp(min=0) + res.double())
    h = torch.empty((T, N), device="cuda")
    a, b = (torch.empty((T, N), dtype=BF, device="cuda") for _ in range(2))
    bsq.gated_linear_into(x, w, v, h, "relu", a, b)
    assert torch.equal(h, (z.clamp(min=0) * u).float())
    assert torch.equal(a, z.float().to(BF)) and torch.equal(b, u.float().to(BF))
    d = torch.randint(-1, 2, (T, N), generator=g, device="cuda").to(BF)
    dx, dw, db = bsq.linear_backward(d, x, w)
    assert torch.equal(dx, (d.double() @ w.double()).float().to(BF))
    assert torch.equal(dw, (d.double().T @ x.double()).float().to(BF))
    assert torch.equal(db, d.double().sum(0).float())
    one = torch.ones((T, N), dtype=BF, device="cuda")
    dx, dg, du = bsq.gated_linear_backward(d, x, w, v, one, -one, "identity")
    assert torch.equal(dx, (-d.double() @ w.double() + d.double() @ v.double()).float().to(BF))
    assert torch.equal(dg, (-d.double().T @ x.double()).float().to(BF))
    assert torch.equal(du, (d.double().T @ x.double()).float().to(BF))


# which of the outputs are on 16-byte rows (bit 0: y or h, 1: z or gate, 2: up): a warp's stores go two ways in turn
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows16", range(8))
@pytest.mark.parametrize("N", [520, 515])
def test_outputs_on_rows_of_different_alignment(bsq, N, rows16, dtype):
    # small whole numbers, exact in BF16: sums up to 16, products up to 256
    T, K = 2500, 16
    g = gen(N, rows16, 50)
    x, w, v = (torch.randint(-1, 2, s, generator=g, device="cuda").to(BF) for s in ((T, K), (N, K), (N, K)))
    a, u = x.double() @ w.double().T, x.double() @ v.double().T

    def out(bit, t):
        whole = rows16 >> bit & 1
        return strided((T, N), t, pad=(-N) % 8 if whole else 3, offset=0 if whole else 1, fill=float("nan"))

    (y, yb), (z, zb), (s, sb) = out(0, dtype), out(1, BF), out(2, BF)
    bsq.linear_into(x, w, y, None, None, "relu", z)
    assert torch.equal(z.double(), a) and torch.equal(y.double(), a.clamp(min=0))
    y.fill_(float("nan"))
    z.fill_(float("nan"))
    bsq.gated_linear_into(x, w, v, y, "relu", z, s)
    assert torch.equal(z.double(), a) and torch.equal(s.double(), u) and torch.equal(y.double(), a.clamp(min=0) * u)
    for m, b in ((y, yb), (z, zb), (s, sb)):
        Guard(m, b).check()


@pytest.mark.parametrize("T", [3, 200])
def test_values_that_are_not_finite_stay_in_their_rows(bsq, T):
    g = gen(T)
    x, wg, wu = operands(g, T, 300, 128, 2)
    clean = bsq.gated_linear(x, wg, wu), bsq.linear(x, wg, None, None, "gelu")
    x[1, 5] = float("nan")
    wg[7, 3] = float("inf")
    for got, want in zip((bsq.gated_linear(x, wg, wu), bsq.linear(x, wg, None, None, "gelu")), clean):
        assert torch.isnan(got[1]).all()
        keep = torch.ones((T, 300), dtype=torch.bool, device="cuda")
        keep[1] = False
        keep[:, 7] = False
        assert torch.equal(got[keep], want[keep])
    z = bsq.linear(x, wg)
    rows = [i for i in range(T) if i != 1]
    assert torch.equal(z[rows, 7].float(), torch.where(x[rows, 3] > 0, float("inf"), -float("inf")))


# tiles of 64 to 256 columns and 64 to 256 rows, whole and in parts
@pytest.mark.parametrize("T,N,K", [(40, 6000, 264), (40, 1000, 4104), (257, 4100, 264), (40, 1537, 4104), (257, 6000, 1000), (40, 6000, 4104),
                                   (520, 4100, 1000), (40, 2500, 8200), (1030, 3001, 1000), (40, 4100, 8200), (520, 6000, 1000),
                                   (40, 2500, 20000), (100, 513, 4104), (150, 2050, 8200), (190, 1000, 20000), (70, 2500, 264)])
def test_tiles_of_every_size(bsq, T, N, K):
    # -1, 0, 1: every sum is exact in FP32, and a result is rounded once
    g = gen(T, N, K, 91)
    x, w, v = (torch.randint(-1, 2, s, generator=g, device="cuda").to(BF) for s in ((T, K), (N, K), (N, K)))
    a, u = x.double() @ w.double().T, x.double() @ v.double().T
    for dtype in (BF, F32):
        res = torch.randint(-99, 100, (T, N), generator=g, device="cuda").to(dtype)
        z = torch.empty((T, N), dtype=BF, device="cuda")
        y = torch.empty((T, N), dtype=dtype, device="cuda")
        bsq.linear_into(x, w, y, None, res, "relu", z)
        assert torch.equal(y, (a.clamp(min=0) + res.double()).to(dtype)) and torch.equal(z, a.to(BF))
        h, gate, up = torch.empty_like(y), torch.empty_like(z), torch.empty_like(z)
        bsq.gated_linear_into(x, w, v, h, "relu", gate, up)
        assert torch.equal(h, (a.clamp(min=0) * u).to(dtype)) and torch.equal(gate, z) and torch.equal(up, u.to(BF))


@pytest.mark.parametrize("T,N,K", [(2600, 2600, 8200), (9000, 72, 264), (40, 9000, 1032)])
def test_gradients_of_many_tiles(bsq, T, N, K):
    # dx and dw in one launch, or in two; -1, 0, 1, so that every sum is exact
    g = gen(T, N, K, 90)
    x, w, v, d = (torch.randint(-1, 2, s, generator=g, device="cuda").to(BF) for s in ((T, K), (N, K), (N, K), (T, N)))
    dx, dw, db = bsq.linear_backward(d, x, w)
    xf, wf, vf, df = (t.double() for t in (x, w, v, d))
    assert torch.equal(dx, (df @ wf).float().to(BF)) and torch.equal(dw, (df.T @ xf).float().to(BF))
    assert torch.equal(db, df.sum(0).float())
    one = torch.ones((T, N), dtype=BF, device="cuda")
    dx, dg, du = bsq.gated_linear_backward(d, x, w, v, one, -one, "identity")
    assert torch.equal(dx, (df @ vf - df @ wf).float().to(BF))
    assert torch.equal(dg, -(df.T @ xf).float().to(BF)) and torch.equal(du, (df.T @ xf).float().to(BF))


@pytest.mark.parametrize("pad", [0, 3])
def test_results_of_more_than_2_31_elements(bsq, pad):
    # whole numbers; the last rows and columns lie past 2^31 elements
    T, N, K = 70001, 32776, 8
    g = gen(pad, 60)
    x, w, v = (torch.randint(-1, 2, s, generator=g, device="cuda").to(BF) for s in ((T, K), (N, K), (N, K)))
    y, z, u = (torch.full((T, N + pad), 77.0, dtype=BF, device="cuda")[:, :N] for _ in range(3))
    tail = slice(T - 300, T)
    a, b = x[tail].double() @ w.double().T, x[tail].double() @ v.double().T
    bsq.linear_into(x, w, y, None, None, "relu", z)
    assert torch.equal(z[tail].double(), a) and torch.equal(y[tail].double(), a.clamp(min=0))
    bsq.gated_linear_into(x, w, v, y, "relu", z, u)
    assert torch.equal(z[tail].double(), a) and torch.equal(u[tail].double(), b) and torch.equal(y[tail].double(), a.clamp(min=0) * b)
    # gradients: dy is 1 in the last row and 0 elsewhere
    y.zero_()
    y[-1] = 1.0
    z[tail] = a.to(BF)
    dx, dw, db = bsq.linear_backward(y, x, w, z, "relu")
    s = (a[-1] > 0).double()
    assert torch.equal(dx[-1], (s @ w.double()).float().to(BF)) and not dx[:-1].any()
    assert torch.equal(dw, (s[:, None] * x[-1].double()).to(BF)) and torch.equal(db, s.float())


@pytest.mark.parametrize("name", ACTS)
def test_large_values(bsq, name):
    # pre-activations from -1e4 to 1e4 through a product with the unit matrix
    v = torch.cat([torch.linspace(-12, 12, 200), torch.tensor([-1e4, -100.0, -50.0, 0.0, -0.0, 50.0, 100.0, 1e4])]).to(BF).cuda()
    n = v.numel()
    x = torch.zeros((n, n), dtype=BF, device="cuda")
    x.diagonal().copy_(v)
    eye = torch.eye(n, dtype=BF, device="cuda")
    want, tol, _, _ = linear_ref(x, eye, None, None, name, F32)
    assert_close(bsq.linear(x, eye, None, None, name, F32), want, tol, name)
    dy = torch.ones((n, n), dtype=BF, device="cuda")
    xr, xt, *_ = linear_grad_ref(dy, x, eye, x, name)
    assert_close(bsq.linear_backward(dy, x, eye, x, name)[0], xr, xt, name)


@pytest.mark.parametrize("name", ACTS)
def test_the_types_lowest_and_highest_values(bsq, name):
    # pre-activations at BF16's ends: the activation is 0 or the value itself, its slope 0 or 1
    top = torch.finfo(BF).max
    v = torch.tensor([-top, -1e30, 1e30, top], dtype=BF, device="cuda").repeat(20)
    n = v.numel()
    x = torch.zeros((n, n), dtype=BF, device="cuda")
    x.diagonal().copy_(v)
    eye = torch.eye(n, dtype=BF, device="cuda")
    want = v.float() if name == "identity" else v.float().clamp(min=0)
    for T in (1, 3, n):
        got = bsq.linear(x[:T], eye, None, None, name, F32)
        assert torch.equal(got.diagonal(), want[:T]) and int((got != 0).sum()) == int((want[:T] != 0).sum())
        dx = bsq.linear_backward(torch.ones((T, n), dtype=BF, device="cuda"), x[:T], eye, x[:T].contiguous(), name)[0]
        slope = torch.ones(n, device="cuda") if name == "identity" else (v > 0).float()
        assert torch.equal(dx.float().diagonal(), slope[:T])


# what the choice of a kernel goes by: 4 and 5, 16 and 17, 128 and 129 tokens, products of 4096 and 16384 elements
@pytest.mark.parametrize("T,N,K", [(4, 5, 8), (5, 1, 8), (5, 3276, 64), (5, 3277, 64), (16, 1024, 200), (17, 240, 72), (17, 241, 72),
                                   (128, 1, 16), (128, 32, 1000), (128, 33, 32), (129, 1, 8), (129, 32, 32), (300, 3, 8), (4, 8000, 1032)])
def test_sizes_at_the_borders(bsq, T, N, K):
    g = gen(T, N, K, 77)
    x, w, v = operands(g, T, N, K, 2)
    bias = randn(g, N, dtype=F32)
    want, tol, _, _ = linear_ref(x, w, bias, None, "gelu_tanh", BF)
    assert_close(bsq.linear(x, w, bias, None, "gelu_tanh"), want, tol, "y")
    want, tol, *_ = gated_ref(x, w, v, "silu", BF)
    assert_close(bsq.gated_linear(x, w, v), want, tol, "h")
    dy, a, b = (randn(g, T, N) for _ in range(3))
    want = linear_grad_ref(dy, x, w, a, "gelu")
    for got, r, t, what in zip(bsq.linear_backward(dy, x, w, a, "gelu"), want[::2], want[1::2], ("dx", "dw", "dbias")):
        assert_close(got, r, t, what)
    want = gated_grad_ref(dy, x, w, v, a, b, "silu")
    for got, r, t, what in zip(bsq.gated_linear_backward(dy, x, w, v, a, b), want[::2], want[1::2], ("dx", "dw_gate", "dw_up")):
        assert_close(got, r, t, what)


def test_gradients_against_differences(bsq):
    # the loss sum(c * f) of the forward calls in FP64, moved along a direction
    from _linear_ref import act
    g = gen(9)
    T, N, K = 70, 90, 64
    x, wg, wu = operands(g, T, N, K, 2)
    c = randn(g, T, N)
    a, u = (torch.empty((T, N), dtype=BF, device="cuda") for _ in range(2))
    bsq.gated_linear_into(x, wg, wu, torch.empty_like(a), "silu", a, u)
    got = bsq.gated_linear_backward(c, x, wg, wu, a, u)
    at = [t.double() for t in (x, wg, wu)]

    def loss(t):
        return float((c.double() * act("silu", t[0] @ t[1].T)[0] * (t[0] @ t[2].T)).sum())

    for i, dt in enumerate(got):
        v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-6
        moved = [[t + s * step * v if k == i else t for k, t in enumerate(at)] for s in (1, -1)]
        slope = (loss(moved[0]) - loss(moved[1])) / (2 * step)
        # the gradient's BF16 parts: gate and up as they were kept, dgate and dup, and its own rounding; independent,
        # so their sum along a random direction stays within 6 of its deviations (2^-9 each, four of them)
        scale = float((dt.double().square().sum() * v.square().mean()).sqrt())
        assert abs(float((dt.double() * v).sum()) - slope) <= 6 * 2 * 2.0 ** -9 * scale * 2
