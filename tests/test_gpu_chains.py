"""Steps of product, gradient and update with nothing between them: each call reads what
the one right before it wrote, weights among them, and gives what it gives with a
wait after every call."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    yield b
    b.sync_status()


def run(bsq, T, D, N, act, wait):
    g = torch.Generator(device="cuda").manual_seed(T + D + N)
    x = torch.randn((T, D), generator=g, device="cuda").to(BF)
    w = (torch.randn((N, D), generator=g, device="cuda") * D ** -0.5).to(BF)
    wu = (torch.randn((N, D), generator=g, device="cuda") * D ** -0.5).to(BF)
    bias = torch.randn(N, generator=g, device="cuda")
    y, z, h, a, u = (torch.empty((T, N), dtype=BF, device="cuda") for _ in range(5))
    dx, dw, dwg, dwu = (torch.empty_like(t) for t in (x, w, w, wu))
    dbias = torch.empty_like(bias)
    first, second = bsq.AdamWList([w, bias], [dw, dbias]), bsq.AdamWList([w, wu], [dwg, dwu], 8)
    keep = []
    for k in range(1, 9):
        bsq.linear_into(x, w, y, bias, None, act, z)
        wait()
        bsq.linear_backward_into(y, x, w, dx, dw, dbias, z, act)
        wait()
        bsq.adamw_step(first, 1e-2, k)
        wait()
        bsq.gated_linear_into(x, w, wu, h, "silu", a, u)
        wait()
        bsq.gated_linear_backward_into(h, x, w, wu, a, u, dx, dwg, dwu)
        wait()
        bsq.adamw_step(second, 1e-2, k, seed=k)
        wait()
        keep += [t.clone() for t in (y, h, dx, dbias)] if k in (1, 8) else []
        wait()
    torch.cuda.synchronize()
    return [*keep, dw, dwg, dwu, w, wu, bias]


# one token to several tiles; sums over K and over the rows in parts
@pytest.mark.parametrize("T,D,N", [(1, 4096, 2048), (2, 2048, 2048), (4, 1024, 1032), (5, 2048, 2040), (60, 64, 72), (130, 1024, 1000),
                                   (500, 4000, 704), (1021, 2040, 1531), (2100, 1024, 4104)])
def test_steps_in_a_row(bsq, T, D, N):
    for act in ("identity", "gelu"):
        want = run(bsq, T, D, N, act, torch.cuda.synchronize)
        assert all(torch.isfinite(t).all() for t in want)
        for _ in range(3):
            got = run(bsq, T, D, N, act, lambda: None)
            assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("T", [1, 2, 3, 40])
@pytest.mark.parametrize("fmt", ["mxfp8_e4m3", "nvfp4"])
def test_quantized_weights_of_the_step_before(bsq, fmt, T):
    g = torch.Generator(device="cuda").manual_seed(T)
    D, N = 2048, 1024
    x, _ = bsq.quantize(torch.randn((T, D), generator=g, device="cuda").to(BF), fmt)
    start = (torch.randn((N, D), generator=g, device="cuda") * D ** -0.5).to(BF)
    grad = torch.randn((N, D), generator=g, device="cuda").to(BF)

    def go(wait):
        w, out = start.clone(), []
        lists = bsq.AdamWList([w], [grad])
        q = bsq.empty(fmt, N, D)
        y = torch.empty((T, N), dtype=BF, device="cuda")
        for k in range(1, 9):
            bsq.adamw_step(lists, 1e-1, k)
            wait()
            bsq.quantize_into(w, fmt, "row", q, None)
            wait()
            bsq.gemm_linear_into(x, q, y, None, None, "silu")
            wait()
            out.append(y.clone())
        torch.cuda.synchronize()
        return out

    want = go(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(go(lambda: None), want))


# dbias beside dx and dw, beside either, alone, of few and many tiles: the same bits
@pytest.mark.parametrize("T,D,N", [(130, 8, 5000), (300, 64, 20000), (1021, 2040, 1531), (4500, 512, 96), (8192, 1024, 6000)])
def test_dbias_is_the_same_beside_every_product(bsq, T, D, N):
    g = torch.Generator(device="cuda").manual_seed(T)
    x, w, dy, z = (torch.randint(-2, 3, s, generator=g, device="cuda").to(BF) for s in ((T, D), (N, D), (T, N), (T, N)))
    want = (dy.double() * (z > 0).double()).sum(0)
    for use_x, use_w in ((1, 1), (1, 0), (0, 1), (0, 0)):
        db = torch.full((N,), float("nan"), device="cuda")
        bsq.linear_backward_into(dy, x, w, torch.empty_like(x) if use_x else None, torch.empty_like(w) if use_w else None, db, z, "relu")
        assert torch.equal(db.double(), want)
