"""Operands and results of more than 2^31 elements in products with an epilogue and
their gradients: whole numbers, so that every sum is exact."""
import pytest
import torch

from _ops_ref import Guard, strided

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    yield b
    b.sync_status()
    torch.cuda.empty_cache()


def whole(g, *shape):
    return torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8).to(BF)


@pytest.mark.parametrize("pad", [0, 3])
def test_block_scaled_results(bsq, pad):
    T, N, K = 70001, 32776, 64
    g = torch.Generator(device="cuda").manual_seed(pad)
    x, w, v = whole(g, T, K), whole(g, N, K), whole(g, N, K)
    A, B, C = (bsq.quantize(t, "mxfp8_e4m3")[0] for t in (x, w, v))
    y, z, u = (torch.full((T, N + pad), 77.0, dtype=BF, device="cuda")[:, :N] for _ in range(3))
    tails = [slice(0, 300), slice(65400, 65700), slice(T - 300, T)]

    def want(t):
        return x[t].double() @ w.double().T, x[t].double() @ v.double().T

    bsq.gemm_linear_into(A, B, y, None, None, "relu", z)
    for t in tails:
        a, _ = want(t)
        assert torch.equal(z[t].double(), a) and torch.equal(y[t].double(), a.clamp(min=0))
    bsq.gemm_gated_into(A, B, C, y, "relu", z, u)
    for t in tails:
        a, b = want(t)
        assert torch.equal(z[t].double(), a) and torch.equal(u[t].double(), b)
        assert torch.equal(y[t], (a.clamp(min=0) * b).float().to(BF))


# one and two tokens on the CUDA cores, few and some on the tensor cores
@pytest.mark.parametrize("T", [1, 2, 8, 40])
def test_weights(bsq, T):
    N, K = 600001, 8192
    g = torch.Generator(device="cuda").manual_seed(T)
    x, w = whole(g, T, K), whole(g, N, K)
    tail = slice(N - 500, N)
    want = x.double() @ w[tail].double().T
    A, B = (bsq.quantize(t, "mxfp8_e4m3")[0] for t in (x, w))
    y, buf = strided((T, N), F32, pad=3, fill=float("nan"))
    bsq.gemm_linear_into(A, B, y)
    assert torch.equal(y[:, tail].double(), want)
    Guard(y, buf).check()
    h = bsq.gemm_gated(A, B, B, "identity", F32)
    assert torch.equal(h[:, tail].double(), want * want)
    del A, B, h
    y.fill_(float("nan"))
    bsq.linear_into(x, w, y)
    assert torch.equal(y[:, tail].double(), want)
    Guard(y, buf).check()
    h = bsq.gated_linear(x, w, w, "identity", F32)
    assert torch.equal(h[:, tail].double(), want * want)
    # gradients that come from the last rows of w alone, and go there
    dy = torch.zeros((T, N), dtype=BF, device="cuda")
    dy[:, tail] = whole(g, T, 500)
    dx, dw, _ = bsq.linear_backward(dy, x, w, bias=False)
    assert torch.equal(dx, (dy[:, tail].double() @ w[tail].double()).float().to(BF))
    assert torch.equal(dw[tail], (dy[:, tail].double().T @ x.double()).float().to(BF)) and not dw[:N - 500].any()


def test_gated_gradient(bsq):
    T, N, K = 70001, 32776, 8
    g = torch.Generator(device="cuda").manual_seed(7)
    x, w, v = whole(g, T, K), whole(g, N, K), whole(g, N, K)
    dh, gate, up = (torch.zeros((T, N), dtype=BF, device="cuda") for _ in range(3))
    dh[-1], gate[-1], up[-1] = 1.0, whole(g, N), whole(g, N)
    dx, dg, du = bsq.gated_linear_backward(dh, x, w, v, gate, up, "relu")
    a = (gate[-1] > 0).double() * up[-1].double()
    u = gate[-1].double().clamp(min=0)
    assert torch.equal(dx[-1], (a @ w.double() + u @ v.double()).float().to(BF)) and not dx[:-1].any()
    assert torch.equal(dg.double(), a[:, None] * x[-1].double()) and torch.equal(du.double(), u[:, None] * x[-1].double())
