"""Long sums of block-scaled products with an epilogue, of operands of one sign, where
what a truncated addition loses adds up: FP32 results keep their accuracy whatever
K, and sums of whole numbers are exact, in one accumulator or several."""
import pytest
import torch

from _ops_ref import U, assert_close

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# An accumulator takes 128 products of the tensor cores: 16 stages of 8 in FP8 (K = 4096), 32 of 4 in FP4 (8192).  Each
# addition is truncated, off by at most an ulp (2 U) of the sum so far; of operands that are alike along K that sum grows
# evenly, to half of the whole in the mean (1.1: unevenness).  The accumulators are added in FP32: U each of the sum so
# far.  Scales and products of a block are exact, and so are MXFP4's sums.
PER_SUM = 1.1 * 128 / 2 * 2 * U


def bound(parts):
    return PER_SUM + (parts + 2) * U


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    yield b
    b.sync_status()


def operand(bsq, g, rows, cols, fmt):
    q, _ = bsq.quantize(torch.rand((rows, cols), generator=g, device="cuda").to(BF), fmt)
    return q, bsq.dequantize(q)


def product(x, w):
    """x w^T in FP64, some rows of w at a time"""
    xd = x.double()
    return torch.cat([xd @ w[i:i + 2048].double().T for i in range(0, w.shape[0], 2048)], 1)


# as many tiles as pairs of SMs, so that the sum over K stays in one part
@pytest.mark.parametrize("fmt", ["mxfp8_e4m3", "mxfp8_e5m2", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,N,K", [(4864, 1024, 65536), (20, 19456, 32768), (2, 300, 65536), (300, 600, 65536)])
def test_linear(bsq, fmt, T, N, K):
    g = torch.Generator(device="cuda").manual_seed(T)
    (A, x), (B, w) = operand(bsq, g, T, K, fmt), operand(bsq, g, N, K, fmt)
    want = product(x, w)
    got = bsq.gemm_linear(A, B, out_dtype=F32)
    assert_close(got, want, bound(K / 4096) * want, fmt)
    z = torch.empty((T, N), dtype=BF, device="cuda")
    y = torch.empty((T, N), dtype=F32, device="cuda")
    res = torch.full_like(y, -0.5)
    bsq.gemm_linear_into(A, B, y, None, res, "relu", z)
    assert torch.equal(y, got + res) and torch.equal(z, got.to(BF))


@pytest.mark.parametrize("fmt", ["mxfp8_e4m3", "nvfp4"])
@pytest.mark.parametrize("T,N,K", [(4864, 512, 65536), (100, 9728, 32768), (300, 200, 65536)])
def test_gated(bsq, fmt, T, N, K):
    g = torch.Generator(device="cuda").manual_seed(T + 1)
    (A, x), (B, w), (C, v) = (operand(bsq, g, n, K, fmt) for n in (T, N, N))
    a, u = product(x, w), product(x, v)
    h = bsq.gemm_gated(A, B, C, "identity", F32)
    assert_close(h, a * u, (2.02 * bound(K / 4096) + U) * a * u, fmt)


# -1, 0, 1: every sum is exact; K on both sides of an accumulator's end, and several accumulators of a BF16 result
@pytest.mark.parametrize("fmt", ["mxfp8_e4m3", "mxfp4"])
@pytest.mark.parametrize("T,N,K", [(4864, 1024, 4096), (4864, 1024, 4128), (4800, 1000, 8224), (4864, 1024, 66592), (20, 19456, 12320),
                                   (20, 19400, 66592), (9, 19456, 8192)])
def test_whole_numbers(bsq, fmt, T, N, K):
    g = torch.Generator(device="cuda").manual_seed(K)
    x, w = (torch.randint(-1, 2, s, generator=g, device="cuda").to(BF) for s in ((T, K), (N, K)))
    A, B = (bsq.quantize(t, fmt)[0] for t in (x, w))
    want = product(x, w)
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(bsq.gemm_linear(A, B, out_dtype=F32).double(), want)
    assert torch.equal(bsq.gemm_linear(A, B), want.float().to(BF))
    if T > 32:
        n = N // 2 // 8 * 8
        w2 = w[n:2 * n].contiguous()
        C, D = (bsq.quantize(t, fmt)[0] for t in (w[:n].contiguous(), w2))
        for dtype in (F32, BF):
            gate, up = (torch.empty((T, n), dtype=BF, device="cuda") for _ in range(2))
            h = torch.empty((T, n), dtype=dtype, device="cuda")
            bsq.gemm_gated_into(A, C, D, h, "relu", gate, up)
            assert torch.equal(h, (want[:, :n].clamp(min=0) * want[:, n:2 * n]).float().to(dtype))
            assert torch.equal(gate, want[:, :n].float().to(BF)) and torch.equal(up, want[:, n:2 * n].float().to(BF))
