"""Numbers of tokens on both sides of every choice that products with an epilogue make, with
bias, pre-activation and residual, and the residual's own place as the output on every path."""
import pytest
import torch

from _linear_ref import gated_ref, linear_ref
from _ops_ref import ACC, U, Guard, assert_close, strided

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    yield b
    b.sync_status()


def gen(*seed):
    return torch.Generator(device="cuda").manual_seed(hash(seed) & 0xFFFFFFFF)


def quantized(bsq, g, rows, cols, fmt, scale=1.0):
    v = (torch.randn((rows, cols), generator=g, device="cuda") * scale).to(BF)
    v[:, ::32] *= 8
    v *= torch.rand((rows, 1), generator=g, device="cuda").to(BF) + 0.25
    q, _ = bsq.quantize(v, fmt)
    return q, bsq.dequantize(q)


TOKENS = [1, 2, 3, 7, 8, 9, 15, 16, 17, 24, 25, 31, 32, 33, 40, 64, 65, 127, 128, 129]


# K in one part and in several
@pytest.mark.parametrize("fmt", ["mxfp8_e4m3", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("N,K", [(300, 544), (264, 8192)])
def test_gemm_linear(bsq, N, K, T, fmt):
    g = gen(T, N, K)
    A, x = quantized(bsq, g, T, K, fmt)
    B, w = quantized(bsq, g, N, K, fmt, K ** -0.5)
    bias = torch.randn(N, generator=g, device="cuda")
    for dtype, pad in ((BF, 4), (F32, 4), (BF, 1), (F32, 3)):
        res = torch.randn((T, N), generator=g, device="cuda").to(dtype)
        y, ybuf = strided((T, N), dtype, pad=pad, fill=float("nan"))
        z, zbuf = strided((T, N), BF, pad=pad, fill=float("nan"))
        bsq.gemm_linear_into(A, B, y, bias, res, "silu", z)
        want, tol, zw, zt = linear_ref(x, w, bias, res, "silu", dtype)
        assert_close(y, want, tol, "y")
        assert_close(z, zw, zt, "z")
        Guard(y, ybuf).check()
        Guard(z, zbuf).check()


@pytest.mark.parametrize("fmt", ["mxfp8_e4m3", "nvfp4"])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("N,K", [(300, 544), (264, 8192)])
def test_gemm_gated(bsq, N, K, T, fmt):
    g = gen(T, N, K, 1)
    A, x = quantized(bsq, g, T, K, fmt)
    (B, w), (C, v) = (quantized(bsq, g, N, K, fmt, s * K ** -0.5) for s in (1, 9))
    for dtype, pad in ((BF, 4), (F32, 1)):
        h, hbuf = strided((T, N), dtype, pad=pad, fill=float("nan"))
        (a, abuf), (u, ubuf) = (strided((T, N), BF, pad=k, fill=float("nan")) for k in (pad, 4))
        bsq.gemm_gated_into(A, B, C, h, "silu", a, u)
        want, tol, aw, at, uw, ut = gated_ref(x, w, v, "silu", dtype)
        for got, ref, t, buf in ((h, want, tol, hbuf), (a, aw, at, abuf), (u, uw, ut, ubuf)):
            assert_close(got, ref, t)
            Guard(got, buf).check()


# CUDA cores; few tokens; tiles of 128 and of 256 columns; each in one part and in several
PLACES = [(1, 300, 1024), (2, 300, 4128), (3, 300, 544), (20, 300, 8192), (32, 2000, 1056), (33, 300, 544), (60, 2051, 8192), (130, 1000, 8192),
          (300, 6000, 8192), (2100, 2500, 1056), (1100, 1000, 14336)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,N,K", PLACES)
def test_the_residuals_own_place(bsq, T, N, K, dtype):
    g = gen(T, N, K, 2)
    bias = torch.randn(N, generator=g, device="cuda")
    calls = []
    for fmt in ("mxfp8_e4m3", "nvfp4"):
        A, B = quantized(bsq, g, T, K, fmt)[0], quantized(bsq, g, N, K, fmt, K ** -0.5)[0]
        calls.append(lambda y, r, z, A=A, B=B: bsq.gemm_linear_into(A, B, y, bias, r, "gelu", z))
    x, w = (torch.randn((n, K), generator=g, device="cuda").to(BF) for n in (T, N))
    calls.append(lambda y, r, z: bsq.linear_into(x, w, y, bias, r, "gelu", z))
    for call in calls:
        for pad, offset in ((-N % 8, 0), (8 - N % 8, 8), (3, 1)):
            for z in (None, torch.empty((T, N), dtype=BF, device="cuda")):
                r, rbuf = strided((T, N), dtype, pad=pad, offset=offset, gen=g)
                y, ybuf = strided((T, N), dtype, pad=pad, offset=offset, fill=float("nan"))
                call(y, r, z)
                call(r, r, z)
                assert torch.equal(r, y)
                Guard(r, rbuf).check()
                Guard(y, ybuf).check()


@pytest.mark.parametrize("fmt", ["mxfp8_e4m3", "mxfp8_e5m2", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,N,K", [(1, 300, 1024), (9, 300, 8192), (40, 300, 8192), (300, 520, 1024), (520, 1000, 256), (1100, 2500, 4128)])
def test_without_an_epilogue(bsq, fmt, T, N, K):
    # element by element, against the exact product and the bare one
    g = gen(T, N, K, 3)
    (A, x), (B, w) = quantized(bsq, g, T, K, fmt), quantized(bsq, g, N, K, fmt)
    xd, wd = x.double(), w.double()
    tol = (ACC + U) * (xd.abs() @ wd.abs().T)
    got = bsq.gemm_linear(A, B, out_dtype=F32)
    assert_close(got, xd @ wd.T, tol)
    assert_close(got, bsq.gemm(A, B, F32).double(), 2 * tol)
