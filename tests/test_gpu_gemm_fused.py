"""Products of block-scaled operands with an epilogue, against FP64 over the
exactly dequantized operands: every format, few rows to several tiles, sums in
parts, rows off 16-byte boundaries, and scales that differ between the two
projections of a gated layer."""
import pytest
import torch

from _linear_ref import ACTS, gated_ref, linear_ref
from _ops_ref import Guard, assert_close, strided

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FORMATS = [("mxfp8_e4m3", "mxfp8_e4m3"), ("mxfp8_e5m2", "mxfp8_e4m3"), ("mxfp4", "mxfp4"), ("nvfp4", "nvfp4")]
SIZES = [(1, 5, 32), (3, 130, 96), (2, 70, 1056), (1, 4096, 8192), (4, 300, 4128), (5, 40, 64), (100, 700, 2080), (130, 257, 544), (257, 384, 1024), (300, 1000, 4128), (700, 264, 256)]


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    yield b
    b.sync_status()


def quantized(bsq, g, rows, cols, fmt, scale):
    v = (torch.randn((rows, cols), generator=g, device="cuda") * scale).to(BF)
    v[:, ::32] *= 8                                   # blocks and rows of different size
    v *= torch.rand((rows, 1), generator=g, device="cuda").to(BF) + 0.25
    q, _ = bsq.quantize(v, fmt)
    return q, bsq.dequantize(q)


@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("T,N,K", SIZES)
def test_gemm_linear(bsq, T, N, K, fa, fb):
    g = torch.Generator(device="cuda").manual_seed(T + N + K)
    A, x = quantized(bsq, g, T, K, fa, 1.0)
    B, w = quantized(bsq, g, N, K, fb, K ** -0.5)
    for i, name in enumerate(ACTS):
        dtype = [BF, F32][i % 2]
        bias = [None, torch.randn(N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda").to(BF)][i % 3]
        res = torch.randn((T, N), generator=g, device="cuda").to(dtype) if i > 1 else None
        y, ybuf = strided((T, N), dtype, pad=(-N) % 8 if i < 3 else 1, offset=0 if i < 3 else 1, fill=float("nan"))
        z, zbuf = strided((T, N), BF, pad=(-N) % 8 if i % 2 else 3, fill=float("nan"))
        keep = i != 2
        bsq.gemm_linear_into(A, B, y, bias, res, name, z if keep else None)
        want, tol, zw, zt = linear_ref(x, w, bias, res, name, dtype)
        assert_close(y, want, tol, f"y {name}")
        Guard(y, ybuf).check()
        if keep:
            assert_close(z, zw, zt, f"z {name}")
            Guard(z, zbuf).check()


@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("T,N,K", SIZES)
def test_gemm_gated(bsq, T, N, K, fa, fb):
    g = torch.Generator(device="cuda").manual_seed(T + N + K + 1)
    A, x = quantized(bsq, g, T, K, fa, 1.0)
    G, wg = quantized(bsq, g, N, K, fb, K ** -0.5)
    B, wu = quantized(bsq, g, N, K, fb, 37 * K ** -0.5)     # NVFP4: another tensor scale
    for i, name in enumerate(ACTS):
        dtype = [BF, F32][i % 2]
        h, hbuf = strided((T, N), dtype, pad=(-N) % 8 if i < 3 else 1, offset=0 if i < 3 else 1, fill=float("nan"))
        a, abuf = strided((T, N), BF, pad=(-N) % 8 if i % 2 else 3, fill=float("nan"))
        u, ubuf = strided((T, N), BF, pad=(-N) % 8, fill=float("nan"))
        keep = i != 2
        bsq.gemm_gated_into(A, G, B, h, name, a if keep else None, u if keep else None)
        want, tol, aw, at, uw, ut = gated_ref(x, wg, wu, name, dtype)
        assert_close(h, want, tol, f"h {name}")
        Guard(h, hbuf).check()
        if keep:
            assert_close(a, aw, at, "gate")
            assert_close(u, uw, ut, "up")
            Guard(a, abuf).check()
            Guard(u, ubuf).check()


# the smaller sizes above have tiles of 128 columns; these of 256, whole and in parts
@pytest.mark.parametrize("fa,fb", [FORMATS[0], FORMATS[3]])
@pytest.mark.parametrize("T,N,K", [(2050, 2500, 2080), (100, 4096, 14336), (60, 2051, 8192)])
def test_wide_tiles_and_long_sums(bsq, T, N, K, fa, fb):
    test_gemm_linear(bsq, T, N, K, fa, fb)
    test_gemm_gated(bsq, T, N, K, fa, fb)


@pytest.mark.parametrize("fmt", ["mxfp8_e4m3", "mxfp8_e5m2", "mxfp4"])
@pytest.mark.parametrize("T", [1, 4, 9, 200])
def test_scales_far_from_one(bsq, fmt, T):
    # one operand's scales near 2^100, the other's near 2^-100, and a row whose scales are NaN
    g = torch.Generator(device="cuda").manual_seed(5)
    A, x = quantized(bsq, g, T, 96, fmt, 2.0 ** 100)
    v = torch.randn((140, 96), generator=g, device="cuda") * 2.0 ** -100
    v[7, 40] = float("nan")
    B, _ = bsq.quantize(v.to(BF), fmt)
    w = bsq.dequantize(B)
    got = bsq.gemm_linear(A, B, out_dtype=F32)
    assert torch.isnan(got[:, 7]).all()
    rows = [i for i in range(140) if i != 7]
    want, tol, _, _ = linear_ref(x.double(), w[rows].double(), None, None, "identity", F32)
    assert_close(got[:, rows], want, tol)


@pytest.mark.parametrize("fmt", ["mxfp8_e4m3", "mxfp4", "nvfp4"])
def test_without_an_epilogue_it_is_the_gemm(bsq, fmt):
    g = torch.Generator(device="cuda").manual_seed(3)
    for T, N, K in ((300, 520, 1024), (520, 1000, 256)):
        A, _ = quantized(bsq, g, T, K, fmt, 1.0)
        B, _ = quantized(bsq, g, N, K, fmt, 1.0)
        want = bsq.gemm(A, B, F32)
        got = bsq.gemm_linear(A, B, out_dtype=F32)
        # the sum over K may come in parts
        assert (got.double() - want.double()).abs().max() <= 1e-5 * K * float(want.abs().max())
        assert torch.equal(bsq.gemm_linear(A, B, activation="relu", out_dtype=F32), got.clamp(min=0))
