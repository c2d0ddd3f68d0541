"""FP64 references and error bounds for the linear layers, the gated feed-forward
and AdamW (U, UB: FP32's and BF16's unit roundoff)."""
import math

import numpy as np
import torch

from _ops_ref import ACC, U, UB, round_out

ACTS = ("identity", "relu", "silu", "gelu", "gelu_tanh")
STEEPEST = 1.13           # of any activation: gelu's slope at sqrt(2) is 1.1289


def act(name, z):
    """act(z), act'(z) and the factor of U in act's own relative error, in FP64.

    silu: exp2's argument is off by 2 U |z| (two roundings), which is the relative error it brings
    to the exponential; ex2, the sum, rcp and the product some 10 U.  gelu_tanh: the same with the
    argument 2 t, itself a few roundings.  gelu: erfc's argument is off by U 2 |z|, which moves erfc by
    2 z^2 U of itself where z is negative; erfcf itself 6 ulp."""
    if name == "identity":
        return z, torch.ones_like(z), torch.zeros_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double(), torch.zeros_like(z)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s)), 2 * z.abs() + 12
    if name == "gelu":
        c = torch.special.ndtr(z)
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), 2 * z * z + 24
    k = math.sqrt(2 / math.pi)
    t = k * (z + 0.044715 * z ** 3)
    s = torch.sigmoid(2 * t)
    return z * s, s + 2 * z * s * (1 - s) * k * (1 + 3 * 0.044715 * z * z), 16 * t.abs() + 12


TINY = 1e-30              # results and factors that FP32 flushes


def product(x, w):
    """x w^T and the bound of its FP32 sum on the tensor cores"""
    xd, wd = x.double(), w.double()
    return xd @ wd.T, ACC * (xd.abs() @ wd.abs().T)


def linear_ref(x, w, bias, residual, name, dtype):
    """(y, its bound, z, its bound)"""
    z, e = product(x, w)
    if bias is not None:
        z = z + bias.double()
        e = e + U * z.abs()
    y, _, rel = act(name, z)
    tol = STEEPEST * e + rel * U * y.abs() + TINY
    if residual is not None:
        y = y + residual.double()
        tol = tol + U * y.abs()
    return y, 1.01 * tol + 1.01 * round_out(dtype, y), z, 1.01 * e + 1.01 * UB * z.abs() + TINY


def gated_ref(x, wg, wu, name, dtype):
    a, ea = product(x, wg)
    u, eu = product(x, wu)
    f, _, rel = act(name, a)
    ef = STEEPEST * ea + rel * U * f.abs() + TINY
    h = f * u
    tol = ef * (u.abs() + eu) + f.abs() * eu + U * h.abs() + TINY
    return h, 1.01 * tol + 1.01 * round_out(dtype, h), a, 1.01 * (ea + UB * a.abs()) + TINY, u, 1.01 * (eu + UB * u.abs()) + TINY


def slope_error(z):
    """|error of act'(z)|: a sum of terms of at most 1 + 2 |z|^3 / e^(z^2 / 2) and the like, each with its
    argument's error; below 40 U everywhere, and growing with z^2 where gelu's terms cancel"""
    return (40 + 8 * z * z) * U


def linear_grad_ref(dy, x, w, z, name):
    """dx, dw, dbias and their bounds"""
    d = dy.double()
    if name == "identity":
        dz, e = d, torch.zeros_like(d)
    else:
        _, slope, _ = act(name, z.double())
        dz, e = d * slope, d.abs() * slope_error(z.double()) + U * (d * slope).abs()
    return _products(dz, e, x, w, name != "identity")


def _products(dz, e, x, w, rounded):
    xd, wd = x.double(), w.double()
    dx, dw, db = dz @ wd, dz.T @ xd, dz.sum(0)
    ez = e + (UB * dz.abs() if rounded else 0)
    tx = ez @ wd.abs() + ACC * (dz.abs() @ wd.abs())
    tw = ez.T @ xd.abs() + ACC * (dz.abs().T @ xd.abs())
    tb = e.sum(0) + (dz.shape[0] + 8) * U * dz.abs().sum(0)
    return (dx, 1.01 * tx + 1.01 * UB * dx.abs() + TINY, dw, 1.01 * tw + 1.01 * UB * dw.abs() + TINY, db, 1.01 * tb + TINY)


def gated_grad_ref(dh, x, wg, wu, gate, up, name):
    d, a, u = dh.double(), gate.double(), up.double()
    f, slope, rel = act(name, a)
    da, du = d * u * slope, d * f
    ea = (d * u).abs() * slope_error(a) + 3 * U * da.abs()
    eu = d.abs() * (rel * U * f.abs() + TINY) + U * du.abs()
    x1, t1, g, tg, _, _ = _products(da, ea, x, wg, True)
    x2, t2, v, tv, _, _ = _products(du, eu, x, wu, True)
    dx = x1 + x2
    t = t1 + t2
    return dx, t + 1.01 * UB * dx.abs(), g, tg, v, tv


# ------------------------------------------------------------------------ AdamW
F = np.float32


def mix(x):
    x = x.astype(np.uint32)
    with np.errstate(over="ignore"):
        x = x ^ (x >> np.uint32(16))
        x = x * np.uint32(0x7FEB352D)
        x = x ^ (x >> np.uint32(15))
        x = x * np.uint32(0x846CA68B)
        return x ^ (x >> np.uint32(16))


def random_bits(seed, step, tensor, n, start=0):
    """of the elements from `start` on, which do not pass a multiple of 2^32"""
    key = mix(np.array([tensor ^ (seed & 0xFFFFFFFF)]))
    key = mix(key ^ np.uint32(seed >> 32))
    key = mix(key ^ np.uint32(step & 0xFFFFFFFF))
    with np.errstate(over="ignore"):
        key = key + np.uint32(start >> 32) * np.uint32(0x9E3779B9)
    return mix(np.arange(start & 0xFFFFFFFF, (start & 0xFFFFFFFF) + n, dtype=np.uint64).astype(np.uint32) ^ key)


def e4m3_values():
    """The value of every E4M3 code (0x7F, 0xFF: NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


E4M3 = e4m3_values()


def decode(codes, scales):
    s = np.ldexp(np.ones(len(scales)), scales.astype(int) - 127)
    s[scales == 255] = np.nan
    return (E4M3[codes] * np.repeat(s, 32)[:len(codes)]).astype(F)


def encode(x, bits, root):
    """Codes and scales of x (FP32) from the definition; bits: 16 random bits each, or None."""
    n = len(x)
    pad = np.zeros(-(-n // 32) * 32, F)
    pad[:n] = x
    b = pad.reshape(-1, 32)
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.abs(b).max(1)
        bad = ~np.isfinite(amax)
        most = (amax * F(8 / 7)).astype(F)
        _, e = np.frexp(most)                                   # in [2^(e-1), 2^e)
        e = np.where(np.isinf(most), 129, e)                    # past FP32's range: in [2^128, 2^129)
        e = np.where(amax == 0, -127, np.maximum(e.astype(int) - 1 - 8, -127))
        y = np.abs(b).astype(np.float64) * np.ldexp(1.0, -e)[:, None]
    y = np.where(np.isfinite(y), y, 0).reshape(-1)[:n]
    grid = E4M3[:127]                                           # 0 .. 448, ascending
    if bits is None:
        y = np.minimum(y, 448)
        hi = np.minimum(np.searchsorted(grid, y), 126)
        lo = np.maximum(hi - 1, 0)
        up = (grid[hi] - y < y - grid[lo]) | ((grid[hi] - y == y - grid[lo]) & (hi % 2 == 0)) | (grid[hi] == y)
        code = np.where(up, hi, lo)
    else:
        # below 2^-6 2^-6 is added first, in FP32; the 16 bits meet the 16 highest of the 20 that are cut
        low = np.where(y < 2.0 ** -6, 2.0 ** -6, 0)
        v = (y.astype(F) + low.astype(F)).astype(F)
        w = (v.view(np.uint32) + (bits.astype(np.uint32) << np.uint32(4))) & np.uint32(0xFFF00000)
        v = np.minimum(w.view(F) - low.astype(F), 448)
        code = np.searchsorted(grid, v.astype(np.float64))
        assert (grid[code] == v).all()
    if root:
        code = np.where((x != 0) & (code == 0), 1, code)
    else:
        code = np.where(np.signbit(x), code | 0x80, code)
    code = np.where(np.repeat(bad, 32)[:n], 0x7F, code)
    return code.astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def adamw_ref(p, g, state, lr, step, betas, eps, wd, factor=None, seed=None, tensor=0, p_bf16=False, start=0):
    """One step in FP32, each operation rounded, as numpy does it; returns (p, copy, state), p before its rounding to
    nearest (BF16 with a seed: rounded)."""
    b1, b2 = betas
    x = g.astype(F)
    if factor is not None:
        x = x * F(factor)
    if len(state) == 2:
        m, v = state
    else:
        m, v = decode(state[0], state[1]), decode(state[2], state[3])
        v = v * v
    with np.errstate(all="ignore"):
        m = F(b1) * m + F(1 - b1) * x
        v = F(b2) * v + (F(1 - b2) * x) * x
        r = np.sqrt(v)
        d = r * F(1 / math.sqrt(1 - b2 ** step)) + F(eps)
        q = F(1 - lr * wd) * p.astype(F) - F(lr / (1 - b1 ** step)) * (m / d)
    assert m.dtype == v.dtype == q.dtype == F
    copy = q
    bits = None if seed is None else random_bits(seed, step, tensor, len(p), start)
    if len(state) == 2:
        out = (m, v)
    else:
        out = (*encode(m, None if bits is None else bits & np.uint32(0xFFFF), False),
               *encode(r, None if bits is None else bits >> np.uint32(16), True))
    if bits is not None and p_bf16:
        with np.errstate(over="ignore"):
            w = q.view(np.uint32) + ((bits * np.uint32(0x9E3779B1)) >> np.uint32(16))
        q = np.where(np.isfinite(q), (w & np.uint32(0xFFFF0000)).view(F), q)
    return q, copy, out
