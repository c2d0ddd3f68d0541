"""AdamW bit for bit where a quotient is infinite, tiny or zero while the second
moments are ordinary, and with an eps or a bias correction far from 1."""
import numpy as np
import pytest
import torch

from _linear_ref import adamw_ref

pytestmark = pytest.mark.gpu
F = np.float32


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    return b


def host(t):
    return t.cpu().numpy()


def bits(x):
    """FP32 by its bits, every NaN as one"""
    x = np.ascontiguousarray(x)
    return np.where(np.isnan(x), np.uint32(0x7FC00000), x.view(np.uint32)) if x.dtype == F else x


def step(bsq, p, g, state, number=10, betas=(0.5, 0.5), eps=1e-8, wd=0.1, lr=0.5, shift=0):
    """One step of a tensor that starts `shift` elements off its boundary, against numpy"""
    def dev(x):
        t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
        return torch.cat([t[:1].repeat(shift), t])[shift:] if shift else t

    pt, gt, st = dev(p), dev(g), tuple(dev(s) for s in state)
    bsq.adamw_step(bsq.AdamWList([pt], [gt], [st]), lr, number, betas, eps, wd)
    want, _, new = adamw_ref(p, g, state, lr, number, betas, eps, wd)
    for a, b in zip(st, new):
        assert np.array_equal(bits(host(a)), bits(b))
    got = host(pt)
    bad = np.flatnonzero(bits(got) != bits(want))
    assert bad.size == 0, (bad.size, got[bad[:3]], want[bad[:3]])
    return got


def floats(rng, n, low, high):
    """Random mantissas and signs, exponents low .. high (below -126: not normal)"""
    return np.ldexp((1 + rng.random(n)) * rng.choice([-1, 1], n), rng.integers(low, high + 1, n)).astype(F)


N = 8192


@pytest.mark.parametrize("shift", [0, 1])
def test_infinite_first_moments(bsq, shift):
    rng = np.random.default_rng(1)
    m, v, p, g = floats(rng, N, -3, 3), np.abs(floats(rng, N, -3, 3)), floats(rng, N, -3, 3), np.zeros(N, F)
    m[::5], m[1::7] = np.inf, -np.inf
    p[::11] = 0
    got = step(bsq, p, g, (m, v), shift=shift)
    assert np.isinf(got[::35]).all() and not np.isnan(got).any()


@pytest.mark.parametrize("shift", [0, 1])
def test_quotients_past_the_largest_number(bsq, shift):
    rng = np.random.default_rng(2)
    m, v = floats(rng, N, 70, 127), np.abs(floats(rng, N, -80, -40))
    got = step(bsq, floats(rng, N, -3, 3), np.zeros(N, F), (m, v), eps=0.0, shift=shift)
    assert np.isinf(got).any() and not np.isnan(got).any()


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("eps", [0.0, 1e-8, 1.0])
def test_tiny_first_moments(bsq, eps, shift):
    # where m came down by half a step; p at 0, so that the quotient's last bit shows
    rng = np.random.default_rng(3)
    for low, high in ((-149, -80), (-110, -85), (-92, -88)):
        m, v = floats(rng, N, low, high), np.abs(floats(rng, N, -60, 40))
        p = np.zeros(N, F)
        p[::3] = floats(rng, len(p[::3]), -140, -60)
        for beta1 in (0.5, 0.0):
            g = np.zeros(N, F) if beta1 else m
            step(bsq, p, g, (m, v), betas=(beta1, 0.5), eps=eps, shift=shift)


def test_zeros_of_either_sign(bsq):
    rng = np.random.default_rng(4)
    m, p = rng.choice([F(0), F(-0.0), F(1), F(2.0 ** -149)], N), rng.choice([F(0), F(-0.0), F(1)], N)
    step(bsq, p, rng.choice([F(0), F(-0.0)], N), (m, np.full(N, 2, F)))
    step(bsq, p, rng.choice([F(0), F(-0.0)], N), (m, rng.choice([F(0), F(2)], N)), eps=0.0)


@pytest.mark.parametrize("eps,beta2,number", [(1e10, 0.5, 10), (1e12, 0.5, 10), (1e30, 0.5, 10), (3e38, 0.5, 10), (1e300, 0.5, 10),
                                              (1e-8, 1 - 1e-6, 1), (1e-8, 1 - 1e-7, 1), (1e-8, 1 - 1e-15, 1), (0.0, 0.9999, 2)])
def test_eps_and_bias_corrections_far_from_one(bsq, eps, beta2, number):
    rng = np.random.default_rng(5)
    v = np.abs(floats(rng, N, -90, 120))
    v[::2] = np.abs(floats(rng, len(v[::2]), -30, 10))
    with np.errstate(over="ignore"):
        for low, high in ((-126, 127), (-20, 20), (70, 90)):
            step(bsq, np.zeros(N, F), np.zeros(N, F), (floats(rng, N, low, high), v), number, (0.5, beta2), eps)


@pytest.mark.parametrize("seed", range(3))
def test_tiny_first_moments_in_8_bits(bsq, seed):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 127, N).astype(np.uint8)
    low = rng.integers(0, 60, N // 32).astype(np.uint8)
    high = rng.integers(100, 130, N // 32).astype(np.uint8)
    g = np.zeros(N, F)
    step(bsq, g.copy(), g, (codes | (rng.integers(0, 2, N) << 7).astype(np.uint8), low, np.maximum(codes, 1), high), betas=(0.9, 0.999))
