"""The global gradient norm and clipping against FP64: empty and odd tensors,
both types, addresses without alignment, lists longer than one launch takes,
in place and into copies, and norms that are zero, infinite or NaN."""
import math

import pytest
import torch

from _ops_ref import U, UB, assert_close

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    return b


def tensors(sizes, seed, packed, scale=1.0):
    """Gradients of the sizes, alternately BF16 and FP32; packed: back to back in one buffer a type."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out, at = [], {BF: 1, F32: 1}
    pool = {t: torch.full((sum(sizes) + 8,), float("nan"), dtype=t, device="cuda") for t in (BF, F32)}
    for i, n in enumerate(sizes):
        t = BF if i % 2 == 0 else F32
        if packed:
            v = pool[t][at[t]:at[t] + n]
            at[t] += n
        else:
            v = torch.empty(n, dtype=t, device="cuda")
        v.copy_(torch.randn(n, generator=g, device="cuda") * scale)
        out.append(v)
    return out


def norm_ref(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


# squares and runs of at most 128 of them in FP32: 129 U on the sum, half of it on the norm, its
# own rounding; the factor: the quotient, the sum with eps and the norm's error; the product
REL_NORM = 66 * U
REL_FACTOR = REL_NORM + 3 * U


def check(bsq, grads, max_norm, inplace, eps=1e-6):
    before = [g.clone() for g in grads]
    ref = norm_ref(before)
    assert abs(float(bsq.grad_norm(grads)) - ref) <= REL_NORM * ref
    outs = None if inplace else [torch.full_like(g, float("nan")) for g in grads]
    norm = bsq.clip_grad_norm(bsq.GradList(grads, outs), max_norm, eps)
    assert abs(float(norm) - ref) <= REL_NORM * ref
    factor = min(1.0, max_norm / (ref + eps))
    for b, g, o in zip(before, grads, grads if inplace else outs):
        want = b.double() * factor
        assert_close(o, want, (REL_FACTOR + 2 * U + (1.01 * UB if b.dtype == BF else 0)) * want.abs() + 1e-38, "clipped")
        if not inplace:
            assert torch.equal(b, g)
        if factor == 1.0:
            assert torch.equal(o, b)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("sizes", [[1], [0, 3, 0], [7, 1, 2, 33], [16384, 16385, 16383, 5], [100003, 8, 8, 70000],
                                   [1 + i % 37 for i in range(33)], [3 + 5 * (i % 11) for i in range(1025)],
                                   [1] * 2500, [3_000_001, 2_000_003]])
def test_norm_and_clip(bsq, sizes, packed, inplace):
    check(bsq, tensors(sizes, len(sizes), packed), 0.5, inplace)
    check(bsq, tensors(sizes, len(sizes), packed, 1e-4), 1e6, inplace)


def test_outputs_at_other_alignments_and_nothing_else_written(bsq):
    g = torch.randn(10007, device="cuda").bfloat16()
    f = torch.randn(5003, device="cuda")
    for shift in range(8):
        ob = torch.full((10007 + 32,), float("nan"), dtype=BF, device="cuda")
        of = torch.full((5003 + 32,), float("nan"), dtype=F32, device="cuda")
        grads = [g[shift:], f[shift:]]
        outs = [ob[9:9 + 10007 - shift], of[6:6 + 5003 - shift]]
        bsq.clip_grad_norm(bsq.GradList(grads, outs), 1.0)
        factor = min(1.0, 1.0 / (norm_ref(grads) + 1e-6))
        for b, o in zip(grads, outs):
            want = b.double() * factor
            assert_close(o, want, (REL_FACTOR + 2 * U + (1.01 * UB if b.dtype == BF else 0)) * want.abs(), "clipped")
        assert torch.isnan(ob[:9]).all() and torch.isnan(ob[9 + 10007 - shift:]).all()
        assert torch.isnan(of[:6]).all() and torch.isnan(of[6 + 5003 - shift:]).all()


def test_zero_infinite_and_nan_norms(bsq):
    z = [torch.zeros(1000, device="cuda"), torch.zeros(7, dtype=BF, device="cuda")]
    assert float(bsq.clip_grad_norm(z, 1.0)) == 0 and all((t == 0).all() for t in z)
    g = [torch.ones(1000, device="cuda"), torch.ones(7, dtype=BF, device="cuda")]
    g[0][17] = float("inf")
    assert float(bsq.clip_grad_norm(g, 1.0)) == float("inf")      # factor 0: finite gradients 0, inf * 0 NaN
    assert torch.isnan(g[0][17]) and int((g[0] == 0).sum()) == 999 and (g[1] == 0).all()
    g = [torch.ones(1000, device="cuda"), torch.ones(7, dtype=BF, device="cuda")]
    g[1][3] = float("nan")
    assert math.isnan(float(bsq.clip_grad_norm(g, 1.0)))
    assert all(torch.isnan(t).all() for t in g)
    g = [torch.full((100,), 3.0, device="cuda")]
    assert float(bsq.clip_grad_norm(g, 0.0)) == 30.0 and (g[0] == 0).all()
    g = [torch.full((100,), 3.0, device="cuda")]
    bsq.clip_grad_norm(g, float("inf"))
    assert (g[0] == 3.0).all()


def test_same_bits_every_time(bsq):
    g = tensors([100003, 65537, 5, 3_000_001], 3, True)
    want = float(bsq.grad_norm(g))
    assert all(float(bsq.grad_norm(g)) == want for _ in range(5))


def test_refusals(bsq):
    g = torch.ones(8, device="cuda")
    bad = [lambda: bsq.GradList([]), lambda: bsq.GradList([g.half()]), lambda: bsq.GradList([g[::2]]),
           lambda: bsq.GradList([g.cpu()]), lambda: bsq.GradList([g], [g[:4]]), lambda: bsq.GradList([g], [g.bfloat16()]),
           lambda: bsq.GradList([g], []), lambda: bsq.clip_grad_norm([g], -1.0),
           lambda: bsq.clip_grad_norm([g], float("nan")), lambda: bsq.clip_grad_norm([g], 1.0, eps=-1.0),
           lambda: bsq.clip_grad_norm_into([g], 1.0, torch.zeros(2, device="cuda"))]
    for i, c in enumerate(bad):
        with pytest.raises(bsq.BsqError):
            c()
            pytest.fail(f"case {i} was not refused")
