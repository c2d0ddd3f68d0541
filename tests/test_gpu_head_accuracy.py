"""How exact the linear cross entropy and its gradient are, with bounds near
what their sums can hold: the K = 512 read-out of the tensor cores' sums in
the loss and in the gradient's logits, long sums into dh and dw, the target's entry
of g; and values of dloss and logits that are not finite."""
import math

import pytest
import torch

from _ops_ref import U, UB, assert_close

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# A tensor core's FP32 sum drops less than one unit in the last place at each of the 32 additions
# (16 products each) of K = 512.  Over terms of one sign and like size the sum after j of them is
# j / 32 of the whole, so what is lost is below sum_j 2^-23 j / 32 = 16.5 * 2^-23 of the whole:
# 2.0e-6.  (One accumulator for K = 4096, 256 additions, loses up to eight times that.)
CHUNK = 16.5 * 2.0 ** -23


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    return b


@pytest.mark.parametrize("T", [40, 300])
def test_loss_of_long_sums_of_one_sign(bsq, T):
    # every logit is a sum of 4096 positive products: a bias of the sum is a bias of lse
    V, D = 333, 4096
    g = torch.Generator(device="cuda").manual_seed(T)
    h = (torch.rand((T, D), generator=g, device="cuda") + 0.5).to(BF)
    w = ((torch.rand((V, D), generator=g, device="cuda") + 0.5) / 64).to(BF)
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    _, lse = bsq.linear_cross_entropy(h, w, targets)
    z = h.double() @ w.double().T
    want = torch.logsumexp(z, 1)
    # the chunk's loss, 8 chunks added in FP32, the parts' exponentials and sums (64 U), the sum m + log s
    tol = (CHUNK + 8 * U) * z.amax(1) + 64 * U + U * want.abs()
    assert_close(lse, want, tol, "lse")


@pytest.mark.parametrize("T", [40, 300])
def test_gradient_of_confident_targets(bsq, T):
    # 1 - p of the target from 1e-3 to 1e-6: p - 1 cancels, so an error of the logit of 1e-5 is an
    # error of the gradient's largest entry of as much or more
    V, D = 2000, 4096
    g = torch.Generator(device="cuda").manual_seed(T)
    w = (torch.randn((V, D), generator=g, device="cuda") * D ** -0.5).to(BF)
    targets = torch.randperm(V, generator=g, device="cuda")[:T]
    left = torch.logspace(-3, -6, T, device="cuda")                # 1 - p
    h = ((V / left).log()[:, None] * w[targets].float()).to(BF)
    _, lse = bsq.linear_cross_entropy(h, w, targets)
    dh, dw = bsq.linear_cross_entropy_backward(h, w, targets, lse, torch.ones(T, device="cuda"))
    hd, wd = h.double(), w.double()
    z, mag = hd @ wd.T, hd.abs() @ wd.abs().T
    far = z - lse.double()[:, None]
    p = far.exp()
    gr = p - torch.nn.functional.one_hot(targets, V)
    # the logit (chunks, and 8 of them added), z - lse and the exponential (4 U of the argument, 8 U),
    # the rounding of g to BF16
    dg = p * ((CHUNK + 8 * U) * mag + 4 * U * far.abs() + 8 * U) + (UB + 4 * U) * gr.abs()
    long = 1e-5                                                     # of dh's and dw's own sums, as in the other tests
    want, tol = gr @ wd, dg @ wd.abs() + long * (gr.abs() @ wd.abs())
    assert_close(dh, want, 1.01 * tol + 1.01 * UB * want.abs(), "dh")
    want, tol = gr.T @ hd, dg.T @ hd.abs() + long * (gr.abs().T @ hd.abs())
    assert_close(dw, want, 1.01 * tol + 1.01 * UB * want.abs(), "dw")


def mean_bias(got, want):
    """Mean relative error, and five standard deviations of what BF16 outputs rounded to nearest leave
    of it (each at most UB off, uniformly: UB / sqrt(3))."""
    return float((got.double() / want - 1).mean()), 5 * UB / math.sqrt(3 * got.numel())


def g_rounded(h, w, lse):
    """exp(z - lse) as it enters the products: in BF16 (dloss is 1 here, so nothing is scaled)."""
    return (h.double() @ w.double().T - lse.double()[:, None]).exp().to(BF).double()


# dh and dw keep an accumulator for K = 4096 at most: 256 additions, sum_j 2^-23 j / 256
LONG = 128.5 * 2.0 ** -23


def test_dw_over_many_tokens_is_not_biased(bsq):
    # dw[v] is a sum over 200003 tokens of terms of one sign (the target's column is left out)
    T, V, D = 200003, 2100, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    h = (torch.rand((T, D), generator=g, device="cuda") + 0.5).to(BF)
    w = (torch.randn((V, D), generator=g, device="cuda") * 0.02).to(BF)
    targets = torch.zeros(T, dtype=torch.int64, device="cuda")
    _, lse = bsq.linear_cross_entropy(h, w, targets)
    dw = torch.empty_like(w)
    bsq.linear_cross_entropy_backward_into(h, w, targets, lse, torch.ones(T, device="cuda"), None, dw)
    want = 0
    for at in range(0, T, 32768):
        want = want + g_rounded(h[at:at + 32768], w, lse[at:at + 32768]).T @ h[at:at + 32768].double()
    bias, noise = mean_bias(dw[1:], want[1:])
    # the logits (their |h w| sum to 1.3 here), the sum's own loss, its 49 chunks added in FP32
    assert abs(bias) < noise + 1.3 * CHUNK + LONG + U * math.sqrt(49), bias


def test_dh_over_a_large_vocabulary_is_not_biased(bsq):
    # dh[t] is a sum over 131072 columns, of one sign (the target's row of w is 0); 76 tiles, so that
    # the sum is not split.  128 of its rows are looked at.  w's columns differ in size, so that dh's
    # elements do not lie within one rounding step of each other.
    T, V, D = 1024, 131072, 4864
    g = torch.Generator(device="cuda").manual_seed(2)
    h = (torch.randn((T, D), generator=g, device="cuda") * 0.02).to(BF)
    size = (1 + torch.rand(D, generator=g, device="cuda")) / 96
    w = ((torch.rand((V, D), generator=g, device="cuda") + 0.5) * size).to(BF)
    w[0] = 0
    targets = torch.zeros(T, dtype=torch.int64, device="cuda")
    _, lse = bsq.linear_cross_entropy(h, w, targets)
    dh = torch.empty_like(h)
    bsq.linear_cross_entropy_backward_into(h, w, targets, lse, torch.ones(T, device="cuda"), dh, None)
    want = 0
    for at in range(0, V, 8192):
        want = want + g_rounded(h[:128], w[at:at + 8192], lse[:128]) @ w[at:at + 8192].double()
    bias, noise = mean_bias(dh[:128], want)
    # the logits (their |h w| sum to 1.3 here), the sum's own loss, its 32 chunks added in FP32
    assert abs(bias) < noise + 1.3 * CHUNK + LONG + U * math.sqrt(32), bias


@pytest.mark.parametrize("T", [9, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_dloss_that_is_not_finite(bsq, T, bad):
    g = torch.Generator(device="cuda").manual_seed(T)
    V, D = 500, 64
    h = torch.randn((T, D), generator=g, device="cuda").to(BF)
    w = (torch.randn((V, D), generator=g, device="cuda") / 8).to(BF)
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    targets[2] = -100
    _, lse = bsq.linear_cross_entropy(h, w, targets)
    # every token's (one loss scale for all): the gradient says so
    dh, dw = bsq.linear_cross_entropy_backward(h, w, targets, lse, torch.full((T,), bad, device="cuda"))
    counts = torch.ones(T, dtype=torch.bool, device="cuda")
    counts[2] = False
    assert not torch.isfinite(dh[counts]).any() and (dh[2] == 0).all() and not torch.isfinite(dw).any()
    # one token's: its row of dh and dw, not the other rows
    dloss = torch.rand(T, generator=g, device="cuda")
    dloss[4] = 0
    clean = bsq.linear_cross_entropy_backward(h, w, targets, lse, dloss)
    dloss[4] = bad
    dh, dw = bsq.linear_cross_entropy_backward(h, w, targets, lse, dloss)
    assert not torch.isfinite(dh[4]).any() and not torch.isfinite(dw).any()
    dh[4] = clean[0][4]
    assert torch.equal(dh, clean[0])
    # that of a token that does not count is nobody's
    dloss[4], dloss[2] = 0, bad
    assert all(torch.equal(a, b) for a, b in zip(bsq.linear_cross_entropy_backward(h, w, targets, lse, dloss), clean))


@pytest.mark.parametrize("T", [5, 200])
def test_infinite_logits(bsq, T):
    # exp(inf) is inf: lse = inf, the loss of another target inf, that of the column itself inf - inf
    V, D = 1000, 64
    g = torch.Generator(device="cuda").manual_seed(T)
    h = torch.randn((T, D), generator=g, device="cuda").to(BF)
    w = torch.randn((V, D), generator=g, device="cuda").to(BF)
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    h[:, 0] = 1
    w[700, 0] = -float("inf")                       # a logit of -inf: exp is 0
    targets[1], targets[2] = 700, 0
    want = torch.logsumexp(h.double() @ w.double().T, 1)
    loss, lse = bsq.linear_cross_entropy(h, w, targets)
    assert torch.isfinite(lse).all() and (lse.double() - want).abs().max() < 1e-4
    assert loss[1] == float("inf") and torch.isfinite(loss[targets != 700]).all()
    w[300, 0] = float("inf")                        # and one of +inf
    targets[targets == 300] = 301
    targets[3] = 300
    loss, lse = bsq.linear_cross_entropy(h, w, targets)
    assert (lse == float("inf")).all()
    assert torch.isnan(loss[3]) and (loss[targets != 300] == float("inf")).all()


def test_a_single_row_has_no_pitch(bsq):
    # one token of a buffer whose rows are not whole vectors, and one column of such a head
    g = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn((5, 20), generator=g, device="cuda").to(BF)[:1, :16]
    w = torch.randn((7, 16), generator=g, device="cuda").to(BF)
    target, dloss = torch.tensor([2], device="cuda"), torch.ones(1, device="cuda")
    want = bsq.linear_cross_entropy(h.contiguous(), w, target)
    got = bsq.linear_cross_entropy(h, w, target)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dh, dw = torch.empty((3, 20), dtype=BF, device="cuda")[:1, :16], torch.empty_like(w)
    bsq.linear_cross_entropy_backward_into(h, w, target, want[1], dloss, dh, dw)
    wh, ww = bsq.linear_cross_entropy_backward(h.contiguous(), w, target, want[1], dloss)
    assert torch.equal(dh, wh) and torch.equal(dw, ww)
    one = torch.randn((2, 20), generator=g, device="cuda").to(BF)[:1, :16]
    assert torch.equal(bsq.linear_cross_entropy(h, one, target * 0)[1],
                       bsq.linear_cross_entropy(h.contiguous(), one.contiguous(), target * 0)[1])


@pytest.mark.parametrize("T,V,D", [(40, 20000, 256), (100, 20000, 256), (300, 20000, 256), (1200, 20000, 256),
                                   (300, 700, 64), (2000, 257, 320), (1200, 1500, 2104), (17000, 1100, 64)])
def test_gradient_keeps_the_targets_entry(bsq, T, V, D):
    # p - 1 is the largest entry of a row of g by far, and enters dh and dw in full: what is left of the
    # rounding of g are the other entries' errors, which are independent and small
    g = torch.Generator(device="cuda").manual_seed(T + V)
    w = (torch.randn((V, D), generator=g, device="cuda") * D ** -0.5).to(BF)
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    targets[T // 2:T // 2 + 9] = targets[3]                       # tokens that share a target
    h = (torch.randn((T, D), generator=g, device="cuda") + 10 * torch.rand((T, 1), generator=g, device="cuda")
         * w[targets].float()).to(BF)
    targets[1] = -100
    _, lse = bsq.linear_cross_entropy(h, w, targets)
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    hd, wd = h.double(), w.double()
    p = (hd @ wd.T - lse.double()[:, None]).exp()
    scale = torch.where(targets >= 0, dloss.double(), 0.0)[:, None]
    others = p.scatter(1, targets.clamp(min=0)[:, None], 0.0) * scale
    gr = scale * (p - torch.nn.functional.one_hot(targets.clamp(min=0), V))
    both = bsq.linear_cross_entropy_backward(h, w, targets, lse, dloss)
    for got, want, rest in ((both[0], gr @ wd, others.square() @ wd.square()),
                            (both[1], gr.T @ hd, others.square().T @ hd.square())):
        # before the outputs' rounding: each other entry rounded to BF16 (UB / sqrt(3) of it, independent),
        # the target's logit and sums (4e-6).  Two values e apart are rounded to neighbours one unit (at most
        # 2 UB) apart with a chance of e / unit: sqrt(e 2 UB) of mean square
        norm = want.norm()
        e = UB / math.sqrt(3) * float(rest.sum().sqrt() / norm) + 4e-6
        apart = float((got.double() - want.to(BF).double()).norm() / norm)
        assert apart <= 1.5 * math.sqrt(e * 2 * UB), (apart, e)
    # each gradient alone: the same bits
    one, two = torch.empty_like(both[0]), torch.empty_like(both[1])
    bsq.linear_cross_entropy_backward_into(h, w, targets, lse, dloss, one, None)
    bsq.linear_cross_entropy_backward_into(h, w, targets, lse, dloss, None, two)
    assert torch.equal(one, both[0]) and torch.equal(two, both[1])


@pytest.mark.parametrize("T,V,D", [(50, 3000, 136), (100, 3000, 136), (700, 3000, 136), (9000, 3000, 136),
                                   (1025, 20000, 2104), (40000, 3000, 8)])
def test_gradient_of_one_target_for_all(bsq, T, V, D):
    # every token has the same target: dw's row of it is a sum over all of them, in a fixed order
    g = torch.Generator(device="cuda").manual_seed(T)
    h = torch.randn((T, D), generator=g, device="cuda").to(BF)
    w = (torch.randn((V, D), generator=g, device="cuda") * 0.1).to(BF)
    targets = torch.full((T,), 2999, device="cuda")
    _, lse = bsq.linear_cross_entropy(h, w, targets)
    dloss = torch.ones(T, device="cuda")
    dh, dw = bsq.linear_cross_entropy_backward(h, w, targets, lse, dloss)
    p = (h.double() @ w.double().T - lse.double()[:, None]).exp()
    p[:, 2999] -= 1
    want = p.T @ h.double()
    # the row's own rounding, its entries (4e-6: logits and sums) and the rounding of the correction (UB^2)
    tol = 1.01 * UB * want[2999].abs() + (4e-6 + UB * UB) * (p[:, 2999].abs() @ h.double().abs())
    assert_close(dw[2999], want[2999], tol, "dw of the target")
    for _ in range(3):
        again = bsq.linear_cross_entropy_backward(h, w, targets, lse, dloss)
        assert torch.equal(again[0], dh) and torch.equal(again[1], dw)
