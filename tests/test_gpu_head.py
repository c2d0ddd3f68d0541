"""The softmax cross entropy of a linear head and its gradient against FP64
with bounds from the formula: one token and one column, odd vocabularies, row
pitches, tokens that do not count, several pieces of the vocabulary, large
logits, and the gradient also against differences."""
import pytest
import torch

from _ops_ref import Guard, assert_close, head_grad_ref, head_ref, strided

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    return b


def make(T, V, D, seed, pad=0, scale=1.0, wscale=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h, _ = strided((T, D), BF, pad, pad, gen=g, scale=scale)
    w, _ = strided((V, D), BF, pad, pad, gen=g, scale=wscale or D ** -0.5)
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    return h, w, targets, g


SHAPES = [(1, 1, 8), (1, 2, 16), (2, 5, 24), (7, 255, 64), (1, 50021, 512), (129, 256, 72), (128, 257, 136),
          (300, 1000, 1000), (5, 5003, 4096), (513, 777, 320), (1000, 130, 64), (256, 4096, 256), (2050, 2051, 128)]


@pytest.mark.parametrize("T,V,D", SHAPES)
@pytest.mark.parametrize("pad", [0, 8])
def test_forward_and_gradient(bsq, T, V, D, pad):
    h, w, targets, g = make(T, V, D, T + V, pad)
    if T > 3:
        targets[1], targets[2], targets[3] = -100, V, -(1 << 40)
    loss = torch.full((T,), float("nan"), device="cuda")
    lse = torch.full((T,), float("nan"), device="cuda")
    bsq.linear_cross_entropy_into(h, w, targets, loss, lse)
    rl, rz, tl, tz = head_ref(h, w, targets)
    assert_close(lse, rz, tz, "lse")
    assert_close(loss, rl, tl, "loss")
    if T > 3:
        assert (loss[1:4] == 0).all()
    dloss = torch.randn(T, generator=g, device="cuda") / T
    dh, hbuf = strided((T, D), BF, pad, pad, fill=float("nan"))
    dw, wbuf = strided((V, D), BF, pad, pad, fill=float("nan"))
    bsq.linear_cross_entropy_backward_into(h, w, targets, lse, dloss, dh, dw)
    rh, th, rw, tw = head_grad_ref(h, w, targets, lse, dloss)
    assert_close(dh, rh, th, "dh")
    assert_close(dw, rw, tw, "dw")
    Guard(dh, hbuf).check()
    Guard(dw, wbuf).check()
    if T > 3:
        assert (dh[1:4] == 0).all()
    # each gradient alone: the same bits
    one, two = torch.empty_like(dh), torch.empty_like(dw)
    bsq.linear_cross_entropy_backward_into(h, w, targets, lse, dloss, one, None)
    bsq.linear_cross_entropy_backward_into(h, w, targets, lse, dloss, None, two)
    assert torch.equal(one, dh) and torch.equal(two, dw)


@pytest.mark.parametrize("T", [15, 16, 17, 63, 64, 65, 100, 127, 255, 256, 257])
def test_token_counts_around_the_tiles(bsq, T):
    # the token counts at which a tile's shape or the products' order changes, over vocabularies
    # that end inside a tile
    for V, D in ((1, 8), (333, 200), (4501, 136)):
        h, w, targets, g = make(T, V, D, T + V)
        targets[T // 2] = -1
        loss, lse = bsq.linear_cross_entropy(h, w, targets)
        rl, rz, tl, tz = head_ref(h, w, targets)
        assert_close(lse, rz, tz, "lse")
        assert_close(loss, rl, tl, "loss")
        dloss = torch.rand(T, generator=g, device="cuda")
        dh, hbuf = strided((T, D), BF, 8, 8, fill=float("nan"))
        dw, wbuf = strided((V, D), BF, 8, 8, fill=float("nan"))
        bsq.linear_cross_entropy_backward_into(h, w, targets, lse, dloss, dh, dw)
        rh, th, rw, tw = head_grad_ref(h, w, targets, lse, dloss)
        assert_close(dh, rh, th, "dh")
        assert_close(dw, rw, tw, "dw")
        Guard(dh, hbuf).check()
        Guard(dw, wbuf).check()


@pytest.mark.parametrize("T,V,D", [(5180, 300, 72), (2304, 257, 600), (2048, 2049, 8), (130, 9001, 64)])
def test_sums_split_over_the_tokens_or_the_vocabulary(bsq, T, V, D):
    for pad in (0, 8):
        test_forward_and_gradient(bsq, T, V, D, pad)


def test_several_pieces_of_the_vocabulary(bsq):
    # more tokens than one 256 MB piece of the whole vocabulary holds: 3 pieces
    T, V, D = 70001, 5003, 16
    h, w, targets, g = make(T, V, D, 9)
    loss, lse = bsq.linear_cross_entropy(h, w, targets)
    rl, rz, tl, tz = head_ref(h, w, targets)
    assert_close(lse, rz, tz, "lse")
    assert_close(loss, rl, tl, "loss")
    del rl, rz, tl, tz
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    dh, dw = bsq.linear_cross_entropy_backward(h, w, targets, lse, dloss)
    for lo in (0, T - 4096):                              # rows of dh are independent
        at = slice(lo, lo + 4096)
        rh, th, _, _ = head_grad_ref(h[at], w, targets[at], lse[at], dloss[at])
        assert_close(dh[at], rh, th, "dh")
    ref, tol = 0, 0
    for lo in range(0, T, 8192):
        at = slice(lo, lo + 8192)
        _, _, rw, tw = head_grad_ref(h[at], w, targets[at], lse[at], dloss[at])
        ref, tol = ref + rw, tol + tw                     # each block's bound covers its share of the rounding
    assert_close(dw, ref, tol, "dw")


def test_several_pieces_one_gradient_at_a_time(bsq):
    # the pieces' kernels follow each other differently where one gradient is left out: the same bits
    T, V, D = 70001, 5003, 16
    h, w, targets, _ = make(T, V, D, 10)
    _, lse = bsq.linear_cross_entropy(h, w, targets)
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    dh, dw = bsq.linear_cross_entropy_backward(h, w, targets, lse, dloss)
    one, two = torch.empty_like(dh), torch.empty_like(dw)
    for _ in range(3):
        bsq.linear_cross_entropy_backward_into(h, w, targets, lse, dloss, one.fill_(0), None)
        bsq.linear_cross_entropy_backward_into(h, w, targets, lse, dloss, None, two.fill_(0))
        assert torch.equal(one, dh) and torch.equal(two, dw)


@pytest.mark.parametrize("scale", [30.0, 3000.0, 1e18])
def test_large_logits(bsq, scale):
    # exponentials that overflow without the maximum taken out; one-hot softmax rows
    T, V, D = 40, 700, 64
    h, w, targets, g = make(T, V, D, 4, scale=scale)
    loss, lse = bsq.linear_cross_entropy(h, w, targets)
    rl, rz, tl, tz = head_ref(h, w, targets)
    assert_close(lse, rz, tz, "lse")
    assert_close(loss, rl, tl, "loss")
    assert torch.isfinite(loss).all()


def test_nothing_counts_and_zero_weights(bsq):
    T, V, D = 33, 300, 64
    h, w, targets, g = make(T, V, D, 5)
    none = torch.full_like(targets, -100)
    loss, lse = bsq.linear_cross_entropy(h, w, none)
    assert (loss == 0).all()
    dh, dw = bsq.linear_cross_entropy_backward(h, w, none, lse, torch.ones(T, device="cuda"))
    assert (dh == 0).all() and (dw == 0).all()
    dh, dw = bsq.linear_cross_entropy_backward(h, w, targets, lse, torch.zeros(T, device="cuda"))
    assert (dh == 0).all() and (dw == 0).all()


def test_nan_and_inf_stay_in_their_rows(bsq):
    T, V, D = 300, 500, 64
    h, w, targets, g = make(T, V, D, 6)
    h[5, 3], h[290, 0] = float("nan"), float("inf")
    loss, lse = bsq.linear_cross_entropy(h, w, targets)
    assert torch.isnan(loss[5]) and not torch.isfinite(lse[290])
    good = torch.ones(T, dtype=torch.bool, device="cuda")
    good[5] = good[290] = False
    rl, rz, tl, tz = head_ref(h[good], w, targets[good])
    assert_close(loss[good], rl, tl, "loss")
    # a token that does not count and whose state is not finite gives no gradient
    targets[5] = targets[290] = -100
    h2 = h.clone()
    h2[5], h2[290] = 0, 0
    dloss = torch.ones(T, device="cuda")
    dh, _ = bsq.linear_cross_entropy_backward(h, w, targets, lse, dloss)
    assert (dh[5] == 0).all() and (dh[290] == 0).all()
    lse2 = bsq.linear_cross_entropy(h2, w, targets)[1]
    want = bsq.linear_cross_entropy_backward(h2, w, targets, lse2, dloss)[0]
    assert torch.equal(dh, want)


@pytest.mark.parametrize("T", [5, 200])
@pytest.mark.parametrize("where", [0, 256, 700])
def test_columns_of_nan_reach_every_loss(bsq, T, where):
    # whole tiles of logits without a number beside tiles with some
    h, w, targets, _ = make(T, 1000, 64, 8)
    w[where:where + 256] = float("nan")
    loss, lse = bsq.linear_cross_entropy(h, w, targets)
    assert torch.isnan(lse).all() and torch.isnan(loss).all()


def test_gradient_against_differences(bsq):
    T, V, D, step = 19, 101, 40, 1e-4
    h, w, targets, g = make(T, V, D, 7)
    targets[4] = -100
    dloss = torch.rand(T, generator=g, device="cuda")
    _, lse = bsq.linear_cross_entropy(h, w, targets)
    dh, dw = bsq.linear_cross_entropy_backward(h, w, targets, lse, dloss)
    _, th, _, tw = head_grad_ref(h, w, targets, lse, dloss)

    def f(h, w):
        return (head_ref(h, w, targets)[0] * dloss.double()).sum()
    H, W = h.double(), w.double()
    for grad, tol, at in ((dh, th, 0), (dw, tw, 1)):
        d = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        want = ((f(H + step * d, W) - f(H - step * d, W)) if at == 0 else (f(H, W + step * d) - f(H, W - step * d)))
        assert abs(want / (2 * step) - (grad.double() * d).sum()) <= (tol * d.abs()).sum() + 1e-5 * d.abs().sum()


def test_refusals(bsq):
    T, V, D = 4, 10, 16
    h = torch.zeros((T, D), dtype=BF, device="cuda")
    w = torch.zeros((V, D), dtype=BF, device="cuda")
    t = torch.zeros(T, dtype=torch.int64, device="cuda")
    f = torch.zeros(T, device="cuda")
    wide = torch.zeros((V, D + 4), dtype=BF, device="cuda")
    off = torch.zeros(V * D + 8, dtype=BF, device="cuda")
    L, B = bsq.linear_cross_entropy, bsq.linear_cross_entropy_backward_into
    bad = [lambda: L(h.float(), w.float(), t), lambda: L(h.half(), w.half(), t), lambda: L(h, w[:, :8], t),
           lambda: L(h, w, t.int()), lambda: L(h, w, t[:3]), lambda: L(h[:, :12], w[:, :12], t),
           lambda: L(h, wide[:, :D], t), lambda: L(h, off[1:1 + V * D].view(V, D), t), lambda: L(h[:0], w, t[:0]),
           lambda: L(h, w[:0], t), lambda: L(h.cpu(), w, t), lambda: B(h, w, t, f, f, None, None),
           lambda: B(h, w, t, f, f, h.float(), None), lambda: B(h, w, t, f, f, None, w[:9]),
           lambda: B(h, w, t, f, f, None, wide[:, :D]), lambda: B(h, w, t, f[:2], f, h, None),
           lambda: B(h, w, t, f, f.bfloat16(), h, None)]
    for i, c in enumerate(bad):
        with pytest.raises(bsq.BsqError):
            c()
            pytest.fail(f"case {i} was not refused")
