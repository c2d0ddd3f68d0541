"""Sums that hold every element: inputs whose sums are whole numbers, exact in
FP32 in whatever order, so that one element left out or taken twice is far
outside the few roundings that remain.  (The bounds for random inputs grow with
the number of terms, and pass a single element of a long row.)"""
import pytest
import torch

from _ops_ref import U, UB, strided

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    return b


# rows of one warp and of many, at the ends of what a group of threads holds, odd ones between
COLS = [1, 7, 24, 100, 257, 1000, 2047, 4096, 4104, 8191, 8192, 8200, 14336, 16383, 16384, 16400, 20000, 40001, 70000]
SIDES = [(0, 0), (5, 1)]


def rows_of(C):
    return [3] if C > 20000 else [3, 700]


def edges(C, g):
    """Columns to look at: both ends of the row and of the vectors there, powers of two, and some others."""
    at = {c for e in (0, 1, 3, 4, 7, 8, 9, 15, 16, 31, 32) for c in (e, C - 1 - e)}
    at |= {c for p in range(5, 17) for c in (2 ** p - 1, 2 ** p)}
    at |= set(torch.randint(0, C, (24,), generator=g, device="cuda").tolist())
    return sorted(c for c in at if 0 <= c < C)


def plus_minus(R, C, g):
    """Rows of as many 1 as -1 (and a 0 where C is odd), in random places."""
    v = torch.ones(C, device="cuda")
    v[C // 2:] = -1
    if C % 2:
        v[C - 1] = 0
    return v[torch.rand((R, C), generator=g, device="cuda").argsort(1)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C", COLS)
@pytest.mark.parametrize("pad,offset", SIDES)
def test_norm_statistics(bsq, C, dtype, pad, offset):
    g = torch.Generator(device="cuda").manual_seed(C)
    for R in rows_of(C):
        x, _ = strided((R, C), dtype, pad, offset, fill=0.0)
        if C > 1:
            x.copy_(plus_minus(R, C, g))
            _, mean, rstd = bsq.layer_norm(x, eps=0.0)
            assert (mean == 0).all()
            want = (C / (C - C % 2)) ** 0.5
            # the quotient, the sum's product with 1 / C, the root: a few U; one element more or less: 1 / (2 C)
            assert 16 * U < 0.5 / C and ((rstd.double() - want).abs() <= 8 * U * want).all(), (R, rstd)
    # all but one element 0: the mean is that element's share
    at = edges(C, g)
    x, _ = strided((len(at), C), dtype, pad, offset, fill=0.0)
    x[torch.arange(len(at), device="cuda"), torch.tensor(at, device="cuda")] = 4096.0
    _, mean, _ = bsq.layer_norm(x)
    assert ((mean.double() - 4096.0 / C).abs() <= 3 * U * 4096.0 / C).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C", COLS)
@pytest.mark.parametrize("pad,offset", SIDES)
def test_norm_gradient_sums(bsq, C, dtype, pad, offset):
    g = torch.Generator(device="cuda").manual_seed(C + 1)
    # column sums: whole numbers below 2^24
    for R in rows_of(C):
        x, _ = strided((R, C), dtype, pad, offset, fill=0.0)
        dy, _ = strided((R, C), dtype, pad, offset, fill=0.0)
        for t in (x, dy):
            t.copy_(torch.randint(-4, 5, (R, C), generator=g, device="cuda"))
        zero, one = torch.zeros(R, device="cuda"), torch.ones(R, device="cuda")
        dx, dw, db = bsq.layer_norm_backward(dy, x, None, zero, one)
        assert torch.equal(dw.double(), (dy.double() * x.double()).sum(0)) and torch.equal(db.double(), dy.double().sum(0))
        if dtype == F32:
            # the rows' sums too are whole numbers; dx is a few roundings of numbers up to 4 (1 + 2 + 4 * 2)
            s1, s2 = dy.double().mean(1, keepdim=True), (dy.double() * x.double()).mean(1, keepdim=True)
            want = dy.double() - s1 - x.double() * s2
            tol = 4 * U * (dy.double().abs() + s1.abs() + 3 * (x.double() * s2).abs()) + 1e-30
            assert ((dx.double() - want).abs() <= tol).all()
    # dy 0 but at one column, x of 1 and -1: elsewhere dx is -2 shares of that column, or 0
    at = edges(C, g)
    R = len(at)
    rows, cols = torch.arange(R, device="cuda"), torch.tensor(at, device="cuda")
    x, _ = strided((R, C), dtype, pad, offset, fill=0.0)
    dy, _ = strided((R, C), dtype, pad, offset, fill=0.0)
    x.copy_(torch.where(torch.rand((R, C), generator=g, device="cuda") < 0.5, 1.0, -1.0))
    dy[rows, cols] = 4096.0
    dx, _, _ = bsq.layer_norm_backward(dy, x, None, torch.zeros(R, device="cuda"), torch.ones(R, device="cuda"))
    share = 4096.0 / C
    like = x.double() == x.double()[rows, cols][:, None]
    want = torch.where(like, -2.0 * share, 0.0)
    want[rows, cols] += 4096.0
    tol = (UB if dtype == BF else 4 * U) * want.abs() + 4 * U * share + 4 * U * dy.double()
    assert ((dx.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,C", [(37, 3, 2047), (37, 3, 2046), (5, 11, 7168), (40, 1, 100), (3, 2, 20001), (1, 8, 7)])
def test_combine_gradient_dot_products(bsq, T, k, C, dtype):
    g = torch.Generator(device="cuda").manual_seed(C)
    ids = torch.randint(-1, 5, (T, k), generator=g, device="cuda")
    plan = bsq.moe_sort(ids, 5)

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").to(dtype)
    dout, rows = whole(T, C), whole(T * k, C)
    _, dweights = bsq.moe_combine_backward(dout, rows, torch.ones((T, k), device="cuda"), plan)
    slot = plan.slot_row.long()
    want = (rows.double()[slot.clamp(min=0)] * dout.double()[:, None, :]).sum(2)
    assert torch.equal(dweights.double(), torch.where(slot >= 0, want, 0.0))


@pytest.mark.parametrize("T", [1, 100, 129, 300])
@pytest.mark.parametrize("V", [1, 255, 256, 257, 5003, 50021])
def test_every_vocabulary_row_enters_the_loss(bsq, T, V):
    # h is 40 times the unit vector of one row of w, whose logit is 40 and the others' far below: lse without
    # that row would be lower by several units
    D = 64
    g = torch.Generator(device="cuda").manual_seed(V + T)
    w = torch.nn.functional.normalize(torch.randn((V, D), generator=g, device="cuda"), dim=1).to(BF)
    at = edges(V, g) if V > 1 else [0]
    for lo in range(0, len(at), T):
        cols = torch.tensor((at[lo:lo + T] + at * T)[:T], device="cuda")
        h = (40 * w[cols].float()).to(BF)
        _, lse = bsq.linear_cross_entropy(h, w, torch.zeros(T, dtype=torch.int64, device="cuda"))
        z = h.double() @ w.double().T
        want = torch.logsumexp(z, 1)
        without = torch.logsumexp(z.scatter(1, cols[:, None], -float("inf")), 1)
        assert (want - without).min() > 0.1 and ((lse.double() - want).abs() <= 1e-4).all()


def test_every_element_enters_the_norm_of_gradients(bsq):
    g = torch.Generator(device="cuda").manual_seed(0)
    for dtype, n in ((BF, 40003), (F32, 20003), (BF, 16384), (F32, 8193), (BF, 5), (F32, 1)):
        for shift in (0, 1):
            t = torch.zeros(n + shift, dtype=dtype, device="cuda")[shift:]
            grads = bsq.GradList([torch.zeros(3, dtype=BF, device="cuda"), t, torch.zeros(70000, device="cuda")])
            for at in edges(n, g):
                t[at] = -24.0
                assert float(bsq.clip_grad_norm(grads, 6.0, eps=0.0)) == 24.0
                assert float(t[at]) == -6.0 and int((t != 0).sum()) == 1
                t[at] = 0
