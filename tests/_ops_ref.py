"""FP64 references and error bounds for the operators around the layer.

U is FP32's unit roundoff (half an ulp, relative: 24 significant bits), UB BF16's.  Every bound is
worked out from the formula: a sum of n terms in FP32, in whatever order,
differs from the exact one by at most (depth) * U * (sum of the magnitudes),
where depth is the longest chain of additions (n at most)."""
import numpy as np
import torch

U, UB = 2.0 ** -24, 2.0 ** -8


def round_out(dtype, ref):
    """Rounding of the result at its store."""
    return (UB if dtype == torch.bfloat16 else U) * ref.abs()


def assert_close(got, ref, tol, what=""):
    got, ref = got.double(), ref.double()
    finite = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaNs differ"
    inf = ~finite & ~torch.isnan(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    err = (got - ref).abs()
    bad = finite & ~(err <= tol)
    if bad.any():
        i = int(torch.argmax((torch.where(finite, err / (tol + 1e-300), torch.zeros_like(err))).flatten()))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; worst: got "
                             f"{got.flatten()[i].item()!r}, want {ref.flatten()[i].item()!r}, tol "
                             f"{(tol.flatten()[i] if tol.numel() > 1 else tol).item()!r}")


def strided(shape, dtype, pad=0, offset=0, fill=None, gen=None, scale=1.0):
    """A CUDA matrix whose row pitch is cols + pad and whose first element lies
    `offset` elements into its allocation; the elements around it are NaN."""
    R, C = shape
    buf = torch.full((offset + R * (C + pad) + 64,), float("nan"), dtype=dtype, device="cuda")
    m = buf[offset:offset + R * (C + pad)].view(R, C + pad)[:, :C]
    if fill is not None:
        m.fill_(fill)
    else:
        m.copy_(torch.randn((R, C), generator=gen, device="cuda") * scale)
    return m, buf


class Guard:
    """The elements of a strided() buffer outside its matrix are unchanged (NaN)."""

    def __init__(self, m, buf):
        self.m, self.buf = m, buf

    def check(self):
        inside = torch.zeros(self.buf.numel(), dtype=torch.bool, device="cuda")
        at = (self.m.data_ptr() - self.buf.data_ptr()) // self.buf.element_size()
        R, C = self.m.shape
        ld = self.m.stride(0) if R > 1 else C
        idx = at + torch.arange(R, device="cuda")[:, None] * ld + torch.arange(C, device="cuda")
        inside[idx.flatten()] = True
        assert torch.isnan(self.buf[~inside]).all(), "written outside the output"


# ------------------------------------------------------------------ expert sort
def plan_ref(ids: np.ndarray, E: int):
    """offsets, slot_row, row_slot from the definition (numpy's stable sort)."""
    flat = ids.reshape(-1).astype(np.int64)
    valid = (flat >= 0) & (flat < E)
    slots = np.flatnonzero(valid)
    order = slots[np.argsort(flat[slots], kind="stable")]
    offsets = np.zeros(E + 1, np.int64)
    offsets[1:] = np.cumsum(np.bincount(flat[slots], minlength=E))
    row_slot = np.full(flat.size, -1, np.int32)
    row_slot[:order.size] = order
    slot_row = np.full(flat.size, -1, np.int32)
    slot_row[order] = np.arange(order.size)
    return offsets, slot_row.reshape(ids.shape), row_slot


def combine_ref(rows, weights, slot_row):
    """(sum_j w rows, sum_j |w rows|) in FP64 over the slots that are not left out."""
    T, k = slot_row.shape
    out = torch.zeros((T, rows.shape[1]), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for j in range(k):
        here = slot_row[:, j] >= 0
        v = rows.double()[slot_row[here, j].long()]
        if weights is not None:
            v = v * weights.double()[here, j][:, None]
        out[here] += v
        mag[here] += v.abs()
    return out, mag


# ------------------------------------------------------------------- layer norm
def norm_ref(x, w, b, eps):
    xd = x.double()
    C = x.shape[1]
    mean = xd.mean(1, keepdim=True)
    c = xd - mean
    var = c.square().mean(1, keepdim=True)
    rstd = 1 / (var + eps).sqrt()
    wd = w.double() if w is not None else torch.ones(C, dtype=torch.float64, device="cuda")
    bd = b.double() if b is not None else torch.zeros(C, dtype=torch.float64, device="cuda")
    y = c * rstd * wd + bd
    # mean's error e1: a sum of C terms; the deviations sum to 0, so var takes e1^2 and its own
    # sum's rounding; depth of a sum: at most C terms
    d = C + 8
    e1 = d * U * xd.abs().mean(1, keepdim=True)
    rel = (d / 2 + 8) * U + e1 * e1 / (2 * (var + eps))
    tol = wd.abs() * rstd * e1 + (y - bd).abs() * rel + 2 * U * (y.abs() + (y - bd).abs()) + round_out(x.dtype, y)
    return y, mean[:, 0], rstd[:, 0], tol, (e1 + U * mean.abs())[:, 0], (rstd * (rel + 3 * U))[:, 0]


def norm_grad_ref(dy, x, w, mean, rstd):
    R, C = x.shape
    wd = w.double() if w is not None else torch.ones(C, dtype=torch.float64, device="cuda")
    r = rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * r
    dyd = dy.double()
    g = dyd * wd
    s1, s2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - s1 - xh * s2)
    a1, a2 = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    d = C + 10                                     # depth of a row's sums, and the few roundings of each term
    tol = r * U * (d * (a1 + xh.abs() * a2) + 8 * (g.abs() + s1.abs() + (xh * s2).abs())) + round_out(x.dtype, dx)
    dw, db = (dyd * xh).sum(0), dyd.sum(0)
    return dx, tol, dw, (R + 8) * U * (dyd * xh).abs().sum(0), db, (R + 8) * U * dyd.abs().sum(0)


# ------------------------------------------------------- linear cross entropy
ACC = 1e-5        # FP32 tensor-core accumulation: at most ACC * sum |a b|, the bound of the GEMM tests


def head_ref(h, w, targets):
    V = w.shape[0]
    z = h.double() @ w.double().T
    lse = torch.logsumexp(z, 1)
    counts = (targets >= 0) & (targets < V)
    hit = z.gather(1, targets.clamp(0, V - 1)[:, None])[:, 0]
    loss = torch.where(counts, lse - hit, torch.zeros_like(lse))
    mag = (h.double().abs() @ w.double().abs().T).amax(1)
    # logsumexp moves by at most the largest change of a logit; its sum and its logarithm add
    # relative errors of the sum (depth 600 bounds any tiling here) that enter lse absolutely
    tol = ACC * mag + 600 * U + 4 * U * (lse.abs() + mag)
    return loss, lse, torch.where(counts, 2 * tol, torch.zeros_like(tol)), tol


def head_grad_ref(h, w, targets, lse, dloss):
    V = w.shape[0]
    hd, wd = h.double(), w.double()
    z = hd @ wd.T
    mag = hd.abs() @ wd.abs().T
    counts = (targets >= 0) & (targets < V)
    s = torch.where(counts, dloss.double(), torch.zeros_like(dloss, dtype=torch.float64))[:, None]
    p = (z - lse.double()[:, None]).exp()
    one = torch.nn.functional.one_hot(targets.clamp(0, V - 1), V).double()
    g = s * (p - one)
    # g's error: the logit's through exp, the exponential's own (argument rounding: 4 U |z - lse|;
    # 8 U for the rest), the rounding to BF16
    dg = s.abs() * p * (ACC * mag + 4 * U * (z - lse.double()[:, None]).abs() + 8 * U) + (UB + 4 * U) * g.abs()
    dh, dw = g @ wd, g.T @ hd
    tol_h = dg @ wd.abs() + ACC * (g.abs() @ wd.abs()) + 1.01 * UB * dh.abs() + 1e-38
    tol_w = dg.T @ hd.abs() + ACC * (g.abs().T @ hd.abs()) + 1.01 * UB * dw.abs() + 1e-38
    return dh, 1.01 * tol_h, dw, 1.01 * tol_w
