"""Tokens sorted by expert and back: the sort exact, the row movements against
FP64 with bounds from their formulas, at odd sizes, pitches and addresses,
with slots left out, and the gradients also against differences."""
import numpy as np
import pytest
import torch

from _ops_ref import U, Guard, assert_close, combine_ref, plan_ref, round_out, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    return b


def make_ids(T, k, E, seed, dropped=0.0, dtype=np.int64):
    rng = np.random.default_rng(seed)
    p = 1.0 / np.arange(1, E + 1) ** 1.1
    ids = rng.choice(E, size=(T, k), p=p / p.sum()).astype(dtype)
    out = rng.random((T, k)) < dropped
    ids[out] = rng.choice(np.array([-1, -100, E, E + 7, 2 ** 31 - 1], dtype), size=int(out.sum()))
    return ids


def check_plan(plan, ids, E):
    offsets, slot_row, row_slot = plan_ref(ids, E)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.slot_row.cpu().numpy(), slot_row)
    assert np.array_equal(plan.row_slot.cpu().numpy(), row_slot)


@pytest.mark.parametrize("T,k,E,dropped", [
    (1, 1, 1, 0.0), (1, 8, 64, 0.0), (3, 2, 5, 0.4), (31, 1, 2, 0.0), (33, 7, 9, 0.1), (128, 8, 256, 0.0),
    (1023, 1, 33, 0.2), (1025, 1, 1024, 0.0), (4096, 8, 64, 0.02), (3001, 5, 1023, 0.5), (40001, 7, 17, 0.05),
    (5, 256, 300, 0.0), (140000, 1, 3, 0.0), (70000, 8, 256, 0.01), (200, 3, 4, 1.0)])
def test_sort_is_exact(bsq, T, k, E, dropped):
    ids = make_ids(T, k, E, 1, dropped)
    plan = bsq.moe_sort(torch.from_numpy(ids).cuda(), E)
    check_plan(plan, ids, E)
    ids32 = ids.astype(np.int32)
    check_plan(bsq.moe_sort(torch.from_numpy(ids32).cuda(), E), ids32, E)


def test_sort_of_ids_beyond_32_bits_and_of_one_expert(bsq):
    ids = np.full((300, 4), 2, np.int64)
    check_plan(bsq.moe_sort(torch.from_numpy(ids).cuda(), 3), ids, 3)
    ids[::3, 1] = (1 << 32) + 2                        # its low word is a valid id
    ids[::5, 2] = -(1 << 32)
    check_plan(bsq.moe_sort(torch.from_numpy(ids).cuda(), 3), ids, 3)


CASES = [(1, 1, 1, 1, 0.0), (1, 8, 64, 7168, 0.0), (2, 3, 4, 8, 0.0), (7, 2, 5, 33, 0.3), (130, 8, 16, 2048, 0.05),
         (257, 3, 13, 2047, 0.1), (64, 4, 8, 1, 0.0), (50, 5, 6, 130, 1.0), (33, 12, 40, 520, 0.2),
         (19, 17, 3, 96, 0.1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,E,C,dropped", CASES)
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1)])
def test_dispatch_gather_combine(bsq, T, k, E, C, dropped, dtype, pad, offset):
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + C)
    ids = make_ids(T, k, E, 2, dropped)
    x, _ = strided((T, C), dtype, pad, offset, gen=g)
    x[T // 2, C // 2] = float("inf")
    rows, buf = strided((T * k, C), dtype, pad, offset, fill=float("nan"))
    plan = bsq.moe_plan(T, k, E)
    bsq.moe_dispatch_into(x, torch.from_numpy(ids).cuda(), plan, rows)
    check_plan(plan, ids, E)
    slot = plan.row_slot.long()
    want = torch.where((slot >= 0)[:, None], x[slot.clamp(min=0) // k], torch.zeros((), dtype=dtype, device="cuda"))
    assert torch.equal(rows, want)
    Guard(rows, buf).check()
    again, buf = strided((T * k, C), dtype, pad + 1, offset, fill=float("nan"))
    assert torch.equal(bsq.moe_gather_into(x, plan, again), want)
    Guard(again, buf).check()

    y, _ = strided((T * k, C), dtype, pad, offset, gen=g)
    y[int(plan.offsets[-1]):] = float("nan")            # rows that hold no slot are not read
    w = torch.rand((T, k), generator=g, device="cuda") + 0.1
    w[plan.slot_row < 0] = float("nan")                 # nor are the weights of slots left out
    for weights in (w, None):
        out, buf = strided((T, C), dtype, pad, offset, fill=float("nan"))
        bsq.moe_combine_into(y, weights, plan, out)
        ref, mag = combine_ref(y, weights, plan.slot_row)
        assert_close(out, ref, (k + 1) * U * mag + round_out(dtype, ref), "combine")
        Guard(out, buf).check()
    assert torch.equal(bsq.moe_dispatch_backward(y, plan), out)


# even widths that are not whole 16-byte vectors, and rows that start between them
PAIRS = [(70, 4, 9, 1030, 0.1), (3, 2, 4, 2, 0.0), (300, 9, 20, 62, 0.2), (2000, 3, 8, 1764, 0.5)]


@pytest.mark.parametrize("T,k,E,C,dropped", PAIRS)
@pytest.mark.parametrize("pad,offset", [(0, 0), (2, 2), (6, 4)])
def test_pairs(bsq, T, k, E, C, dropped, pad, offset):
    test_dispatch_gather_combine(bsq, T, k, E, C, dropped, torch.bfloat16, pad, offset)
    test_combine_backward(bsq, T, k, E, C, dropped, torch.bfloat16, pad, offset)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,E,C,dropped", CASES)
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1)])
def test_combine_backward(bsq, T, k, E, C, dropped, dtype, pad, offset):
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + C + 1)
    plan = bsq.moe_sort(torch.from_numpy(make_ids(T, k, E, 3, dropped)).cuda(), E)
    total = int(plan.offsets[-1])
    y, _ = strided((T * k, C), dtype, pad, offset, gen=g)
    y[total:] = float("nan")
    dout, _ = strided((T, C), dtype, pad, offset, gen=g)
    w = torch.rand((T, k), generator=g, device="cuda")
    w[plan.slot_row < 0] = float("nan")
    drows, buf = strided((T * k, C), dtype, pad, offset, fill=float("nan"))
    dw = torch.full((T, k), float("nan"), device="cuda")
    bsq.moe_combine_backward_into(dout, y, w, plan, drows, dw)
    slot = plan.row_slot[:total].long()
    ref = dout.double()[slot // k] * w.double().flatten()[slot][:, None]
    assert_close(drows[:total], ref, U * ref.abs() + 1.01 * round_out(dtype, ref), "drows")
    assert (drows[total:] == 0).all()
    Guard(drows, buf).check()
    prod = dout.double()[slot // k] * y.double()[:total]
    ref_w = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref_w)
    ref_w[slot] = prod.sum(1)
    mag[slot] = prod.abs().sum(1)
    assert_close(dw.flatten(), ref_w, (C + 8) * U * mag, "dweights")
    only, none = bsq.moe_combine_backward_into(dout, None, w, plan, torch.empty_like(drows), None)
    assert none is None and torch.equal(only, drows)


def test_gradients_against_differences(bsq):
    # combine is linear in the rows and in the weights: <grad, d> equals half the difference of
    # sum(out * dout) at +d and -d, up to the outputs' rounding
    g = torch.Generator(device="cuda").manual_seed(5)
    T, k, E, C = 37, 3, 6, 75
    plan = bsq.moe_sort(torch.from_numpy(make_ids(T, k, E, 6, 0.2)).cuda(), E)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    y, dy, w, dwt, dout = rnd(T * k, C), rnd(T * k, C), rnd(T, k), rnd(T, k), rnd(T, C)
    drows, dweights = bsq.moe_combine_backward(dout, y, w, plan)
    f = lambda y, w: (bsq.moe_combine(y, w, plan).double() * dout.double()).sum()  # noqa: E731
    _, mag = combine_ref(y.abs() + dy.abs(), w.abs() + dwt.abs(), plan.slot_row)
    tol = ((k + 2) * U * mag * dout.abs().double()).sum() * 2
    assert abs((f(y + dy, w) - f(y - dy, w)) / 2 - (drows.double() * dy).sum()) <= tol
    assert abs((f(y, w + dwt) - f(y, w - dwt)) / 2 - (dweights.double() * dwt).sum()) <= tol + (C + 8) * tol
    # and the gather's: <moe_dispatch_backward(d), x> = <d, moe_gather(x)>
    x = rnd(T, C)
    left = (bsq.moe_dispatch_backward(dy, plan).double() * x.double()).sum()
    right = (dy.double() * bsq.moe_gather(x, plan).double()).sum()
    _, mag = combine_ref(dy.abs(), None, plan.slot_row)
    assert abs(left - right) <= ((k + 2) * U * mag * x.abs().double()).sum()


def test_refusals(bsq):
    T, k, E, C = 4, 2, 3, 16
    ids = torch.zeros((T, k), dtype=torch.int64, device="cuda")
    x = torch.zeros((T, C), dtype=torch.bfloat16, device="cuda")
    plan = bsq.moe_sort(ids, E)
    rows = torch.zeros((T * k, C), dtype=torch.bfloat16, device="cuda")
    bad = [lambda: bsq.moe_sort(ids.float(), E), lambda: bsq.moe_sort(ids[:, 0], E), lambda: bsq.moe_sort(ids, 0),
           lambda: bsq.moe_sort(ids, 1025), lambda: bsq.moe_sort(ids[:, ::2], E),
           lambda: bsq.moe_dispatch(x.half(), ids, E), lambda: bsq.moe_dispatch(x[:3], ids, E),
           lambda: bsq.moe_dispatch(x.t(), ids, E), lambda: bsq.moe_dispatch(x.cpu(), ids, E),
           lambda: bsq.moe_dispatch(x[:1].expand(T, C), ids, E),
           lambda: bsq.moe_gather_into(x, plan, rows.float()), lambda: bsq.moe_gather_into(x, plan, rows[1:]),
           lambda: bsq.moe_combine(rows, torch.zeros((T, k), dtype=torch.bfloat16, device="cuda"), plan),
           lambda: bsq.moe_combine(rows, torch.zeros((T, k + 1), device="cuda"), plan),
           lambda: bsq.moe_combine_backward_into(x, None, None, plan, rows, None),
           lambda: bsq.moe_combine_backward_into(x, None, torch.zeros((T, k), device="cuda"), plan, rows,
                                                 torch.zeros((T, k), device="cuda")),
           lambda: bsq.moe_sort(torch.zeros((0, k), dtype=torch.int64, device="cuda"), E)]
    for i, f in enumerate(bad):
        with pytest.raises(bsq.BsqError):
            f()
            pytest.fail(f"case {i} was not refused")
