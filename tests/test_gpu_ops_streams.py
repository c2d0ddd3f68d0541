"""The operators one after another without waiting for any of them, on one
stream and on two: kernels that start beside the ones before them, and memory
that the next call takes over, must not change a bit."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    return b


def head(bsq, g, rng):
    T, V, D = rng.choice([1, 60, 129, 700, 2050]), rng.choice([260, 3000, 9000]), 8 * rng.choice([8, 20, 64])
    h, w = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((T, D), (V, D)))
    t = torch.randint(-1, V, (T,), generator=g, device="cuda")
    dloss = torch.rand(T, generator=g, device="cuda")

    def call():
        loss, lse = bsq.linear_cross_entropy(h, w, t)
        return (loss, lse, *bsq.linear_cross_entropy_backward(h, w, t, lse, dloss))
    return call


def norm(bsq, g, rng):
    R, C = rng.choice([1, 300, 310, 2000]), rng.choice([17, 1000, 2047, 4096, 9000])
    x = torch.randn((R, C), generator=g, device="cuda").to(rng.choice([torch.bfloat16, torch.float32]))
    w, b = (torch.randn(C, generator=g, device="cuda") for _ in range(2))

    def call():
        y, mean, rstd = bsq.layer_norm(x, w, b)
        return (y, mean, rstd, *bsq.layer_norm_backward(y, x, w, mean, rstd))
    return call


def experts(bsq, g, rng):
    T, k, E, C = rng.choice([1, 33, 1500, 6000]), rng.choice([1, 2, 5]), rng.choice([5, 64]), rng.choice([64, 130, 1023])
    x = torch.randn((T, C), generator=g, device="cuda").bfloat16()
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda")
    w = torch.rand((T, k), generator=g, device="cuda")

    def call():
        rows, plan = bsq.moe_dispatch(x, ids, E)
        out = bsq.moe_combine(rows, w, plan)
        return (rows, plan.offsets, plan.slot_row, out, *bsq.moe_combine_backward(out, rows, w, plan))
    return call


def clip(bsq, g, rng):
    grads = [torch.randn(rng.randint(1, 100000), generator=g, device="cuda").to(rng.choice([torch.bfloat16, torch.float32]))
             for _ in range(rng.choice([1, 5, 40, 200]))]

    def call():
        outs = [t.clone() for t in grads]
        return (bsq.clip_grad_norm(outs, 0.5), *outs)
    return call


@pytest.mark.parametrize("streams", [1, 2])
def test_calls_in_any_order_without_waiting(bsq, streams):
    g, rng = torch.Generator(device="cuda").manual_seed(3), random.Random(streams)
    calls = [make(bsq, g, rng) for _ in range(8) for make in (head, norm, experts, clip)]
    want = []
    for call in calls:
        out = call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    on = [torch.cuda.current_stream()] if streams == 1 else [torch.cuda.Stream() for _ in range(streams)]
    for _ in range(3):
        order = rng.sample(range(len(calls)), len(calls))
        torch.cuda.synchronize()
        got = {}
        for n, i in enumerate(order):
            with torch.cuda.stream(on[n % streams]):
                got[i] = calls[i]()
        torch.cuda.synchronize()
        for i in order:
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i])), i
    bsq.sync_status()
