"""The operators together with the quantize and the grouped GEMM, as the
example runs them: the first step's loss, gradients and norm against the same
step in FP64 with the weights the library holds, then the loss falls; the same
step on a side stream; and the operators captured in a CUDA graph."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    return b


def step_fp64(block, ids, weights):
    """Loss, head, gamma and beta gradients and their norm in FP64 (autograd), experts as dequantized."""
    import block_scaled_precision_03_gb300 as bsq
    x = block.x.double()
    gamma, beta = (p.double().requires_grad_() for p in (block.gamma, block.beta))
    head = block.head.double().requires_grad_()
    c = x - x.mean(1, keepdim=True)
    y = c / (c.square().mean(1, keepdim=True) + 1e-5).sqrt() * gamma + beta
    out = torch.zeros_like(x)
    for e in range(block.experts):
        w = bsq.dequantize(block.forward_w[e]).double()
        for j in range(block.k):
            here = ids[:, j] == e
            out = out + torch.where(here[:, None], weights[:, j].double()[:, None] * (y @ w.T), 0.0)
    z = (x + out) @ head.T
    n = block.targets >= 0
    loss = torch.nn.functional.cross_entropy(z[n], block.targets[n])
    loss.backward()
    grads = [head.grad, gamma.grad, beta.grad]
    return loss.detach(), grads, torch.sqrt(sum(g.square().sum() for g in grads))


def test_first_step_against_fp64_and_the_loss_falls(bsq):
    from moe_step import MoeBlock
    block = MoeBlock()
    with torch.no_grad():
        ids, weights = block.route(bsq.layer_norm(block.x, block.gamma, block.beta)[0])
    loss64, grads64, norm64 = step_fp64(block, ids, weights)
    loss, norm = block.step(max_norm=float("inf"))
    # activations are rounded to BF16 and E4M3 (2^-4 a value), gradients to E5M2 (2^-3) on the way:
    # independent roundings, so the relative error of a sum's norm stays at that of its terms
    assert abs(float(loss) - float(loss64)) < 2.0 ** -6 * float(loss64)
    for got, want in zip(block.grads, grads64):
        assert float((got.double() - want).norm()) < 2.0 ** -3 * float(want.norm())
    assert abs(float(norm) - float(norm64)) < 2.0 ** -4 * float(norm64)
    losses = [float(block.step()[0]) for _ in range(15)]
    assert losses[-1] < 0.9 * float(loss)
    bsq.sync_status()


def make(bsq, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, k, E, C, V = 300, 4, 16, 256, 777

    def randn(*s):
        return torch.randn(s, generator=g, device="cuda")
    return {"x": randn(T, C).bfloat16(), "ids": torch.randint(-1, E, (T, k), generator=g, device="cuda"),
            "w": torch.rand((T, k), generator=g, device="cuda"), "gamma": randn(C), "head": (randn(V, C) * 0.1).bfloat16(),
            "t": torch.randint(-1, V, (T,), generator=g, device="cuda"), "E": E}


def calls(bsq, i, stream=None):
    """Every operator once, each on what the one before left; returns all outputs."""
    rows, plan = bsq.moe_dispatch(i["x"], i["ids"], i["E"], stream=stream)
    out = bsq.moe_combine(rows, i["w"], plan, stream=stream)
    y, mean, rstd = bsq.layer_norm(out, i["gamma"], None, stream=stream)
    loss, lse = bsq.linear_cross_entropy(y, i["head"], i["t"], stream=stream)
    dh, dw = bsq.linear_cross_entropy_backward(y, i["head"], i["t"], lse, i["w"][:, 0].contiguous(), stream=stream)
    dx, dg, db = bsq.layer_norm_backward(dh, out, i["gamma"], mean, rstd, stream=stream)
    drows, dweights = bsq.moe_combine_backward(dx, rows, i["w"], plan, stream=stream)
    dtok = bsq.moe_dispatch_backward(drows, plan, stream=stream)
    grads = bsq.GradList([dw.view(-1), dg, db, dtok.view(-1)], [torch.empty_like(t) for t in
                                                               (dw.view(-1), dg, db, dtok.view(-1))])
    norm = bsq.clip_grad_norm(grads, 0.1, stream=stream)
    return [rows, plan.offsets, plan.slot_row, plan.row_slot, out, y, mean, rstd, loss, lse, dh, dw, dx, dg, db, drows,
            dweights, dtok, norm, *grads.outs]


def test_on_another_stream_and_every_time_the_same_bits(bsq):
    i = make(bsq)
    want = [t.clone() for t in calls(bsq, i)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = calls(bsq, i, stream=s)
        # work on the current stream meanwhile must not get at their workspaces
        noise = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
        s.synchronize()
        assert all(torch.equal(a.view(-1).view(torch.uint8), b.view(-1).view(torch.uint8)) for a, b in zip(got, want))
        del noise


def test_graph_replay_equals_stream_launch(bsq):
    i = make(bsq, 1)
    want = [t.clone() for t in calls(bsq, i)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = calls(bsq, i)
    for _ in range(2):
        for t in got:
            t.view(-1).view(torch.uint8).fill_(0xAB)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(-1).view(torch.uint8), b.view(-1).view(torch.uint8)) for a, b in zip(got, want))
    # a second input through the same graph
    j = make(bsq, 2)
    for name in ("x", "ids", "w", "gamma", "head", "t"):
        i[name].copy_(j[name])
    want = [t.clone() for t in calls(bsq, j)]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(-1).view(torch.uint8), b.view(-1).view(torch.uint8)) for a, b in zip(got, want))
    bsq.sync_status()
