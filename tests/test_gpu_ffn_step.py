"""The feed-forward block as the example runs it: the first step's loss and
gradients against the same step in FP64, the update that follows against the
formula; the step on another stream and captured in a CUDA graph; and the
operators in any order, without waiting, on one stream and on two."""
import os
import random
import sys

import pytest
import torch

from _linear_ref import act

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    yield b
    b.sync_status()


def step_fp64(block):
    """Loss and gradients (in the block's order) in FP64, by autograd of the formulas."""
    p = [t.double().requires_grad_() for t in block.params]
    w_gate, w_up, w_down, head, bias, gamma, beta = p
    x = block.x.double()
    c = x - x.mean(1, keepdim=True)
    y = c / (c.square().mean(1, keepdim=True) + 1e-5).sqrt() * gamma + beta
    a = y @ w_gate.T
    out = x + (a * torch.sigmoid(a) * (y @ w_up.T)) @ w_down.T + bias
    n = block.targets >= 0
    loss = torch.nn.functional.cross_entropy((out @ head.T)[n], block.targets[n])
    loss.backward()
    return loss.detach(), [t.grad for t in p]


@pytest.mark.parametrize("mxfp8", [False, True])
def test_a_step_against_fp64(bsq, mxfp8):
    from ffn_step import FeedForward
    block = FeedForward(mxfp8=mxfp8)
    want_loss, want = step_fp64(block)
    loss, norm = block.gradients()
    # BF16: some ten roundings of 2^-9 (root mean square below that) between the input and a gradient, independent; E4M3
    # operands: 2^-4 a value, half of that in the mean, in four of them
    rel = 2.0 ** -3 if mxfp8 else 10 ** 0.5 * 2.0 ** -8
    assert abs(float(loss) - float(want_loss)) < rel / 4 * float(want_loss)
    for i, (got, ref) in enumerate(zip(block.grads, want)):
        assert float((got.double() - ref).norm()) < rel * float(ref.norm()), i
    total = torch.sqrt(sum(g.double().square().sum() for g in block.grads))
    assert abs(float(norm) - float(total)) < 1e-5 * float(total)
    # the update behind it: m = (1 - b1) g, v = (1 - b2) g^2, so that every parameter moves by lr g / (|g| + eps)
    before = [p.double() for p in block.params]
    bsq.adamw_step(block.adam, 1e-3, 1, weight_decay=0.0, norm=norm, max_norm=0.5, seed=3)
    factor = min(1.0, 0.5 / (float(norm) + 1e-6))
    for b, p, g in zip(before, block.params, block.grads):
        g = g.double() * factor
        ref = b - 1e-3 * g / (g.abs() + 1e-8)
        # BF16 parameters are rounded stochastically: by less than a step (2^-7)
        step = (2.0 ** -7 if p.dtype == BF else 2.0 ** -23) * ref.abs().clamp(min=1e-30) + 1e-8
        assert ((p.double() - ref).abs() <= step * 1.001 + 1e-9).all()
    for _ in range(3):
        block.step()
    assert all(torch.isfinite(p).all() for p in block.params)


def inputs(T=300, D=256, N=392, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=g, device="cuda").bfloat16()
    return {"x": randn(T, D), "wg": randn(N, D), "wu": randn(N, D), "wd": randn(D, N), "b": randn(D), "dy": randn(T, D)}


def calls(bsq, i, stream=None):
    """The block forward and backward, and on MXFP8 operands forward; returns all outputs."""
    T, N = i["x"].shape[0], i["wg"].shape[0]
    h, gate, up = (torch.empty((T, N), dtype=BF, device="cuda") for _ in range(3))
    bsq.gated_linear_into(i["x"], i["wg"], i["wu"], h, "gelu_tanh", gate, up, stream=stream)
    z = torch.empty_like(i["dy"])
    y = torch.empty_like(z)
    bsq.linear_into(h, i["wd"], y, i["b"], i["x"], "silu", z, stream=stream)
    dh, dwd, db = bsq.linear_backward(i["dy"], h, i["wd"], z, "silu", stream=stream)
    dx, dwg, dwu = bsq.gated_linear_backward(dh, i["x"], i["wg"], i["wu"], gate, up, "gelu_tanh", stream=stream)
    q = [bsq.empty("mxfp8_e4m3", *t.shape) for t in (i["x"], i["wg"], i["wu"])]
    for t, o in zip((i["x"], i["wg"], i["wu"]), q):
        bsq.quantize_into(t, "mxfp8_e4m3", "row", o, None, stream)
    h8 = bsq.gemm_gated(*q, stream=stream)
    y8 = bsq.gemm_linear(q[0], q[1], None, None, "relu", stream=stream)
    return [h, gate, up, y, z, dh, dwd, db, dx, dwg, dwu, h8, y8]


def same(a, b):
    return all(torch.equal(s.contiguous().view(-1).view(torch.uint8), t.contiguous().view(-1).view(torch.uint8)) for s, t in zip(a, b))


# one token, few, small gradients, one tile, several, and sums in parts
SHAPES = [(1, 256, 392), (3, 64, 40), (7, 256, 104), (60, 512, 392), (300, 256, 392), (520, 4096, 136)]


@pytest.mark.parametrize("shape", SHAPES)
def test_on_another_stream_and_every_time_the_same_bits(bsq, shape):
    i = inputs(*shape)
    want = [t.clone() for t in calls(bsq, i)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = calls(bsq, i)
        noise = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
        s.synchronize()
        assert same(got, want)
        del noise
        got = calls(bsq, i, stream=s)
        s.synchronize()
        assert same(got, want)


@pytest.mark.parametrize("shape", SHAPES)
def test_graph_replay_equals_stream_launch(bsq, shape):
    i = inputs(*shape, seed=1)
    want = [t.clone() for t in calls(bsq, i)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = calls(bsq, i)
    again = torch.cuda.CUDAGraph()
    with torch.cuda.graph(again, stream=side):
        other = calls(bsq, i)
    for _ in range(2):
        for t in got + other:
            t.view(-1).view(torch.uint8).fill_(0xAB)
        # two graphs and calls of the stream itself beside one another
        with torch.cuda.stream(side):
            again.replay()
        graph.replay()
        direct = calls(bsq, i)
        torch.cuda.synchronize()
        assert same(got, want) and same(other, want) and same(direct, want)
    j = inputs(*shape, seed=2)
    for name in i:
        i[name].copy_(j[name])
    want = [t.clone() for t in calls(bsq, j)]
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, want)


def optimizer(bsq, g, rng):
    n = [rng.randint(1, 50000) for _ in range(rng.choice([1, 5, 40]))]
    p_type = rng.choice([BF, F32])
    start = [torch.randn(k, generator=g, device="cuda").to(p_type) for k in n]
    grads = [torch.randn(k, generator=g, device="cuda").to(p_type) for k in n]
    bits, seed = rng.choice([8, 32]), rng.choice([None, 5])

    def call():
        params = [t.clone() for t in start]
        states = bsq.adamw_states(params, bits)
        lists = bsq.AdamWList(params, grads, states)
        norm = bsq.grad_norm(grads)
        for t in (1, 2):
            bsq.adamw_step(lists, 1e-2, t, norm=norm, max_norm=1.0, seed=seed)
        return [*params, *(x for st in states for x in st)]
    return call


@pytest.mark.parametrize("streams", [1, 2])
def test_calls_in_any_order_without_waiting(bsq, streams):
    g, rng = torch.Generator(device="cuda").manual_seed(3), random.Random(streams)
    every = [(lambda i=inputs(*s, seed=k): calls(bsq, i)) for k, s in enumerate(SHAPES * 2)]
    every += [optimizer(bsq, g, rng) for _ in range(8)]
    want = []
    for call in every:
        out = call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    on = [torch.cuda.current_stream()] if streams == 1 else [torch.cuda.Stream() for _ in range(streams)]
    for _ in range(3):
        order = rng.sample(range(len(every)), len(every))
        torch.cuda.synchronize()
        got = {}
        for n, i in enumerate(order):
            with torch.cuda.stream(on[n % streams]):
                got[i] = every[i]()
        torch.cuda.synchronize()
        for i in order:
            assert same(got[i], want[i]), i


@pytest.mark.parametrize("T,D", [(1, 2048), (2, 1024), (4, 1024), (20, 1024), (60, 64), (200, 512), (600, 512)])
def test_every_call_reads_what_the_one_before_wrote(bsq, T, D):
    # calls that start beside the one before them, each on its results, over two buffers that are written again and
    # again: the same as with a wait after each of them
    g = torch.Generator(device="cuda").manual_seed(T)
    w = [(torch.randn((D, D), generator=g, device="cuda") * D ** -0.5).to(BF) for _ in range(3)]
    start = torch.randn((T, D), generator=g, device="cuda").to(BF)

    def chain(wait):
        a, b, c, dw = start.clone(), torch.empty_like(start), torch.empty_like(start), torch.empty_like(w[0])
        weights = [t.clone() for t in w]
        lists = bsq.AdamWList(weights, [dw] * 3, 8)
        q = bsq.empty("mxfp8_e4m3", T, D)
        qw = bsq.empty("mxfp8_e4m3", D, D)
        for k in range(1, 16):
            bsq.linear_into(a, weights[0], b, None, a, "gelu")
            wait()
            bsq.gated_linear_into(b, weights[1], weights[2], a)
            wait()
            bsq.linear_backward_into(a, b, weights[0], c, dw)
            wait()
            bsq.adamw_step(lists, 1e-2, k, weight_decay=0.1, seed=1)
            wait()
            bsq.layer_norm_into(c, None, None, 1e-5, b)
            wait()
            bsq.quantize_into(b, "mxfp8_e4m3", "row", q, None)
            bsq.quantize_into(weights[k % 3], "mxfp8_e4m3", "row", qw, None)
            wait()
            bsq.gemm_linear_into(q, qw, a)
            wait()
            bsq.gemm_gated_into(q, qw, qw, b)
            wait()
            bsq.layer_norm_into(b, None, None, 1e-5, a)
            wait()
        torch.cuda.synchronize()
        return [a, b, c, dw, *weights]

    want = chain(torch.cuda.synchronize)
    assert all(torch.isfinite(t).all() for t in want)
    for _ in range(4):
        assert same(chain(lambda: None), want)


def test_forward_and_backward_are_those_of_autograd(bsq):
    # the formulas once more, as torch differentiates them
    i = inputs(130, 64, 72)
    for name in ("identity", "relu", "silu", "gelu", "gelu_tanh"):
        x, wg, wu = (i[k].double().requires_grad_() for k in ("x", "wg", "wu"))
        a, u = x @ wg.T, x @ wu.T
        h = act(name, a)[0] * u
        dh = i["dy"][:, :1].double().expand(130, 72).contiguous()
        h.backward(dh)
        got = bsq.gated_linear_backward(dh.to(BF), i["x"], i["wg"], i["wu"], a.detach().to(BF), u.detach().to(BF), name)
        # gate and up rounded to BF16, then dgate and dup, then the results: independent, 2^-9 in the mean
        for d, t in zip(got, (x, wg, wu)):
            assert float((d.double() - t.grad).norm()) < 4 * 2.0 ** -8 * float(t.grad.norm()), name
