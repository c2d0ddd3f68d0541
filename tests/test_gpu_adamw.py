"""AdamW against a restatement in numpy, bit for bit: every pair of types, moments
in 32 and 8 bits, rounded to nearest and stochastically, odd and empty tensors, any
alignment, lists longer than one launch takes, clipping in the same pass, the step's
number on the device; and what the stochastic rounding is for."""
import math

import numpy as np
import pytest
import torch

from _linear_ref import E4M3, adamw_ref, decode

pytestmark = pytest.mark.gpu
BF, F32, F32N = torch.bfloat16, torch.float32, np.float32
HYPER = dict(lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    return b


def pieces(sizes, dtype, offset, values):
    """Tensors of the sizes one behind another in a buffer, the first `offset` elements into it, 3 apart."""
    buf = torch.full((sum(sizes) + 3 * len(sizes) + offset + 64,), float("nan") if dtype.is_floating_point else 0xAB, dtype=dtype,
                     device="cuda")
    out, at = [], offset
    for n, v in zip(sizes, values):
        out.append(buf[at:at + n])
        out[-1].copy_(v)
        at += n + 3
    return out


def make(bsq, sizes, p_type, g_type, bits, offset, seed, scale=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(n, s):
        return torch.randn(n, generator=g, device="cuda") * s

    params = pieces(sizes, p_type, offset, [randn(n, 0.3) for n in sizes])
    grads = pieces(sizes, g_type, offset, [randn(n, scale) for n in sizes])
    if bits == 32:
        ms = pieces(sizes, F32, offset, [randn(n, scale) for n in sizes])
        vs = pieces(sizes, F32, offset, [randn(n, scale).square() for n in sizes])
        states = list(zip(ms, vs))
    else:
        blocks = [-(-n // 32) for n in sizes]

        def codes(top):
            c = [torch.randint(0, 0x7F, (n,), generator=g, device="cuda").byte() for n in sizes]
            return [x | (torch.randint(0, 2, x.shape, generator=g, device="cuda").byte() << 7) for x in c] if top else c

        scales = [[torch.randint(108, 114, (n,), generator=g, device="cuda").byte() for n in blocks] for _ in range(2)]
        cols = [pieces(sizes, torch.uint8, offset, codes(True)), pieces(blocks, torch.uint8, 0, scales[0]),
                pieces(sizes, torch.uint8, offset, codes(False)), pieces(blocks, torch.uint8, 0, scales[1])]
        states = list(zip(*cols))
    return params, grads, states


def host(t):
    return t.float().cpu().numpy() if t.dtype == BF else t.cpu().numpy()


def equal(a, b):
    return np.array_equal(a, b, equal_nan=a.dtype.kind == "f")


def to(x, dtype):
    return host(torch.from_numpy(np.ascontiguousarray(x)).to(dtype))


def check(bsq, params, grads, states, step=7, seed=None, norm=None, max_norm=None, copies=None, device=False):
    lists = bsq.AdamWList(params, grads, states, copies)
    before = [(host(p), host(g), tuple(host(s) for s in st)) for p, g, st in zip(params, grads, states)]
    factor = None
    if norm is not None:
        factor = np.minimum(np.float32(max_norm) / (np.float32(float(norm)) + np.float32(1e-6)), np.float32(1))
    bsq.adamw_step(lists, HYPER["lr"], step, HYPER["betas"], HYPER["eps"], HYPER["weight_decay"], norm=norm,
                   max_norm=max_norm, seed=seed)
    for i, (p, g, st) in enumerate(before):
        q, copy, state = adamw_ref(p, g, st, HYPER["lr"], step, HYPER["betas"], HYPER["eps"], HYPER["weight_decay"], factor, seed, i,
                                   params[i].dtype == BF)
        for k, (a, b) in enumerate(zip(states[i], state)):
            assert equal(host(a), b), f"tensor {i}: moments {k}: {int((host(a) != b).sum())} of {len(b)} differ"
        assert equal(host(params[i]), to(q, params[i].dtype)), f"tensor {i}: parameters"
        assert equal(host(grads[i]), g)
        if copies is not None and copies[i] is not None:
            assert equal(host(copies[i]), to(copy, BF)), f"tensor {i}: copy"


SIZES = [[1], [31], [32, 0, 33], [7, 8, 9, 64, 127], [2048, 2047, 2049], [5000, 1, 4096 + 40], [100003]]


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("seed", [None, 0x123456789ABC])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_type,g_type", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
def test_step(bsq, p_type, g_type, bits, seed, offset):
    for i, sizes in enumerate(SIZES):
        params, grads, states = make(bsq, sizes, p_type, g_type, bits, offset, i)
        check(bsq, params, grads, states, step=1 + 3 * i, seed=seed)


# only the moments on 16-byte boundaries: parameters, gradients and copies each somewhere else
@pytest.mark.parametrize("seed", [None, 99])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_type,g_type", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
def test_parameters_off_16_byte_boundaries(bsq, p_type, g_type, bits, seed):
    for sizes in ([70000, 255, 4096], [1025, 2048]):
        for at, (p_off, g_off, c_off) in enumerate([(1, 0, 2), (2, 1, 0), (0, 2, 1), (3, 3, 3), (0, 0, 1)]):
            params, grads, states = make(bsq, sizes, p_type, g_type, bits, 0, at)
            params, grads = pieces(sizes, p_type, p_off, params), pieces(sizes, g_type, g_off, grads)
            copies = pieces(sizes, BF, c_off, [torch.zeros(n, device="cuda") for n in sizes]) if at % 2 == 0 else None
            check(bsq, params, grads, states, seed=seed, copies=copies)


@pytest.mark.parametrize("bits", [32, 8])
def test_several_steps_from_nothing(bsq, bits):
    g = torch.Generator(device="cuda").manual_seed(1)
    params = [torch.randn(n, generator=g, device="cuda") for n in (1000, 77)]
    states = bsq.adamw_states(params, bits)
    for step in range(1, 6):
        grads = [torch.randn(p.shape, generator=g, device="cuda") * 10.0 ** -step for p in params]
        check(bsq, params, grads, states, step=step, seed=step)


@pytest.mark.parametrize("bits", [32, 8])
def test_copies_and_clipping(bsq, bits):
    sizes = [3000, 50]
    params, grads, states = make(bsq, sizes, F32, BF, bits, 0, 5)
    copies = [torch.full((3000,), float("nan"), dtype=BF, device="cuda"), None]
    norm = bsq.grad_norm(grads)
    check(bsq, params, grads, states, norm=norm, max_norm=0.25, copies=copies, seed=9)
    check(bsq, params, grads, states, norm=norm, max_norm=1e9, copies=copies)
    check(bsq, params, grads, states, norm=torch.zeros(1, device="cuda"), max_norm=0.0)


@pytest.mark.parametrize("seed", [None, 77])
def test_a_tensor_of_more_than_2_32_elements(bsq, seed):
    n, tail, step = (1 << 32) + 5003, 5003, 3
    param, grad = (torch.zeros(n, dtype=BF, device="cuda") for _ in range(2))
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    (p,), (g,), (st,) = make(bsq, [tail], BF, BF, 8, 0, 5)
    first = 1 << 32
    for whole, part in ((param, p), (grad, g), (m, st[0]), (v, st[2])):
        whole[first:] = part
    ms[first // 32:], vs[first // 32:] = st[1], st[3]
    bsq.adamw_step(bsq.AdamWList([param], [grad], [(m, ms, v, vs)]), HYPER["lr"], step, HYPER["betas"], HYPER["eps"],
                   HYPER["weight_decay"], seed=seed)
    q, _, state = adamw_ref(host(p), host(g), tuple(host(s) for s in st), HYPER["lr"], step, HYPER["betas"], HYPER["eps"],
                            HYPER["weight_decay"], None, seed, 0, True, first)
    assert equal(host(param[first:]), to(q, BF))
    for got, want in zip((m[first:], ms[first // 32:], v[first:], vs[first // 32:]), state):
        assert equal(host(got), want)
    # everything before is 0 and stays so
    assert not param[:4096].any() and not param[first - 4096:first].any() and not m[:first].any() and not v[:first].any()


def test_many_tensors(bsq):
    sizes = [1 + i % 40 for i in range(1000)]
    params, grads, states = make(bsq, sizes, F32, F32, 8, 0, 2)
    check(bsq, params, grads, states, seed=4)
    # both kinds of moments in one list
    a, b = make(bsq, [100, 200], BF, F32, 32, 0, 3), make(bsq, [300, 70], F32, BF, 8, 0, 4)
    check(bsq, a[0] + b[0], a[1] + b[1], a[2] + b[2], seed=1)


def test_step_and_rate_on_the_device(bsq):
    # the scalars come from FP32 there: 1 - beta^t to 4 roundings, the quotient and its root; the update to 8 U more
    for step in (1, 2, 100, 100000):
        params, grads, states = make(bsq, [3000], F32, F32, 32, 0, step)
        other = [p.clone() for p in params], [tuple(s.clone() for s in st) for st in states]
        t, lr = torch.tensor([step], device="cuda"), torch.tensor([HYPER["lr"]], dtype=F32, device="cuda")
        before = params[0].clone()
        bsq.adamw_step(bsq.AdamWList(params, grads, states), HYPER["lr"], step, HYPER["betas"], HYPER["eps"], HYPER["weight_decay"])
        bsq.adamw_step(bsq.AdamWList(other[0], grads, other[1]), lr, t, HYPER["betas"], HYPER["eps"], HYPER["weight_decay"])
        assert all(torch.equal(a, b) for a, b in zip(states[0], other[1][0]))
        moved = (params[0] - before).abs()
        assert ((params[0] - other[0][0]).abs() <= 16 * 2.0 ** -24 * (moved + before.abs() * HYPER["lr"]) + 2.0 ** -23 * before.abs()).all()


def test_a_captured_step_counts_on(bsq):
    g = torch.Generator(device="cuda").manual_seed(0)
    params = [torch.randn(500, generator=g, device="cuda").to(BF)]
    grads = [torch.randn(500, generator=g, device="cuda").to(BF)]
    lists = bsq.AdamWList(params, grads, 8)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    start = params[0].clone()

    def one():
        step.add_(1)
        bsq.adamw_step(lists, 1e-2, step, seed=3)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        one()
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    got = params[0].clone(), [s.clone() for s in lists.states[0]]
    params[0].copy_(start)
    step.zero_()
    for s in lists.states[0]:
        s.zero_()
    for _ in range(4):
        one()
    assert int(step) == 4 and torch.equal(params[0], got[0]) and all(torch.equal(a, b) for a, b in zip(lists.states[0], got[1]))


@pytest.mark.parametrize("bits", [32, 8])
def test_values_that_are_not_finite(bsq, bits):
    for p_type in (F32, BF):
        params, grads, states = make(bsq, [200], p_type, F32, bits, 0, 8)
        grads[0][40], grads[0][100], params[0][150], params[0][160] = float("nan"), float("inf"), float("inf"), float("nan")
        check(bsq, params, grads, states, seed=2)
    params, grads, states = make(bsq, [200], F32, F32, bits, 0, 8)
    grads[0][40] = float("nan")
    grads[0][100] = float("inf")
    clean = [t.clone() for t in (*params, *states[0])]
    check(bsq, params, grads, states, seed=2)
    if bits == 8:
        # their blocks of 32 are NaN from then on, the others are as they would be
        assert (states[0][1][[1, 3]] == 255).all() and (states[0][0][32:64] == 0x7F).all() and (states[0][2][96:128] == 0x7F).all()
        assert torch.isfinite(params[0][:40]).all() and torch.isfinite(params[0][101:]).all()
        grads[0][40] = grads[0][100] = 0
        bsq.adamw_step(bsq.AdamWList(params, grads, states), 1e-3, 8)
        assert torch.isnan(params[0][32:64]).all() and torch.isfinite(params[0][128:]).all()
    assert torch.isfinite(clean[0]).all()


def test_extreme_blocks(bsq):
    # zeros, the smallest and largest magnitudes, and elements far below their block's largest
    m = torch.zeros(256, device="cuda")
    v = torch.zeros(256, device="cuda")
    m[32:64] = 1e-45
    m[64:96] = 3e38
    m[96] = 1.0
    m[97:128] = 2.0 ** -torch.arange(1, 32, device="cuda").float()
    m[128:160] = 448.0
    v[32:64] = 1e-45
    v[64:96] = 3e38
    v[96] = 1.0
    v[97:128] = 4.0 ** -torch.arange(1, 32, device="cuda").float()
    p, g = torch.ones(256, device="cuda"), torch.zeros(256, device="cuda")
    for seed in (None, 5):
        states = bsq.adamw_states([p], 8)
        lists = bsq.AdamWList([p], [g], states)
        # moments come to the 8 bits by a step from FP32: beta = 0 takes them from the gradient
        grad = m.clone()
        lists = bsq.AdamWList([p.clone()], [grad], states)
        bsq.adamw_step(lists, 0.0, 1, betas=(0.0, 0.0), seed=seed)
        want = adamw_ref(host(p), host(grad), tuple(np.zeros(k, np.uint8) for k in (256, 8, 256, 8)), 0.0, 1, (0.0, 0.0), 1e-8, 0.01,
                         None, seed)[2]
        for a, b in zip(states[0], want):
            assert equal(host(a), b)
        # a second moment that is not 0 has a code that is not
        assert torch.equal(states[0][2] != 0, grad * grad != 0)


def test_stochastic_rounding_moves_as_it_should_on_average(bsq):
    # v decays by 0.1% a step: to nearest its codes never move, stochastically they follow on average
    n, steps = 1 << 16, 200
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    codes = torch.randint(40, 0x70, (n,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).byte()
    codes[::32] = 0x7E                                  # keeps every block's scale for a while
    scales = torch.full((n // 32,), 120, dtype=torch.uint8, device="cuda")
    kept, ratio = [], []
    for seed in (None, 11):
        state = [(torch.zeros_like(codes), torch.zeros_like(scales), codes.clone(), scales.clone())]
        lists = bsq.AdamWList([p], [g], state)
        for t in range(1, steps + 1):
            bsq.adamw_step(lists, 0.0, t, seed=seed)
        kept.append(float((state[0][2] == codes).float().mean()))
        r = decode(host(state[0][2]), host(state[0][3])) / decode(host(codes), host(scales))
        ratio.append(float(np.mean(r)))
    want = 0.999 ** (steps / 2)
    assert kept[0] > 0.95 and ratio[0] > 0.99
    # a step's rounding has a deviation of at most half a step, 2^-4 of the value; 200 of them and 65536 elements
    assert abs(ratio[1] - want) <= 6 * 2.0 ** -4 * math.sqrt(steps / n)
    assert E4M3[0x7E] == 448


def test_root_and_quotient_are_correctly_rounded(bsq):
    # with beta1 = 0 and beta2 = 1/2 far from the first step, weight decay and eps 0 and lr 1, p' = -(g / sqrt(v / 2 + g^2 / 2)):
    # every mantissa of v under two exponents with a g that does not reach it, then random quotients
    grid = (np.arange(1 << 23, dtype=np.uint32) | (np.uint32(127) << np.uint32(23))).view(F32N)
    rng = np.random.default_rng(0)
    for k, (v, g) in enumerate([(grid, np.full(1 << 23, 2.0 ** -40, F32N)), (grid * F32N(2), np.full(1 << 23, 2.0 ** -40, F32N)),
                                (grid, (1 + rng.random(1 << 23)).astype(F32N) * F32N(2.0 ** -30)),
                                (rng.random(1 << 23).astype(F32N) * F32N(1e-10), rng.standard_normal(1 << 23).astype(F32N) * F32N(1e-5)),
                                (np.ldexp(grid, rng.integers(-140, 120, 1 << 23)).astype(F32N), np.full(1 << 23, 0.75, F32N))]):
        p = torch.zeros(1 << 23, device="cuda")
        m, vt = torch.zeros(1 << 23, device="cuda"), torch.from_numpy(v.copy()).cuda()
        bsq.adamw_step(bsq.AdamWList([p], [torch.from_numpy(g).cuda()], [(m, vt)]), 1.0, 100, betas=(0.0, 0.5), eps=0.0, weight_decay=0.0)
        with np.errstate(over="ignore"):
            want = F32N(0.5) * v + (F32N(0.5) * g) * g
            q = F32N(0) - F32N(1) * (g / np.sqrt(want))
        assert np.array_equal(host(vt), want) and np.array_equal(host(m), g)
        got = host(p)
        assert np.array_equal(got, q), (k, int((got != q).sum()))


def test_refusals(bsq):
    p, g = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    m, v = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    ok = bsq.AdamWList([p], [g], [(m, v)])
    c, s = torch.zeros(64, dtype=torch.uint8, device="cuda"), torch.zeros(2, dtype=torch.uint8, device="cuda")
    bad = [lambda: bsq.AdamWList([], []), lambda: bsq.AdamWList([p], []), lambda: bsq.AdamWList([p], [g[:3]]),
           lambda: bsq.AdamWList([p.half()], [g]), lambda: bsq.AdamWList([p], [g[::2]]), lambda: bsq.AdamWList([p.cpu()], [g]),
           lambda: bsq.AdamWList([p], [g], 16), lambda: bsq.AdamWList([p], [g], [(m,)]),
           lambda: bsq.AdamWList([p], [g], [(m, v.to(BF))]), lambda: bsq.AdamWList([p], [g], [(c, s[:1], c, s)]),
           lambda: bsq.AdamWList([p], [g], copies=[p]), lambda: bsq.AdamWList([p], [g], copies=[]),
           lambda: bsq.adamw_step(ok, -1.0, 1), lambda: bsq.adamw_step(ok, 1e-3, 0),
           lambda: bsq.adamw_step(ok, float("nan"), 1), lambda: bsq.adamw_step(ok, 1e-3, 1, betas=(1.0, 0.9)),
           lambda: bsq.adamw_step(ok, 1e-3, 1, betas=(0.9, -0.1)), lambda: bsq.adamw_step(ok, 1e-3, 1, eps=float("inf")),
           lambda: bsq.adamw_step(ok, 1e-3, 1, weight_decay=-1.0), lambda: bsq.adamw_step(ok, 1e-3, 1, max_norm=1.0),
           lambda: bsq.adamw_step(ok, 1e-3, 1, norm=torch.ones(1, device="cuda")),
           lambda: bsq.adamw_step(ok, 1e-3, 1, norm=torch.ones(2, device="cuda"), max_norm=1.0),
           lambda: bsq.adamw_step(ok, torch.ones(1, device="cuda").double(), 1),
           lambda: bsq.adamw_step(ok, 1e-3, torch.ones(1, device="cuda"))]
    for i, f in enumerate(bad):
        with pytest.raises(bsq.BsqError):
            f()
            pytest.fail(f"case {i} was not refused")
    assert (p == 1).all() and (m == 0).all()
