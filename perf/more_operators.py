"""The dense feed-forward block of a training or serving step, and the optimizer
that updates its weights: what is measured.

Three operators, each in a plain form (elementary torch operations in FP32,
rounded once at the end) and as the calls a user makes of the library:

  linear  act(x w^T + bias) + residual in one kernel, forward (BF16 operands, or
          MXFP8 codes and scales) and backward (dx, dw, dbias)
  gated   act(x wg^T) * (x wu^T), both projections in one kernel, forward (BF16
          or MXFP8) and backward (dx, dwg, dwu)
  adamw   one AdamW step over many tensors, moments in FP32 or in 8 bits (E4M3
          codes with one E8M0 scale for 32), with the gradients' clipping

A case is a dict of plain values; its "op" says which pass it is.  Sizes are
those of this repository's own workloads (hidden 4096, an MLP width of 14336,
8192 rows, a layer's 243 M weights) or generic ones."""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
BETAS, ADAM_EPS, DECAY, LR, MAX_NORM, CLIP_EPS = (0.9, 0.999), 1e-8, 0.1, 1e-3, 1.0, 1e-6
MOST_FLOPS = 8 * 8192 * 4096 * 14336


def listed():
    return [
        # the down projection of one decoded token, added to its residual stream: the weights are read once
        {"name": "linear, one token", "op": "linear", "tokens": 1, "cols": 14336, "out": 4096, "dtype": "bf16",
         "act": "identity", "bias": False, "residual": True, "keep": False},
        # a small ragged batch through a biased layer, its pre-activation kept for the backward pass
        {"name": "linear, odd", "op": "linear", "tokens": 1021, "cols": 2040, "out": 1531, "dtype": "bf16",
         "act": "gelu", "bias": True, "residual": False, "keep": True},
        # the down projection of a training batch, added to the residual stream
        {"name": "linear, batch", "op": "linear", "tokens": 8192, "cols": 14336, "out": 4096, "dtype": "bf16",
         "act": "identity", "bias": False, "residual": True, "keep": False},
        # the up projection of a biased MLP on MXFP8 operands, which the quantize calls left
        {"name": "linear, MXFP8 batch", "op": "linear", "tokens": 8192, "cols": 4096, "out": 14336, "dtype": "mxfp8",
         "act": "gelu_tanh", "bias": True, "residual": False, "keep": False},
        # the backward pass of a biased up projection
        {"name": "linear gradient, batch", "op": "linear_grad", "tokens": 8192, "cols": 4096, "out": 14336,
         "dtype": "bf16", "act": "gelu_tanh", "bias": True},
        # one decoded token through the gated half of an MLP: both weights are read once
        {"name": "gated, one token", "op": "gated", "tokens": 1, "cols": 4096, "width": 14336, "dtype": "bf16",
         "act": "silu", "keep": False},
        # a training batch, with what the backward pass takes
        {"name": "gated, batch", "op": "gated", "tokens": 8192, "cols": 4096, "width": 14336, "dtype": "bf16",
         "act": "silu", "keep": True},
        # a prompt on MXFP8 operands
        {"name": "gated, MXFP8 prompt", "op": "gated", "tokens": 2048, "cols": 4096, "width": 14336,
         "dtype": "mxfp8", "act": "silu", "keep": False},
        # the backward pass of the training batch
        {"name": "gated gradient, batch", "op": "gated_grad", "tokens": 8192, "cols": 4096, "width": 14336,
         "dtype": "bf16", "act": "silu"},
        # an adapter's many small tensors, off 16-byte boundaries: latency
        {"name": "adamw, small tensors", "op": "adamw", "tensors": 61, "elements": 200003, "param": "f32",
         "grad": "f32", "bits": 32, "aligned": False, "clip": False, "stochastic": False},
        # one layer of the repository's MLP and projection shapes: BF16 weights and gradients, FP32 moments
        {"name": "adamw, one layer", "op": "adamw", "tensors": 12, "elements": 243300000, "param": "bf16",
         "grad": "bf16", "bits": 32, "aligned": True, "clip": True, "stochastic": False},
        # the same layer with moments in 8 bits, weights and moments rounded stochastically
        {"name": "adamw, one layer, 8 bits", "op": "adamw", "tensors": 12, "elements": 243300000, "param": "bf16",
         "grad": "bf16", "bits": 8, "aligned": True, "clip": True, "stochastic": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "gated", "gated", "gated_grad", "adamw", "adamw"])
    if op == "adamw":
        n = _log(rng, 1, 400)
        return {"op": op, "tensors": n, "elements": n + _log(rng, 1000, 200000000), "param": rng.choice(["bf16", "f32"]),
                "grad": rng.choice(["bf16", "f32"]), "bits": rng.choice([8, 32]), "aligned": rng.random() < 0.6,
                "clip": rng.random() < 0.5, "stochastic": rng.random() < 0.5}
    gated = op.startswith("gated")
    case = {"op": op, "tokens": _log(rng, 1, 8192)}
    mx = not op.endswith("grad") and rng.random() < 0.35
    case["cols"] = 32 * _log(rng, 2, 448) if mx else 8 * _log(rng, 8, 1792)
    wide = _log(rng, 33, 14336)
    per = {"linear": 2, "linear_grad": 4, "gated": 4, "gated_grad": 8}[op] * case["tokens"] * case["cols"]
    wide = max(33, min(wide, MOST_FLOPS // per))
    if rng.random() < 0.6:
        wide = max(40, wide // 8 * 8)
    case["width" if gated else "out"] = wide
    case["dtype"] = "mxfp8" if mx else "bf16"
    case["act"] = rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]) if gated else \
        rng.choice(["identity", "identity", "relu", "silu", "gelu", "gelu_tanh"])
    if not gated:
        case["bias"] = rng.random() < 0.6
    if op == "linear":
        case["residual"] = rng.random() < 0.5
    if not op.endswith("grad"):
        case["keep"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _power(byte):
    """2^(byte - 127)"""
    bits = byte.to(torch.int32)
    return torch.where(bits == 0, torch.full_like(bits, 1 << 22), bits << 23).view(torch.float32)


def _mxfp8(x):
    """x [rows, cols] as the library's MXFP8 E4M3 tensors hold it: codes uint8 [rows * cols], and one E8M0 byte for 32
    in 512-byte tiles of 128 rows x 4 scale columns."""
    R, C = x.shape
    S = C // 32
    amax = x.reshape(R, S, 32).abs().amax(2)
    byte = ((amax.view(torch.int32) >> 23) - 8).clamp(min=0)
    v = (x.reshape(R, S, 32) * _power(254 - byte)[:, :, None]).clamp(-448, 448)
    codes = v.to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1)
    tiles = torch.zeros((-(-R // 128) * 128, -(-S // 4) * 4), dtype=torch.uint8, device=x.device)
    tiles[:R, :S] = byte.to(torch.uint8)
    tiles = tiles.reshape(tiles.shape[0] // 128, 4, 32, tiles.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return {"codes": codes, "scales": tiles.reshape(-1).contiguous(), "rows": R, "cols": C}


def _values(q, dtype):
    """The values that codes and scales stand for."""
    R, C = q["rows"], q["cols"]
    S = C // 32
    tiles = q["scales"].reshape(-(-R // 128), -(-S // 4), 32, 4, 4).permute(0, 3, 2, 1, 4)
    byte = tiles.reshape(-(-R // 128) * 128, -(-S // 4) * 4)[:R, :S]
    v = q["codes"].view(torch.float8_e4m3fn).to(dtype).reshape(R, S, 32)
    return (v * _power(byte).to(dtype)[:, :, None]).reshape(R, C)


def _starts(case):
    """Where each tensor starts (a multiple of 32 elements, aligned: of 256), its length, and the pool's length."""
    n, total = case["tensors"], case["elements"]
    share = [1.0 + 40.0 * (i % 3 == 0) + 7.0 * (i % 4 == 1) for i in range(n)]
    sizes = [max(1, int(total * s / sum(share))) for s in share]
    sizes[0] += max(0, total - sum(sizes))
    pitch, at, spans = 256 if case["aligned"] else 32, 0, []
    for k in sizes:
        spans.append((at, k))
        at += -(-k // pitch) * pitch
    return spans, at


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "adamw":
        return _prepare_adamw(s, case, seed, g)
    T, D = case["tokens"], case["cols"]
    x = _normal(g, (T, D))
    F = case["width"] if op.startswith("gated") else case["out"]
    names = ["w_gate", "w_up"] if op.startswith("gated") else ["w"]
    ws = {k: _normal(g, (F, D), D ** -0.5) for k in names}
    if case["dtype"] == "mxfp8":
        s["x"] = _mxfp8(x)
        for k in names:
            s[k] = _mxfp8(ws[k])
        if own:
            import block_scaled_precision_03_gb300 as bsq
            for k in ["x"] + names:
                q = s[k]
                s[k] = bsq.QTensor(bsq.MXFP8_E4M3, q["rows"], q["cols"], q["codes"], q["scales"], None)
    else:
        s["x"] = x.bfloat16()
        for k in names:
            s[k] = ws[k].bfloat16()

    def out(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "linear":
        s["bias"] = 0.1 * _normal(g, (F,)) if case["bias"] else None
        s["residual"] = _normal(g, (T, F)).bfloat16() if case["residual"] else None
        s["y"], s["z"] = out(T, F), out(T, F) if case["keep"] else None
    elif op == "gated":
        s["h"] = out(T, F)
        s["gate"], s["up"] = (out(T, F) if case["keep"] else None for _ in range(2))
    elif op == "linear_grad":
        s["dy"] = _normal(g, (T, F), 1e-3).bfloat16()
        # a quarter of the tokens is padding, whose gradient is 0
        s["dy"][torch.rand((T,), generator=g, device="cuda") < 0.25] = 0
        bias = 0.1 * _normal(g, (F,))
        s["z"] = None if case["act"] == "identity" else (s["x"].float() @ s["w"].float().T + bias).bfloat16()
        s["dx"], s["dw"] = out(T, D), out(F, D)
        s["dbias"] = out(F, dtype=torch.float32) if case["bias"] else None
    else:
        s["dh"] = _normal(g, (T, F), 1e-3).bfloat16()
        s["dh"][torch.rand((T,), generator=g, device="cuda") < 0.25] = 0
        s["gate"], s["up"] = ((s["x"].float() @ s[k].float().T).bfloat16() for k in names)
        s["dx"], s["dw_gate"], s["dw_up"] = out(T, D), out(F, D), out(F, D)
    return s


def _prepare_adamw(s, case, seed, g):
    spans, n = _starts(case)
    shift = 0 if case["aligned"] else 1
    live = torch.zeros(n, dtype=torch.bool, device="cuda")
    for at, k in spans:
        live[at:at + k] = True

    def pool(dtype, values):
        p = torch.zeros(n + shift, dtype=dtype, device="cuda")
        p[shift:] = torch.where(live, values, torch.zeros_like(values)).to(dtype)
        return p

    s["p"] = pool(DT[case["param"]], 0.02 * _normal(g, (n,)))
    size = 10.0 ** (-4 - 2 * torch.rand(n // 32, generator=g, device="cuda"))       # gradients differ from block to block
    size = size.repeat_interleave(32)
    s["g"] = pool(DT[case["grad"]], _normal(g, (n,)) * size)
    m = torch.where(live, 0.3 * _normal(g, (n,)) * size, torch.zeros_like(size))
    r = torch.where(live, (0.7 + 0.6 * torch.rand(n, generator=g, device="cuda")) * size, torch.zeros_like(size))
    if case["bits"] == 32:
        s["m"], s["v"] = m, r * r
    else:
        for k, x in (("m", m), ("v", r)):           # the second moment is held as its root
            amax = x.abs().reshape(-1, 32).amax(1)
            byte = (((amax * (8 / 7)).view(torch.int32) >> 23) - 8).clamp(min=0)
            codes = (x.reshape(-1, 32) * _power(254 - byte)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[k], s[k + "_scales"] = codes.view(torch.uint8).reshape(-1), byte.to(torch.uint8)
    s["norm"] = s["g"].float().square().sum().sqrt().reshape(1) if case["clip"] else None
    if s["norm"] is not None:
        s["norm"] += 2.0                            # of more gradients than these
    s["t"], s["seed"] = 100, seed
    if case["stochastic"]:
        # which tensor a block of 32 elements belongs to, and its place there
        s["tensor"] = torch.zeros(n // 32, dtype=torch.int64, device="cuda")
        s["place"] = torch.zeros(n // 32, dtype=torch.int64, device="cuda")
        for i, (at, k) in enumerate(spans):
            b = -(-k // 32)
            s["tensor"][at // 32:at // 32 + b] = i
            s["place"][at // 32:at // 32 + b] = 32 * torch.arange(b, device="cuda")
    if own:
        import block_scaled_precision_03_gb300 as bsq
        if case["bits"] == 32:
            states = [(s["m"][a:a + k], s["v"][a:a + k]) for a, k in spans]
        else:
            states = [(s["m"][a:a + k], s["m_scales"][a // 32:a // 32 + -(-k // 32)],
                       s["v"][a:a + k], s["v_scales"][a // 32:a // 32 + -(-k // 32)]) for a, k in spans]
        s["list"] = bsq.AdamWList([s["p"][shift + a:shift + a + k] for a, k in spans],
                                  [s["g"][shift + a:shift + a + k] for a, k in spans], states)
    return s


# ------------------------------------------------------------ plain forms
def _act(name, z):
    if name == "identity":
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z / (1 + (-z).exp())
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z / (1 + (-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)).exp())


def _act_grad(name, z):
    if name == "identity":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        q = 1 / (1 + (-z).exp())
        return q * (1 + z * (1 - q))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * (-0.5 * z * z).exp() / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    q = 1 / (1 + (-2 * c * (z + 0.044715 * z * z * z)).exp())
    return q + 2 * c * z * q * (1 - q) * (1 + 3 * 0.044715 * z * z)


def _operand(v):
    return _values(v, torch.float32) if isinstance(v, dict) else v.float()


def _plain_linear(s):
    z = _operand(s["x"]) @ _operand(s["w"]).T
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(s["case"]["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.bfloat16(), "z": z.bfloat16() if s["z"] is not None else None}


def _plain_linear_grad(s):
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_grad(s["case"]["act"], s["z"].float())
    return {"dx": (dz @ s["w"].float()).bfloat16(), "dw": (dz.T @ s["x"].float()).bfloat16(),
            "dbias": dz.sum(0) if s["dbias"] is not None else None}


def _plain_gated(s):
    x = _operand(s["x"])
    a, u = x @ _operand(s["w_gate"]).T, x @ _operand(s["w_up"]).T
    h = (_act(s["case"]["act"], a) * u).bfloat16()
    return {"h": h, "gate": a.bfloat16(), "up": u.bfloat16()} if s["gate"] is not None else {"h": h}


def _plain_gated_grad(s):
    a, u, dh, x = s["gate"].float(), s["up"].float(), s["dh"].float(), s["x"].float()
    da, du = dh * u * _act_grad(s["case"]["act"], a), dh * _act(s["case"]["act"], a)
    return {"dx": (da @ s["w_gate"].float() + du @ s["w_up"].float()).bfloat16(),
            "dw_gate": (da.T @ x).bfloat16(), "dw_up": (du.T @ x).bfloat16()}


def _mix(x):
    """A permutation of the 32-bit integers, held in int64 (multiply and xor-shift, the constants of C. Wellons'
    lowbias32)."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random(s, t):
    """32 random bits for every element, as [blocks, 32]: from the seed, the step, the tensor's place in the list and
    the element's in the tensor (below 2^32 here)."""
    seed = s["seed"]
    key = _mix(s["tensor"] ^ (seed & 0xFFFFFFFF))
    key = _mix(key ^ (seed >> 32) & 0xFFFFFFFF)
    key = _mix(key ^ (t & 0xFFFFFFFF))
    at = s["place"][:, None] + torch.arange(32, device=key.device)
    return _mix(at ^ key[:, None])


def _to_e4m3(x, bits, keep):
    """Blocks x [blocks, 32] in 8 bits: (codes, scale bytes).  `bits`: 16 random bits of each element (None: to
    nearest); `keep`: what is not 0 stays so."""
    amax = x.abs().amax(1)
    byte = (((amax * (8 / 7)).view(torch.int32) >> 23) - 8).clamp(min=0)
    y = x.abs() * _power(254 - byte)[:, None]
    if bits is not None:
        low = torch.where(y < 2.0 ** -6, 2.0 ** -6, 0.0)        # below 2^-6 the steps stay 2^-9
        w = (y + low).view(torch.int32) + (bits << 4).to(torch.int32)
        y = (w & ~0xFFFFF).view(torch.float32) - low
    codes = y.clamp(max=448).to(torch.float8_e4m3fn)
    if keep:
        codes = torch.where((x != 0) & (codes.view(torch.uint8) == 0), torch.ones_like(codes.view(torch.uint8)),
                            codes.view(torch.uint8))
    else:
        codes = codes.view(torch.uint8) | ((x < 0).to(torch.uint8) << 7)
    return codes.reshape(-1), byte.to(torch.uint8)


def _hyper(t):
    """The step's scalars, in 64 bits: 1 - beta, the weights' factor, the step's size and 1 / sqrt(1 - beta2^t)."""
    b1, b2 = BETAS
    return 1 - b1, 1 - b2, 1 - LR * DECAY, LR / (1 - b1 ** t), 1 / math.sqrt(1 - b2 ** t)


def _plain_adamw(s):
    case = s["case"]
    shift = 0 if case["aligned"] else 1
    s["t"] += 1
    c1, c2, decay, size, root = _hyper(s["t"])
    p, g = s["p"][shift:].float(), s["g"][shift:].float()
    if s["norm"] is not None:
        g = g * (torch.full_like(s["norm"], MAX_NORM) / (s["norm"] + CLIP_EPS)).clamp(max=1.0)
    if case["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m, r = ((s[k].view(torch.float8_e4m3fn).float().reshape(-1, 32) * _power(s[k + "_scales"])[:, None]).reshape(-1)
                for k in ("m", "v"))
        v = r * r
    m = BETAS[0] * m + c1 * g
    v = BETAS[1] * v + c2 * g * g
    r = v.sqrt()
    p = decay * p - size * (m / (r * root + ADAM_EPS))
    bits = _random(s, s["t"]) if case["stochastic"] else None
    if case["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        for k, x, b in (("m", m, 0), ("v", r, 16)):
            u = None if bits is None else bits >> b & 0xFFFF
            codes, byte = _to_e4m3(x.reshape(-1, 32), u, k == "v")
            s[k].copy_(codes)
            s[k + "_scales"].copy_(byte)
    if bits is not None and case["param"] == "bf16":
        w = p.view(torch.int32) + (bits.reshape(-1) * 0x9E3779B1 >> 16 & 0xFFFF).to(torch.int32)
        p = (w & ~0xFFFF).view(torch.float32)
    s["p"][shift:] = p.to(s["p"].dtype)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    if s["case"]["bits"] == 32:
        return {"p": s["p"], "m": s["m"], "v": s["v"]}
    # the numbers that codes and scales stand for
    return {"p": s["p"], "m": s["m"].view(torch.float8_e4m3fn), "m_scales": s["m_scales"].view(torch.float8_e8m0fnu),
            "v": s["v"].view(torch.float8_e4m3fn), "v_scales": s["v_scales"].view(torch.float8_e8m0fnu)}


# ------------------------------------------------------- the library's calls
def _own(s):
    import block_scaled_precision_03_gb300 as bsq
    case = s["case"]
    op, mx = case["op"], case.get("dtype") == "mxfp8"
    if op == "linear":
        call = bsq.gemm_linear_into if mx else bsq.linear_into
        call(s["x"], s["w"], s["y"], s["bias"], s["residual"], case["act"], s["z"])
        return {"y": s["y"], "z": s["z"]}
    if op == "linear_grad":
        bsq.linear_backward_into(s["dy"], s["x"], s["w"], s["dx"], s["dw"], s["dbias"], s["z"], case["act"])
        return {"dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"]}
    if op == "gated":
        call = bsq.gemm_gated_into if mx else bsq.gated_linear_into
        call(s["x"], s["w_gate"], s["w_up"], s["h"], case["act"], s["gate"], s["up"])
        return {"h": s["h"], "gate": s["gate"], "up": s["up"]} if s["gate"] is not None else {"h": s["h"]}
    if op == "gated_grad":
        bsq.gated_linear_backward_into(s["dh"], s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"], s["dx"],
                                       s["dw_gate"], s["dw_up"], case["act"])
        return {"dx": s["dx"], "dw_gate": s["dw_gate"], "dw_up": s["dw_up"]}
    s["t"] += 1
    bsq.adamw_step(s["list"], LR, s["t"], BETAS, ADAM_EPS, DECAY, norm=s["norm"],
                   max_norm=MAX_NORM if s["norm"] is not None else None, clip_eps=CLIP_EPS,
                   seed=s["seed"] if case["stochastic"] else None)
    return _adamw_outputs(s)


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "linear_grad": _plain_linear_grad, "gated": _plain_gated,
            "gated_grad": _plain_gated_grad, "adamw": _plain_adamw}[state["case"]["op"]](state)


def work(case):
    """Bytes with every input read once and every output written once, and the operations of the formula."""
    op = case["op"]
    if op == "adamw":
        n = sum(k for _, k in _starts(case)[0])
        state = 16 if case["bits"] == 32 else 4 * (1 + 1 / 32)
        return {"bytes": n * (2 * SIZE[case["param"]] + SIZE[case["grad"]] + state), "flops": 14 * n}
    T, D = case["tokens"], case["cols"]
    e = 33 / 32 if case["dtype"] == "mxfp8" else 2
    if op == "linear":
        N = case["out"]
        return {"bytes": e * (T + N) * D + 2 * T * N * (1 + case["residual"] + case["keep"]) + 4 * N * case["bias"],
                "flops": 2 * T * N * D}
    if op == "linear_grad":
        N = case["out"]
        return {"bytes": 4 * (T + N) * D + 2 * T * N * (1 + (case["act"] != "identity")) + 4 * N * case["bias"],
                "flops": 4 * T * N * D}
    F = case["width"]
    if op == "gated":
        return {"bytes": e * (T + 2 * F) * D + 2 * T * F * (3 if case["keep"] else 1), "flops": 4 * T * F * D}
    return {"bytes": 4 * (T + 2 * F) * D + 6 * T * F, "flops": 8 * T * F * D}


# --------------------------------------------------- definitions in 64 bits
def _exact_act(name, z):
    """(act(z), act'(z))"""
    if name == "identity":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.relu(z), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if name == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1 - q)
    if name == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 0.134145 * z * z)


def _exact_matrix(v):
    if isinstance(v, dict):
        return _values(v, torch.float64)
    if hasattr(v, "codes"):
        return _values({"codes": v.codes, "scales": v.scales, "rows": v.rows, "cols": v.cols}, torch.float64)
    return v.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "adamw":
        return _exact_adamw(s)
    x = _exact_matrix(s["x"])
    if op == "linear":
        z = x @ _exact_matrix(s["w"]).T
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act(case["act"], z)[0]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"y": y, "z": z if s["z"] is not None else None}
    if op == "linear_grad":
        dz = s["dy"].double()
        if s["z"] is not None:
            dz = dz * _exact_act(case["act"], s["z"].double())[1]
        return {"dx": dz @ s["w"].double(), "dw": dz.T @ x, "dbias": dz.sum(0) if s["dbias"] is not None else None}
    if op == "gated":
        a, u = x @ _exact_matrix(s["w_gate"]).T, x @ _exact_matrix(s["w_up"]).T
        h = _exact_act(case["act"], a)[0] * u
        return {"h": h, "gate": a, "up": u} if s["gate"] is not None else {"h": h}
    f, d = _exact_act(case["act"], s["gate"].double())
    dh = s["dh"].double()
    da, du = dh * s["up"].double() * d, dh * f
    dx = da @ s["w_gate"].double()
    dx += du @ s["w_up"].double()
    return {"dx": dx, "dw_gate": da.T @ x, "dw_up": du.T @ x}


def _exact_adamw(s):
    case, n = s["case"], s["m"].numel()
    t = s["t"] + 1
    shift = 0 if case["aligned"] else 1
    out = {k: [] for k in _adamw_outputs(s)}
    out["p"].append(torch.zeros(shift, dtype=torch.float64, device="cuda"))
    factor = 1.0 if s["norm"] is None else min(1.0, MAX_NORM / (float(s["norm"]) + CLIP_EPS))
    for a in range(0, n, 1 << 26):                              # pieces of whole blocks
        b = min(n, a + (1 << 26))
        g = s["g"][shift + a:shift + b].double() * factor
        if case["bits"] == 32:
            m, v = s["m"][a:b].double(), s["v"][a:b].double()
        else:
            m, v = (s[k][a:b].view(torch.float8_e4m3fn).double() *
                    torch.exp2(s[k + "_scales"][a // 32:b // 32].double() - 127).repeat_interleave(32) for k in ("m", "v"))
            v = v ** 2
        m = BETAS[0] * m + (1 - BETAS[0]) * g
        v = BETAS[1] * v + (1 - BETAS[1]) * g ** 2
        up = (m / (1 - BETAS[0] ** t)) / ((v / (1 - BETAS[1] ** t)).sqrt() + ADAM_EPS)
        p = s["p"][shift + a:shift + b].double()
        p = p - LR * DECAY * p - LR * up
        bits = None
        if case["stochastic"]:
            part = {"seed": s["seed"], "tensor": s["tensor"][a // 32:b // 32], "place": s["place"][a // 32:b // 32]}
            bits = _random(part, t).reshape(-1)
        if bits is not None and case["param"] == "bf16":
            u = ((bits * 0x9E3779B1 >> 16) & 0xFFFF) / 65536
            step = torch.exp2(torch.floor(torch.log2(p.abs().clamp(min=1e-300))) - 7)
            p = torch.sign(p) * torch.floor(p.abs() / step + u) * step
        out["p"].append(p)
        if case["bits"] == 32:
            out["m"].append(m)
            out["v"].append(v)
            continue
        for k, w, low in (("m", m, 0), ("v", v.sqrt(), 16)):
            w = w.reshape(-1, 32)
            e = torch.floor(torch.log2(w.abs().amax(1, keepdim=True).clamp(min=1e-300) * 8 / 7)) - 8
            e = e.clamp(min=-127)
            y = w.abs() * torch.exp2(-e)
            step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
            u = 0.5 if bits is None else (((bits >> low) & 0xFFFF) / 65536).reshape(-1, 32)
            code = torch.floor(y / step + u) * step if bits is not None else torch.round(y / step) * step
            code = code.clamp(max=448)
            if k == "v":
                code = torch.where(w != 0, code.clamp(min=2.0 ** -9), code)
            out[k].append((code * torch.sign(w)).reshape(-1))
            out[k + "_scales"].append(torch.exp2(e).reshape(-1))
    return {k: torch.cat(v) for k, v in out.items()}
