"""The operators around a block-scaled linear layer that a training or serving
step of a mixture-of-experts language model also runs: what is measured.

Four operators, each in a plain form (elementary torch operations in FP32,
rounded once at the end) and as the calls a user makes of the library:

  moe   tokens sorted by expert, gathered into the ragged batch a grouped GEMM
        takes, and combined back with the routing weights; both gradients
  norm  layer norm, forward and backward (with the weight's and bias's gradient)
  head  softmax cross entropy of a linear head over a vocabulary, without
        keeping the logits, and its gradient
  clip  the global norm of many gradients, and their clipped copies

A case is a dict of plain values; its "op" says which pass it is.  Sizes are
those of this repository's own workloads (hidden 4096 and 7168, 8192 rows, 64
experts with 32768 expert rows drawn Zipf(1.1), an MLP width of 14336) or
generic ones."""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
NORM_EPS = 1e-5
CLIP_EPS = 1e-6
IGNORED = -100


def listed():
    return [
        # one token of a decoding request goes to its experts: latency only
        {"name": "moe dispatch, one token", "op": "dispatch", "tokens": 1, "k": 8, "experts": 64, "cols": 7168,
         "dtype": "bf16", "dropped": 0.0},
        # the tokens of a training or prompt batch: 32768 expert rows of 7168, the grouped GEMM's batch
        {"name": "moe dispatch, batch", "op": "dispatch", "tokens": 4096, "k": 8, "experts": 64, "cols": 7168,
         "dtype": "bf16", "dropped": 0.0},
        # a ragged batch whose row pitch has no alignment, with tokens over the experts' capacity left out
        {"name": "moe combine, odd", "op": "combine", "tokens": 1021, "k": 3, "experts": 13, "cols": 2047,
         "dtype": "bf16", "dropped": 0.1},
        # the backward pass of the batch: expert rows' and routing weights' gradients
        {"name": "moe combine gradient, batch", "op": "combine_grad", "tokens": 4096, "k": 8, "experts": 64,
         "cols": 7168, "dtype": "bf16", "dropped": 0.02},
        # one token of a decoding request: latency only
        {"name": "layer norm, one token", "op": "norm", "rows": 1, "cols": 7168, "dtype": "bf16"},
        # the input of the 8192 x 4096 quantize of a training step
        {"name": "layer norm, batch", "op": "norm", "rows": 8192, "cols": 4096, "dtype": "bf16"},
        # its backward pass
        {"name": "layer norm gradient, batch", "op": "norm_grad", "rows": 8192, "cols": 4096, "dtype": "bf16"},
        # the score of a few tokens (a short answer's likelihood): the head's weights are read once
        {"name": "head loss, few tokens", "op": "head", "tokens": 7, "vocab": 50021, "cols": 4096},
        # the loss of a training batch
        {"name": "head loss, batch", "op": "head", "tokens": 8192, "vocab": 65536, "cols": 4096},
        # its gradient with respect to the hidden states and the head's weights
        {"name": "head gradient, batch", "op": "head_grad", "tokens": 8192, "vocab": 65536, "cols": 4096},
        # a small model's or an adapter's many small gradients, packed without alignment
        {"name": "clip, small tensors", "op": "clip", "tensors": 61, "elements": 200003, "aligned": False,
         "scale": 0.05},
        # one layer of the repository's MLP and projection shapes, BF16 weights and FP32 vectors
        {"name": "clip, one layer", "op": "clip", "tensors": 12, "elements": 243300000, "aligned": True,
         "scale": 0.001},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "norm", "norm_grad", "head", "head_grad",
                     "clip"])
    if op in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        cols = _log(rng, 33, 7168 if dtype == "bf16" else 3584)
        if rng.random() < 0.6:
            cols = max(8, cols // 8 * 8)
        experts = _log(rng, 1, 256)
        return {"op": op, "tokens": _log(rng, 1, 4096), "k": min(experts, rng.randint(1, 8)), "experts": experts,
                "cols": cols, "dtype": dtype, "dropped": rng.choice([0.0, 0.05, 0.5])}
    if op in ("norm", "norm_grad"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        cols = _log(rng, 17, 14336)
        if rng.random() < 0.6:
            cols = max(8, cols // 8 * 8)
        most = 8192 * 4096 * 2 // (SIZE[dtype] * cols)
        return {"op": op, "rows": _log(rng, 1, min(most, 32768)), "cols": cols, "dtype": dtype}
    if op in ("head", "head_grad"):
        return {"op": op, "tokens": _log(rng, 1, 8192), "vocab": _log(rng, 257, 65536),
                "cols": 8 * _log(rng, 8, 512)}
    n = _log(rng, 1, 400)
    return {"op": op, "tensors": n, "elements": n + _log(rng, 1000, 200000000), "aligned": rng.random() < 0.5,
            "scale": rng.choice([0.05, 1e-6])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _routing(case, g):
    """Expert ids [tokens, k] (distinct per token, Zipf(1.1) over the experts), with a share of the
    slots left out (-1: over capacity, or a padding token), and softmax weights."""
    T, k, E = case["tokens"], case["k"], case["experts"]
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    rank = torch.arange(1, E + 1, device="cuda", dtype=torch.float32)
    score = -1.1 * rank.log() - (-u.log()).log()
    top, ids = score.topk(k, dim=1)
    weights = torch.softmax(top, dim=1)
    left_out = torch.rand((T, k), generator=g, device="cuda") < case["dropped"]
    return ids.masked_fill(left_out, -1), weights


def _plan(ids, E):
    """Plain form of the sort: ids [T, k] -> (offsets [E + 1], slot_row [T, k], row_slot [T k])."""
    T, k = ids.shape
    n = T * k
    flat = ids.reshape(-1)
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, torch.full_like(flat, E))
    hit = torch.arange(E + 1, device=ids.device)[:, None] == key
    upto = hit.cumsum(1, dtype=torch.int32)
    counts = upto[:, -1]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = counts[:E].cumsum(0)
    place = offsets[key] + upto.gather(0, key[None])[0] - 1
    to = torch.where(valid, place, torch.full_like(place, n))
    row_slot = torch.full((n + 1,), -1, dtype=torch.int32, device=ids.device)
    row_slot[to] = torch.arange(n, device=ids.device, dtype=torch.int32)
    row_slot[n] = -1
    slot_row = torch.where(valid, place, torch.full_like(place, -1)).to(torch.int32).reshape(T, k)
    return offsets, slot_row, row_slot[:n]


def _clip_sizes(case):
    """Element counts and types of the gradients: a few large matrices and many vectors, every fifth FP32."""
    n, total = case["tensors"], case["elements"]
    share = [1.0 + 40.0 * (i % 3 == 0) + 7.0 * (i % 4 == 1) for i in range(n)]
    sizes = [max(1, int(total * s / sum(share))) for s in share]
    sizes[0] += max(0, total - sum(sizes))
    return sizes, ["f32" if i % 5 == 4 else "bf16" for i in range(n)]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
        T, k, E, C, dt = case["tokens"], case["k"], case["experts"], case["cols"], DT[case["dtype"]]
        s["ids"], s["weights"] = _routing(case, g)
        n = T * k
        if op == "dispatch":
            s["x"] = _normal(g, (T, C), dt)
            s["offsets"] = torch.empty(E + 1, dtype=torch.int64, device="cuda")
            s["slot_row"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
            s["row_slot"] = torch.empty(n, dtype=torch.int32, device="cuda")
            s["out"] = torch.empty((n, C), dtype=dt, device="cuda")
        else:
            s["offsets"], s["slot_row"], s["row_slot"] = _plan(s["ids"], E)
            s["rows"] = _normal(g, (n, C), dt)
            if op == "combine_grad":
                s["dout"] = _normal(g, (T, C), dt)
                s["drows"] = torch.empty((n, C), dtype=dt, device="cuda")
                s["dweights"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
            else:
                s["out"] = torch.empty((T, C), dtype=dt, device="cuda")
    elif op in ("norm", "norm_grad"):
        R, C, dt = case["rows"], case["cols"], DT[case["dtype"]]
        row = torch.rand((R, 1), generator=g, device="cuda") * 3 + 0.2
        s["x"] = (_normal(g, (R, C), torch.float32) * row + 0.3).to(dt)
        s["weight"] = 1 + 0.1 * _normal(g, (C,), torch.float32)
        s["bias"] = 0.1 * _normal(g, (C,), torch.float32)
        if op == "norm":
            s["y"] = torch.empty((R, C), dtype=dt, device="cuda")
            s["mean"] = torch.empty(R, dtype=torch.float32, device="cuda")
            s["rstd"] = torch.empty(R, dtype=torch.float32, device="cuda")
        else:
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = 1 / (xf.var(1, unbiased=False) + NORM_EPS).sqrt()
            s["dy"] = _normal(g, (R, C), dt)
            s["dx"] = torch.empty((R, C), dtype=dt, device="cuda")
            s["dweight"] = torch.empty(C, dtype=torch.float32, device="cuda")
            s["dbias"] = torch.empty(C, dtype=torch.float32, device="cuda")
    elif op in ("head", "head_grad"):
        T, V, D = case["tokens"], case["vocab"], case["cols"]
        s["w"] = (0.02 * torch.randn((V, D), generator=g, device="cuda")).to(torch.bfloat16)
        targets = torch.randint(0, V, (T,), generator=g, device="cuda")
        # a partly trained model: the target's logit is raised by 0 to about 13 where cols = 4096
        pull = 8 * torch.rand((T, 1), generator=g, device="cuda")
        s["h"] = (_normal(g, (T, D), torch.float32) + pull * s["w"][targets].float()).to(torch.bfloat16)
        skip = torch.rand((T,), generator=g, device="cuda") < 0.05
        skip[0] = False
        s["targets"] = targets.masked_fill(skip, IGNORED)
        if op == "head":
            s["loss"] = torch.empty(T, dtype=torch.float32, device="cuda")
            s["lse"] = torch.empty(T, dtype=torch.float32, device="cuda")
        else:
            s["lse"] = torch.logsumexp(s["h"].float() @ s["w"].float().T, 1)
            n = (s["targets"] >= 0).sum()
            s["dloss"] = (torch.ones(T, device="cuda") / n).float()
            s["dh"] = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
            s["dw"] = torch.empty((V, D), dtype=torch.bfloat16, device="cuda")
    else:
        sizes, types = _clip_sizes(case)
        pitch = 256 if case["aligned"] else 1          # elements between the starts of two tensors: a multiple of this
        at, spans = {"bf16": 0, "f32": 0}, []
        for n, t in zip(sizes, types):
            spans.append((t, at[t], n))
            at[t] += -(-n // pitch) * pitch
        used = [t for t in ("bf16", "f32") if at[t]]
        s["grads"] = {t: torch.zeros(at[t], dtype=DT[t], device="cuda") for t in used}
        s["out"] = {t: torch.zeros(at[t], dtype=DT[t], device="cuda") for t in used}
        for t in used:
            s["grads"][t].normal_(generator=g).mul_(case["scale"])
            end = 0
            for u, a, n in spans:
                if u == t:
                    s["grads"][t][end:a] = 0
                    end = a + n
            s["grads"][t][end:] = 0
        s["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
        if own:
            import block_scaled_precision_03_gb300 as bsq
            s["list"] = bsq.GradList([s["grads"][t][a:a + n] for t, a, n in spans],
                                     [s["out"][t][a:a + n] for t, a, n in spans])
    return s


# ------------------------------------------------------------ plain forms
def _plain_dispatch(s):
    T, k = s["ids"].shape
    n = T * k
    offsets, slot_row, row_slot = _plan(s["ids"], s["case"]["experts"])
    rows = s["x"][(row_slot.clamp(min=0) // k).long()]
    rows = torch.where((row_slot >= 0)[:, None], rows, torch.zeros_like(rows))
    return {"rows": rows, "offsets": offsets, "slot_row": slot_row, "row_slot": row_slot}


def _plain_combine(s, weighted):
    here = s["slot_row"] >= 0
    rows = s["rows"][s["slot_row"].clamp(min=0).long()].float()
    if weighted:
        rows = rows * s["weights"][:, :, None]
    return torch.where(here[:, :, None], rows, torch.zeros_like(rows)).sum(1).to(s["rows"].dtype)


def _plain_combine_grad(s):
    k = s["weights"].shape[1]
    here = s["slot_row"] >= 0
    slot = s["row_slot"].clamp(min=0).long()
    d = s["dout"].float()
    drows = d[slot // k] * s["weights"].reshape(-1)[slot][:, None]
    drows = torch.where((s["row_slot"] >= 0)[:, None], drows, torch.zeros_like(drows)).to(s["rows"].dtype)
    rows = s["rows"][s["slot_row"].clamp(min=0).long()].float()
    dweights = (rows * d[:, None, :]).sum(2)
    return {"drows": drows, "dweights": torch.where(here, dweights, torch.zeros_like(dweights))}


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = 1 / (c.square().mean(1, keepdim=True) + NORM_EPS).sqrt()
    y = c * rstd * s["weight"] + s["bias"]
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_grad(s):
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["weight"]
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}


def _plain_head(s):
    logits = s["h"].float() @ s["w"].float().T
    most = logits.max(1, keepdim=True).values
    lse = (logits - most).exp().sum(1).log() + most[:, 0]
    counts = s["targets"] >= 0
    hit = logits.gather(1, s["targets"].clamp(min=0)[:, None])[:, 0]
    return {"loss": torch.where(counts, lse - hit, torch.zeros_like(lse)), "lse": lse}


def _plain_head_grad(s):
    h, w = s["h"].float(), s["w"].float()
    p = (h @ w.T - s["lse"][:, None]).exp()
    counts = s["targets"] >= 0
    at = s["targets"].clamp(min=0)[:, None]
    p.scatter_(1, at, p.gather(1, at) - 1)
    p *= torch.where(counts, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    return {"dh": (p @ w).to(s["h"].dtype), "dw": (p.T @ h).to(s["w"].dtype)}


def _plain_clip(s):
    norm = sum(v.float().square().sum() for v in s["grads"].values()).sqrt()
    factor = (1.0 / (norm + CLIP_EPS)).clamp(max=1.0)
    return {"norm": norm.reshape(1), **{t: (v.float() * factor).to(v.dtype) for t, v in s["grads"].items()}}


# ------------------------------------------------------- the library's calls
def _own(s):
    import block_scaled_precision_03_gb300 as bsq
    op = s["case"]["op"]
    if op in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
        plan = bsq.MoePlan(s["case"]["experts"], s["offsets"], s["slot_row"], s["row_slot"])
        if op == "dispatch":
            bsq.moe_dispatch_into(s["x"], s["ids"], plan, s["out"])
            return {"rows": s["out"], "offsets": s["offsets"], "slot_row": s["slot_row"], "row_slot": s["row_slot"]}
        if op == "dispatch_grad":
            return bsq.moe_combine_into(s["rows"], None, plan, s["out"])
        if op == "combine":
            return bsq.moe_combine_into(s["rows"], s["weights"], plan, s["out"])
        bsq.moe_combine_backward_into(s["dout"], s["rows"], s["weights"], plan, s["drows"], s["dweights"])
        return {"drows": s["drows"], "dweights": s["dweights"]}
    if op == "norm":
        bsq.layer_norm_into(s["x"], s["weight"], s["bias"], NORM_EPS, s["y"], s["mean"], s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_grad":
        bsq.layer_norm_backward_into(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"],
                                     s["dbias"])
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if op == "head":
        bsq.linear_cross_entropy_into(s["h"], s["w"], s["targets"], s["loss"], s["lse"])
        return {"loss": s["loss"], "lse": s["lse"]}
    if op == "head_grad":
        bsq.linear_cross_entropy_backward_into(s["h"], s["w"], s["targets"], s["lse"], s["dloss"], s["dh"], s["dw"])
        return {"dh": s["dh"], "dw": s["dw"]}
    bsq.clip_grad_norm_into(s["list"], 1.0, s["norm"], CLIP_EPS)
    return {"norm": s["norm"], **s["out"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "dispatch":
        return _plain_dispatch(state)
    if op in ("dispatch_grad", "combine"):
        return _plain_combine(state, op == "combine")
    return {"combine_grad": _plain_combine_grad, "norm": _plain_norm, "norm_grad": _plain_norm_grad,
            "head": _plain_head, "head_grad": _plain_head_grad, "clip": _plain_clip}[op](state)


def work(case):
    """Bytes with every input read once and every output written once, and the operations of the formula."""
    op = case["op"]
    if op in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
        T, k, E, C, e = case["tokens"], case["k"], case["experts"], case["cols"], SIZE[case["dtype"]]
        n = T * k
        sent = n * (1 - case["dropped"])
        if op == "dispatch":
            return {"bytes": T * C * e + n * C * e + n * 16 + (E + 1) * 8, "flops": 0}
        if op == "combine_grad":
            return {"bytes": T * C * e + sent * C * e + n * C * e + n * 16, "flops": 3 * sent * C}
        return {"bytes": sent * C * e + T * C * e + n * (8 if op == "combine" else 4), "flops": 2 * sent * C}
    if op == "norm":
        R, C, e = case["rows"], case["cols"], SIZE[case["dtype"]]
        return {"bytes": 2 * R * C * e + 8 * C + 8 * R, "flops": 8 * R * C}
    if op == "norm_grad":
        R, C, e = case["rows"], case["cols"], SIZE[case["dtype"]]
        return {"bytes": 3 * R * C * e + 12 * C + 8 * R, "flops": 15 * R * C}
    if op == "head":
        T, V, D = case["tokens"], case["vocab"], case["cols"]
        return {"bytes": 2 * (T + V) * D + 16 * T, "flops": 2 * T * V * D}
    if op == "head_grad":
        # the logits are not kept: they are computed again, and go into two products
        T, V, D = case["tokens"], case["vocab"], case["cols"]
        return {"bytes": 4 * (T + V) * D + 16 * T, "flops": 6 * T * V * D}
    sizes, types = _clip_sizes(case)
    return {"bytes": sum(2 * n * SIZE[t] for n, t in zip(sizes, types)), "flops": 3 * sum(sizes)}


# --------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
        T, k, E, C = case["tokens"], case["k"], case["experts"], case["cols"]
        ids = s["ids"].reshape(-1).tolist()
        order = sorted((i for i, e in enumerate(ids) if 0 <= e < E), key=lambda i: (ids[i], i))
        slot = torch.tensor(order, dtype=torch.int64, device="cuda")
        m = len(order)
        if op == "dispatch":
            rows = torch.zeros((T * k, C), dtype=torch.float64, device="cuda")
            rows[:m] = s["x"].double()[slot // k]
            return {"rows": rows, "offsets": None, "slot_row": None, "row_slot": None}
        y = s["rows"][:m].double()
        w = s["weights"].double().reshape(-1)[slot]
        if op == "combine_grad":
            d = s["dout"].double()[slot // k]
            drows = torch.zeros((T * k, C), dtype=torch.float64, device="cuda")
            drows[:m] = d * w[:, None]
            dweights = torch.zeros(T * k, dtype=torch.float64, device="cuda")
            dweights[slot] = (d * y).sum(1)
            return {"drows": drows, "dweights": dweights.reshape(T, k)}
        out = torch.zeros((T, C), dtype=torch.float64, device="cuda")
        out.index_add_(0, slot // k, y * w[:, None] if op == "combine" else y)
        return out
    if op in ("norm", "norm_grad"):
        x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
        C = case["cols"]
        if op == "norm":
            mean = x.sum(1) / C
            rstd = ((x * x).sum(1) / C - mean * mean + NORM_EPS).rsqrt()
            return {"y": (x - mean[:, None]) * rstd[:, None] * w + b, "mean": mean, "rstd": rstd}
        mean, rstd, dy = s["mean"].double(), s["rstd"].double(), s["dy"].double()
        xh = (x - mean[:, None]) * rstd[:, None]
        a = (dy @ w) / C
        c = ((dy * xh) @ w) / C
        dx = (dy * w - a[:, None] - xh * c[:, None]) * rstd[:, None]
        return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, xh), "dbias": dy.sum(0)}
    if op in ("head", "head_grad"):
        T, V, D = case["tokens"], case["vocab"], case["cols"]
        if op == "head":
            parts, hit = [], torch.zeros(T, dtype=torch.float64, device="cuda")
            for a in range(0, V, 8192):
                z = s["h"].double() @ s["w"][a:a + 8192].double().T
                parts.append(torch.logsumexp(z, 1))
                inside = (s["targets"] >= a) & (s["targets"] < a + z.shape[1])
                hit += torch.where(inside, z.gather(1, (s["targets"] - a).clamp(0, z.shape[1] - 1)[:, None])[:, 0], 0.0)
            lse = torch.logsumexp(torch.stack(parts), 0)
            return {"loss": torch.where(s["targets"] >= 0, lse - hit, 0.0), "lse": lse}
        if 6 * T * V * D > 1.4e13:
            return None
        h = s["h"].double()
        scale = torch.where(s["targets"] >= 0, s["dloss"].double(), 0.0)
        dh, dw = torch.zeros((T, D), dtype=torch.float64, device="cuda"), []
        for a in range(0, V, 8192):
            w = s["w"][a:a + 8192].double()
            p = torch.exp(h @ w.T - s["lse"].double()[:, None])
            p -= (s["targets"][:, None] == torch.arange(a, a + w.shape[0], device="cuda")).double()
            p *= scale[:, None]
            dh += p @ w
            dw.append(p.T @ h)
        return {"dh": dh, "dw": torch.cat(dw)}
    squares = [float((v.double() ** 2).sum()) for v in s["grads"].values()]
    norm = math.sqrt(math.fsum(squares))
    factor = min(1.0, 1.0 / (norm + CLIP_EPS))
    return {"norm": torch.tensor([norm], dtype=torch.float64), **{t: v.double() * factor for t, v in s["grads"].items()}}
