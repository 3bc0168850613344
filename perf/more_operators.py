"""Measured cases of products with an epilogue, of their gradients, and of the router with scores, bias and groups.

  linear nt     y = f(x w^T + bias) + residual, with what f was applied to where a backward pass wants it; w one matrix, or one per
                group of rows
  linear nn     dx = (dy w) * f'(z), the gradient of what f was applied to one layer below, and of that layer's bias
  linear grad   dz = dy * f'(z) and the gradient of the bias, where no product comes before
  route         scores of the experts (softmax or sigmoid), a bias for the choice, the best groups of experts, the best experts in
                them, their weights, the rows sorted by expert, and the logits' gradient

``run`` computes a case either in plain torch operations (``own`` false) or through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "relu2", "gelu", "gelu_tanh", "silu"]


def listed():
    return [
        # one token on its way through a projection: the smallest call, where latency counts
        {"name": "nt one token", "op": "nt", "type": "f16", "groups": 0, "empty": 0, "rows": 1, "n": 2048, "k": 1024, "act": "silu",
         "bias": True, "residual": True, "keep": False},
        # a decode step of 64 sequences, a projection back into the residual stream: bound by the weights' bytes
        {"name": "nt decode step", "op": "nt", "type": "bf16", "groups": 0, "empty": 0, "rows": 64, "n": 8192, "k": 4096, "act": "none",
         "bias": True, "residual": True, "keep": False},
        # a mid-size batch, rows and columns in no whole tiles, in training
        {"name": "nt ragged batch", "op": "nt", "type": "f16", "groups": 0, "empty": 0, "rows": 3000, "n": 5000, "k": 4096, "act": "gelu",
         "bias": True, "residual": False, "keep": True},
        # a training batch of 16384 rows through a wide layer's first half
        {"name": "nt large batch", "op": "nt", "type": "bf16", "groups": 0, "empty": 0, "rows": 16384, "n": 4096, "k": 4096,
         "act": "gelu_tanh", "bias": True, "residual": False, "keep": True},
        # 4096 rows with four of 32 experts each, the experts' first half: short contractions, so the epilogue shows
        {"name": "nt experts", "op": "nt", "type": "bf16", "groups": 32, "empty": 0, "rows": 16384, "n": 2048, "k": 1024, "act": "relu2",
         "bias": False, "residual": False, "keep": True},
        # the large batch backwards, down to the first half's bias
        {"name": "nn large batch", "op": "nn", "type": "bf16", "groups": 0, "empty": 0, "rows": 16384, "n": 4096, "k": 4096,
         "act": "gelu_tanh", "bias": True},
        # the experts backwards; two saw no row
        {"name": "nn experts", "op": "nn", "type": "f16", "groups": 32, "empty": 2, "rows": 16384, "n": 1024, "k": 2048, "act": "relu2",
         "bias": True},
        # the gradient through a last activation and its bias, at a training batch's size: bound by its bytes
        {"name": "grad training step", "op": "grad", "type": "bf16", "groups": 0, "empty": 0, "rows": 16384, "n": 4096, "act": "gelu",
         "bias": True},
        # the same for a small ragged step of eight groups, two of them empty
        {"name": "grad small ragged", "op": "grad", "type": "f16", "groups": 8, "empty": 2, "rows": 777, "n": 1000, "act": "silu",
         "bias": True},
        # the router of a decode step: 256 experts in eight groups, four of them kept
        {"name": "route decode step", "op": "route", "type": "f32", "rows": 64, "experts": 256, "top": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5, "grad": False},
        # the same router in a training step, with the gradient of its logits
        {"name": "route training step", "op": "route", "type": "bf16", "rows": 16384, "experts": 256, "top": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5, "grad": True},
        # softmax scores within the three best of eight groups, by each group's best expert
        {"name": "route softmax groups", "op": "route", "type": "f32", "rows": 2048, "experts": 64, "top": 6, "score": "softmax",
         "bias": False, "groups": 8, "top_groups": 3, "group_top": 1, "renorm": False, "scale": 16.0, "grad": True},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return int(round(float(np.exp(rng.uniform(np.log(low), np.log(high))))))


def draw(rng):
    op = rng.choice(["nt", "nt", "nn", "grad", "route", "route"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        experts = groups * max(2, _spread(rng, 16, 512) // groups)
        top_groups = rng.randint(1, groups)
        score = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "type": rng.choice(["f32", "bf16", "f16"]), "rows": _spread(rng, 1, 16384), "experts": experts,
                "top": rng.randint(1, min(8, top_groups * (experts // groups))), "score": score, "bias": rng.random() < 0.6,
                "groups": groups, "top_groups": top_groups, "group_top": rng.choice([1, 2]), "renorm": rng.random() < 0.5,
                "scale": rng.choice([1.0, 2.5]), "grad": rng.random() < 0.5}
    n, k = min(8 * _spread(rng, 16, 1024), 4096), min(8 * _spread(rng, 16, 512), 4096)
    groups = rng.choice([0, 0, _spread(rng, 2, 64)])
    groups = min(groups, 32 * 4096 * 4096 // (n * k))
    case = {"op": op, "type": rng.choice(["f16", "bf16"]), "groups": groups, "empty": rng.randint(0, groups // 2),
            "rows": _spread(rng, 1, 16384), "n": n, "act": rng.choice(ACTS), "bias": rng.random() < 0.7}
    if op != "grad":
        case["k"] = k
    if op == "grad":
        case["act"], case["bias"] = rng.choice(ACTS[1:]), True
    if op == "nt":
        case["residual"], case["keep"] = rng.random() < 0.5, rng.random() < 0.5
    return case


def _sizes(case, seed):
    """Rows of each group: the active ones get one each and an uneven share of the rest; which are empty goes by the seed."""
    rs = np.random.RandomState(seed % (1 << 31))
    live = min(case["rows"], case["groups"] - case["empty"])
    share = np.exp(0.5 * rs.standard_normal(live))
    rows = 1 + rs.multinomial(case["rows"] - live, share / share.sum())
    sizes = np.zeros(case["groups"], dtype=np.int64)
    sizes[rs.permutation(case["groups"])[:live]] = rows
    return sizes


def _normal(gen, shape, scale, kind):
    return torch.empty(shape, dtype=kind, device=DEVICE).normal_(0.0, scale, generator=gen)


def _buffer(size):
    return torch.empty(size, dtype=torch.uint8, device=DEVICE)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    op, kind, rows = case["op"], TYPES[case["type"]], case["rows"]
    s = dict(case)
    if op == "route":
        s["logits"] = _normal(gen, (rows, case["experts"]), 1.5, kind)
        # a bias that training has moved in small steps
        s["shift"] = _normal(gen, (case["experts"],), 0.05, torch.float32) if case["bias"] else None
        s["dweights"] = _normal(gen, (rows, case["top"]), 1.0, torch.float32)
        if own:
            from dense_fp16_gemm_03_gb300 import ragged
            s["workspace"] = _buffer(ragged.gemm_route_workspace_size(rows, case["experts"], case["top"]))
        return s
    n, k, groups = case["n"], case.get("k", 0), case["groups"]
    s["offsets"] = None
    if groups:
        sizes = _sizes(case, seed)
        s["most"] = int(sizes.max())  # a plain form pads each group to the longest
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).to(DEVICE)
    stack = (groups,) if groups else ()
    if op == "nt":
        s["x"] = _normal(gen, (rows, k), 1.0, kind)
        s["b"] = _normal(gen, stack + (n,), 0.1, kind) if case["bias"] else None
        s["r"] = _normal(gen, (rows, n), 1.0, kind) if case["residual"] else None
    else:
        s["dy"] = _normal(gen, (rows, n), 1.0, kind)
        s["z"] = _normal(gen, (rows, k if op == "nn" else n), 1.0, kind) if case["act"] != "none" else None
    if op != "grad":
        s["w"] = _normal(gen, stack + (n, k), (k if op == "nt" else n) ** -0.5, kind)
    if own:
        from dense_fp16_gemm_03_gb300 import linear
        s["workspace"] = _buffer(linear.gemm_linear_workspace_size(max(groups, 1), rows, n, k))
    return s


# ------------------------------------------------------------------ plain

def _f(act, z):
    if act == "relu":
        return torch.relu(z)
    if act == "relu2":
        return torch.relu(z) * torch.relu(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _df(act, z):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return 2 * torch.relu(z)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _groups_of(s):
    t = torch.arange(s["rows"], device=DEVICE)
    return (t[:, None] >= s["offsets"][None, 1:]).sum(1)


def _cells(s, g):
    """Each row's place in [groups, most] padded rows."""
    return g * s["most"] + torch.arange(s["rows"], device=DEVICE) - s["offsets"].long()[g]


def _padded(s, rows, at):
    out = torch.zeros((s["groups"] * s["most"], rows.shape[1]), dtype=rows.dtype, device=DEVICE)
    out[at] = rows
    return out.view(s["groups"], s["most"], rows.shape[1])


def _product(s, a, w, at):
    if not s["groups"]:
        return a @ w
    return torch.bmm(_padded(s, a, at), w).view(-1, w.shape[2])[at]


def _plain_linear(s):
    kind, act, op = TYPES[s["type"]], s["act"], s["op"]
    g = _groups_of(s) if s["groups"] else None
    at = _cells(s, g) if s["groups"] else None
    if op == "nt":
        z = _product(s, s["x"].float(), s["w"].float().transpose(-1, -2), at)
        if s["b"] is not None:
            b = s["b"].float()
            z = z + (b[g] if s["groups"] else b)
        y = _f(act, z)
        if s["r"] is not None:
            y = y + s["r"].float()
        return {"y": y.to(kind), "z": z.to(kind)} if s["keep"] else {"y": y.to(kind)}
    d = s["dy"].float() if op == "grad" else _product(s, s["dy"].float(), s["w"].float(), at)
    if s["z"] is not None:
        d = d * _df(act, s["z"].float())
    out = {"dx": d.to(kind)}
    if s["bias"]:
        if s["groups"]:
            out["dbias"] = _padded(s, d, at).sum(1, dtype=torch.float64).float()
        else:
            out["dbias"] = d.sum(0, dtype=torch.float64).float()
    return out


def _plain_route(s):
    rows, experts, top, groups = s["rows"], s["experts"], s["top"], s["groups"]
    z = s["logits"].double()  # a choice goes by differences that 32 bits round away
    if s["score"] == "softmax":
        e = torch.exp(z - z.max(1, keepdim=True).values)
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-z))
    c = p + s["shift"].double() if s["shift"] is not None else p
    if groups > 1:
        best = torch.sort(c.view(rows, groups, experts // groups), dim=2, descending=True, stable=True).values
        best = best[:, :, :s["group_top"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        of = torch.arange(experts, device=DEVICE) // (experts // groups)
        c = torch.where((kept[:, :, None] == of[None, None, :]).any(1), c, -torch.inf)
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :top]
    p = p.float()
    w = torch.gather(p, 1, ids)
    total = w.sum(1, keepdim=True) if s["renorm"] else torch.ones_like(w[:, :1])
    weights = s["scale"] * w / total
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = (flat[:, None] == torch.arange(experts, device=DEVICE)[None, :]).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    position = torch.empty_like(order)
    position[order] = torch.arange(rows * top, device=DEVICE)
    out = {"ids": ids.int(), "weights": weights, "offsets": offsets.int(), "order": order.int(),
           "position": position.view(rows, top).int()}
    if s["grad"]:
        dw = s["scale"] * s["dweights"] / total
        if s["renorm"]:
            dw = dw - (dw * w).sum(1, keepdim=True) / total
        if s["score"] == "sigmoid":
            out["dlogits"] = torch.zeros_like(p).scatter_(1, ids, dw * w * (1 - w))
        else:
            dp = torch.zeros_like(p).scatter_(1, ids, dw)
            out["dlogits"] = p * (dp - (dw * w).sum(1, keepdim=True))
    return out


# -------------------------------------------------------------------- own

def _own_linear(s):
    from dense_fp16_gemm_03_gb300 import linear
    ws = s["workspace"]
    if s["op"] == "nt":
        r = linear.gemm_linear_nt(s["x"], s["w"], bias=s["b"], residual=s["r"], act=s["act"], offsets=s["offsets"], keep=s["keep"],
                                  workspace=ws)
        return {"y": r[0], "z": r[1]} if s["keep"] else {"y": r}
    if s["op"] == "nn":
        r = linear.gemm_linear_nn(s["dy"], s["w"], z=s["z"], act=s["act"], offsets=s["offsets"], bias_grad=s["bias"], workspace=ws)
    else:
        r = linear.gemm_linear_grad(s["dy"], z=s["z"], act=s["act"], offsets=s["offsets"], bias_grad=s["bias"], workspace=ws)
    return {"dx": r[0], "dbias": r[1]} if s["bias"] else {"dx": r}


def _own_route(s):
    from dense_fp16_gemm_03_gb300 import ragged
    r = ragged.gemm_route_scored(s["logits"], s["top"], score=s["score"], bias=s["shift"], groups=s["groups"], top_groups=s["top_groups"],
                                 group_top=s["group_top"], renorm=s["renorm"], scale=s["scale"], workspace=s["workspace"])
    out = {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "order": r.order, "position": r.position}
    if s["grad"]:
        out["dlogits"] = ragged.gemm_route_scored_grad(s["logits"], r.ids, s["dweights"], score=s["score"], renorm=s["renorm"],
                                                       scale=s["scale"])
    return out


def run(state):
    if own:
        return _own_route(state) if state["op"] == "route" else _own_linear(state)
    return _plain_route(state) if state["op"] == "route" else _plain_linear(state)


def work(case):
    rows = case["rows"]
    if case["op"] == "route":
        experts, top = case["experts"], case["top"]
        moved = rows * experts * TYPES[case["type"]].itemsize + rows * top * 16 + 4 * (experts + 1)
        if case["bias"]:
            moved += 4 * experts
        if case["grad"]:
            moved += rows * top * 4 + rows * experts * 4  # the choice and the logits stay known from the forward pass
        return {"bytes": moved, "flops": rows * experts * (8 if case["grad"] else 5)}
    n = case["n"]
    live = min(rows, case["groups"] - case["empty"]) if case["groups"] else 1
    if case["op"] == "grad":
        return {"bytes": 6 * rows * n + 4 * max(case["groups"], 1) * n, "flops": 10 * rows * n}
    k = case["k"]
    moved = 2 * rows * (n + k) + 2 * live * n * k
    if case["op"] == "nt":
        moved += 2 * rows * n * (int(case["residual"]) + int(case["keep"])) + (2 * live * n if case["bias"] else 0)
    else:
        moved += (2 * rows * k if case["act"] != "none" else 0) + (4 * max(case["groups"], 1) * k if case["bias"] else 0)
    return {"bytes": moved, "flops": 2 * rows * n * k}


# ------------------------------------------------------------------ exact

def _exact_act(act, z):
    """f(z) and f'(z) in 64 bits."""
    half = torch.special.erfc(-z / math.sqrt(2)) / 2
    sig = torch.where(z >= 0, 1 / (1 + torch.exp(-z.abs())), torch.exp(-z.abs()) / (1 + torch.exp(-z.abs())))
    if act == "relu":
        return z.clamp(min=0), torch.where(z > 0, 1.0, 0.0).double()
    if act == "relu2":
        return z.clamp(min=0) ** 2, 2 * z.clamp(min=0)
    if act == "gelu":
        return z * half, half + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        return z * sig, sig + z * sig * (1 - sig)
    if act == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        s = torch.sigmoid(u)
        return z * s, s + z * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)
    return z, torch.ones_like(z)


def _exact_linear(case, s):
    op, act = case["op"], case["act"]
    ends = s["offsets"].cpu().tolist() if case["groups"] else [0, case["rows"]]
    out = {}
    for g in range(len(ends) - 1):
        lo, hi = ends[g], ends[g + 1]
        part = {}
        if op == "nt":
            w, b = (s["w"][g] if case["groups"] else s["w"]), s["b"]
            z = s["x"][lo:hi].double() @ w.double().T
            if b is not None:
                z = z + (b[g] if case["groups"] else b).double()
            y = _exact_act(act, z)[0]
            part["y"] = y + s["r"][lo:hi].double() if s["r"] is not None else y
            if case["keep"]:
                part["z"] = z
        else:
            d = s["dy"][lo:hi].double()
            if op == "nn":
                d = d @ (s["w"][g] if case["groups"] else s["w"]).double()
            if s["z"] is not None:
                d = d * _exact_act(act, s["z"][lo:hi].double())[1]
            part["dx"] = d
            if case["bias"]:
                part["dbias"] = d.sum(0, keepdim=True)
        for name, v in part.items():
            out.setdefault(name, []).append(v)
    out = {name: torch.cat(v) for name, v in out.items()}
    if "dbias" in out and not case["groups"]:
        out["dbias"] = out["dbias"][0]
    return out


def _exact_route(case, s):
    z = s["logits"].double().cpu().numpy()
    rows, experts = z.shape
    if case["score"] == "softmax":
        p = np.exp(z - np.log(np.exp(z).sum(1, keepdims=True)))
    else:
        p = 0.5 * (1 + np.tanh(z / 2))
    c = p.copy()
    if s["shift"] is not None:
        c += s["shift"].double().cpu().numpy()
    size = experts // case["groups"]
    if case["groups"] > 1:
        score = np.sort(c.reshape(rows, -1, size), axis=2)[:, :, size - case["group_top"]:].sum(2)
        rank = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1, kind="stable")
        c[np.repeat(rank >= case["top_groups"], size, axis=1)] = -np.inf
    ids = np.argsort(-c, axis=1, kind="stable")[:, :case["top"]]
    chosen = np.take_along_axis(p, ids, 1)
    total = chosen.sum(1, keepdims=True)
    w = case["scale"] * (chosen / total if case["renorm"] else chosen)
    out = {"ids": None, "weights": w, "offsets": None, "order": None, "position": None}
    if case["grad"]:
        # d loss / d logit by the chain rule through every weight: first to the scores, then to the logits
        d = s["dweights"].double().cpu().numpy()
        dp = np.zeros_like(p)
        for j in range(case["top"]):
            if not case["renorm"]:
                np.put_along_axis(dp, ids[:, j:j + 1], case["scale"] * d[:, j:j + 1], 1)
                continue
            for i in range(case["top"]):  # d w_i / d p_j
                at = np.take_along_axis(dp, ids[:, j:j + 1], 1)
                step = d[:, i:i + 1] * case["scale"] * (float(i == j) / total - chosen[:, i:i + 1] / total ** 2)
                np.put_along_axis(dp, ids[:, j:j + 1], at + step, 1)
        if case["score"] == "softmax":
            out["dlogits"] = p * (dp - (p * dp).sum(1, keepdims=True))
        else:
            out["dlogits"] = dp * p * (1 - p)
    return out


def exact(case, seed):
    """The definition in 64 bits, group by group."""
    s = prepare(case, seed)
    return _exact_route(case, s) if case["op"] == "route" else _exact_linear(case, s)
