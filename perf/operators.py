"""Measured cases of the products whose second matrix depends on the row, and of the router that feeds them.

  grouped nt / nn / tn   rows sorted by group: the forward product with each group's weights, the gradient of its rows, and the
                         gradient of the weights
  lora                   a shared projection with a low-rank adapter of each row's own beside it
  route                  top-k of the experts' logits: the choice, its weights, the rows sorted by expert, and the logits' gradient

``run`` computes a case either in plain torch operations in 32 bits (``own`` false) or through the package's entry points.
"""
import numpy as np
import torch

own = False

DEVICE = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token that goes to two experts of eight: the smallest call, where latency counts
        {"name": "nt one token", "op": "nt", "type": "f16", "groups": 8, "empty": 6, "rows": 2, "n": 2048, "k": 1024},
        # a decode step of 32 sequences, eight experts each: a few rows for nearly every expert, bound by the weights' bytes
        {"name": "nt decode step", "op": "nt", "type": "bf16", "groups": 64, "empty": 4, "rows": 256, "n": 2048, "k": 4096},
        # a ragged mid-size batch, rows and columns in no whole tiles
        {"name": "nt ragged batch", "op": "nt", "type": "f16", "groups": 16, "empty": 1, "rows": 3000, "n": 5000, "k": 4096},
        # a prompt or a training batch of 16384 rows over 32 experts
        {"name": "nt large batch", "op": "nt", "type": "bf16", "groups": 32, "empty": 0, "rows": 16384, "n": 4096, "k": 4096},
        # the same batch backwards: the gradient of the rows
        {"name": "nn large batch", "op": "nn", "type": "bf16", "groups": 32, "empty": 0, "rows": 16384, "n": 4096, "k": 4096},
        # and of the weights, in the weights' type
        {"name": "tn large batch", "op": "tn", "type": "bf16", "groups": 32, "empty": 0, "rows": 16384, "n": 4096, "k": 4096,
         "out": "bf16"},
        # a small ragged step's weight gradient in 32 bits, for accumulation; two experts saw no row
        {"name": "tn small ragged f32", "op": "tn", "type": "f16", "groups": 8, "empty": 2, "rows": 777, "n": 1000, "k": 520,
         "out": "f32"},
        # one token of one request
        {"name": "lora one token", "op": "lora", "type": "f16", "rows": 1, "n": 4096, "k": 4096, "adapters": 8, "rank": 16,
         "requests": 1},
        # a decode step of 64 requests, nearly each with an adapter of its own
        {"name": "lora decode step", "op": "lora", "type": "bf16", "rows": 64, "n": 8192, "k": 4096, "adapters": 64, "rank": 16,
         "requests": 64},
        # 16 prompts together, 8192 tokens in all
        {"name": "lora prompts", "op": "lora", "type": "bf16", "rows": 8192, "n": 8192, "k": 4096, "adapters": 16, "rank": 64,
         "requests": 16},
        # the router of a decode step
        {"name": "route decode step", "op": "route", "type": "f32", "rows": 64, "experts": 64, "top": 8, "renorm": True,
         "grad": False},
        # the router of a training step, with the gradient of its logits
        {"name": "route training step", "op": "route", "type": "bf16", "rows": 16384, "experts": 128, "top": 8, "renorm": False,
         "grad": True},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return int(round(float(np.exp(rng.uniform(np.log(low), np.log(high))))))


def draw(rng):
    op = rng.choice(["nt", "nt", "nn", "tn", "lora", "route"])
    if op == "route":
        experts = _spread(rng, 8, 256)
        return {"op": op, "type": rng.choice(["f32", "bf16", "f16"]), "rows": _spread(rng, 1, 16384), "experts": experts,
                "top": rng.randint(1, min(8, experts)), "renorm": rng.random() < 0.5, "grad": rng.random() < 0.5}
    kind = rng.choice(["f16", "bf16"])
    n, k = 8 * _spread(rng, 16, 1024), 8 * _spread(rng, 16, 512)
    if op == "lora":
        rows = _spread(rng, 1, 4096)
        return {"op": op, "type": kind, "rows": rows, "n": n, "k": k, "adapters": _spread(rng, 1, 64),
                "rank": 8 * rng.randint(1, 8), "requests": min(rows, _spread(rng, 1, 128))}
    groups = _spread(rng, 2, 64)
    n, k = min(n, 4096), min(k, 4096)
    groups = min(groups, 32 * 4096 * 4096 // (n * k))
    case = {"op": op, "type": kind, "groups": groups, "empty": rng.randint(0, groups // 2), "rows": _spread(rng, 1, 16384), "n": n, "k": k}
    if op == "tn":
        case["out"] = rng.choice([kind, "f32"])
    return case


def _active(case):
    """How many groups have rows."""
    return min(case["rows"], case["groups"] - case["empty"])


def _sizes(case, seed):
    """Rows of each group: the active ones get one each and an uneven share of the rest; which are empty goes by the seed."""
    rs = np.random.RandomState(seed % (1 << 31))
    live = _active(case)
    share = np.exp(0.5 * rs.standard_normal(live))
    rows = 1 + rs.multinomial(case["rows"] - live, share / share.sum())
    sizes = np.zeros(case["groups"], dtype=np.int64)
    sizes[rs.permutation(case["groups"])[:live]] = rows
    return sizes


def _normal(gen, shape, scale, kind):
    out = torch.empty(shape, dtype=kind, device=DEVICE)
    return out.normal_(0.0, scale, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    op, kind = case["op"], TYPES[case["type"]]
    s = dict(case)
    if op == "route":
        rows, experts, top = case["rows"], case["experts"], case["top"]
        s["logits"] = _normal(gen, (rows, experts), 1.5, kind)
        s["dweights"] = _normal(gen, (rows, top), 1.0, torch.float32)
        if own:
            from dense_fp16_gemm_03_gb300 import ragged
            s["workspace"] = _buffer(ragged.gemm_route_workspace_size(rows, experts, top))
        return s
    rows, n, k = case["rows"], case["n"], case["k"]
    if op == "lora":
        rs = np.random.RandomState(seed % (1 << 31))
        count, rank = case["adapters"], case["rank"]
        # contiguous requests of about equal length, each with an adapter of the pool; one in sixteen has none
        which = rs.permutation(max(count, case["requests"]))[: case["requests"]] % count
        which[rs.uniform(size=case["requests"]) < 1.0 / 16] = -1
        ids = which[(np.arange(rows) * case["requests"]) // rows]
        s["ids"] = torch.from_numpy(ids.astype(np.int32)).to(DEVICE)
        s["x"] = _normal(gen, (rows, k), 1.0, kind)
        s["w"] = _normal(gen, (n, k), k ** -0.5, kind)
        s["a"] = _normal(gen, (count, rank, k), k ** -0.5, kind)
        s["b"] = _normal(gen, (count, n, rank), rank ** -0.5, kind)
        s["scale"] = torch.rand((count,), generator=gen, device=DEVICE) + 0.5
        if own:
            from dense_fp16_gemm_03_gb300 import ragged
            s["workspace"] = _buffer(ragged.gemm_lora_workspace_size(rows, n, k, rank, count))
        return s
    groups = case["groups"]
    sizes = _sizes(case, seed)
    s["most"] = int(sizes.max())  # a plain form pads each group to the longest
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).to(DEVICE)
    if op in ("nt", "tn"):
        s["x"] = _normal(gen, (rows, k), 1.0, kind)
    if op in ("nn", "tn"):
        s["dy"] = _normal(gen, (rows, n), 1.0, kind)
    if op in ("nt", "nn"):
        s["w"] = _normal(gen, (groups, n, k), k ** -0.5, kind)
    if own:
        from dense_fp16_gemm_03_gb300 import ragged
        s["workspace"] = _buffer(ragged.gemm_grouped_workspace_size(groups, rows, n, k))
    return s


def _buffer(size):
    return torch.empty(size, dtype=torch.uint8, device=DEVICE)


def _cells(s):
    """Each row's place in [groups, most] padded rows."""
    t = torch.arange(s["rows"], device=DEVICE)
    g = (t[:, None] >= s["offsets"][None, 1:]).sum(1)
    return g * s["most"] + t - s["offsets"].long()[g]


def _padded(s, rows, at):
    out = torch.zeros((s["groups"] * s["most"], rows.shape[1]), dtype=torch.float32, device=DEVICE)
    out[at] = rows.float()
    return out.view(s["groups"], s["most"], rows.shape[1])


def _plain_grouped(s):
    at = _cells(s)
    if s["op"] == "nt":
        y = torch.bmm(_padded(s, s["x"], at), s["w"].float().transpose(1, 2))
        return y.view(-1, s["n"])[at].to(s["x"].dtype)
    if s["op"] == "nn":
        dx = torch.bmm(_padded(s, s["dy"], at), s["w"].float())
        return dx.view(-1, s["k"])[at].to(s["dy"].dtype)
    dw = torch.bmm(_padded(s, s["dy"], at).transpose(1, 2), _padded(s, s["x"], at))
    return dw.to(TYPES[s["out"]])


def _plain_lora(s):
    x, count, rank = s["x"].float(), s["adapters"], s["rank"]
    u = (x @ s["a"].float().view(count * rank, s["k"]).T).view(-1, count, rank)
    mine = s["ids"][:, None] == torch.arange(count, device=DEVICE)[None, :]
    u = u * (mine * s["scale"][None, :])[:, :, None]
    delta = u.view(-1, count * rank) @ s["b"].float().permute(0, 2, 1).reshape(count * rank, s["n"])
    return (x @ s["w"].float().T + delta).to(s["x"].dtype)


def _plain_route(s):
    rows, experts, top = s["rows"], s["experts"], s["top"]
    logits = s["logits"].float()
    e = torch.exp(logits - logits.max(1, keepdim=True).values)
    p = e / e.sum(1, keepdim=True)
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top]
    weights = torch.gather(p, 1, ids)
    if s["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = (flat[:, None] == torch.arange(experts, device=DEVICE)[None, :]).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    position = torch.empty_like(order)
    position[order] = torch.arange(rows * top, device=DEVICE)
    out = {"ids": ids.int(), "weights": weights, "offsets": offsets.int(), "order": order.int(),
           "position": position.view(rows, top).int()}
    if s["grad"]:
        inner = (weights * s["dweights"]).sum(1, keepdim=True)
        if s["renorm"]:
            dl = torch.zeros_like(p).scatter_(1, ids, weights * (s["dweights"] - inner))
        else:
            dl = p * (torch.zeros_like(p).scatter_(1, ids, s["dweights"]) - inner)
        out["dlogits"] = dl
    return out


def _own(s):
    from dense_fp16_gemm_03_gb300 import ragged
    ws = s["workspace"]
    if s["op"] == "nt":
        return ragged.gemm_grouped_nt(s["x"], s["w"], s["offsets"], workspace=ws)
    if s["op"] == "nn":
        return ragged.gemm_grouped_nn(s["dy"], s["w"], s["offsets"], workspace=ws)
    if s["op"] == "tn":
        return ragged.gemm_grouped_tn(s["dy"], s["x"], s["offsets"], dtype=TYPES[s["out"]], workspace=ws)
    if s["op"] == "lora":
        return ragged.gemm_lora_nt(s["x"], s["w"], s["a"], s["b"], s["ids"], s["scale"], workspace=ws)
    r = ragged.gemm_route_topk(s["logits"], s["top"], renorm=s["renorm"], workspace=ws)
    out = {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "order": r.order, "position": r.position}
    if s["grad"]:
        out["dlogits"] = ragged.gemm_route_topk_grad(s["logits"], r.ids, r.weights, s["dweights"], renorm=s["renorm"])
    return out


def run(state):
    if own:
        return _own(state)
    if state["op"] == "lora":
        return _plain_lora(state)
    if state["op"] == "route":
        return _plain_route(state)
    return _plain_grouped(state)


def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "route":
        rows, experts, top = case["rows"], case["experts"], case["top"]
        moved = rows * experts * size + rows * top * 16 + 4 * (experts + 1)
        if case["grad"]:
            moved += rows * top * 4 + rows * experts * 4  # the choice and the logits stay known from the forward pass
        return {"bytes": moved, "flops": rows * experts * (6 if case["grad"] else 3)}
    rows, n, k = case["rows"], case["n"], case["k"]
    if case["op"] == "lora":
        # the adapters that some request has, by expectation: each is read once
        used = min(case["adapters"], case["requests"] * 15 / 16)
        rank = case["rank"]
        return {"bytes": 2 * (rows * (k + n) + n * k + used * rank * (k + n)) + 4 * rows,
                "flops": 2 * rows * n * k + 2 * rows * rank * (k + n) * 15 / 16}
    flops = 2 * rows * n * k
    if case["op"] == "tn":
        out = 4 if case["out"] == "f32" else 2
        return {"bytes": 2 * rows * (n + k) + out * case["groups"] * n * k, "flops": flops}
    return {"bytes": 2 * rows * (n + k) + 2 * _active(case) * n * k, "flops": flops}


def exact(case, seed):
    """The definition in 64 bits, group by group and request by request."""
    s = prepare(case, seed)
    if case["op"] == "route":
        z = s["logits"].cpu().numpy() if case["type"] == "f32" else s["logits"].float().cpu().numpy()
        z = z.astype(np.float64)
        top = case["top"]
        p = np.exp(z) / np.exp(z).sum(1, keepdims=True)
        ids = np.argsort(-z, axis=1, kind="stable")[:, :top]
        w = np.take_along_axis(p, ids, 1)
        if case["renorm"]:
            w = w / w.sum(1, keepdims=True)
        out = {"ids": None, "weights": w, "offsets": None, "order": None, "position": None}
        if case["grad"]:
            # d loss / d logit by the chain rule through every weight
            d = s["dweights"].cpu().numpy().astype(np.float64)
            dl = np.zeros_like(p)
            for j in range(top):
                for i in range(top if case["renorm"] else 1):
                    if case["renorm"]:
                        np.put_along_axis(dl, ids[:, i:i + 1], np.take_along_axis(dl, ids[:, i:i + 1], 1)
                                          + d[:, j:j + 1] * w[:, j:j + 1] * (float(i == j) - w[:, i:i + 1]), 1)
                    else:
                        dl -= d[:, j:j + 1] * w[:, j:j + 1] * p
                        np.put_along_axis(dl, ids[:, j:j + 1], np.take_along_axis(dl, ids[:, j:j + 1], 1)
                                          + d[:, j:j + 1] * w[:, j:j + 1], 1)
            out["dlogits"] = dl
        return out
    if case["op"] == "lora":
        x = s["x"].double()
        y = x @ s["w"].double().T
        ids = s["ids"].cpu().numpy()
        for i in sorted(set(ids[ids >= 0].tolist())):
            at = torch.from_numpy(np.nonzero(ids == i)[0]).to(DEVICE)
            y[at] += float(s["scale"][i]) * ((x[at] @ s["a"][i].double().T) @ s["b"][i].double().T)
        return y
    ends = s["offsets"].cpu().numpy().tolist()
    rows, n, k = case["rows"], case["n"], case["k"]
    shape = {"nt": (rows, n), "nn": (rows, k), "tn": (case["groups"], n, k)}[case["op"]]
    out = torch.zeros(shape, dtype=torch.float64, device=DEVICE)
    for g in range(case["groups"]):
        lo, hi = ends[g], ends[g + 1]
        if lo == hi:
            continue
        if case["op"] == "nt":
            out[lo:hi] = s["x"][lo:hi].double() @ s["w"][g].double().T
        elif case["op"] == "nn":
            out[lo:hi] = s["dy"][lo:hi].double() @ s["w"][g].double()
        else:
            out[g] = s["dy"][lo:hi].double().T @ s["x"][lo:hi].double()
    return out
