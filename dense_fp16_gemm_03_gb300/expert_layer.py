"""An expert layer and an adapted projection, run with the ragged products as a model would: forward, backward, decode.

    python -m dense_fp16_gemm_03_gb300.expert_layer [--rows 4096] [--width 1024] [--hidden 2048] [--experts 32] [--top 4]
                                                    [--groups 8] [--top-groups 4] [--shared 2048]

The layer sends every row to ``top`` experts, each a product of its own, a square of the positive part, and a product
back, and adds their results weighted by the router:

    l = x . router^T;  w, e = top-k of softmax(l), w divided by their sum
    out[t] = sum_j w[t, j] relu(x[t] . up[e_tj]^T)^2 . down[e_tj]^T

The grouped products, the router and its gradient are this package's; what is between them (gathering rows, the
activation, adding rows up) is plain torch.  ``SharedExpertLayer`` has the activations in the products, a router that scores
by sigmoid, chooses with a bias within the best groups of experts, and an expert that every row shares.  ``adapted`` is a
projection with a low-rank adapter per row.
"""
import argparse
import time

import torch

from . import gemm, linear, ragged


class ExpertLayer:
    """Weights, and the workspaces a program keeps for them: router [experts, width], up [experts, hidden, width],
    down [experts, width, hidden]."""

    def __init__(self, width, hidden, experts, top, rows, dtype=torch.bfloat16, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(shape, scale):
            return torch.empty(shape, dtype=dtype, device=device).normal_(0.0, scale, generator=gen)

        self.width, self.hidden, self.experts, self.top = width, hidden, experts, top
        self.router = normal((experts, width), width ** -0.5)
        self.up = normal((experts, hidden, width), width ** -0.5)
        self.down = normal((experts, width, hidden), hidden ** -0.5)

        def buffer(size):
            return torch.empty(size, dtype=torch.uint8, device=device)

        # one buffer for all grouped calls: they follow one another on a stream
        self.work = buffer(max(ragged.gemm_grouped_workspace_size(experts, rows * top, hidden, width),
                               ragged.gemm_grouped_workspace_size(experts, rows * top, width, hidden)))
        self.route_work = buffer(ragged.gemm_route_workspace_size(rows, experts, top))

    def forward(self, x):
        """out [rows, width], and what the backward pass needs."""
        logits = x.float() @ self.router.float().T
        r = ragged.gemm_route_topk(logits, self.top, workspace=self.route_work)
        # choices t * top + j by expert; a choice of -1 (an expert at -infinity) stands past the last group's rows
        token = (r.order.clamp(min=0) // self.top).long()
        xs = x[token]
        h = ragged.gemm_grouped_nt(xs, self.up, r.offsets, workspace=self.work)
        a = torch.relu(h).square()
        ys = ragged.gemm_grouped_nt(a, self.down, r.offsets, workspace=self.work)
        # [rows, top, width]; nothing where there is no choice (a weight of 0 would not keep row 0's infinities out)
        mine = torch.where((r.position >= 0)[:, :, None], ys[r.position.clamp(min=0).long()].float(), 0.0)
        out = (r.weights[:, :, None] * mine).sum(1).to(x.dtype)
        return out, (x, logits, r, token, xs, h, a, mine)

    def backward(self, dout, saved):
        """Gradients of x, router, up and down."""
        x, logits, r, token, xs, h, a, mine = saved
        dmine = r.weights[:, :, None] * dout.float()[:, None, :]
        dweights = (mine * dout.float()[:, None, :]).sum(2)
        # rows sorted by expert are gathered by `order`, rows as they came by `position`: nothing waits for the GPU (a
        # training step can be captured), and no sum depends on the order of atomics
        dys = torch.where((r.order >= 0)[:, None], dmine.reshape(-1, self.width)[r.order.clamp(min=0).long()], 0.0).to(xs.dtype)
        da = ragged.gemm_grouped_nn(dys, self.down, r.offsets, workspace=self.work)
        ddown = ragged.gemm_grouped_tn(dys, a, r.offsets, dtype=torch.float32, workspace=self.work)
        dh = (da.float() * 2 * torch.relu(h.float())).to(h.dtype)
        dup = ragged.gemm_grouped_tn(dh, xs, r.offsets, dtype=torch.float32, workspace=self.work)
        dxs = ragged.gemm_grouped_nn(dh, self.up, r.offsets, workspace=self.work)
        dlogits = ragged.gemm_route_topk_grad(logits, r.ids, r.weights, dweights)
        dmine_x = torch.where((r.position >= 0)[:, :, None], dxs[r.position.clamp(min=0).long()].float(), 0.0)
        dx = dlogits @ self.router.float() + dmine_x.sum(1)
        return dx.to(x.dtype), dlogits.T @ x.float(), dup, ddown


class SharedExpertLayer(ExpertLayer):
    """An expert layer with a shared expert of `shared` hidden columns beside the routed ones:

        l = x . router^T;  s = sigmoid(l);  e = top-k of s + balance within the best groups of experts
        w = scale s[e] / sum of s[e]
        out[t] = sum_j w[t, j] relu(x[t] . up[e_tj]^T)^2 . down[e_tj]^T + gelu(x[t] . w1^T + b1) . w2^T + b2

    The activations, the biases and the sum with the routed experts are in the products' epilogues, their gradients in those of
    the products backwards."""

    def __init__(self, width, hidden, experts, top, rows, shared, groups=1, top_groups=None, scale=1.0, dtype=torch.bfloat16, seed=0,
                 device="cuda"):
        super().__init__(width, hidden, experts, top, rows, dtype=dtype, seed=seed, device=device)
        gen = torch.Generator(device=device).manual_seed(seed + 1)

        def normal(shape, scale):
            return torch.empty(shape, dtype=dtype, device=device).normal_(0.0, scale, generator=gen)

        self.groups, self.top_groups, self.scale = groups, groups if top_groups is None else top_groups, scale
        self.balance = torch.zeros(experts, device=device)
        self.w1, self.b1 = normal((shared, width), width ** -0.5), normal((shared,), 0.1)
        self.w2, self.b2 = normal((width, shared), shared ** -0.5), normal((width,), 0.1)
        sizes = [linear.gemm_linear_workspace_size(experts, rows * top, hidden, width),
                 linear.gemm_linear_workspace_size(experts, rows * top, width, hidden),
                 linear.gemm_linear_workspace_size(1, rows, shared, width), linear.gemm_linear_workspace_size(1, rows, width, shared),
                 ragged.gemm_grouped_workspace_size(1, rows, shared, width), ragged.gemm_grouped_workspace_size(1, rows, width, shared),
                 self.work.numel()]
        self.work = torch.empty(max(sizes), dtype=torch.uint8, device=device)

    def forward(self, x):
        """out [rows, width], and what the backward pass needs."""
        logits = x.float() @ self.router.float().T
        r = ragged.gemm_route_scored(logits, self.top, score="sigmoid", bias=self.balance, groups=self.groups, top_groups=self.top_groups,
                                     scale=self.scale, workspace=self.route_work)
        token = (r.order.clamp(min=0) // self.top).long()
        xs = x[token]
        a, h = linear.gemm_linear_nt(xs, self.up, act="relu2", offsets=r.offsets, keep=True, workspace=self.work)
        ys = ragged.gemm_grouped_nt(a, self.down, r.offsets, workspace=self.work)
        mine = torch.where((r.position >= 0)[:, :, None], ys[r.position.clamp(min=0).long()].float(), 0.0)
        routed = (r.weights[:, :, None] * mine).sum(1).to(x.dtype)
        s, z = linear.gemm_linear_nt(x, self.w1, bias=self.b1, act="gelu", keep=True, workspace=self.work)
        out = linear.gemm_linear_nt(s, self.w2, bias=self.b2, residual=routed, workspace=self.work)
        return out, (x, logits, r, token, xs, h, a, mine, s, z)

    def backward(self, dout, saved):
        """Gradients of x, router, up, down, w1, b1, w2 and b2."""
        x, logits, r, token, xs, h, a, mine, s, z = saved
        rows = x.shape[0]
        every = torch.arange(2, dtype=torch.int32, device=x.device) * rows  # all rows as one group
        _, db2 = linear.gemm_linear_grad(dout, bias_grad=True, workspace=self.work)
        dw2 = ragged.gemm_grouped_tn(dout, s, every, dtype=torch.float32, workspace=self.work)[0]
        dz, db1 = linear.gemm_linear_nn(dout, self.w2, z=z, act="gelu", bias_grad=True, workspace=self.work)
        dw1 = ragged.gemm_grouped_tn(dz, x, every, dtype=torch.float32, workspace=self.work)[0]
        dshared = linear.gemm_linear_nn(dz, self.w1, workspace=self.work)
        dmine = r.weights[:, :, None] * dout.float()[:, None, :]
        dweights = (mine * dout.float()[:, None, :]).sum(2)
        dys = torch.where((r.order >= 0)[:, None], dmine.reshape(-1, self.width)[r.order.clamp(min=0).long()], 0.0).to(xs.dtype)
        ddown = ragged.gemm_grouped_tn(dys, a, r.offsets, dtype=torch.float32, workspace=self.work)
        dh = linear.gemm_linear_nn(dys, self.down, z=h, act="relu2", offsets=r.offsets, workspace=self.work)
        dup = ragged.gemm_grouped_tn(dh, xs, r.offsets, dtype=torch.float32, workspace=self.work)
        dxs = ragged.gemm_grouped_nn(dh, self.up, r.offsets, workspace=self.work)
        dlogits = ragged.gemm_route_scored_grad(logits, r.ids, dweights, score="sigmoid", scale=self.scale)
        dmine_x = torch.where((r.position >= 0)[:, :, None], dxs[r.position.clamp(min=0).long()].float(), 0.0)
        dx = dlogits @ self.router.float() + dmine_x.sum(1) + dshared.float()
        return dx.to(x.dtype), dlogits.T @ x.float(), dup, ddown, dw1, db1, dw2, db2

    def rebalance(self, routing, rate=1e-3):
        """Moves the experts' bias a step towards those with fewer rows than the mean."""
        counts = torch.diff(routing.offsets).float()
        self.balance += rate * torch.sign(counts.mean() - counts)


def adapted(x, w, a, b, ids, scale):
    """A shared projection of rows that belong to many requests, each with an adapter of its own."""
    size = ragged.gemm_lora_workspace_size(x.shape[0], w.shape[0], x.shape[1], a.shape[1], a.shape[0])
    return ragged.gemm_lora_nt(x, w, a, b, ids, scale, workspace=torch.empty(size, dtype=torch.uint8, device=x.device))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("rows", 4096), ("width", 1024), ("hidden", 2048), ("experts", 32), ("top", 4), ("groups", 8),
                          ("top-groups", 4), ("shared", 2048)):
        ap.add_argument("--" + name, type=int, default=default)
    args = ap.parse_args()
    layer = ExpertLayer(args.width, args.hidden, args.experts, args.top, args.rows)
    x = torch.randn(args.rows, args.width, device="cuda").bfloat16()
    dout = torch.randn_like(x)

    def timed(name, f, n=20):
        for _ in range(3):
            r = f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            r = f()
        torch.cuda.synchronize()
        print("%-32s %9.1f us" % (name, (time.perf_counter() - t) / n * 1e6))
        return r

    _, saved = timed("expert layer, forward", lambda: layer.forward(x))
    timed("expert layer, backward", lambda: layer.backward(dout, saved))
    one = x[:1].contiguous()
    timed("expert layer, one token", lambda: layer.forward(one))
    both = SharedExpertLayer(args.width, args.hidden, args.experts, args.top, args.rows, args.shared, groups=args.groups,
                             top_groups=args.top_groups)
    _, saved = timed("with a shared expert, forward", lambda: both.forward(x))
    timed("with a shared expert, backward", lambda: both.backward(dout, saved))
    timed("with a shared expert, one token", lambda: both.forward(one))
    rank, adapters = 16, 64
    a = (torch.randn(adapters, rank, args.width, device="cuda") * args.width ** -0.5).bfloat16()
    b = (torch.randn(adapters, args.hidden, rank, device="cuda") * rank ** -0.5).bfloat16()
    rows = x[:64].contiguous()
    ids = torch.arange(rows.shape[0], dtype=torch.int32, device="cuda") % adapters
    scale = torch.ones(adapters, device="cuda")
    timed("adapted projection, 64 rows", lambda: adapted(rows, layer.up[0], a, b, ids, scale))
    status, code = gemm.gemm_f16_take_device_error()
    if status != gemm.GEMM_OK:
        raise SystemExit("device error word 0x%x" % code)


if __name__ == "__main__":
    main()
