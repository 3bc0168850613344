"""An expert layer and an adapted projection, run with the ragged products as a model would: forward, backward, decode.

    python -m dense_fp16_gemm_03_gb300.expert_layer [--rows 4096] [--width 1024] [--hidden 2048] [--experts 32] [--top 4]

The layer sends every row to ``top`` experts, each a product of its own, a square of the positive part, and a product
back, and adds their results weighted by the router:

    l = x . router^T;  w, e = top-k of softmax(l), w divided by their sum
    out[t] = sum_j w[t, j] relu(x[t] . up[e_tj]^T)^2 . down[e_tj]^T

The grouped products, the router and its gradient are this package's; what is between them (gathering rows, the
activation, adding rows up) is plain torch.  ``adapted`` is a projection with a low-rank adapter per row.
"""
import argparse
import time

import torch

from . import gemm, ragged


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


def adapted(x, w, a, b, ids, scale):
    """A shared projection of rows that belong to many requests, each with an adapter of its own."""
    size = ragged.gemm_lora_workspace_size(x.shape[0], w.shape[0], x.shape[1], a.shape[1], a.shape[0])
    return ragged.gemm_lora_nt(x, w, a, b, ids, scale, workspace=torch.empty(size, dtype=torch.uint8, device=x.device))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("rows", 4096), ("width", 1024), ("hidden", 2048), ("experts", 32), ("top", 4)):
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
        print("%-28s %9.1f us" % (name, (time.perf_counter() - t) / n * 1e6))
        return r

    _, saved = timed("expert layer, forward", lambda: layer.forward(x))
    timed("expert layer, backward", lambda: layer.backward(dout, saved))
    one = x[:1].contiguous()
    timed("expert layer, one token", lambda: layer.forward(one))
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
