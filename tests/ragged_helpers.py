"""Plain 64-bit implementations of the ragged products and the router, and operands on which the tensor
cores' sums are exact, for the GPU tests."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from dense_fp16_gemm_03_gb300 import gemm as G  # noqa: E402
from dense_fp16_gemm_03_gb300 import ragged as R  # noqa: E402

KINDS = {"f16": torch.float16, "bf16": torch.bfloat16}
# relative half step of the type: a correctly rounded result is off by at most this times its binade
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8 / 2}


def require_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    R.lib()


def no_device_error(stream=None):
    st, code = G.gemm_f16_take_device_error(stream)
    assert st == G.GEMM_OK, "device error word 0x%x" % code


def eighths(rng, shape, kind):
    """Integers in [-8, 8] over 8: exact in both types, and every sum of up to 2^17 products is exact in fp32."""
    return torch.from_numpy(rng.integers(-8, 9, size=shape).astype(np.float32) / 8).to(kind)


def small_ints(rng, shape, kind, most):
    return torch.from_numpy(rng.integers(-most, most + 1, size=shape).astype(np.float32)).to(kind)


def offsets_of(sizes, head=0):
    return torch.tensor(np.concatenate([[head], head + np.cumsum(sizes)]).astype(np.int32))


def grouped_ref(op, first, second, offsets, groups):
    """In float64 on the host; offsets as the header defines them (clamped, running maximum)."""
    rows = first.shape[0]
    ends = np.maximum.accumulate(np.clip(offsets.cpu().numpy().astype(np.int64), 0, rows))
    a, b = first.double(), second.double()
    if op == "nt":
        out = torch.zeros((rows, second.shape[1]), dtype=torch.float64)
    elif op == "nn":
        out = torch.zeros((rows, second.shape[2]), dtype=torch.float64)
    else:
        out = torch.zeros((groups, first.shape[1], second.shape[1]), dtype=torch.float64)
    for g in range(groups):
        lo, hi = int(ends[g]), int(ends[g + 1])
        if lo == hi:
            continue
        if op == "nt":
            out[lo:hi] = a[lo:hi] @ b[g].T
        elif op == "nn":
            out[lo:hi] = a[lo:hi] @ b[g]
        else:
            out[g] = a[lo:hi].T @ b[lo:hi]
    return out


def grouped_run(op, first, second, offsets, dtype=None, workspace=True, stream=None, out=None):
    """The package's call on device copies of host operands; returns the host result."""
    f, s, o = first.cuda(), second.cuda(), offsets.cuda()
    groups, rows = offsets.shape[0] - 1, first.shape[0]
    n, k = (second.shape[1], second.shape[2]) if op != "tn" else (first.shape[1], second.shape[1])
    ws = torch.full((R.gemm_grouped_workspace_size(groups, rows, n, k),), 0xA5, dtype=torch.uint8, device="cuda") if workspace else None
    if op == "nt":
        y = R.gemm_grouped_nt(f, s, o, y=out, workspace=ws, stream=stream)
    elif op == "nn":
        y = R.gemm_grouped_nn(f, s, o, dx=out, workspace=ws, stream=stream)
    else:
        y = R.gemm_grouped_tn(f, s, o, dw=out, dtype=dtype, workspace=ws, stream=stream)
    no_device_error(stream)
    return y.cpu()


def grouped_operands(op, rng, sizes, n, k, kind, extra=0, draw=eighths):
    """(first, second) of a grouped call with sum(sizes) + extra rows."""
    rows, groups = int(sum(sizes)) + extra, len(sizes)
    x = draw(rng, (rows, k), kind)
    dy = draw(rng, (rows, n), kind)
    if op == "tn":
        return dy, x
    w = draw(rng, (groups, n, k), kind)
    return (x if op == "nt" else dy), w


def lora_ref(x, w, a, b, ids, scale):
    y = x.double() @ w.double().T
    for i in range(a.shape[0]):
        at = torch.nonzero(ids == i).flatten()
        if len(at):
            s = 1.0 if scale is None else float(scale[i])
            y[at] += s * (x[at].double() @ a[i].double().T) @ b[i].double().T
    return y


def lora_run(x, w, a, b, ids, scale=None, stream=None):
    rows, k = x.shape
    ws = torch.full((R.gemm_lora_workspace_size(rows, w.shape[0], k, a.shape[1], a.shape[0]),), 0xA5, dtype=torch.uint8,
                    device="cuda")
    y = R.gemm_lora_nt(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(), None if scale is None else scale.cuda(),
                       workspace=ws, stream=stream)
    no_device_error(stream)
    return y.cpu()


def route_ref(logits, top, renorm):
    """The header's definition in float64: a dict of numpy arrays."""
    z = logits.double().numpy()
    rows, experts = z.shape
    ids = np.full((rows, top), -1, dtype=np.int32)
    weights = np.zeros((rows, top))
    for t in range(rows):
        rank = [(1 if np.isnan(v) else 2, 0.0 if np.isnan(v) else v) for v in z[t]]
        order = sorted((e for e in range(experts) if z[t, e] != -np.inf), key=lambda e: (-rank[e][0], -rank[e][1], e))
        pick = order[:top]
        ids[t, : len(pick)] = pick
        with np.errstate(all="ignore"):
            m = np.nanmax(z[t]) if not np.all(np.isnan(z[t])) else np.nan
            p = np.where(z[t] == -np.inf, 0.0, np.exp(z[t] - m)) if m != -np.inf else np.where(np.isnan(z[t]), np.nan, 0.0)
            s = p.sum()
            if pick:
                w = p[pick] / (s if not renorm or np.isnan(s) else p[pick].sum())
                weights[t, : len(pick)] = w
    flat = ids.reshape(-1)
    order = np.argsort(np.where(flat < 0, experts, flat), kind="stable").astype(np.int32)
    live = int((flat >= 0).sum())
    position = np.full(rows * top, -1, dtype=np.int32)
    position[order[:live]] = np.arange(live)
    order[live:] = -1
    counts = np.bincount(flat[flat >= 0], minlength=experts)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return {"ids": ids, "weights": weights, "offsets": offsets, "order": order, "position": position.reshape(rows, top)}


def route_run(logits, top, renorm=True, stream=None):
    rows, experts = logits.shape
    ws = torch.full((max(1, R.gemm_route_workspace_size(rows, experts, top)),), 0xA5, dtype=torch.uint8, device="cuda")
    r = R.gemm_route_topk(logits.cuda(), top, renorm=renorm, workspace=ws, stream=stream)
    no_device_error(stream)
    return r
