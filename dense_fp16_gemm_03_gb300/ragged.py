"""ctypes binding of include/gemm_ragged.h (same entry-point names): grouped
products by expert with their gradients, low-rank adapters beside a shared
projection, and the experts' router.

Argument marshalling only, as in ``gemm``: every step runs in the CUDA library,
a missing library raises, and there is no fallback.  Operands are contiguous
CUDA tensors; a call runs on ``stream`` (a torch.cuda.Stream, a raw integer, or
None for the current torch stream).  Outputs that are not given are allocated
on the current torch stream; workspaces are the caller's (sizes from the
``*_workspace_size`` functions, any contents, one call at a time).
"""
import collections
import ctypes

from . import gemm as _gemm
from .gemm import GemmError, gemm_f16_take_device_error  # noqa: F401  (the same errors, the same device word)

DTYPE_F16 = 0
DTYPE_BF16 = 1
DTYPE_F32 = 2

MAX_GROUPS = 1024
MAX_RANK = 128
MAX_EXPERTS = 1024
MAX_TOP = 32

# every symbol the public header declares
EXPORTED = [
    "gemm_grouped_workspace_size", "gemm_grouped_nt", "gemm_grouped_nn", "gemm_grouped_tn", "gemm_grouped_stall_test",
    "gemm_lora_workspace_size", "gemm_lora_nt",
    "gemm_route_workspace_size", "gemm_route_topk", "gemm_route_topk_grad",
]

Routing = collections.namedtuple("Routing", ["ids", "weights", "offsets", "order", "position"])

_lib = None


def lib():
    """The library of ``gemm.lib()`` with this header's signatures."""
    global _lib
    if _lib is not None:
        return _lib
    L = _gemm.lib()
    i32, i64, u32, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_size_t
    psz, dt = ctypes.POINTER(ctypes.c_size_t), ctypes.c_int
    sig = {
        "gemm_grouped_workspace_size": [i64, i64, i64, i64, psz],
        "gemm_grouped_nt": [dt, i64, i64, i64, i64, vp, vp, vp, vp, vp, sz, vp],
        "gemm_grouped_nn": [dt, i64, i64, i64, i64, vp, vp, vp, vp, vp, sz, vp],
        "gemm_grouped_tn": [dt, dt, i64, i64, i64, i64, vp, vp, vp, vp, vp, sz, vp],
        "gemm_grouped_stall_test": [i32, dt, i64, i64, i64, i64, vp, vp, vp, vp, vp, sz, u32, ctypes.c_longlong, vp],
        "gemm_lora_workspace_size": [i64, i64, i64, i64, i64, psz],
        "gemm_lora_nt": [dt, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "gemm_route_workspace_size": [i64, i64, i64, psz],
        "gemm_route_topk": [dt, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "gemm_route_topk_grad": [dt, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.restype = ctypes.c_int
        f.argtypes = args
    _lib = L
    return L


def _check(status, where):
    if status != _gemm.GEMM_OK:
        raise GemmError(status, where)


def _dtype(t, f32=False):
    torch = _gemm._tm()
    if t is torch.float16:
        return DTYPE_F16
    if t is torch.bfloat16:
        return DTYPE_BF16
    if f32 and t is torch.float32:
        return DTYPE_F32
    raise ValueError("operands must be float16 or bfloat16%s, got %s" % (" or float32" if f32 else "", t))


def _need(t, what, shape, dtype, device):
    """`t` must be a contiguous CUDA tensor of this shape, type and device."""
    if (tuple(t.shape) != tuple(shape) or t.dtype is not dtype or not t.is_cuda or t.device != device
            or not t.is_contiguous()):
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s" % (what, dtype, list(shape), device))


def _operand(t, what, dims):
    if t.dim() != dims or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor with %d dimensions" % (what, dims))
    if t.device.index != _gemm._tm().cuda.current_device():
        raise ValueError("%s must be on the current device" % what)


def _out(t, what, shape, dtype, device):
    if t is None:
        return _gemm._tm().empty(shape, dtype=dtype, device=device)
    _need(t, what, shape, dtype, device)
    return t


def _workspace(ws):
    if ws is None:
        return None, 0
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _size(name, *args):
    b = ctypes.c_size_t()
    _check(getattr(lib(), name)(*args, ctypes.byref(b)), name)
    return b.value


# ------------------------------------------------------------ grouped products

def gemm_grouped_workspace_size(groups, rows, n, k):
    return _size("gemm_grouped_workspace_size", groups, rows, n, k)


def _offsets(offsets, device):
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must hold groups + 1 numbers")
    _need(offsets, "offsets", offsets.shape, _gemm._tm().int32, device)
    return offsets.shape[0] - 1


def gemm_grouped_nt(x, w, offsets, y=None, workspace=None, stream=None):
    """y[t] = x[t] . w[g]^T for the rows t in [offsets[g], offsets[g + 1]); rows of no group are zero.

    x [rows, k], w [groups, n, k], offsets [groups + 1] int32 on the device; returns y [rows, n]."""
    _operand(x, "x", 2)
    groups, rows, k = _offsets(offsets, x.device), x.shape[0], x.shape[1]
    if w.dim() != 3:
        raise ValueError("w must be [groups, n, k]")
    n = w.shape[1]
    _need(w, "w", (groups, n, k), x.dtype, x.device)
    kind = _dtype(x.dtype)
    y = _out(y, "y", (rows, n), x.dtype, x.device)
    ws, ws_bytes = _workspace(workspace)
    _check(lib().gemm_grouped_nt(kind, groups, rows, n, k, offsets.data_ptr(), x.data_ptr(), w.data_ptr(), y.data_ptr(), ws,
                                 ws_bytes, _gemm._stream(stream)), "gemm_grouped_nt")
    return y


def gemm_grouped_nn(dy, w, offsets, dx=None, workspace=None, stream=None):
    """dx[t] = dy[t] . w[g]: the gradient of gemm_grouped_nt's rows.  dy [rows, n]; returns dx [rows, k]."""
    _operand(dy, "dy", 2)
    groups, rows, n = _offsets(offsets, dy.device), dy.shape[0], dy.shape[1]
    if w.dim() != 3:
        raise ValueError("w must be [groups, n, k]")
    k = w.shape[2]
    _need(w, "w", (groups, n, k), dy.dtype, dy.device)
    kind = _dtype(dy.dtype)
    dx = _out(dx, "dx", (rows, k), dy.dtype, dy.device)
    ws, ws_bytes = _workspace(workspace)
    _check(lib().gemm_grouped_nn(kind, groups, rows, n, k, offsets.data_ptr(), dy.data_ptr(), w.data_ptr(), dx.data_ptr(), ws,
                                 ws_bytes, _gemm._stream(stream)), "gemm_grouped_nn")
    return dx


def gemm_grouped_tn(dy, x, offsets, dw=None, dtype=None, workspace=None, stream=None):
    """dw[g] = dy_g^T . x_g: the gradient of gemm_grouped_nt's weights, zero for a group without rows.

    dy [rows, n], x [rows, k]; returns dw [groups, n, k] in `dtype` (the operands' type, or torch.float32)."""
    _operand(dy, "dy", 2)
    groups, rows, n = _offsets(offsets, dy.device), dy.shape[0], dy.shape[1]
    if x.dim() != 2:
        raise ValueError("x must be [rows, k]")
    k = x.shape[1]
    _need(x, "x", (rows, k), dy.dtype, dy.device)
    kind = _dtype(dy.dtype)
    if dtype is None:
        dtype = dy.dtype if dw is None else dw.dtype
    if dtype is not dy.dtype and dtype is not _gemm._tm().float32:
        raise ValueError("dw must have the operands' type or float32")
    dw = _out(dw, "dw", (groups, n, k), dtype, dy.device)
    ws, ws_bytes = _workspace(workspace)
    _check(lib().gemm_grouped_tn(kind, _dtype(dtype, f32=True), groups, rows, n, k, offsets.data_ptr(), dy.data_ptr(),
                                 x.data_ptr(), dw.data_ptr(), ws, ws_bytes, _gemm._stream(stream)), "gemm_grouped_tn")
    return dw


def gemm_grouped_stall_test(mode, first, second, offsets, out, workspace, skip_fill, wait_limit_cycles, stream=None):
    """Status of the failure-detection launch (mode 0, 1, 2: nt, nn, tn)."""
    groups, rows = offsets.shape[0] - 1, first.shape[0]
    n, k = (second.shape[1], second.shape[2]) if mode < 2 else (first.shape[1], second.shape[1])
    ws, ws_bytes = _workspace(workspace)
    return lib().gemm_grouped_stall_test(mode, _dtype(first.dtype), groups, rows, n, k, offsets.data_ptr(), first.data_ptr(),
                                         second.data_ptr(), out.data_ptr(), ws, ws_bytes, skip_fill, wait_limit_cycles,
                                         _gemm._stream(stream))


# ------------------------------------------------------------------- adapters

def gemm_lora_workspace_size(rows, n, k, rank, adapters):
    return _size("gemm_lora_workspace_size", rows, n, k, rank, adapters)


def gemm_lora_nt(x, w, a, b, ids, scale=None, y=None, workspace=None, stream=None):
    """y[t] = x[t] . w^T + scale[i] (x[t] . a[i]^T) . b[i]^T with i = ids[t]; no adapter where ids[t] is not in [0, adapters).

    x [rows, k], w [n, k], a [adapters, rank, k], b [adapters, n, rank], ids [rows] int32, scale [adapters] float32 or
    None for 1; returns y [rows, n].  The workspace (gemm_lora_workspace_size) is required."""
    torch = _gemm._tm()
    _operand(x, "x", 2)
    rows, k = x.shape
    if w.dim() != 2 or a.dim() != 3:
        raise ValueError("w must be [n, k] and a [adapters, rank, k]")
    n, adapters, rank = w.shape[0], a.shape[0], a.shape[1]
    _need(w, "w", (n, k), x.dtype, x.device)
    _need(a, "a", (adapters, rank, k), x.dtype, x.device)
    _need(b, "b", (adapters, n, rank), x.dtype, x.device)
    _need(ids, "ids", (rows,), torch.int32, x.device)
    if scale is not None:
        _need(scale, "scale", (adapters,), torch.float32, x.device)
    kind = _dtype(x.dtype)
    y = _out(y, "y", (rows, n), x.dtype, x.device)
    ws, ws_bytes = _workspace(workspace)
    _check(lib().gemm_lora_nt(kind, rows, n, k, rank, adapters, x.data_ptr(), w.data_ptr(), a.data_ptr(), b.data_ptr(),
                              ids.data_ptr(), None if scale is None else scale.data_ptr(), y.data_ptr(), ws, ws_bytes,
                              _gemm._stream(stream)), "gemm_lora_nt")
    return y


# --------------------------------------------------------------------- router

def gemm_route_workspace_size(rows, experts, top):
    return _size("gemm_route_workspace_size", rows, experts, top)


def gemm_route_topk(logits, top, renorm=True, out=None, workspace=None, stream=None):
    """The `top` largest logits of each row and the rows sorted by expert, as a Routing.

    logits [rows, experts] float16, bfloat16 or float32; returns ids, weights and position [rows, top], offsets
    [experts + 1] and order [rows * top] (choices t * top + j sorted by expert).  The weights are softmax(logits) at
    ids, divided by their sum if `renorm`.  `out`: a Routing of tensors to write into."""
    torch = _gemm._tm()
    _operand(logits, "logits", 2)
    rows, experts = logits.shape
    kind = _dtype(logits.dtype, f32=True)
    dev = logits.device
    top = int(top)
    shapes = Routing((rows, top), (rows, top), (experts + 1,), (rows * top,), (rows, top))
    kinds = Routing(torch.int32, torch.float32, torch.int32, torch.int32, torch.int32)
    if top < 1 or top > experts:
        raise ValueError("top must be in [1, experts]")
    given = out if out is not None else Routing(None, None, None, None, None)
    r = Routing(*(_out(t, name, shape, k, dev) for t, name, shape, k in zip(given, Routing._fields, shapes, kinds)))
    ws, ws_bytes = _workspace(workspace)
    _check(lib().gemm_route_topk(kind, rows, experts, top, int(bool(renorm)), logits.data_ptr(), r.ids.data_ptr(),
                                 r.weights.data_ptr(), r.offsets.data_ptr(), r.order.data_ptr(), r.position.data_ptr(), ws,
                                 ws_bytes, _gemm._stream(stream)), "gemm_route_topk")
    return r


def gemm_route_topk_grad(logits, ids, weights, dweights, renorm=True, dlogits=None, stream=None):
    """The gradient of the logits [rows, experts] float32 from that of gemm_route_topk's weights."""
    torch = _gemm._tm()
    _operand(logits, "logits", 2)
    rows, experts = logits.shape
    kind = _dtype(logits.dtype, f32=True)
    if ids.dim() != 2:
        raise ValueError("ids must be [rows, top]")
    top = ids.shape[1]
    _need(ids, "ids", (rows, top), torch.int32, logits.device)
    _need(weights, "weights", (rows, top), torch.float32, logits.device)
    _need(dweights, "dweights", (rows, top), torch.float32, logits.device)
    dlogits = _out(dlogits, "dlogits", (rows, experts), torch.float32, logits.device)
    _check(lib().gemm_route_topk_grad(kind, rows, experts, top, int(bool(renorm)), logits.data_ptr(), ids.data_ptr(),
                                      weights.data_ptr(), dweights.data_ptr(), dlogits.data_ptr(), _gemm._stream(stream)),
           "gemm_route_topk_grad")
    return dlogits
