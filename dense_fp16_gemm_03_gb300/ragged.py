"""ctypes binding of include/gemm_ragged.h (same entry-point names): grouped
products by expert with their gradients, low-rank adapters beside a shared
projection, and the experts' router.

Argument marshalling only, as in ``gemm`` (that of the router with scores in
csrc/binding.cpp): every step runs in the CUDA library,
a missing library raises, and there is no fallback.  Operands are contiguous
CUDA tensors; a call runs on ``stream`` (a torch.cuda.Stream, a raw integer, or
None for the current torch stream).  Outputs that are not given are allocated
on the current torch stream; workspaces are the caller's (sizes from the
``*_workspace_size`` functions, any contents, one call at a time).
"""
import collections
import ctypes

from . import _binding
from . import gemm as _gemm
from .gemm import GemmError, gemm_f16_take_device_error  # noqa: F401  (the same errors, the same device word)

DTYPE_F16 = 0
DTYPE_BF16 = 1
DTYPE_F32 = 2

MAX_GROUPS = 1024
MAX_RANK = 128
MAX_EXPERTS = 1024
MAX_TOP = 32
MAX_ROUTE_GROUPS = 32

ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}

LORA_BESIDE = 0
LORA_TENSOR_CORES = 1

# every symbol the public header declares
EXPORTED = [
    "gemm_grouped_workspace_size", "gemm_grouped_nt", "gemm_grouped_nn", "gemm_grouped_tn", "gemm_grouped_stall_test",
    "gemm_lora_workspace_size", "gemm_lora_way", "gemm_lora_nt", "gemm_lora_stall_test",
    "gemm_route_workspace_size", "gemm_route_topk", "gemm_route_topk_grad", "gemm_route_scored", "gemm_route_scored_grad",
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
        "gemm_lora_way": [i64, i64, i64, i64, i64, i32, ctypes.POINTER(i32)],
        "gemm_lora_nt": [dt, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "gemm_lora_stall_test": [dt, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, sz, u32, ctypes.c_longlong, vp],
        "gemm_route_workspace_size": [i64, i64, i64, psz],
        "gemm_route_topk": [dt, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "gemm_route_topk_grad": [dt, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp],
        "gemm_route_scored": [dt, dt, i64, i64, i64, i64, i64, i32, i32, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "gemm_route_scored_grad": [dt, dt, i64, i64, i64, i32, ctypes.c_float, vp, vp, vp, vp, vp],
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


def _need(t, what, shape, dtype, dev):
    """`t` must be a contiguous tensor of this shape and type on CUDA device number `dev`."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on cuda:%d" % (what, dtype, list(shape), dev))


def _operand(t, what, dims):
    """The device number of a contiguous tensor on the current CUDA device."""
    dev = t.get_device()
    if dev < 0 or t.dim() != dims or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor with %d dimensions" % (what, dims))
    if dev != _gemm._tm()._C._cuda_getDevice():
        raise ValueError("%s must be on the current device" % what)
    return dev


_devices = {}


def _empty(shape, dtype, dev):
    # (a device object at hand is quicker than Tensor.new_empty by more than a microsecond)
    device = _devices.get(dev)
    if device is None:
        device = _devices[dev] = _gemm._tm().device("cuda", dev)
    return _gemm._tm().empty(shape, dtype=dtype, device=device)


def _out(t, what, shape, dtype, dev):
    if t is None:
        return _empty(shape, dtype, dev)
    _need(t, what, shape, dtype, dev)
    return t


def _workspace(ws, dev):
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on cuda:%d" % dev)
    return ws.data_ptr(), ws.nbytes


def _stream(stream, dev):
    if stream is None:
        return _gemm._tm()._C._cuda_getCurrentRawStream(dev)
    return _gemm._stream(stream)


def _size(name, *args):
    b = ctypes.c_size_t()
    _check(getattr(lib(), name)(*args, ctypes.byref(b)), name)
    return b.value


# ------------------------------------------------------------ grouped products

def gemm_grouped_workspace_size(groups, rows, n, k):
    return _size("gemm_grouped_workspace_size", groups, rows, n, k)


def _offsets(offsets, dev):
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must hold groups + 1 numbers")
    _need(offsets, "offsets", offsets.shape, _gemm._tm().int32, dev)
    return offsets.shape[0] - 1


def gemm_grouped_nt(x, w, offsets, y=None, workspace=None, stream=None):
    """y[t] = x[t] . w[g]^T for the rows t in [offsets[g], offsets[g + 1]); rows of no group are zero.

    x [rows, k], w [groups, n, k], offsets [groups + 1] int32 on the device; returns y [rows, n]."""
    dev, kind = _operand(x, "x", 2), x.dtype
    groups = _offsets(offsets, dev)
    rows, k = x.shape
    if w.dim() != 3:
        raise ValueError("w must be [groups, n, k]")
    n = w.shape[1]
    _need(w, "w", (groups, n, k), kind, dev)
    code = _dtype(kind)
    y = _out(y, "y", (rows, n), kind, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    st = lib().gemm_grouped_nt(code, groups, rows, n, k, offsets.data_ptr(), x.data_ptr(), w.data_ptr(), y.data_ptr(), ws,
                               ws_bytes, _stream(stream, dev))
    _check(st, "gemm_grouped_nt")
    return y


def gemm_grouped_nn(dy, w, offsets, dx=None, workspace=None, stream=None):
    """dx[t] = dy[t] . w[g]: the gradient of gemm_grouped_nt's rows.  dy [rows, n]; returns dx [rows, k]."""
    dev, kind = _operand(dy, "dy", 2), dy.dtype
    groups = _offsets(offsets, dev)
    rows, n = dy.shape
    if w.dim() != 3:
        raise ValueError("w must be [groups, n, k]")
    k = w.shape[2]
    _need(w, "w", (groups, n, k), kind, dev)
    code = _dtype(kind)
    dx = _out(dx, "dx", (rows, k), kind, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    st = lib().gemm_grouped_nn(code, groups, rows, n, k, offsets.data_ptr(), dy.data_ptr(), w.data_ptr(), dx.data_ptr(), ws,
                               ws_bytes, _stream(stream, dev))
    _check(st, "gemm_grouped_nn")
    return dx


def gemm_grouped_tn(dy, x, offsets, dw=None, dtype=None, workspace=None, stream=None):
    """dw[g] = dy_g^T . x_g: the gradient of gemm_grouped_nt's weights, zero for a group without rows.

    dy [rows, n], x [rows, k]; returns dw [groups, n, k] in `dtype` (the operands' type, or torch.float32)."""
    dev, kind = _operand(dy, "dy", 2), dy.dtype
    groups = _offsets(offsets, dev)
    rows, n = dy.shape
    if x.dim() != 2:
        raise ValueError("x must be [rows, k]")
    k = x.shape[1]
    _need(x, "x", (rows, k), kind, dev)
    code = _dtype(kind)
    if dtype is None:
        dtype = kind if dw is None else dw.dtype
    if dtype is not kind and dtype is not _gemm._tm().float32:
        raise ValueError("dw must have the operands' type or float32")
    dw = _out(dw, "dw", (groups, n, k), dtype, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    st = lib().gemm_grouped_tn(code, _dtype(dtype, f32=True), groups, rows, n, k, offsets.data_ptr(), dy.data_ptr(),
                               x.data_ptr(), dw.data_ptr(), ws, ws_bytes, _stream(stream, dev))
    _check(st, "gemm_grouped_tn")
    return dw


def gemm_grouped_stall_test(mode, first, second, offsets, out, workspace, skip_fill, wait_limit_cycles, stream=None):
    """Status of the failure-detection launch (mode 0, 1, 2: nt, nn, tn)."""
    dev = _operand(first, "first", 2)
    groups, rows = _offsets(offsets, dev), first.shape[0]
    n, k = (second.shape[1], second.shape[2]) if mode < 2 else (first.shape[1], second.shape[1])
    _need(second, "second", (groups, n, k) if mode < 2 else (rows, k), first.dtype, dev)
    _need(out, "out", ((rows, n), (rows, k), (groups, n, k))[mode], first.dtype, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    return lib().gemm_grouped_stall_test(mode, _dtype(first.dtype), groups, rows, n, k, offsets.data_ptr(), first.data_ptr(),
                                         second.data_ptr(), out.data_ptr(), ws, ws_bytes, skip_fill, wait_limit_cycles,
                                         _stream(stream, dev))


# ------------------------------------------------------------------- adapters

def gemm_lora_workspace_size(rows, n, k, rank, adapters):
    return _size("gemm_lora_workspace_size", rows, n, k, rank, adapters)


def gemm_lora_way(rows, n, k, rank, adapters, num_sms=0):
    """LORA_BESIDE or LORA_TENSOR_CORES: how a call of these sizes runs, on the current device or on one of `num_sms` SMs."""
    way = ctypes.c_int32()
    _check(lib().gemm_lora_way(rows, n, k, rank, adapters, num_sms, ctypes.byref(way)), "gemm_lora_way")
    return way.value


def _lora_sizes(x, w, a, b, ids, scale):
    """Device number, rows, n, k, rank and adapters of a call, its operands checked."""
    torch = _gemm._tm()
    dev, kind = _operand(x, "x", 2), x.dtype
    rows, k = x.shape
    if w.dim() != 2 or a.dim() != 3:
        raise ValueError("w must be [n, k] and a [adapters, rank, k]")
    n = w.shape[0]
    adapters, rank, _ = a.shape
    _need(w, "w", (n, k), kind, dev)
    _need(a, "a", (adapters, rank, k), kind, dev)
    _need(b, "b", (adapters, n, rank), kind, dev)
    _need(ids, "ids", (rows,), torch.int32, dev)
    if scale is not None:
        _need(scale, "scale", (adapters,), torch.float32, dev)
    return dev, rows, n, k, rank, adapters


def gemm_lora_nt(x, w, a, b, ids, scale=None, y=None, workspace=None, stream=None):
    """y[t] = x[t] . w^T + scale[i] (x[t] . a[i]^T) . b[i]^T with i = ids[t]; no adapter where ids[t] is not in [0, adapters).

    x [rows, k], w [n, k], a [adapters, rank, k], b [adapters, n, rank], ids [rows] int32, scale [adapters] float32 or
    None for 1; returns y [rows, n].  The workspace (gemm_lora_workspace_size) is required."""
    dev, rows, n, k, rank, adapters = _lora_sizes(x, w, a, b, ids, scale)
    kind = x.dtype
    code = _dtype(kind)
    y = _out(y, "y", (rows, n), kind, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    st = lib().gemm_lora_nt(code, rows, n, k, rank, adapters, x.data_ptr(), w.data_ptr(), a.data_ptr(), b.data_ptr(),
                            ids.data_ptr(), None if scale is None else scale.data_ptr(), y.data_ptr(), ws, ws_bytes,
                            _stream(stream, dev))
    _check(st, "gemm_lora_nt")
    return y


def gemm_lora_stall_test(x, w, a, b, ids, y, workspace, skip_fill, wait_limit_cycles, scale=None, stream=None):
    """Status of the failure-detection launch."""
    dev, rows, n, k, rank, adapters = _lora_sizes(x, w, a, b, ids, scale)
    _need(y, "y", (rows, n), x.dtype, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    return lib().gemm_lora_stall_test(_dtype(x.dtype), rows, n, k, rank, adapters, x.data_ptr(), w.data_ptr(), a.data_ptr(),
                                      b.data_ptr(), ids.data_ptr(), None if scale is None else scale.data_ptr(), y.data_ptr(),
                                      ws, ws_bytes, skip_fill, wait_limit_cycles, _stream(stream, dev))


# --------------------------------------------------------------------- router

def gemm_route_workspace_size(rows, experts, top):
    return _size("gemm_route_workspace_size", rows, experts, top)


def _routing(out, rows, experts, top, dev):
    """A Routing to write into: `out`, checked, or a new one."""
    torch = _gemm._tm()
    i32 = torch.int32
    shape, f32 = (rows, top), torch.float32
    if out is None:  # (five allocations are quicker than views of one)
        r = Routing(_empty(shape, i32, dev), _empty(shape, f32, dev), _empty((experts + 1,), i32, dev),
                    _empty((rows * top,), i32, dev), _empty(shape, i32, dev))
    else:
        r = out
        _need(r.ids, "ids", shape, i32, dev)
        _need(r.weights, "weights", shape, f32, dev)
        _need(r.offsets, "offsets", (experts + 1,), i32, dev)
        _need(r.order, "order", (rows * top,), i32, dev)
        _need(r.position, "position", shape, i32, dev)
    return r


def gemm_route_topk(logits, top, renorm=True, out=None, workspace=None, stream=None):
    """The `top` largest logits of each row and the rows sorted by expert, as a Routing.

    logits [rows, experts] float16, bfloat16 or float32; returns ids, weights and position [rows, top], offsets
    [experts + 1] and order [rows * top] (choices t * top + j sorted by expert).  The weights are softmax(logits) at
    ids, divided by their sum if `renorm`.  `out`: a Routing of tensors to write into.  The workspace
    (gemm_route_workspace_size) is required above 64 rows."""
    dev = _operand(logits, "logits", 2)
    rows, experts = logits.shape
    code = _dtype(logits.dtype, f32=True)
    top = int(top)
    if top < 1 or top > experts:
        raise ValueError("top must be in [1, experts]")
    r = _routing(out, rows, experts, top, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    st = lib().gemm_route_topk(code, rows, experts, top, 1 if renorm else 0, logits.data_ptr(), r.ids.data_ptr(),
                               r.weights.data_ptr(), r.offsets.data_ptr(), r.order.data_ptr(), r.position.data_ptr(), ws,
                               ws_bytes, _stream(stream, dev))
    _check(st, "gemm_route_topk")
    return r


def gemm_route_topk_grad(logits, ids, weights, dweights, renorm=True, dlogits=None, stream=None):
    """The gradient of the logits [rows, experts] float32 from that of gemm_route_topk's weights."""
    torch = _gemm._tm()
    dev = _operand(logits, "logits", 2)
    rows, experts = logits.shape
    code = _dtype(logits.dtype, f32=True)
    if ids.dim() != 2:
        raise ValueError("ids must be [rows, top]")
    shape = ids.shape
    _need(ids, "ids", (rows, shape[1]), torch.int32, dev)
    _need(weights, "weights", shape, torch.float32, dev)
    _need(dweights, "dweights", shape, torch.float32, dev)
    dlogits = _out(dlogits, "dlogits", (rows, experts), torch.float32, dev)
    st = lib().gemm_route_topk_grad(code, rows, experts, shape[1], 1 if renorm else 0, logits.data_ptr(), ids.data_ptr(),
                                    weights.data_ptr(), dweights.data_ptr(), dlogits.data_ptr(), _stream(stream, dev))
    _check(st, "gemm_route_topk_grad")
    return dlogits


def _score(score):
    code = ROUTE_SCORES.get(score)
    if code is None:
        raise ValueError("score must be one of %s" % ", ".join(repr(n) for n in ROUTE_SCORES))
    return code


def gemm_route_scored(logits, top, score="sigmoid", bias=None, groups=1, top_groups=None, group_top=2, renorm=True, scale=1.0,
                      out=None, workspace=None, stream=None):
    """The `top` experts of each row with the largest s + bias among those of its best groups, as a Routing.

    s = softmax(logits) or the logits' sigmoid; bias [experts] float32 moves the choice and not the weights.  The experts form
    `groups` (1, 2, 4 ... 32) groups of neighbours; the `top_groups` (None: all) with the largest score are kept, a group's
    score being its largest s + bias (group_top 1) or the sum of its two largest (2).  The weights are scale * s at ids,
    divided by their sum if `renorm`.  `out` (all five tensors) and the workspace as in gemm_route_topk.  Without `out` the five
    lie in one allocation, which lives as long as any of them; clone one that is kept for long by itself."""
    groups = int(groups)
    r = _binding.native().route_scored(logits, int(top), _score(score), bias, groups, groups if top_groups is None else int(top_groups),
                                       group_top, renorm, scale, out, workspace, None if stream is None else _gemm._stream(stream))
    _binding.checked(r, "gemm_route_scored")
    return Routing._make(r) if out is None else out


def gemm_route_scored_grad(logits, ids, dweights, score="sigmoid", renorm=True, scale=1.0, dlogits=None, stream=None):
    """The gradient of the logits [rows, experts] float32 from that of gemm_route_scored's weights."""
    r = _binding.native().route_scored_grad(logits, ids, dweights, _score(score), renorm, scale, dlogits,
                                            None if stream is None else _gemm._stream(stream))
    return _binding.checked(r, "gemm_route_scored_grad")
