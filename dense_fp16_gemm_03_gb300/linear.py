"""ctypes binding of include/gemm_linear.h (same entry-point names): products
with a bias, an activation and a residual in their epilogue, and their gradients.

Argument marshalling only (the calls' in csrc/binding.cpp), with the rules of
``ragged`` for operands, streams, outputs and workspaces.  ``w`` is one matrix [n, k], or with ``offsets`` one per
group of rows [groups, n, k], as the grouped products take them; bias and
dbias then have a line per group.  ``act``: None or "none", "relu", "relu2",
"gelu", "gelu_tanh" or "silu".

A layer y = f(x w^T + bias) and its backward pass:

    y, z = gemm_linear_nt(x, w, bias=bias, act="gelu", keep=True, workspace=ws)
    dz, dbias = gemm_linear_grad(dy, z, act="gelu", bias_grad=True, workspace=ws)
    dx = gemm_linear_nn(dz, w, workspace=ws)
    dw = ragged.gemm_grouped_tn(dz, x, ...)

and where another layer's activation lies below, gemm_linear_nn(dz, w, z=z_below,
act=..., bias_grad=True) gives that layer's dz and dbias at once.
"""
import ctypes

from . import _binding
from . import gemm as _gemm
from .ragged import _dtype, _need, _offsets, _operand, _size, _stream, _workspace

ACTS = {None: 0, "none": 0, "relu": 1, "relu2": 2, "gelu": 3, "gelu_tanh": 4, "silu": 5}

# every symbol the public header declares
EXPORTED = ["gemm_linear_workspace_size", "gemm_linear_nt", "gemm_linear_nn", "gemm_linear_grad", "gemm_linear_stall_test"]

_lib = None
_native = None
_checked = _binding.checked


def _load():
    global _native
    _native = _binding.native()
    return _native


def _raw(stream):
    return None if stream is None else _gemm._stream(stream)


def lib():
    """The library of ``gemm.lib()`` with this header's signatures."""
    global _lib
    if _lib is not None:
        return _lib
    L = _gemm.lib()
    i32, i64, u32, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_size_t
    kind = ctypes.c_int
    sig = {
        "gemm_linear_workspace_size": [i64, i64, i64, i64, ctypes.POINTER(ctypes.c_size_t)],
        "gemm_linear_nt": [kind, kind, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "gemm_linear_nn": [kind, kind, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "gemm_linear_grad": [kind, kind, i64, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp],
        "gemm_linear_stall_test": [i32, kind, kind, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, sz, u32, ctypes.c_longlong, vp],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.restype = ctypes.c_int
        f.argtypes = args
    _lib = L
    return L


def _act(act):
    code = ACTS.get(act)
    if code is None:
        raise ValueError("act must be one of %s" % ", ".join(repr(a) for a in ACTS))
    return code


def _groups(offsets, dev):
    """(number of groups, address of the offsets, leading sizes of what each group has of its own)"""
    if offsets is None:
        return 1, None, ()
    groups = _offsets(offsets, dev)
    return groups, offsets.data_ptr(), (groups,)


def _weights(w, stack):
    """n and k of the weights."""
    shape = w.shape
    if len(shape) != len(stack) + 2:
        raise ValueError("w must be [groups, n, k]" if stack else "w must be [n, k] without offsets")
    return shape[-2], shape[-1]


def _at(t, what, shape, dtype, dev):
    """The address of a tensor that has to be as _need says, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _need(t, what, shape, dtype, dev)
    return t.data_ptr()


def gemm_linear_workspace_size(groups, rows, n, k):
    return _size("gemm_linear_workspace_size", groups, rows, n, k)


def gemm_linear_nt(x, w, bias=None, residual=None, act=None, offsets=None, keep=False, y=None, z=None, workspace=None, stream=None):
    """y = f(x w^T + bias) + residual; with `keep` (y, z), where z = x w^T + bias is what the backward pass needs.

    x [rows, k], w [n, k], bias [n], residual [rows, n] (y may be the residual itself); with offsets [groups + 1] int32 on the
    device w [groups, n, k], bias [groups, n], and rows of no group are zero."""
    r = (_native or _load()).linear_nt(x, w, bias, residual, _act(act), offsets, keep, y, z, workspace, _raw(stream))
    return _checked(r, "gemm_linear_nt")


def gemm_linear_nn(dy, w, z=None, act=None, offsets=None, bias_grad=False, dx=None, dbias=None, workspace=None, stream=None):
    """dx = (dy w) * f'(z), the gradient of z = x w^T + bias one layer below; with `bias_grad` (dx, dbias), dbias the sum of dx
    over the rows (of each group) in float32.

    dy [rows, n], w [n, k] or [groups, n, k], z [rows, k] (not needed without `act`; dx may be z itself)."""
    r = (_native or _load()).linear_nn(dy, w, z, _act(act), offsets, bias_grad, dx, dbias, workspace, _raw(stream))
    return _checked(r, "gemm_linear_nn")


def gemm_linear_grad(dy, z=None, act=None, offsets=None, bias_grad=False, dz=None, dbias=None, workspace=None, stream=None):
    """dz = dy * f'(z); with `bias_grad` (dz, dbias), dbias the sum of dz over the rows (of each group) in float32.

    dy, z [rows, n]; dz may be dy or z.  Without `act` and offsets dz is dy, which is returned as it is unless another dz is given."""
    r = (_native or _load()).linear_grad(dy, z, _act(act), offsets, bias_grad, dz, dbias, workspace, _raw(stream))
    return _checked(r, "gemm_linear_grad")


def gemm_linear_stall_test(mode, first, w, extra, out, dbias, workspace, skip_fill, wait_limit_cycles, act=None, offsets=None, stream=None):
    """Status of the failure-detection launch (mode 0: nt with a residual, 1: nn with z and dbias)."""
    lib()
    dev, kind = _operand(first, "first", 2), first.dtype
    groups, ends, stack = _groups(offsets, dev)
    rows = first.shape[0]
    n, k = _weights(w, stack)
    wp = _at(w, "w", (*stack, first.shape[1], k) if mode else (*stack, n, first.shape[1]), kind, dev)
    shape = (rows, k if mode else n)
    _need(out, "out", shape, kind, dev)
    more = _at(extra, "extra", shape, kind, dev)
    db = _at(dbias, "dbias", (*stack, k), _gemm._tm().float32, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    return _lib.gemm_linear_stall_test(mode, _dtype(kind), _act(act), groups, rows, n, k, ends, first.data_ptr(), wp, more,
                                       out.data_ptr(), db, ws, ws_bytes, skip_fill, wait_limit_cycles, _stream(stream, dev))
