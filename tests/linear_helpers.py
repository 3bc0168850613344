"""Plain 64-bit implementations of the products with an epilogue and of their gradients, with bounds on how far the kernels'
results may be from them."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from dense_fp16_gemm_03_gb300 import gemm as G  # noqa: E402
from dense_fp16_gemm_03_gb300 import linear as L  # noqa: E402
from ragged_helpers import KINDS, eighths, no_device_error, offsets_of, require_gpu  # noqa: E402, F401

ACTS = ["none", "relu", "relu2", "gelu", "gelu_tanh", "silu"]


def value(act, z):
    """f(z) in float64."""
    if act == "relu":
        return z.clamp(min=0)
    if act == "relu2":
        return z.clamp(min=0) ** 2
    if act == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2)) / 2
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def terms(act, z):
    """f'(z) in float64 as the two terms that the kernels add."""
    zero = torch.zeros_like(z)
    if act == "relu":
        return (z > 0).double(), zero
    if act == "relu2":
        return 2 * z.clamp(min=0), zero
    if act == "gelu":
        return torch.special.erfc(-z / math.sqrt(2)) / 2, z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        s = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return s, z * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
    if act == "silu":
        s = torch.sigmoid(z)
        return s, z * s * (1 - s)
    return torch.ones_like(z), zero


def act_error(act, z):
    """A bound on the relative error of f(z), and of each term of f'(z), in fp32 arithmetic: an exponential of a value a that is
    itself rounded a few times in fp32 is off by |a| 2^-22 at most, with |a| up to z^2/2 (gelu), 1.6 |z| + 0.08 |z|^3
    (gelu_tanh) or |z| (silu); the approximate exponential and reciprocal by 2^-22 each, the polynomial by 2^-22, a dozen
    other roundings by 2^-24 each."""
    if act in ("none", "relu", "relu2"):
        return torch.full_like(z, 2.0 ** -23)
    a = {"gelu": z * z / 2, "gelu_tanh": 1.6 * z.abs() + 0.08 * z.abs() ** 3, "silu": z.abs()}[act]
    return (a + 8) * 2.0 ** -22


def flushed(act, z):
    """The approximate exponential and reciprocal give 0 below 2^-126 (their results are e^-a <= 1 and s <= 1, so nothing else is
    flushed): the term without z is off by 2^-126 then, the other by that times what multiplies it."""
    if act in ("none", "relu", "relu2"):
        return torch.zeros_like(z)
    return (1 + z.abs() * (1.6 + 0.22 * z * z if act == "gelu_tanh" else 1.0)) * 2.0 ** -126


def grad_error(act, z):
    """A bound on the error of f'(z): both terms' relative errors, and that of 1 - s, which is off by 2^-22 where s is near 1."""
    a, b = terms(act, z)
    off = act_error(act, z) * (a.abs() + b.abs()) + flushed(act, z)
    if act == "silu":
        off = off + z.abs() * 2.0 ** -21
    if act == "gelu_tanh":
        off = off + z.abs() * (1.6 + 0.22 * z * z) * 2.0 ** -21
    return off


def rounded(kind, ref, off):
    """How far a value within `off` of ref may be from ref once it is rounded to `kind`: half a step of the value, or of the
    smallest normal number below that."""
    info = torch.finfo(kind)
    return off + info.eps / 2 * torch.clamp(ref.abs() + off, min=info.tiny)


def near(got, ref, bound, what):
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    fine = torch.isfinite(ref)
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), what
    over = ((got - ref).abs() > bound) & fine
    if over.any():
        at = tuple(torch.nonzero(over)[0].tolist())
        raise AssertionError("%s: %d of %d values off, first at %s: %r, want %r within %r" % (
            what, int(over.sum()), over.numel(), at, float(got[at]), float(ref[at]), float(bound[at])))


def ends_of(offsets, rows):
    """[(group, first row, end)] as the header defines them."""
    if offsets is None:
        return [(0, 0, rows)]
    e = np.maximum.accumulate(np.clip(offsets.cpu().numpy().astype(np.int64), 0, rows)).tolist()
    return [(g, e[g], e[g + 1]) for g in range(len(e) - 1)]


def nt_ref(x, w, bias, residual, act, offsets):
    """y, a bound on its error before rounding, and z; host tensors, products exact in fp32 by the operands' choice."""
    rows, n = x.shape[0], w.shape[-2]
    y, off, z = (torch.zeros((rows, n), dtype=torch.float64) for _ in range(3))
    for g, lo, hi in ends_of(offsets, rows):
        wg, bg = (w, bias) if offsets is None else (w[g], None if bias is None else bias[g])
        zz = x[lo:hi].double() @ wg.double().T
        if bg is not None:
            zz = zz + bg.double()
        f = value(act, zz)
        z[lo:hi], y[lo:hi], off[lo:hi] = zz, f, act_error(act, zz) * f.abs() + flushed(act, zz) if act != "none" else 0.0
        if residual is not None:
            y[lo:hi] += residual[lo:hi].double()
            off[lo:hi] += y[lo:hi].abs() * 2.0 ** -24 if act != "none" else 0.0
    return y, off, z


def grad_ref(d, z, act, offsets, groups=None):
    """dx = d f'(z) with d in float64, a bound on its error before rounding, dbias and a bound on its error; d of rows of no
    group is left out."""
    rows, cols = d.shape
    dx, off = torch.zeros_like(d), torch.zeros_like(d)
    ends = ends_of(offsets, rows)
    db, db_off = (torch.zeros((len(ends), cols), dtype=torch.float64) for _ in range(2))
    for g, lo, hi in ends:
        dd = d[lo:hi]
        if act != "none":
            a, b = terms(act, z[lo:hi].double())
            v, o = dd * (a + b), dd.abs() * grad_error(act, z[lo:hi].double()) + (dd * (a + b)).abs() * 2.0 ** -23
        else:
            v, o = dd, torch.zeros_like(dd)
        dx[lo:hi], off[lo:hi] = v, o
        db[g] = v.sum(0)
        # a sum of m values in fp32, in any order: m - 1 roundings of partial sums that the sum of magnitudes bounds
        db_off[g] = o.sum(0) + (hi - lo) * 2.0 ** -24 * (v.abs() + o).sum(0)
    if offsets is None:
        db, db_off = db[0], db_off[0]
    return dx, off, db, db_off


def buffer(groups, rows, n, k):
    return torch.full((L.gemm_linear_workspace_size(groups, rows, n, k),), 0xA5, dtype=torch.uint8, device="cuda")


def cuda(t):
    return None if t is None else t.cuda()


def draw(rng, sizes, n, k, kind, grouped, bias=True, residual=True, extra=0):
    """Operands on the host; integers over 8, with weights that keep z small: (x, w, bias, residual, offsets)."""
    rows, groups = int(sum(sizes)) + extra, len(sizes)
    stack = (groups,) if grouped else ()
    x = eighths(rng, (rows, k), kind)
    # few columns of w are not zero, so that z stays within some ten
    w = eighths(rng, stack + (n, k), kind) * (torch.from_numpy(rng.random(stack + (n, k))) < min(1.0, 24.0 / max(k, 1))).to(kind)
    b = eighths(rng, stack + (n,), kind) if bias else None
    r = eighths(rng, (rows, n), kind) if residual else None
    return x, w, b, r, (offsets_of(sizes) if grouped else None)
