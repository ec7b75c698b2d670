"""What stands between the products: layer norm with its gradients, and dropout.

The ``gemm_*`` functions forward to the entry points of the same name
(include/dense_fp32_tiled.h).  ``layer_norm``, ``layer_norm_grad`` and
``dropout`` take torch tensors (bfloat16, float16 or float32); they check
types, layouts, shapes and devices before anything is launched, enqueue on
``stream`` or torch's current stream of the tensors' device, allocate on it,
and raise GemmError on a non-zero status, as the layers of products.py do.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import dense_fp32_tiled_amd as dft

from . import products as pr

VALUE_BF16, VALUE_F16, VALUE_F32 = range(3)

_i32, _i64, _u64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p
_f32, _f64 = ctypes.c_float, ctypes.c_double


class LayerNormArgs(ctypes.Structure):
    """gemm_layer_norm_args."""
    _fields_ = [("value_type", _i32), ("eps", _f32), ("p", _f64), ("seed", _u64), ("offset", _u64), ("step", _vp),
                ("rows", _i64), ("cols", _i64), ("x", _vp), ("ldx", _i64), ("residual", _vp), ("ldr", _i64),
                ("weight", _vp), ("bias", _vp), ("total", _vp), ("ldt", _i64), ("y", _vp), ("ldy", _i64),
                ("mean", _vp), ("rstd", _vp)]


class LayerNormGradArgs(ctypes.Structure):
    """gemm_layer_norm_grad_args."""
    _fields_ = [("value_type", _i32), ("p", _f64), ("seed", _u64), ("offset", _u64), ("step", _vp), ("rows", _i64),
                ("cols", _i64), ("dY", _vp), ("ldy", _i64), ("total", _vp), ("ldt", _i64), ("mean", _vp),
                ("rstd", _vp), ("weight", _vp), ("dstream", _vp), ("lds", _i64), ("dtotal", _vp), ("lddt", _i64),
                ("dx", _vp), ("lddx", _i64), ("dweight", _vp), ("dbias", _vp), ("workspace", _vp),
                ("workspace_bytes", _i64)]


class NormState(NamedTuple):
    """What layer_norm keeps for layer_norm_grad: the rows that were normalised, and their statistics (float32)."""
    total: object
    mean: object
    rstd: object


class NormGrads(NamedTuple):
    """Gradients of layer_norm's x, residual, weight and bias; None where not wanted."""
    x: object
    residual: object
    weight: object
    bias: object


def declare(lib) -> None:
    """Argument and result types of this module's entry points."""
    i = ctypes.c_int
    for name, result, types in (
            ("gemm_layer_norm", i, [ctypes.POINTER(LayerNormArgs), _vp]),
            ("gemm_layer_norm_grad", i, [ctypes.POINTER(LayerNormGradArgs), _vp]),
            ("gemm_layer_norm_grad_workspace_bytes", _i64, [ctypes.POINTER(LayerNormGradArgs), _i32]),
            ("gemm_dropout", i, [i, _i64, _i64, _f64, _u64, _u64, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = result, types


# ---- entry points, same names as the C ABI ----------------------------------------------
def gemm_layer_norm(args: LayerNormArgs, stream=None) -> int:
    return dft.library().gemm_layer_norm(args, stream)


def gemm_layer_norm_grad(args: LayerNormGradArgs, stream=None) -> int:
    return dft.library().gemm_layer_norm_grad(args, stream)


def gemm_layer_norm_grad_workspace_bytes(args: LayerNormGradArgs, num_cus: int) -> int:
    return dft.library().gemm_layer_norm_grad_workspace_bytes(args, num_cus)


def gemm_dropout(value_type, rows, cols, p, seed, offset, step, X, ldx, residual, ldr, Y, ldy, stream=None) -> int:
    return dft.library().gemm_dropout(value_type, rows, cols, p, seed, offset, step, X, ldx, residual, ldr, Y, ldy,
                                      stream)


_NORM_GRADS = frozenset(("x", "residual", "weight", "bias"))


# ---- torch convenience --------------------------------------------------------------------
def _value_type(t, name):
    if pr.torch is None:
        pr._bind()
    if not isinstance(t, pr._Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype = t.dtype
    if dtype is pr._bf16:
        return VALUE_BF16
    if dtype is pr._f16:
        return VALUE_F16
    if dtype is pr._f32:
        return VALUE_F32
    raise TypeError(f"{name} must be bfloat16, float16 or float32, not {dtype}")


def _counter(p, seed, offset, step, device):
    """The seed and step's device pointer, after checks of what draws the mask."""
    if not 0 <= p <= 1:
        raise ValueError(f"p must lie in [0, 1], not {p}")
    if seed is None:
        if p > 0:
            raise ValueError("dropout needs a seed (calls of one seed and offset drop the same elements)")
        seed = 0
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("seed and offset must be unsigned 64-bit numbers")
    return seed, None if step is None else pr._list(step, "step", (1,), pr.torch.int64, device)


def dropout(x, p: float, seed: int, offset: int = 0, residual=None, step=None, out=None, stream=None):
    """x / (1 - p) where kept and 0 where dropped, plus ``residual``, by gemm_dropout.

    x: rows x cols; ``out`` may be x or residual itself.  The mask is a function of seed, offset (plus ``step``, one
    int64 on the device, which a captured graph can count up) and the element's place, and is never stored: the
    gradient for dy is ``dropout(dy, p, seed, offset)``."""
    kind, device = _value_type(x, "x"), pr._gpu(x, "x")
    if stream is not None:
        with pr._current(stream, device):
            return dropout(x, p, seed, offset, residual, step, out)
    rows, cols = x.shape if x.dim() == 2 else (-1, -1)
    dtype = x.dtype
    px, ldx = pr._matrix(x, "x", rows, cols, dtype, device)
    seed, at = _counter(p, seed, offset, step, device)
    pres, ldr = (None, 0) if residual is None else pr._matrix(residual, "residual", rows, cols, dtype, device)
    if out is None:
        out = pr.torch.empty(rows, cols, dtype=dtype, device=device)
        po, ldo = out.data_ptr(), cols if cols > 0 else 1
    else:
        po, ldo = pr._matrix(out, "out", rows, cols, dtype, device)
    pr._run(dft.library().gemm_dropout, "gemm_dropout", device, kind, rows, cols, p, seed, offset, at, px, ldx, pres,
            ldr, po, ldo)
    return out


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, residual=None, p: float = 0.0, seed: int | None = None,
               offset: int = 0, step=None, out=None, total=None, stream=None):
    """(y, NormState): each row of total = dropout(x) + residual normalised, times weight plus bias, by
    gemm_layer_norm.

    x, residual: rows x cols of one type; weight, bias: cols values of it.  Without residual and with p = 0, total is
    x itself; else it is rounded to the type and stored, in ``total`` if given (which may be x or residual itself).
    p, seed, offset and step as in ``dropout``; a p above 0 needs the seed."""
    kind, device = _value_type(x, "x"), pr._gpu(x, "x")
    if stream is not None:
        with pr._current(stream, device):
            return layer_norm(x, weight, bias, eps, residual, p, seed, offset, step, out, total)
    rows, cols = x.shape if x.dim() == 2 else (-1, -1)
    dtype = x.dtype
    px, ldx = pr._matrix(x, "x", rows, cols, dtype, device)
    seed, at = _counter(p, seed, offset, step, device)
    pw = None if weight is None else pr._list(weight, "weight", (cols,), dtype, device)
    pb = None if bias is None else pr._list(bias, "bias", (cols,), dtype, device)
    empty, ld = pr.torch.empty, cols if cols > 0 else 1
    pres = pt = None
    ldr = ldt = ldy = ld
    if residual is not None or p > 0:
        if residual is not None:
            pres, ldr = pr._matrix(residual, "residual", rows, cols, dtype, device)
        if total is None:
            total = empty(rows, cols, dtype=dtype, device=device)
            pt = total.data_ptr()
        else:
            pt, ldt = pr._matrix(total, "total", rows, cols, dtype, device)
    elif total is not None:
        raise ValueError("total is x itself without residual and dropout")
    else:
        total = x
    if out is None:
        out = empty(rows, cols, dtype=dtype, device=device)
        py = out.data_ptr()
    else:
        py, ldy = pr._matrix(out, "out", rows, cols, dtype, device)
    mean, rstd = empty(rows, dtype=pr._f32, device=device), empty(rows, dtype=pr._f32, device=device)
    pr._run(dft.library().gemm_layer_norm, "gemm_layer_norm", device,
            LayerNormArgs(kind, eps, p, seed, offset, at, rows, cols, px, ldx, pres, ldr, pw, pb, pt, ldt, py, ldy,
                          mean.data_ptr(), rstd.data_ptr()))
    return out, NormState(total, mean, rstd)


def layer_norm_grad(dy, state: NormState, weight=None, dtotal=None, p: float = 0.0, seed: int | None = None,
                    offset: int = 0, step=None, want=("x", "residual", "weight", "bias"), workspace=None,
                    stream=None) -> NormGrads:
    """Gradients of layer_norm for y's gradient dy and, where total is used elsewhere too, ``dtotal``, total's
    gradient from there, by gemm_layer_norm_grad.  x's and the residual's are of dy's type (one tensor without
    dropout), weight's and bias's float32.  ``want`` names the ones computed; p, seed, offset and step are the
    forward pass's."""
    kind, device = _value_type(dy, "dy"), pr._gpu(dy, "dy")
    if stream is not None:
        with pr._current(stream, device):
            return layer_norm_grad(dy, state, weight, dtotal, p, seed, offset, step, want, workspace)
    if not _NORM_GRADS.issuperset(want):
        raise ValueError(f"want names 'x', 'residual', 'weight' and 'bias', not {sorted(set(want) - _NORM_GRADS)}")
    rows, cols = dy.shape if dy.dim() == 2 else (-1, -1)
    dtype = dy.dtype
    py, ldy = pr._matrix(dy, "dy", rows, cols, dtype, device)
    seed, at = _counter(p, seed, offset, step, device)
    total, mean, rstd = state
    pt, ldt = pr._matrix(total, "state.total", rows, cols, dtype, device)
    pm = pr._list(mean, "state.mean", (rows,), pr._f32, device)
    ps = pr._list(rstd, "state.rstd", (rows,), pr._f32, device)
    pw = None if weight is None else pr._list(weight, "weight", (cols,), dtype, device)
    pd, lds = (None, 0) if dtotal is None else pr._matrix(dtotal, "dtotal", rows, cols, dtype, device)
    empty, ld = pr.torch.empty, cols if cols > 0 else 1
    dx = dresidual = dweight = dbias = pdx = pdr = pdw = pdb = None
    if "residual" in want or (p == 0 and "x" in want):
        dresidual = empty(rows, cols, dtype=dtype, device=device)
        pdr = dresidual.data_ptr()
    if "x" in want:
        dx = dresidual
        if p > 0:
            dx = empty(rows, cols, dtype=dtype, device=device)
            pdx = dx.data_ptr()
    if "weight" in want:
        dweight = empty(cols, dtype=pr._f32, device=device)
        pdw = dweight.data_ptr()
    if "bias" in want:
        dbias = empty(cols, dtype=pr._f32, device=device)
        pdb = dbias.data_ptr()
    g = LayerNormGradArgs(kind, p, seed, offset, at, rows, cols, py, ldy, pt, ldt, pm, ps, pw, pd, lds, pdr, ld, pdx, ld,
                          pdw, pdb)
    lib = dft.library()
    keep = pr._workspace(g, lib.gemm_layer_norm_grad_workspace_bytes(g, pr._num_cus(device)),
                         "gemm_layer_norm_grad_workspace_bytes", workspace, device)
    pr._run(lib.gemm_layer_norm_grad, "gemm_layer_norm_grad", device, g)
    del keep
    return NormGrads(dx, dresidual if "residual" in want else None, dweight, dbias)
