"""The loss after the last product: cross entropy over a vocabulary, with its gradients, the logits never stored.

The ``gemm_*`` functions forward to the entry points of the same name
(include/dense_fp32_tiled.h).  ``linear_cross_entropy`` and its gradient take
torch tensors; they check types, layouts, shapes and devices before anything is
launched, enqueue on ``stream`` or torch's current stream of the tensors'
device, allocate on it, and raise GemmError on a non-zero status, as the layers
of products.py do.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import dense_fp32_tiled_amd as dft

from . import products as pr

TARGET_I32, TARGET_I64 = 0, 1

_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class CrossEntropyArgs(ctypes.Structure):
    """gemm_cross_entropy_args."""
    _fields_ = [("input_type", _i32), ("target_type", _i32), ("b_transposed", _i32), ("variant", _i32), ("M", _i64),
                ("N", _i64), ("K", _i64), ("piece", _i64), ("A", _vp), ("lda", _i64), ("B", _vp), ("ldb", _i64),
                ("targets", _vp), ("loss", _vp), ("lse", _vp), ("workspace", _vp), ("workspace_bytes", _i64)]


class CrossEntropyGradArgs(ctypes.Structure):
    """gemm_cross_entropy_grad_args."""
    _fields_ = [("input_type", _i32), ("target_type", _i32), ("b_transposed", _i32), ("variant", _i32),
                ("a_grad_type", _i32), ("b_grad_type", _i32), ("M", _i64), ("N", _i64), ("K", _i64), ("piece", _i64),
                ("A", _vp), ("lda", _i64), ("B", _vp), ("ldb", _i64), ("targets", _vp), ("lse", _vp), ("dloss", _vp),
                ("dA", _vp), ("ldda", _i64), ("dB", _vp), ("lddb", _i64), ("workspace", _vp),
                ("workspace_bytes", _i64)]


class CrossEntropyGrads(NamedTuple):
    """Gradients of a and b; None where not wanted."""
    a: object
    b: object


def declare(lib) -> None:
    """Argument and result types of this module's entry points."""
    i, fwd, grad = ctypes.c_int, ctypes.POINTER(CrossEntropyArgs), ctypes.POINTER(CrossEntropyGradArgs)
    for name, result, types in (("gemm_cross_entropy", i, [fwd, _vp]),
                                ("gemm_cross_entropy_workspace_bytes", _i64, [fwd, _i32]),
                                ("gemm_cross_entropy_grad", i, [grad, _vp]),
                                ("gemm_cross_entropy_grad_workspace_bytes", _i64, [grad, _i32])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = result, types


# ---- entry points, same names as the C ABI ----------------------------------------------
def gemm_cross_entropy(args: CrossEntropyArgs, stream=None) -> int:
    return dft.library().gemm_cross_entropy(args, stream)


def gemm_cross_entropy_workspace_bytes(args: CrossEntropyArgs, num_cus: int) -> int:
    return dft.library().gemm_cross_entropy_workspace_bytes(args, num_cus)


def gemm_cross_entropy_grad(args: CrossEntropyGradArgs, stream=None) -> int:
    return dft.library().gemm_cross_entropy_grad(args, stream)


def gemm_cross_entropy_grad_workspace_bytes(args: CrossEntropyGradArgs, num_cus: int) -> int:
    return dft.library().gemm_cross_entropy_grad_workspace_bytes(args, num_cus)


# ---- torch convenience --------------------------------------------------------------------
def _operands(g, a, b, targets, device):
    """Fills in what both passes read; whether b lies a word per row."""
    if a.dim() != 2 or not isinstance(b, pr._Tensor) or b.dim() != 2:
        raise TypeError("a and b must be 2-D tensors")
    dtype = a.dtype
    M, K = a.shape
    N = b.shape[1]
    g.M, g.N, g.K = M, N, K
    g.A, g.lda = pr._matrix(a, "a", M, K, dtype, device)
    transposed = N > 1 and b.stride(1) != 1 and b.stride(0) == 1
    g.b_transposed = transposed
    if transposed:
        g.B, g.ldb = pr._matrix(b.t(), "b.t()", N, K, dtype, device)
    else:
        g.B, g.ldb = pr._matrix(b, "b", K, N, dtype, device)
    if targets is not None:
        wide = getattr(targets, "dtype", None) is pr.torch.int64
        g.target_type = TARGET_I64 if wide else TARGET_I32
        g.targets = pr._list(targets, "targets", (M,), pr.torch.int64 if wide else pr._int32, device)
    return transposed


def linear_cross_entropy(a, b, targets=None, piece: int = 0, workspace=None, stream=None,
                         variant: int = pr.LINEAR_AUTO):
    """(loss, lse), each of a's rows in float32, by gemm_cross_entropy: the cross entropy of softmax(a @ b) with each
    row's target, and the logarithm of the row's sum of exponentials, which the gradient reads.

    a: M x K and b: K x N, both bfloat16 or both float16; b may be the transpose of an N x K matrix (``embedding.t()``).
    targets: M int32 or int64; one outside [0, N) is none, and its loss zero.  Without targets loss is None.  The
    mean over the tokens that count is ``loss.sum() / count``, its gradient's ``dloss`` 1 / count.  ``piece``: words
    at a time (a multiple of 256), which bounds the workspace."""
    kind, device = pr._input_type(a, "a"), pr._gpu(a, "a")
    if stream is not None:
        with pr._current(stream, device):
            return linear_cross_entropy(a, b, targets, piece, workspace, None, variant)
    g = CrossEntropyArgs(input_type=kind, variant=variant, piece=piece)
    _operands(g, a, b, targets, device)
    empty = pr.torch.empty
    lse = empty(g.M, dtype=pr._f32, device=device)
    g.lse = lse.data_ptr()
    loss = None
    if targets is not None:
        loss = empty(g.M, dtype=pr._f32, device=device)
        g.loss = loss.data_ptr()
    lib = dft.library()
    keep = pr._workspace(g, lib.gemm_cross_entropy_workspace_bytes(g, pr._num_cus(device)),
                         "gemm_cross_entropy_workspace_bytes", workspace, device)
    pr._run(lib.gemm_cross_entropy, "gemm_cross_entropy", device, g)
    del keep
    return loss, lse


def linear_cross_entropy_grad(dloss, a, b, targets, lse, want=("a", "b"), a_dtype=None, b_dtype=None, piece: int = 0,
                              workspace=None, stream=None, variant: int = pr.LINEAR_AUTO) -> CrossEntropyGrads:
    """Gradients of ``linear_cross_entropy`` for the loss's gradient dloss (M float32), by gemm_cross_entropy_grad:
    with dz = (softmax(a @ b) - onehot(targets)) * dloss, a's dz @ b^T and b's a^T @ dz, each of the inputs' type or
    ``a_dtype`` / ``b_dtype`` torch.float32; b's lies as b does.  lse is the forward pass's.  ``want`` names the ones
    computed."""
    kind, device = pr._input_type(a, "a"), pr._gpu(a, "a")
    if stream is not None:
        with pr._current(stream, device):
            return linear_cross_entropy_grad(dloss, a, b, targets, lse, want, a_dtype, b_dtype, piece, workspace,
                                             None, variant)
    want = frozenset(want)
    if not want <= {"a", "b"}:
        raise ValueError(f"want names 'a' and 'b', not {sorted(want - {'a', 'b'})}")
    if targets is None:
        raise TypeError("targets must be a torch.Tensor")
    g = CrossEntropyGradArgs(input_type=kind, variant=variant, piece=piece)
    transposed = _operands(g, a, b, targets, device)
    M, N, K = g.M, g.N, g.K
    g.lse = pr._list(lse, "lse", (M,), pr._f32, device)
    g.dloss = pr._list(dloss, "dloss", (M,), pr._f32, device)
    dtype, empty = a.dtype, pr.torch.empty
    types = {None: (dtype, pr.OUTPUT_SAME), dtype: (dtype, pr.OUTPUT_SAME), pr._f32: (pr._f32, pr.OUTPUT_F32)}
    if a_dtype not in types or b_dtype not in types:
        raise TypeError(f"gradients are {dtype} or torch.float32")
    da = db = None
    if "a" in want:
        da = empty(M, K, dtype=types[a_dtype][0], device=device)
        g.dA, g.ldda, g.a_grad_type = da.data_ptr(), max(K, 1), types[a_dtype][1]
    if "b" in want:
        db = empty((N, K) if transposed else (K, N), dtype=types[b_dtype][0], device=device)
        g.dB, g.lddb, g.b_grad_type = db.data_ptr(), max(db.shape[1], 1), types[b_dtype][1]
        if transposed:
            db = db.t()
    lib = dft.library()
    keep = pr._workspace(g, lib.gemm_cross_entropy_grad_workspace_bytes(g, pr._num_cus(device)),
                         "gemm_cross_entropy_grad_workspace_bytes", workspace, device)
    pr._run(lib.gemm_cross_entropy_grad, "gemm_cross_entropy_grad", device, g)
    del keep
    return CrossEntropyGrads(da, db)
