"""Products with an epilogue, their gradients, and tokens sorted by expert.

The ``gemm_*`` functions forward to the entry points of the same name
(include/dense_fp32_tiled.h).  ``linear``, ``grouped_linear``, their
``*_grad`` and the ``expert_*`` functions take torch tensors; like ``matmul``
they check types, layouts, shapes and devices before anything is launched,
enqueue on ``stream`` (a torch.cuda.Stream or raw handle) or torch's current
stream of the tensors' device, and raise GemmError on a non-zero status.  What
they allocate (results, workspaces) is allocated on the stream they run on.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import dense_fp32_tiled_amd as dft

ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)
ACT_NAMES = {ACT_NONE: "none", ACT_RELU: "relu", ACT_GELU: "gelu", ACT_GELU_TANH: "gelu_tanh", ACT_SILU: "silu"}
OUTPUT_SAME, OUTPUT_F32 = 0, 1
LINEAR_AUTO, LINEAR_256x256, LINEAR_128x128, LINEAR_64x64, LINEAR_32x128 = range(5)
LINEAR_COUNT = 5
LINEAR_NAMES = {LINEAR_AUTO: "auto", LINEAR_256x256: "256x256", LINEAR_128x128: "128x128", LINEAR_64x64: "64x64",
                LINEAR_32x128: "32x128"}

_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class LinearArgs(ctypes.Structure):
    """gemm_linear_args."""
    _fields_ = [("input_type", _i32), ("output_type", _i32), ("activation", _i32), ("variant", _i32),
                ("splits", _i32), ("groups", _i32), ("M", _i64), ("N", _i64), ("K", _i64), ("A", _vp), ("lda", _i64),
                ("B", _vp), ("ldb", _i64), ("b_stride", _i64), ("bias", _vp), ("bias_stride", _i64),
                ("offsets", _vp), ("residual", _vp), ("ldr", _i64), ("preact", _vp), ("ldp", _i64), ("D", _vp),
                ("ldd", _i64), ("workspace", _vp), ("workspace_bytes", _i64)]


class LinearGradArgs(ctypes.Structure):
    """gemm_linear_grad_args."""
    _fields_ = [("input_type", _i32), ("activation", _i32), ("a_grad_type", _i32), ("b_grad_type", _i32),
                ("groups", _i32), ("M", _i64), ("N", _i64), ("K", _i64), ("offsets", _vp), ("dY", _vp), ("ldy", _i64),
                ("Z", _vp), ("ldz", _i64), ("A", _vp), ("lda", _i64), ("B", _vp), ("ldb", _i64), ("b_stride", _i64),
                ("dZ", _vp), ("lddz", _i64), ("dA", _vp), ("ldda", _i64), ("dB", _vp), ("lddb", _i64),
                ("db_stride", _i64), ("dbias", _vp), ("workspace", _vp), ("workspace_bytes", _i64)]


class LinearGrads(NamedTuple):
    """Gradients of a, b, bias and of the pre-activation; None where not wanted."""
    a: object
    b: object
    bias: object
    preact: object


def declare(lib) -> None:
    """Argument and result types of this module's entry points."""
    i, p_args, p_grad, p_i32 = ctypes.c_int, ctypes.POINTER(LinearArgs), ctypes.POINTER(LinearGradArgs), ctypes.POINTER(_i32)
    for name, result, types in (
            ("gemm_linear", i, [p_args, _vp]),
            ("gemm_linear_workspace_bytes", _i64, [p_args, _i32]),
            ("gemm_linear_choice", i, [p_args, _i32, p_i32, p_i32]),
            ("gemm_linear_grad", i, [p_grad, _vp]),
            ("gemm_linear_grad_workspace_bytes", _i64, [p_grad, _i32]),
            ("gemm_expert_sort", i, [_i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i64, _vp]),
            ("gemm_expert_sort_workspace_bytes", _i64, [_i64, _i32, _i32]),
            ("gemm_expert_gather", i, [i, _i64, _i64, _i32, _i64, _vp, _i64, _vp, _vp, _i64, _vp]),
            ("gemm_expert_combine", i, [i, _i64, _i64, _i32, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp]),
            ("gemm_expert_combine_grad", i, [i, _i64, _i64, _i32, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64,
                                             _vp, _vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = result, types


# ---- entry points, same names as the C ABI ----------------------------------------------
def gemm_linear(args: LinearArgs, stream=None) -> int:
    return dft.library().gemm_linear(args, stream)


def gemm_linear_workspace_bytes(args: LinearArgs, num_cus: int) -> int:
    return dft.library().gemm_linear_workspace_bytes(args, num_cus)


def gemm_linear_choice(args: LinearArgs, num_cus: int):
    """(status, variant, splits)."""
    v, s = _i32(-1), _i32(-1)
    st = dft.library().gemm_linear_choice(args, num_cus, ctypes.byref(v), ctypes.byref(s))
    return st, v.value, s.value


def gemm_linear_grad(args: LinearGradArgs, stream=None) -> int:
    return dft.library().gemm_linear_grad(args, stream)


def gemm_linear_grad_workspace_bytes(args: LinearGradArgs, num_cus: int) -> int:
    return dft.library().gemm_linear_grad_workspace_bytes(args, num_cus)


def gemm_expert_sort(tokens, top_k, num_experts, experts, offsets, order, position, workspace=None,
                     workspace_bytes=0, stream=None) -> int:
    return dft.library().gemm_expert_sort(tokens, top_k, num_experts, experts, offsets, order, position, workspace,
                                          workspace_bytes, stream)


def gemm_expert_sort_workspace_bytes(tokens: int, top_k: int, num_experts: int) -> int:
    return dft.library().gemm_expert_sort_workspace_bytes(tokens, top_k, num_experts)


def gemm_expert_gather(input_type, tokens, rows, top_k, cols, X, ldx, position, sorted_rows, lds, stream=None) -> int:
    return dft.library().gemm_expert_gather(input_type, tokens, rows, top_k, cols, X, ldx, position, sorted_rows, lds,
                                            stream)


def gemm_expert_combine(input_type, tokens, rows, top_k, cols, Y, ldy, position, weights, out, ldo,
                        stream=None) -> int:
    return dft.library().gemm_expert_combine(input_type, tokens, rows, top_k, cols, Y, ldy, position, weights, out,
                                             ldo, stream)


def gemm_expert_combine_grad(input_type, tokens, rows, top_k, cols, dout, ldd, Y, ldy, position, weights, dY, lddy,
                             dweights, stream=None) -> int:
    return dft.library().gemm_expert_combine_grad(input_type, tokens, rows, top_k, cols, dout, ldd, Y, ldy, position,
                                                  weights, dY, lddy, dweights, stream)


# ---- torch convenience --------------------------------------------------------------------
# A single token's layer takes a few microseconds on the GPU, so what a call costs here counts: torch is bound on
# first use (the package works without it), and every tensor is looked at once.
_ACT_CODES = {name: code for code, name in ACT_NAMES.items()}
_cus: dict[int, int] = {}
torch = None
_Tensor: type = type(None)
_bf16 = _f16 = _f32 = _int32 = None


def _bind():
    global torch, _Tensor, _bf16, _f16, _f32, _int32
    import torch as torch_

    _Tensor, _bf16, _f16, _f32, _int32 = torch_.Tensor, torch_.bfloat16, torch_.float16, torch_.float32, torch_.int32
    torch = torch_


def _num_cus(device) -> int:
    n = _cus.get(device.index)
    if n is None:
        n = _cus[device.index] = torch.cuda.get_device_properties(device).multi_processor_count
    return n


def _input_type(t, name):
    if torch is None:
        _bind()
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype = t.dtype
    if dtype is _bf16:
        return dft.INPUT_BF16
    if dtype is _f16:
        return dft.INPUT_F16
    raise TypeError(f"{name} must be bfloat16 or float16, not {dtype}")


def _act_code(activation):
    code = _ACT_CODES.get(activation)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(_ACT_CODES)}, not {activation!r}")
    return code


def _bad(t, name, dims, dtype, device):
    """What is wrong with a tensor that is not of these dimensions, type and device."""
    if not isinstance(t, _Tensor):
        return TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype or (dims is not None and t.dim() != dims):
        return TypeError(f"{name} must be a {f'{dims}-D ' if dims else ''}{dtype} tensor")
    return ValueError(f"{name} is on {t.device}, expected {device}")


def _matrix(t, name, rows, cols, dtype, device):
    """(device pointer, row pitch) of a rows x cols tensor of that type and device, rows laid out one after another."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.dim() != 2 or t.device != device:
        raise _bad(t, name, 2, dtype, device)
    if t.shape != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if ld < cols or cols == 0 or rows <= 1:
        if rows > 1 and cols > 0:
            raise ValueError(f"{name} has overlapping rows (row stride {ld} < {cols} columns)")
        ld = cols if cols > 1 else 1
    return t.data_ptr(), ld


def _stack(t, name, count, rows, cols, dtype, device):
    """(device pointer, row pitch, elements between matrices) of a count x rows x cols tensor."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.dim() != 3 or t.device != device:
        raise _bad(t, name, 3, dtype, device)
    if t.shape != (count, rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(count, rows, cols)}")
    outer, ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if ld < cols or cols == 0 or rows <= 1:
        if rows > 1 and cols > 0:
            raise ValueError(f"{name} has overlapping rows (row stride {ld} < {cols} columns)")
        ld = cols if cols > 1 else 1
    span = (rows - 1) * ld + cols if rows > 0 else 0
    if count > 1 and outer < span:
        raise ValueError(f"{name} has overlapping matrices (stride {outer} < {span} elements)")
    return t.data_ptr(), ld, outer if count > 1 else max(span, 1)


def _list(t, name, shape, dtype, device):
    """Device pointer of a packed tensor."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.device != device:
        raise _bad(t, name, None, dtype, device)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _gpu(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    return t.device


def _current(stream, device):
    """A context with `stream` torch's current one.  The whole call runs inside it, so that a workspace's memory goes
    back to that stream's pool: from another stream's it could be handed out again while the call's work is queued."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    return torch.cuda.stream(stream)


def _run(entry, what, device, *args):
    """One entry point on the tensors' device, on torch's current stream of it."""
    index = device.index
    handle = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        st = entry(*args, handle)
    else:
        with torch.cuda.device(device):
            st = entry(*args, handle)
    if st != dft.GEMM_OK:
        raise dft.GemmError(st, what)


def _workspace(args, need, what, given, device):
    if need < 0:
        raise dft.GemmError(int(need), what)
    if given is None and need > 0:
        given = torch.empty(need, dtype=torch.uint8, device=device)
    if given is not None:
        if given.device != device:
            raise ValueError(f"workspace is on {given.device}, expected {device}")
        if not given.is_contiguous():
            raise ValueError("workspace must be contiguous")
        args.workspace, args.workspace_bytes = given.data_ptr(), given.numel() * given.element_size()
    return given  # (kept alive by the caller until the launch)


def _linear(a, b, offsets, bias, residual, activation, out, out_dtype, preact, workspace, stream, variant, splits):
    dtype, kind = getattr(a, "dtype", None), _input_type(a, "a")
    device = _gpu(a, "a")
    if stream is not None:
        with _current(stream, device):
            return _linear(a, b, offsets, bias, residual, activation, out, out_dtype, preact, workspace, None,
                           variant, splits)
    grouped = offsets is not None
    if a.dim() != 2 or not isinstance(b, _Tensor) or b.dim() != 2 + grouped:
        raise TypeError(f"a must be a 2-D tensor and b a {2 + grouped}-D one")
    M, K = a.shape
    N = b.shape[-1]
    g = LinearArgs(input_type=kind, activation=_act_code(activation), variant=variant, splits=splits, M=M, N=N, K=K)
    g.A, g.lda = _matrix(a, "a", M, K, dtype, device)
    if grouped:
        groups = b.shape[0]
        if groups < 1:
            raise ValueError("b must have at least one matrix")
        g.groups = groups
        g.B, g.ldb, g.b_stride = _stack(b, "b", groups, K, N, dtype, device)
        g.offsets = _list(offsets, "offsets", (groups + 1,), _int32, device)
        if bias is not None:
            g.bias, g.bias_stride = _matrix(bias, "bias", groups, N, dtype, device)
    else:
        g.B, g.ldb = _matrix(b, "b", K, N, dtype, device)
        if bias is not None:
            g.bias = _list(bias, "bias", (N,), dtype, device)
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype or dtype, device=device)
    elif out_dtype is not None and getattr(out, "dtype", None) is not out_dtype:
        raise TypeError(f"out must be a 2-D {out_dtype} tensor")
    out_type = getattr(out, "dtype", None)
    if out_type is _f32:
        g.output_type = OUTPUT_F32
    elif out_type is not dtype:
        raise TypeError(f"out must be {dtype} or torch.float32")
    g.D, g.ldd = _matrix(out, "out", M, N, out_type, device)
    if residual is not None:
        g.residual, g.ldr = _matrix(residual, "residual", M, N, out_type, device)
    if preact is not None:
        g.preact, g.ldp = _matrix(preact, "preact", M, N, dtype, device)
    lib = dft.library()
    keep = _workspace(g, lib.gemm_linear_workspace_bytes(g, _num_cus(device)), "gemm_linear_workspace_bytes",
                      workspace, device)
    _run(lib.gemm_linear, "gemm_linear", device, g)
    del keep
    return out


def linear(a, b, bias=None, residual=None, activation="none", out=None, out_dtype=None, preact=None, workspace=None,
           stream=None, variant: int = LINEAR_AUTO, splits: int = 0):
    """act(a @ b + bias) + residual, by gemm_linear.

    a: M x K and b: K x N, both bfloat16 or both float16; bias: N values of that type; residual: M x N of the
    output's type (``out`` itself may be given).  The output is of the inputs' type, or ``out_dtype`` torch.float32,
    or ``out``.  ``preact`` (M x N of the inputs' type) receives a @ b + bias, which linear_grad reads.
    activation: "none", "relu", "gelu", "gelu_tanh" or "silu"."""
    return _linear(a, b, None, bias, residual, activation, out, out_dtype, preact, workspace, stream, variant, splits)


def grouped_linear(a, b, offsets, bias=None, residual=None, activation="none", out=None, out_dtype=None, preact=None,
                   workspace=None, stream=None, variant: int = LINEAR_AUTO):
    """``linear`` with one b (G x K x N) and bias (G x N) per group: rows [offsets[g], offsets[g + 1]) of a (offsets:
    G + 1 int32 on the device, as expert_sort gives them).  Rows in no group are left as they were."""
    if offsets is None:
        raise TypeError("offsets must be a torch.Tensor")
    return _linear(a, b, offsets, bias, residual, activation, out, out_dtype, preact, workspace, stream, variant, 1)


def _linear_grad(dy, a, b, offsets, preact, activation, want, a_dtype, b_dtype, workspace, stream):
    dtype, kind = getattr(a, "dtype", None), _input_type(a, "a")
    device = _gpu(a, "a")
    if stream is not None:
        with _current(stream, device):
            return _linear_grad(dy, a, b, offsets, preact, activation, want, a_dtype, b_dtype, workspace, None)
    grouped = offsets is not None
    if a.dim() != 2 or not isinstance(b, _Tensor) or b.dim() != 2 + grouped:
        raise TypeError(f"a must be a 2-D tensor and b a {2 + grouped}-D one")
    want = frozenset(want)
    if not want <= {"a", "b", "bias"}:
        raise ValueError(f"want names 'a', 'b' and 'bias', not {sorted(want - {'a', 'b', 'bias'})}")
    M, K = a.shape
    N = b.shape[-1]
    act = _act_code(activation)
    g = LinearGradArgs(input_type=kind, activation=act, M=M, N=N, K=K)
    g.A, g.lda = _matrix(a, "a", M, K, dtype, device)
    g.dY, g.ldy = _matrix(dy, "dy", M, N, dtype, device)
    groups = 1
    if grouped:
        groups = b.shape[0]
        if groups < 1:
            raise ValueError("b must have at least one matrix")
        g.groups = groups
        g.B, g.ldb, g.b_stride = _stack(b, "b", groups, K, N, dtype, device)
        g.offsets = _list(offsets, "offsets", (groups + 1,), _int32, device)
    else:
        g.B, g.ldb = _matrix(b, "b", K, N, dtype, device)
    types = {None: (dtype, OUTPUT_SAME), dtype: (dtype, OUTPUT_SAME), torch.float32: (torch.float32, OUTPUT_F32)}
    if a_dtype not in types or b_dtype not in types:
        raise TypeError(f"gradients are {dtype} or torch.float32")
    da = db = dbias = None
    dz = dy
    if act != ACT_NONE:
        if preact is None:
            raise ValueError(f"the gradient of {activation} needs preact")
        g.Z, g.ldz = _matrix(preact, "preact", M, N, dtype, device)
        dz = torch.empty(M, N, dtype=dtype, device=device)
        g.dZ, g.lddz = dz.data_ptr(), max(N, 1)
    if "a" in want:
        da = torch.empty(M, K, dtype=types[a_dtype][0], device=device)
        g.dA, g.ldda, g.a_grad_type = da.data_ptr(), max(K, 1), types[a_dtype][1]
    if "b" in want:
        db = torch.empty(b.shape, dtype=types[b_dtype][0], device=device)
        g.dB, g.lddb, g.db_stride, g.b_grad_type = db.data_ptr(), max(N, 1), max(K * N, 1), types[b_dtype][1]
    if "bias" in want:
        dbias = torch.empty((groups, N) if grouped else (N,), dtype=torch.float32, device=device)
        g.dbias = dbias.data_ptr()
    lib = dft.library()
    keep = _workspace(g, lib.gemm_linear_grad_workspace_bytes(g, _num_cus(device)),
                      "gemm_linear_grad_workspace_bytes", workspace, device)
    _run(lib.gemm_linear_grad, "gemm_linear_grad", device, g)
    del keep
    return LinearGrads(da, db, dbias, dz)


def linear_grad(dy, a, b, preact=None, activation="none", want=("a", "b", "bias"), a_dtype=None, b_dtype=None,
                workspace=None, stream=None) -> LinearGrads:
    """Gradients of ``linear`` for the output's gradient dy (M x N, the inputs' type), by gemm_linear_grad:
    preact's dz = dy * act'(preact), a's dz @ b^T, b's a^T @ dz (each of the inputs' type, or ``a_dtype`` /
    ``b_dtype`` torch.float32) and bias's column sums (float32).  ``want`` names the ones computed.  The residual's
    gradient is dy itself, and so is preact's without an activation."""
    return _linear_grad(dy, a, b, None, preact, activation, want, a_dtype, b_dtype, workspace, stream)


def grouped_linear_grad(dy, a, b, offsets, preact=None, activation="none", want=("a", "b", "bias"), a_dtype=None,
                        b_dtype=None, workspace=None, stream=None) -> LinearGrads:
    """Gradients of ``grouped_linear``: b's is G x K x N and bias's G x N (zero for a group without rows); rows in
    no group are left as they were (unset, as they are allocated here)."""
    if offsets is None:
        raise TypeError("offsets must be a torch.Tensor")
    return _linear_grad(dy, a, b, offsets, preact, activation, want, a_dtype, b_dtype, workspace, stream)


def expert_sort(experts, num_experts: int, stream=None):
    """Sorts (token, choice) pairs by expert, by gemm_expert_sort.  experts: tokens x top_k int32; a value outside
    [0, num_experts) drops its pair.  Returns int32 tensors: offsets (num_experts + 1), order (tokens * top_k) and
    position (tokens x top_k)."""
    if torch is None:
        _bind()
    if not isinstance(experts, _Tensor) or experts.dim() != 2:
        raise TypeError("experts must be a 2-D torch.int32 tensor")
    device = _gpu(experts, "experts")
    if stream is not None:
        with _current(stream, device):
            return expert_sort(experts, num_experts)
    tokens, top_k = experts.shape
    src = _list(experts, "experts", (tokens, top_k), _int32, device)
    need = gemm_expert_sort_workspace_bytes(tokens, top_k, num_experts)
    if need < 0:
        raise dft.GemmError(need, "gemm_expert_sort")
    pairs = tokens * top_k
    offsets = torch.empty(num_experts + 1, dtype=_int32, device=device)
    order = torch.empty(pairs, dtype=_int32, device=device)
    position = torch.empty(tokens, top_k, dtype=_int32, device=device)
    space = torch.empty(need // 4, dtype=_int32, device=device) if need else None
    _run(dft.library().gemm_expert_sort, "gemm_expert_sort", device, tokens, top_k, num_experts, src,
         offsets.data_ptr(), order.data_ptr(), position.data_ptr(), space.data_ptr() if need else None, need)
    return offsets, order, position


def _positions(position, device):
    if not isinstance(position, _Tensor) or position.dim() != 2:
        raise TypeError("position must be a 2-D torch.int32 tensor")
    tokens, top_k = position.shape
    return tokens, top_k, _list(position, "position", (tokens, top_k), _int32, device)


def expert_gather(x, position, out=None, stream=None):
    """The tokens' rows in expert order, by gemm_expert_gather: row position[t, j] of the result is x[t].  The
    result has tokens * top_k rows (or ``out``'s); rows that no pair has are left as they were."""
    kind, device = _input_type(x, "x"), _gpu(x, "x")
    if stream is not None:
        with _current(stream, device):
            return expert_gather(x, position, out)
    tokens, top_k, pos = _positions(position, device)
    cols = x.shape[-1] if x.dim() == 2 else -1
    px, ldx = _matrix(x, "x", tokens, cols, x.dtype, device)
    if out is None:
        out = torch.empty(tokens * top_k, cols, dtype=x.dtype, device=device)
    rows = out.shape[0] if isinstance(out, _Tensor) and out.dim() == 2 else -1
    po, ldo = _matrix(out, "out", rows, cols, x.dtype, device)
    _run(dft.library().gemm_expert_gather, "gemm_expert_gather", device, kind, tokens, rows, top_k, cols, px,
         ldx, pos, po, ldo)
    return out


def expert_combine(y, position, weights=None, out=None, stream=None):
    """The experts' rows back in token order, by gemm_expert_combine: result[t] = sum over j of weights[t, j] *
    y[position[t, j]] (weights: tokens x top_k float32, or None for ones: the gradient of expert_gather)."""
    kind, device = _input_type(y, "y"), _gpu(y, "y")
    if stream is not None:
        with _current(stream, device):
            return expert_combine(y, position, weights, out)
    tokens, top_k, pos = _positions(position, device)
    rows, cols = y.shape if y.dim() == 2 else (-1, -1)
    py, ldy = _matrix(y, "y", rows, cols, y.dtype, device)
    pw = None if weights is None else _list(weights, "weights", (tokens, top_k), _f32, device)
    if out is None:
        out = torch.empty(tokens, cols, dtype=y.dtype, device=device)
    po, ldo = _matrix(out, "out", tokens, cols, y.dtype, device)
    _run(dft.library().gemm_expert_combine, "gemm_expert_combine", device, kind, tokens, rows, top_k, cols,
         py, ldy, pos, pw, po, ldo)
    return out


def expert_combine_grad(dout, y, position, weights=None, dy=None, stream=None):
    """Gradients of expert_combine, by gemm_expert_combine_grad: (dy, dweights) with dy[position[t, j]] = weights[t,
    j] * dout[t] and dweights[t, j] = y[position[t, j]] . dout[t] (float32; None without weights).  Rows of dy that
    no pair has are left as they were."""
    kind, device = _input_type(y, "y"), _gpu(y, "y")
    if stream is not None:
        with _current(stream, device):
            return expert_combine_grad(dout, y, position, weights, dy)
    tokens, top_k, pos = _positions(position, device)
    rows, cols = y.shape if y.dim() == 2 else (-1, -1)
    py, ldy = _matrix(y, "y", rows, cols, y.dtype, device)
    pd, ldd = _matrix(dout, "dout", tokens, cols, y.dtype, device)
    pw = pdw = dweights = None
    if weights is not None:
        pw = _list(weights, "weights", (tokens, top_k), _f32, device)
        dweights = torch.empty(tokens, top_k, dtype=torch.float32, device=device)
        pdw = dweights.data_ptr()
    if dy is None:
        dy = torch.empty(rows, cols, dtype=y.dtype, device=device)
    pdy, lddy = _matrix(dy, "dy", rows, cols, y.dtype, device)
    _run(dft.library().gemm_expert_combine_grad, "gemm_expert_combine_grad", device, kind, tokens, rows,
         top_k, cols, pd, ldd, py, ldy, pos, pw, pdy, lddy, pdw)
    return dy, dweights


# ---- a routed layer ---------------------------------------------------------------------------
class ExpertState(NamedTuple):
    """What expert_mlp keeps for expert_mlp_grad."""
    offsets: object
    position: object
    rows: object
    preact: object
    hidden: object
    back: object


def expert_mlp(x, experts, weights, w1, w2, b1=None, b2=None, activation="silu", stream=None):
    """A routed two-layer block: each token's top_k experts applied to it and summed with the router's weights,

        out[t] = sum over j of weights[t, j] * (act(x[t] @ w1[e] + b1[e]) @ w2[e] + b2[e]),  e = experts[t, j]

    x: tokens x D; experts: tokens x top_k int32; weights: tokens x top_k float32; w1: E x D x H; w2: E x H x D;
    b1: E x H; b2: E x D.  Returns (out, state); state is what expert_mlp_grad needs."""
    _input_type(x, "x")
    if not isinstance(w1, _Tensor) or w1.dim() != 3:
        raise TypeError("w1 must be a 3-D tensor")
    device = _gpu(x, "x")
    if stream is not None:
        with _current(stream, device):
            return expert_mlp(x, experts, weights, w1, w2, b1, b2, activation)
    offsets, _, position = expert_sort(experts, w1.shape[0])
    rows = expert_gather(x, position)
    preact = None
    if activation != "none":
        preact = torch.empty(rows.shape[0], w1.shape[2], dtype=x.dtype, device=device)
    hidden = grouped_linear(rows, w1, offsets, bias=b1, activation=activation, preact=preact)
    back = grouped_linear(hidden, w2, offsets, bias=b2)
    out = expert_combine(back, position, weights)
    return out, ExpertState(offsets, position, rows, preact, hidden, back)


class ExpertGrads(NamedTuple):
    x: object
    weights: object
    w1: object
    b1: object
    w2: object
    b2: object


def expert_mlp_grad(dout, state: ExpertState, weights, w1, w2, activation="silu", stream=None) -> ExpertGrads:
    """Gradients of expert_mlp for its output's gradient dout (tokens x D); the biases' are float32."""
    _input_type(dout, "dout")
    if stream is not None:
        with _current(stream, _gpu(dout, "dout")):
            return expert_mlp_grad(dout, state, weights, w1, w2, activation)
    dback, dweights = expert_combine_grad(dout, state.back, state.position, weights)
    g2 = grouped_linear_grad(dback, state.hidden, w2, state.offsets)
    g1 = grouped_linear_grad(g2.a, state.rows, w1, state.offsets, preact=state.preact, activation=activation)
    dx = expert_combine(g1.a, state.position)
    return ExpertGrads(dx, dweights, g1.b, g1.bias, g2.b, g2.bias)
