"""The products with an epilogue and their gradients in float64 on the CPU,
with elementwise error bounds for the GPU's results, and buffers that show a
read or write outside a matrix.

Bounds.  u = 2^-24 is fp32's largest relative rounding error.  A sum of L
products (exact in fp32) in any order is off by at most L * 2u * sum |a b|
(2u: the matrix cores may round each step less tightly than to nearest, but
by less than one step).  Activations have slopes of at most 1.13, so an error
dz of z moves them by at most 1.2 dz; their own evaluation is off by at most
16u |z| (a few roundings of values no larger than |z|, and the library's erf
and exp).  Slopes are at most 1.13 and off by at most 16u * (1 + |z|).  Each
rounding to an output type t adds finfo(t).eps / 2 relative, or half of its
smallest step.
"""

from __future__ import annotations

import math

import torch

import dense_fp32_tiled_amd as dft

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
KINDS = {torch.bfloat16: dft.INPUT_BF16, torch.float16: dft.INPUT_F16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
SMALLEST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half a step at 0


def half_step(x: torch.Tensor, dtype) -> torch.Tensor:
    return x.abs() * (torch.finfo(dtype).eps / 2) + SMALLEST[dtype]


def act(z: torch.Tensor, kind: str) -> torch.Tensor:
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z.clone()


def slope(z: torch.Tensor, kind: str) -> torch.Tensor:
    if kind == "relu":
        return (z > 0).double()
    if kind == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if kind == "silu":
        g = torch.sigmoid(z)
        return g + z * g * (1 - g)
    return torch.ones_like(z)


def ranges(offsets, groups: int, rows: int):
    """(group, lo, hi) of the documented reading of offsets; one matrix: all rows."""
    if offsets is None:
        return [(0, 0, rows)]
    out = []
    for g in range(groups):
        lo = min(max(int(offsets[g]), 0), rows)
        out.append((g, lo, min(max(int(offsets[g + 1]), lo), rows)))
    return out


def forward(a, b, offsets=None, bias=None, residual=None, kind="none", out_dtype=None):
    """((D, its bound), (Z rounded, its bound)) in float64; b: G x K x N, bias: G x N.  Rows in no group are NaN."""
    dtype = a.dtype
    out_dtype = out_dtype or dtype
    A, B = a.double(), b.double()
    M, K, N = a.shape[0], a.shape[1], b.shape[2]
    d, d_tol = torch.full((M, N), math.nan, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    z_out, z_tol = d.clone(), d_tol.clone()
    for g, lo, hi in ranges(offsets, b.shape[0], M):
        z = A[lo:hi] @ B[g]
        size = A[lo:hi].abs() @ B[g].abs()
        if bias is not None:
            z, size = z + bias[g].double(), size + bias[g].double().abs()
        dz = (K + 2) * 2 * U * size
        y = act(z, kind)
        dy = 1.2 * dz + (16 * U * z.abs() if kind != "none" else 0)
        if residual is not None:
            y = y + residual[lo:hi].double()
            dy = dy + 2 * U * (y.abs() + residual[lo:hi].double().abs())
        d[lo:hi], d_tol[lo:hi] = y, dy + half_step(y.abs() + dy, out_dtype)
        z_out[lo:hi], z_tol[lo:hi] = z, dz + half_step(z.abs() + dz, dtype)
    return (d, d_tol), (z_out, z_tol)


def grad(dy, a, b, offsets=None, preact=None, kind="none", a_dtype=None, b_dtype=None):
    """{name: (value, bound)} of dz, a, b and bias in float64; b: G x K x N.  Rows in no group are NaN."""
    dtype = a.dtype
    A, B, DY = a.double(), b.double(), dy.double()
    G, K, N = b.shape
    M = a.shape[0]
    nan = math.nan
    dz, dz_tol = torch.full((M, N), nan, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    da, da_tol = torch.full((M, K), nan, dtype=torch.float64), torch.zeros(M, K, dtype=torch.float64)
    db, db_tol = torch.zeros(G, K, N, dtype=torch.float64), torch.zeros(G, K, N, dtype=torch.float64)
    dbias, dbias_tol = torch.zeros(G, N, dtype=torch.float64), torch.zeros(G, N, dtype=torch.float64)
    for g, lo, hi in ranges(offsets, G, M):
        s, off = DY[lo:hi], torch.zeros(hi - lo, N, dtype=torch.float64)
        if kind != "none":
            z = preact[lo:hi].double()
            s = s * slope(z, kind)
            off = DY[lo:hi].abs() * 16 * U * (1 + z.abs()) + 2 * U * s.abs()
        dz[lo:hi] = s
        rounded = off + (half_step(s.abs() + off, dtype) if kind != "none" else 0)
        dz_tol[lo:hi] = rounded
        big = s.abs() + rounded
        da[lo:hi] = s @ B[g].t()
        t = rounded @ B[g].abs().t() + (N + 2) * 2 * U * (big @ B[g].abs().t())
        da_tol[lo:hi] = t + half_step(da[lo:hi].abs() + t, a_dtype or dtype)
        db[g] = A[lo:hi].t() @ s
        t = A[lo:hi].abs().t() @ rounded + (M + 2) * 2 * U * (A[lo:hi].abs().t() @ big)
        db_tol[g] = t + half_step(db[g].abs() + t, b_dtype or dtype)
        dbias[g] = s.sum(0)
        dbias_tol[g] = off.sum(0) + (M + 2) * 2 * U * (s.abs() + off).sum(0) + SMALLEST[torch.float32]
    return {"dz": (dz, dz_tol), "a": (da, da_tol), "b": (db, db_tol), "bias": (dbias, dbias_tol)}


def assert_within(got: torch.Tensor, want, what):
    value, tol = want
    known = ~torch.isnan(value)
    off = (got.double().cpu() - value).abs()
    bad = known & ~(off <= tol)
    if bool(bad.any()):
        at = bad.nonzero()[0].tolist()
        i = tuple(at)
        raise AssertionError(f"{what}: {int(bad.sum())} of {int(known.sum())} values off, first at {at}: "
                             f"{float(got.double().cpu()[i])} against {float(value[i])} +- {float(tol[i]):.3g}")


class Guarded:
    """A matrix (or stack of them) on the GPU inside a buffer whose every other element is NaN."""

    def __init__(self, value: torch.Tensor, pad: int = 0, offset: int = 0, gap: int = 0, after: int = 16):
        lead = value.shape[:-2]
        rows, cols = value.shape[-2:]
        self.count = lead[0] if lead else 1
        self.shape, self.ld, self.offset = value.shape, max(cols, 1) + pad, offset
        self.stride = max(rows, 1) * self.ld + gap
        self.rows, self.cols = rows, cols
        buf = torch.full((offset + self.count * self.stride + after,), math.nan, dtype=value.dtype)
        self._view(buf).copy_(value.reshape(self.count, rows, cols))
        self.buf = buf.cuda()

    def _view(self, buf):
        return buf.as_strided((self.count, self.rows, self.cols), (self.stride, self.ld, 1), self.offset)

    @property
    def ptr(self):
        return self.buf.data_ptr() + self.offset * self.buf.element_size()

    def value(self):
        return self._view(self.buf.cpu()).reshape(self.shape)

    def assert_rest_untouched(self, what, rows=None):
        """Every element outside the matrix (and outside `rows` of it) is still NaN."""
        buf = self.buf.cpu()
        seen = torch.zeros(buf.shape, dtype=torch.bool)
        view = seen.as_strided((self.count, self.rows, self.cols), (self.stride, self.ld, 1), self.offset)
        if rows is None:
            view[:] = True
        else:
            view[:, rows] = True
        assert bool(torch.isnan(buf[~seen]).all()), f"{what}: a write outside the matrix"


def empty(shape, dtype, **kw):
    return Guarded(torch.full(shape, math.nan, dtype=dtype), **kw)


def workspace(need: int):
    assert need >= 0, need
    return torch.full((need // 4 + 4,), math.nan, dtype=torch.float32, device="cuda") if need else None


def run_forward(lib, a, b, offsets=None, bias=None, residual=None, kind="none", out_dtype=None, keep=False, variant=0,
                splits=0, pad=(0, 0, 0, 0), offset=0, in_place=False):
    """gemm_linear through the C ABI on guarded buffers; b: G x K x N (one matrix when offsets is None)."""
    dtype, (M, K), N = a.dtype, a.shape, b.shape[2]
    out_dtype = out_dtype or dtype
    grouped = offsets is not None
    ga, gb = Guarded(a, pad[0], offset), Guarded(b, pad[1], offset, gap=8 if pad[1] % 8 == 0 else 3)
    gd, gp = empty((M, N), out_dtype, pad=pad[2], offset=offset), empty((M, N), dtype, pad=pad[3], offset=offset)
    g = dft.LinearArgs(input_type=KINDS[dtype], output_type=int(out_dtype == torch.float32),
                       activation=ACTS.index(kind), variant=variant, splits=splits,
                       groups=b.shape[0] if grouped else 0, M=M, N=N, K=K, A=ga.ptr, lda=ga.ld, B=gb.ptr, ldb=gb.ld,
                       b_stride=gb.stride, D=gd.ptr, ldd=gd.ld)
    held = [ga, gb, gd, gp]
    if grouped:
        held.append(torch.tensor(offsets, dtype=torch.int32, device="cuda"))
        g.offsets = held[-1].data_ptr()
    if bias is not None:
        held.append(Guarded(bias, 0, 1))
        g.bias, g.bias_stride = held[-1].ptr, N
    if residual is not None:
        r = gd if in_place else Guarded(residual, pad[2], offset)
        if in_place:
            gd._view(gd.buf).copy_(residual.reshape(1, M, N))
        held.append(r)
        g.residual, g.ldr = r.ptr, r.ld
    if keep:
        g.preact, g.ldp = gp.ptr, gp.ld
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    ws = workspace(lib.gemm_linear_workspace_bytes(g, cus))
    if ws is not None:
        g.workspace, g.workspace_bytes = ws.data_ptr(), ws.numel() * 4
    st = lib.gemm_linear(g, torch.cuda.current_stream().cuda_stream)
    assert st == dft.GEMM_OK, dft.gemm_f32_status_string(st)
    torch.cuda.synchronize()
    rows = None
    if grouped:
        rows = torch.zeros(M, dtype=torch.bool)
        for _, lo, hi in ranges(offsets, b.shape[0], M):
            rows[lo:hi] = True
    gd.assert_rest_untouched("D", None if in_place else rows)
    gp.assert_rest_untouched("Z", rows if keep else torch.zeros(M, dtype=torch.bool))
    return gd.value(), gp.value()


def run_grad(lib, dy, a, b, offsets=None, preact=None, kind="none", a_dtype=None, b_dtype=None,
             want=("a", "b", "bias"), pad=(0, 0, 0, 0), offset=0, in_place=False):
    """gemm_linear_grad through the C ABI on guarded buffers: {name: value}."""
    dtype, (M, K), N, G = a.dtype, a.shape, b.shape[2], b.shape[0]
    a_dtype, b_dtype = a_dtype or dtype, b_dtype or dtype
    grouped = offsets is not None
    ga, gb, gy = Guarded(a, pad[0], offset), Guarded(b, pad[1], offset, gap=8 if pad[1] % 8 == 0 else 3), \
        Guarded(dy, pad[2], offset)
    g = dft.LinearGradArgs(input_type=KINDS[dtype], activation=ACTS.index(kind),
                           a_grad_type=int(a_dtype == torch.float32), b_grad_type=int(b_dtype == torch.float32),
                           groups=G if grouped else 0, M=M, N=N, K=K, dY=gy.ptr, ldy=gy.ld)
    held, out = [ga, gb, gy], {}
    if grouped:
        held.append(torch.tensor(offsets, dtype=torch.int32, device="cuda"))
        g.offsets = held[-1].data_ptr()
    rows = torch.zeros(M, dtype=torch.bool)
    for _, lo, hi in ranges(offsets, G, M):
        rows[lo:hi] = True
    if kind != "none":
        gz = Guarded(preact, pad[2], offset)
        out["dz"] = gy if in_place else empty((M, N), dtype, pad=pad[3], offset=offset)
        held.append(gz)
        g.Z, g.ldz, g.dZ, g.lddz = gz.ptr, gz.ld, out["dz"].ptr, out["dz"].ld
    if "a" in want:
        out["a"] = empty((M, K), a_dtype, pad=pad[0], offset=offset)
        g.B, g.ldb, g.b_stride, g.dA, g.ldda = gb.ptr, gb.ld, gb.stride, out["a"].ptr, out["a"].ld
    if "b" in want:
        out["b"] = empty((G, K, N), b_dtype, pad=pad[1], offset=offset, gap=5)
        g.A, g.lda, g.dB, g.lddb, g.db_stride = ga.ptr, ga.ld, out["b"].ptr, out["b"].ld, out["b"].stride
    if "bias" in want:
        out["bias"] = empty((G, N), torch.float32, pad=0, offset=1)
        g.dbias = out["bias"].ptr
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    ws = workspace(lib.gemm_linear_grad_workspace_bytes(g, cus))
    if ws is not None:
        g.workspace, g.workspace_bytes = ws.data_ptr(), ws.numel() * 4
    st = lib.gemm_linear_grad(g, torch.cuda.current_stream().cuda_stream)
    assert st == dft.GEMM_OK, dft.gemm_f32_status_string(st)
    torch.cuda.synchronize()
    for name, o in out.items():
        o.assert_rest_untouched(name, rows if name == "a" or (name == "dz" and not in_place) else None)
    return {name: o.value() for name, o in out.items()}


def draw(gen, shape, dtype, integer=False, scale=1.0):
    if integer:
        return torch.randint(-3, 4, shape, generator=gen).to(dtype)
    return (torch.randn(shape, generator=gen) * scale).to(dtype)
