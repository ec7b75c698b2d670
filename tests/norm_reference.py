"""Layer norm, its gradients and dropout in float64 on the CPU, with
elementwise error bounds for the GPU's results.

Bounds.  u = 2^-24 is fp32's rounding error.  A row's sum is a chain of at most
8 values per 16-byte piece of a lane, two pieces, then six steps over a wave
and up to 16 waves: fewer than 40 additions for rows of up to 16384 columns;
wider rows add cols / 1024 per lane.  A sum of n terms with chains of d
additions is off by at most d u sum |terms| (and the terms' own errors).  Sums
over rows are bounded by rows additions.  A rounding to type t adds
finfo(t).eps / 2 relative, or half of the type's smallest step."""

from __future__ import annotations

import torch

from linear_reference import SMALLEST, U, half_step

LOW = 0xFFFFFFFF
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def philox(key: int, counter: int):
    """Philox4x32-10 of a 128-bit counter under a 64-bit key, in Python's whole numbers: four words."""
    c = [counter >> 32 * i & LOW for i in range(4)]
    k = [key & LOW, key >> 32]
    for _ in range(10):
        m0, m1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [m1 >> 32 ^ c[1] ^ k[0], m1 & LOW, m0 >> 32 ^ c[3] ^ k[1], m0 & LOW]
        k = [(k[0] + 0x9E3779B9) & LOW, (k[1] + 0xBB67AE85) & LOW]
    return c


def drop_count(p: float) -> int:
    return int(p * 65536 + 0.5)


def keep_row(row: int, cols: int, p: float, seed: int, offset: int) -> torch.Tensor:
    """One row's factors: 0 where dropped, 65536 / (65536 - drop) where kept."""
    drop = drop_count(p)
    if drop == 0:
        return torch.ones(cols, dtype=torch.float64)
    each, out = (cols + 7) // 8, []
    for i in range(each):
        for w in philox(seed, ((offset & (1 << 64) - 1) << 64) + row * each + i):
            out += [w & 0xFFFF, w >> 16]
    return torch.tensor([0.0 if n < drop else 65536 / (65536 - drop) for n in out[:cols]], dtype=torch.float64)


def keep(rows: int, cols: int, p: float, seed: int, offset: int) -> torch.Tensor:
    if drop_count(p) == 0:
        return torch.ones(rows, cols, dtype=torch.float64)
    return torch.stack([keep_row(r, cols, p, seed, offset) for r in range(rows)]) if rows else torch.ones(0, cols)


def chain(cols: int) -> int:
    return 40 + cols // 1024


def dropped(x, factors, residual, dtype):
    """(dropout(x) + residual, its bound): the scale is one rounding, so is each product and the sum."""
    v = torch.where(factors == 0, 0.0, x.double()) * factors
    tol = 2 * U * v.abs()
    if residual is not None:
        v = v + residual.double()
        tol = tol + U * (v.abs() + tol)
    return v, tol + half_step(v.abs() + tol, dtype)


def normed(total, weight, bias, eps):
    """{mean, rstd, y} with bounds, of rows as they are kept."""
    t, n = total.double(), total.shape[1]
    d = chain(n)
    mean = t.mean(1)
    off = (d + 2) * U * t.abs().mean(1) + SMALLEST[torch.float32]  # (sum, 1 / cols, product)
    dev = t - mean[:, None]
    var = dev.square().mean(1)
    # deviations from the computed mean: each off by `off` and one rounding; their squares average var + off^2
    var_off = off.square() + (d + 6) * U * (var + off.square())
    rstd = (var + eps).rsqrt()
    rel = 0.5 * var_off / (var + eps - var_off).clamp(min=torch.finfo(torch.float64).tiny) + 4 * U
    y = dev * rstd[:, None]
    tol = (off[:, None] + U * (dev.abs() + off[:, None])) * rstd[:, None] * (1 + rel[:, None]) + y.abs() * (rel[:, None] + 2 * U)
    if weight is not None:
        w = weight.double()
        y, tol = y * w, tol * w.abs() + 2 * U * (y * w).abs()
    if bias is not None:
        y = y + bias.double()
        tol = tol + 2 * U * (y.abs() + bias.double().abs())
    return {"mean": (mean, off), "rstd": (rstd, rstd * rel), "y": (y, tol + half_step(y.abs() + tol, total.dtype))}


def gradients(dy, total, mean, rstd, weight, dstream, factors):
    """{residual, x, weight, bias} with bounds, for the given statistics."""
    dtype, n, rows = dy.dtype, dy.shape[1], dy.shape[0]
    DY, s, m = dy.double(), rstd.double()[:, None], mean.double()[:, None]
    d = chain(n)
    u = (total.double() - m) * s
    u_off = 2 * U * u.abs()
    g = DY * (weight.double() if weight is not None else 1.0)
    g_off = U * g.abs()
    mg, mgu = g.mean(1, keepdim=True), (g * u).mean(1, keepdim=True)
    mg_off = (d + 4) * U * g.abs().mean(1, keepdim=True)
    mgu_off = (d + 8) * U * (g * u).abs().mean(1, keepdim=True)
    inner = g - mg - u * mgu
    off = g_off + mg_off + u.abs() * mgu_off + u_off * mgu.abs() + 4 * U * (g.abs() + mg.abs() + (u * mgu).abs())
    v = inner * s
    off = off * s + 2 * U * v.abs()
    if dstream is not None:
        v = v + dstream.double()
        off = off + U * (v.abs() + dstream.double().abs())
    x, x_off = v * factors, off * factors + 2 * U * (v * factors).abs()
    size = (DY * u).abs().sum(0)
    return {"residual": (v, off + half_step(v.abs() + off, dtype)), "x": (x, x_off + half_step(x.abs() + x_off, dtype)),
            "weight": ((DY * u).sum(0), (rows + 5) * U * size + SMALLEST[torch.float32]),
            "bias": (DY.sum(0), (rows + 2) * U * DY.abs().sum(0) + SMALLEST[torch.float32])}
