"""The cross entropy over a vocabulary and its gradients in float64, with
elementwise error bounds for the GPU's results.

Bounds.  u = 2^-24 is fp32's rounding error; a logit's sum of K products is off
by at most e = (K + 2) 2u sum |a b| (linear_reference).  exp(z - m) is one
subtraction, one product and the hardware's exp2: relative 3u |z - m| + 4u
beside e.  A row's sum of N such values is a chain of at most N / 32 + 100
additions (16 in a lane, two over a wave, a thread's pieces, ten halvings),
each joining with two more products and exponentials: relative 8u a step is
taken for all of them, with the row's spread of logits s in 3u s.  dZ is
rounded to 16 bits: eps / 2, and where it is held scaled, half of the type's
least step over the scale, which is at least 2^13 / max |dloss|; up to 32 tokens
it is held in two parts, and what is left is (eps / 2)^2."""

from __future__ import annotations

import torch

from linear_reference import SMALLEST, U, half_step


def forward(a, b, targets):
    """{lse, loss} with bounds; b: K x N."""
    A, B = a.double(), b.double()
    K, N = B.shape
    z, size = A @ B, A.abs() @ B.abs()
    e = ((K + 2) * 2 * U * size).amax(1)
    most = z.amax(1)
    lse = torch.logsumexp(z, 1)
    rest = 8 * U * (N / 32 + 100) + 3 * U * (most - z.amin(1) + 2 * e)
    log = lse - most
    out = {"lse": (lse, e + rest + 4 * U * (most.abs() + log))}
    if targets is not None:
        t = targets.long()
        valid = (t >= 0) & (t < N)
        goal = z.gather(1, torch.where(valid, t, 0)[:, None])[:, 0]
        loss = torch.where(valid, lse - goal, 0.0)
        tol = torch.where(valid, 2 * e + rest + 4 * U * ((most - goal).abs() + log), 0.0)
        out["loss"] = (loss, tol)
    return out


def gradients(dloss, a, b, targets, lse, a_dtype=None, b_dtype=None, pieces=1):
    """{a, b} with bounds, for the given lse."""
    dtype = a.dtype
    A, B = a.double(), b.double()
    (K, N), M = B.shape, A.shape[0]
    t = targets.long()
    valid = (t >= 0) & (t < N)
    A = torch.where(valid[:, None], A, 0.0)  # (rows without target have no part, whatever they hold)
    z, e = A @ B, (K + 2) * 2 * U * (A.abs() @ B.abs())
    L = torch.where(valid, lse.double(), 0.0)[:, None]
    p = torch.exp(z - L)
    p_off = p * 1.01 * (e + 3 * U * (z - L).abs() + 4 * U)
    hot = torch.zeros_like(z)
    hot[valid.nonzero()[:, 0], t[valid]] = 1.0
    g = torch.where(valid, dloss.double(), 0.0)[:, None]
    dz = torch.where(valid[:, None], (p - hot) * g, 0.0)
    off = torch.where(valid[:, None], p_off * g.abs() + 3 * U * dz.abs(), 0.0)
    most = float(g.abs().max()) if M else 0.0
    step = torch.finfo(dtype).eps / 2
    if M <= 32:
        step *= step
    off = off + torch.where(valid[:, None], step * (dz.abs() + off) + SMALLEST[dtype] * most / 2 ** 13, 0.0)
    big = dz.abs() + off
    da, db = dz @ B.t(), A.t() @ dz
    da_off = off @ B.abs().t() + (N + 2 + pieces) * 2 * U * (big @ B.abs().t())
    db_off = A.abs().t() @ off + (M + 3) * 2 * U * (A.abs().t() @ big)
    return {"a": (da, da_off + half_step(da.abs() + da_off, a_dtype or dtype)),
            "b": (db, db_off + half_step(db.abs() + db_off, b_dtype or dtype))}
