"""Tokens of very different weights in one batch of the vocabulary's loss: each
token's own row of dA, and the words that light tokens alone have as targets,
against float64 with bounds relative to the token's own weight."""

from __future__ import annotations

import pytest
import torch

import dense_fp32_tiled_amd as dft
from linear_reference import SMALLEST, U, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu(gemm_lib):
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def problem(M, N, K, dtype, seed, transposed=True, size=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    a = (torch.randn(M, K, device="cuda", generator=gen) * size).to(dtype)
    b = (torch.randn(N, K, device="cuda", generator=gen) * 2 * K ** -0.5 / size).to(dtype)
    t = torch.randint(0, N, (M,), device="cuda", generator=gen)
    return a, b.t() if transposed else b.t().contiguous(), t


def bounds(g, a, b, t, lse, dtype, pieces):
    """((dA, bound), (dB, bound)) for fp32 results.  Logits, exponentials and sums as in loss_reference.  dZ's rounding is
    relative to each row's own weight: in fp16 a row is held at a scale of more than 2^12 / g (2^13, but for a factor
    that is not a power of two).  dB takes A's rows scaled so that the largest |g A| of all lies in [2^14 / 4, 2^16) times
    2^14 and every other at its own: an entry is off by 2^-25 of that scale where it is below fp16's normal numbers."""
    A, B = a.double(), b.double()
    (M, K), N = A.shape, B.shape[1]
    valid = (t >= 0) & (t < N)
    A = torch.where(valid[:, None], A, 0.0)
    goal, G = torch.where(valid, t, 0), torch.where(valid, g.double(), 0.0)
    z, e = A @ B, (K + 2) * 2 * U * (A.abs() @ B.abs())
    L = lse.double()[:, None]
    p = torch.exp(z - L)
    hot = torch.zeros_like(z)
    hot[valid.nonzero()[:, 0], goal[valid]] = 1
    dz = (p - hot) * G[:, None]
    step = (torch.finfo(dtype).eps / 2) ** (2 if M <= 32 else 1)
    # (two parts: the second is rounded to the type's least step too)
    least = (2.0 ** -25 / 2 ** 12 if dtype == torch.float16 else SMALLEST[dtype]) * G.abs()[:, None]
    off = p * 1.01 * (e + 3 * U * (z - L).abs() + 4 * U) * G.abs()[:, None] + 3 * U * dz.abs()
    off = off + step * (dz.abs() + off) + least
    big = dz.abs() + off
    da_off = off @ B.abs().t() + (N + 2 + pieces) * 2 * U * (big @ B.abs().t())
    a_off = torch.zeros_like(A)
    if dtype == torch.float16:
        top = (G.abs() * A.abs().amax(1)).max()
        a_off = torch.where(G[:, None] != 0, 2.0 ** -25 * top / 2.0 ** 12 / G.abs().clamp(min=1e-300)[:, None], 0.0).expand_as(A)
    db_off = A.abs().t() @ off + a_off.t() @ big + (M + 3) * 2 * U * (A.abs().t() @ big)
    da, db = dz @ B.t(), A.t() @ dz
    return (da, da_off + half_step(da.abs() + da_off, torch.float32)), (db, db_off + half_step(db.abs() + db_off, torch.float32))


def check(got, want, what):
    value, tol = want
    bad = ~((got.double() - value).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("M", [24, 200])
@pytest.mark.parametrize("ratio", [1e-2, 1e-4, 1e-6, 1e-7, 1e-8, 1e-9])
def test_light_tokens_keep_their_rows(ratio, M, dtype):
    for transposed, piece in ((True, 0), (False, 8192)):
        a, b, t = problem(M, 50000, 72, dtype, M, transposed)
        g = torch.full((M,), ratio, device="cuda")
        g[::8] = 1.0 / M
        g[3::8] *= 0.37
        t[5] = -1
        _, lse = dft.linear_cross_entropy(a, b, t)
        grads = dft.linear_cross_entropy_grad(g, a, b, t, lse, a_dtype=torch.float32, b_dtype=torch.float32, piece=piece)
        da, db = bounds(g, a, b, t, lse, dtype, 7)
        check(grads.a, da, "da")
        check(grads.b, db, "db")
        # in the 2-norm a row is off by its roundings, a few units of 16 bits, whatever its weight
        rel = (grads.a.double() - da[0]).norm(dim=1) / da[0].norm(dim=1).clamp(min=1e-300)
        assert float(rel[t >= 0].max()) <= 2 * torch.finfo(dtype).eps


@pytest.mark.parametrize("size", [1e-3, 100.0])
@pytest.mark.parametrize("M", [24, 200])
def test_every_size_of_the_rows(M, size):
    """Rows of A near both ends of fp16's range beside weights of every size from 1 to 2^-22, both gradients."""
    a, b, t = problem(M, 3000, 136, torch.float16, 7, size=size)
    g = 2.0 ** -(torch.arange(M, device="cuda") % 23).float()
    a[7] = 0
    a[9, 5] = 65504.0 if size > 1 else 2.0 ** -24
    b[5] = 0  # (the large value has no part in the logits)
    _, lse = dft.linear_cross_entropy(a, b, t)
    grads = dft.linear_cross_entropy_grad(g, a, b, t, lse, a_dtype=torch.float32, b_dtype=torch.float32)
    da, db = bounds(g, a, b, t, lse, torch.float16, 1)
    check(grads.a, da, "da")
    check(grads.b, db, "db")


def test_weights_that_nothing_holds():
    """Zero, infinite and NaN weights: a zero one has no part, the others spoil what they are part of and no more."""
    a, b, t = problem(40, 500, 64, torch.float16, 3)
    g = torch.rand(40, device="cuda")
    g[4] = 0.0
    _, lse = dft.linear_cross_entropy(a, b, t)
    clean = dft.linear_cross_entropy_grad(g, a, b, t, lse, a_dtype=torch.float32, b_dtype=torch.float32)
    for x, want in zip(clean, bounds(g, a, b, t, lse, torch.float16, 1)):
        check(x, want, "clean")
    assert float(clean.a[4].abs().max()) == 0
    bad = g.clone()
    bad[7] = float("nan")
    spoilt = dft.linear_cross_entropy_grad(bad, a, b, t, lse, a_dtype=torch.float32, b_dtype=torch.float32)
    rest = torch.arange(40, device="cuda") != 7
    assert bool(spoilt.a[7].isnan().all()) and torch.equal(spoilt.a[rest], clean.a[rest]) and bool(spoilt.b.isnan().all())
    spoilt = dft.linear_cross_entropy_grad(torch.where(rest, g, float("inf")), a, b, t, lse, a_dtype=torch.float32)
    assert not bool(spoilt.a[7].isfinite().any()) and bool(spoilt.a[rest].isfinite().all())
    none = dft.linear_cross_entropy_grad(torch.zeros_like(g), a, b, t, lse)
    assert float(none.a.abs().max()) == 0 == float(none.b.abs().max())


@pytest.mark.parametrize("M", [20, 300])
def test_one_gradient_alone_and_captured(M):
    """The same bits for either gradient alone, and replayed in a graph with other weights."""
    a, b, t = problem(M, 5000, 264, torch.float16, 11)
    g = 2.0 ** -(torch.arange(M, device="cuda") % 30).float()
    _, lse = dft.linear_cross_entropy(a, b, t, piece=2048)

    def both():
        lse = dft.linear_cross_entropy(a, b, t, piece=2048)[1]
        return dft.linear_cross_entropy_grad(g, a, b, t, lse, piece=2048)

    want = both()
    assert torch.equal(dft.linear_cross_entropy_grad(g, a, b, t, lse, want=("a",), piece=2048).a, want.a)
    assert torch.equal(dft.linear_cross_entropy_grad(g, a, b, t, lse, want=("b",), piece=2048).b, want.b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for n in range(4):
        g.copy_(g.roll(1))
        a.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        want = both()
        assert torch.equal(held.a, want.a) and torch.equal(held.b, want.b), n


@pytest.mark.parametrize("M", [20, 100])
@pytest.mark.parametrize("ratio", [1e-2, 1e-5, 1e-8])
def test_words_of_light_tokens_beside_large_values(ratio, M):
    """A heavy token of large values and sure of its word (any other has e^-40 of it), light ones of small values in
    features of their own: dB at a light token's feature and target has that token's term alone, -g a (1 - p).  A is held
    to 2^-24 of its largest value; the target's entry of dZ and the products add 2^-11 and a few 2^-24 each."""
    N, K, heavy = 5000, 128, 200.0
    a, b = torch.zeros(M, K, dtype=torch.float16, device="cuda"), torch.zeros(N, K, dtype=torch.float16, device="cuda")
    small = 0.02 * (1 + torch.arange(1, M, device="cuda") / M)
    light = torch.arange(1, M, device="cuda")
    a[0, 0], b[0, 0] = heavy, 0.2
    a[light, light] = small.half()
    t = torch.cat([torch.zeros(1, device="cuda").long(), 7 + 40 * light])
    g = torch.full((M,), ratio, device="cuda")
    g[0] = 1.0
    _, lse = dft.linear_cross_entropy(a, b.t(), t)
    grads = dft.linear_cross_entropy_grad(g, a, b.t(), t, lse, a_dtype=torch.float32, b_dtype=torch.float32)
    got = grads.b[light, t[light]].double()
    want = -g[light].double() * a[light, light].double() * (1 - torch.exp(-lse[light].double()))
    rel = 2.0 ** -24 * heavy / a[light, light].double() + 2.0 ** -11 + 2.0 ** -20
    assert bool(((got - want).abs() <= rel * want.abs()).all()), ((got / want - 1).abs() / rel).max()
