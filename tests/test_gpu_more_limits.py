"""The norm, dropout and the vocabulary's loss at sizes where a launch takes
several steps, or a matrix several pieces by itself: more rows than a launch has
workgroups for, vocabularies of more than a piece's 2^20 words, contractions of
200001 values."""

from __future__ import annotations

import pytest
import torch

import dense_fp32_tiled_amd as dft
import loss_counted as counted
import mask_reference
import norm_reference as ref
from test_gpu_loss_counted import check

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def gpu(gemm_lib):
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def within(got, want, what):
    value, tol = want
    bad = ~((got.double() - value).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[0].tolist())


# 2^21 workgroups of four rows, of one row in four waves, of one row that is read again (narrower than eight columns)
@pytest.mark.parametrize("rows,cols", [((1 << 23) + 7, 8), ((1 << 21) + 5, 1040), ((1 << 21) + 3, 3)])
def test_more_rows_than_workgroups(rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    p, seed = 0.25, 11
    x = torch.randn(rows, cols, device="cuda", generator=gen, dtype=torch.float32).bfloat16()
    w = (torch.randn(cols, device="cuda", generator=gen) + 1).bfloat16()
    y, state = dft.layer_norm(x, w, eps=EPS, p=p, seed=seed)
    g = dft.layer_norm_grad(y, state, w, p=p, seed=seed, want=("x", "residual"))
    # both ends, and both sides of the last row of the first step
    for part in (slice(0, 50), slice(rows - 2000, rows), slice((1 << 21) - 30, (1 << 21) + 2)):
        # (a row's blocks follow those of all rows before it)
        factors = mask_reference.keep(part.stop - part.start, cols, p, seed, 0, "cuda", first=part.start * -(-cols // 8))
        within(state.total[part], ref.dropped(x[part], factors, None, x.dtype), ("total", part))
        want = ref.normed(state.total[part], w, None, EPS)
        for got, name in ((state.mean, "mean"), (state.rstd, "rstd"), (y, "y")):
            within(got[part], want[name], (name, part))
        want = ref.gradients(y[part], state.total[part], state.mean[part], state.rstd[part], w, None, factors)
        within(g.residual[part], want["residual"], ("residual", part))
        within(g.x[part], want["x"], ("x", part))


@pytest.mark.parametrize("transposed", [False, True], ids=["columns", "rows"])
@pytest.mark.parametrize("size", [(40, 1_200_001, 24), (3, 2_090_000, 16)], ids=lambda s: "x".join(map(str, s)))
def test_words_beyond_a_piece(size, transposed):
    for dtype in (torch.bfloat16, torch.float16):
        check(counted.make(*size, device="cuda"), dtype, transposed)


@pytest.mark.parametrize("transposed", [False, True], ids=["columns", "rows"])
@pytest.mark.parametrize("size,depth", [((5, 700, 12), 200001), ((70, 300, 9), 131080)])
def test_deep_contractions(size, depth, transposed):
    """The counted problem's features at places of a deep contraction, first and last among them; zeros elsewhere."""
    c = counted.make(*size, device="cuda")
    at = torch.linspace(0, depth - 1, c.K, device="cuda").round().long()
    for dtype in (torch.bfloat16, torch.float16):
        small_a, small_b = counted.operands(c, dtype, False)
        a, b = torch.zeros(c.M, depth, dtype=dtype, device="cuda"), torch.zeros(depth, c.N, dtype=dtype, device="cuda")
        a[:, at], b[at] = small_a, small_b
        if transposed:
            b = b.t().contiguous().t()
        loss, lse = dft.linear_cross_entropy(a, b, c.targets)
        want = counted.forward(c)
        counted.assert_tokens(lse, want["lse"], "lse")
        counted.assert_tokens(loss, want["loss"], "loss")
        grads = dft.linear_cross_entropy_grad(c.g, a, b, c.targets, lse)
        want = counted.gradients(c, lse, dtype)
        counted.assert_tokens(grads.a[:, at], want["a"], "a")
        counted.assert_words(c, grads.b[at], want["b"])
        grads.a[:, at], grads.b[at] = 0, 0
        assert float(grads.a.abs().max()) == 0 == float(grads.b.abs().max())
