"""How exact the norm's fp32 results are where the arithmetic can be followed
addition by addition: the mean of 16-bit rows, and the sums over the rows."""

from __future__ import annotations

import math

import pytest
import torch

import dense_fp32_tiled_amd as dft

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu(gemm_lib):
    assert torch.cuda.is_available(), "GPU tests need a GPU"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("cols", [7, 50, 300, 499, 500])
def test_mean_of_16_bit_rows(cols, dtype):
    """Rows of k / 128 whose mean lies in [1/4, 1/2).  The kernel's first mean has 16 significant bits there, multiples of
    2^-17, so each deviation is exact (at most 18 bits), and so is any partial sum of theirs in any order: it is at most
    half of the sum of their magnitudes, below 2^7.  What is left are the division by cols, 2^-24 of a shift below 2^-17,
    and the sum of the two, half a unit, 2^-26."""
    gen = torch.Generator().manual_seed(cols)
    x = torch.randint(-40, 121, (400, cols), generator=gen).double() / 128
    x = x[(x.mean(1) >= 0.25) & (x.mean(1) < 0.5)]
    assert x.shape[0] > 100 and float((x - x.mean(1, keepdim=True)).abs().sum(1).max()) / 2 < 2 ** 7 - 1
    _, state = dft.layer_norm(x.to(dtype).cuda())
    off = (state.mean.cpu().double() - x.mean(1)).abs().max()
    assert float(off) <= 2.0 ** -26 + 2.0 ** -41, float(off) * 2 ** 26


@pytest.mark.parametrize("rows", [1000, 1024, 500])
def test_sums_over_the_rows(rows):
    """The bias's gradient of up to 1024 rows of 513 columns, a row to a workgroup: the join's order alone counts.  An
    addition that makes a sum of n independent values of variance 1 is off by at most 2^-24 of it, evenly spread: variance
    2^-48 n / 3.  A column's 1024 values are added by 32 threads, each in eight chains of four, joined by halves, and so are
    the 32: over all additions the n add up to 32 (8 (2 + 3 + 4) + 3 32) + 5 1024, and the result's variance is 1024.  513
    columns' mean square is within a tenth of its expectation's root (8 standard deviations: 513^-1/2 / 2 each at most)."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    dy, total = (torch.randn(rows, 513, device="cuda", generator=gen) for _ in range(2))
    state = dft.NormState(total, total.mean(1), total.var(1, correction=0).rsqrt())
    exact = dy.double().sum(0)
    got = dft.layer_norm_grad(dy, state, want=("bias",)).bias
    off = float((got.double() - exact).norm() / exact.norm())
    additions = 32 * (8 * (2 + 3 + 4) + 3 * 32) + 5 * 1024
    assert off <= 1.2 * 2.0 ** -24 * math.sqrt(additions / 1024 / 3), off
