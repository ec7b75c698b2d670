"""How exact the norm's fp32 results are where the arithmetic can be followed
addition by addition: the mean of 16-bit rows."""

from __future__ import annotations

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
