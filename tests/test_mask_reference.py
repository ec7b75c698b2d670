"""The many rows' mask against the row-by-row one, whose generator is pinned to
its authors' published numbers."""

from __future__ import annotations

import pytest
import torch

import mask_reference
import norm_reference as ref


@pytest.mark.parametrize("p", [0.1, 0.3, 0.999, 1e-9])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (4, 64), (5, 41), (2, 999)])
@pytest.mark.parametrize("seed,offset", [(0, 0), (0xFEDCBA9876543210, 5 << 33), ((1 << 64) - 1, (1 << 64) - 3), (77, 1 << 63)])
def test_the_same_mask(rows, cols, p, seed, offset):
    assert torch.equal(mask_reference.keep(rows, cols, p, seed, offset), ref.keep(rows, cols, p, seed, offset))


def test_a_row_under_the_mask_of_another_is_seen():
    """What the GPU tests hold the gradients to rejects rows that a workgroup takes second under its first row's mask."""
    gen = torch.Generator().manual_seed(1)
    rows, cols, places = 40, 24, 16
    total, dy = (torch.randn(rows, cols, generator=gen).bfloat16() for _ in range(2))
    mean = total.double().mean(1).float()
    rstd = (total.double().var(1, correction=0) + 1e-5).rsqrt().float()
    masks = mask_reference.keep(rows, cols, 0.3, 9, 2)
    value, tol = ref.gradients(dy, total, mean, rstd, None, None, masks)["x"]
    wrong = ref.gradients(dy, total, mean, rstd, None, None, masks[torch.arange(rows) % places])["x"][0].bfloat16()
    assert bool(((value.bfloat16().double() - value).abs() <= tol).all())
    seen = ((wrong.double() - value).abs() > tol).any(1)
    assert not bool(seen[:places].any()) and bool(seen[places:].all())


def test_rows_of_a_larger_matrix():
    whole = mask_reference.keep(9, 41, 0.3, 5, 7)
    assert torch.equal(mask_reference.keep(3, 41, 0.3, 5, 7, first=6 * 6), whole[6:])
