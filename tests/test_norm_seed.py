"""Dropout without a seed is refused, in the norm and its gradient as in
`dropout` itself: calls that leave it out would all drop the same elements."""

from __future__ import annotations

import pytest
import torch

import dense_fp32_tiled_amd as dft
from dense_fp32_tiled_amd import norms


@pytest.fixture(scope="module", autouse=True)
def bound(gemm_lib):
    with pytest.raises(ValueError, match="GPU"):
        dft.layer_norm(torch.zeros(1, 8))


def test_the_check():
    device = torch.device("cpu")
    for p in (1e-9, 0.1, 1.0):
        with pytest.raises(ValueError, match="seed"):
            norms._counter(p, None, 0, None, device)
        assert norms._counter(p, 0, 0, None, device) == (0, None) and norms._counter(p, 7, 5, None, device) == (7, None)
    assert norms._counter(0.0, None, 0, None, device) == (0, None)
    for bad in (dict(p=-0.1, seed=None), dict(p=2.0, seed=None), dict(p=0.5, seed=-1), dict(p=0.0, seed=None, offset=-1)):
        with pytest.raises(ValueError):
            norms._counter(**{**dict(offset=0, step=None, device=device), **bad})
    with pytest.raises(TypeError):
        norms._counter(0.0, None, 0, torch.zeros(1), device)


@pytest.mark.gpu
def test_the_calls():
    x = torch.randn(4, 40, device="cuda")
    y, state = dft.layer_norm(x)
    for call in (lambda: dft.layer_norm(x, p=0.1), lambda: dft.layer_norm(x, residual=x, p=0.1, offset=3),
                 lambda: dft.layer_norm_grad(x, state, p=0.1)):
        with pytest.raises(ValueError, match="seed"):
            call()
    # without dropout nothing is drawn
    assert torch.equal(dft.layer_norm(x, p=0.0)[0], y) and dft.layer_norm_grad(x, state).x.shape == x.shape
    assert not torch.equal(dft.layer_norm(x, p=0.1, seed=0)[0], y)
