"""The norm's dropout at sizes where a workgroup of the gradient's kernel takes
several rows one after another (its next row read ahead of this one's results),
and the forward pass at the same sizes: every element of every row against
float64 with the mask of that row, beside the stream's gradient and without.

`taken` counts the rows that a workgroup takes, as the C API's workspace tells
it: two sums of cols fp32 values for each workgroup."""

from __future__ import annotations

import pytest
import torch

import dense_fp32_tiled_amd as dft
import mask_reference
import norm_reference as ref

pytestmark = pytest.mark.gpu

EPS, P, SEED, OFFSET = 1e-5, 0.3, 0xFEDCBA9876543210, 5 << 33
KINDS = {torch.bfloat16: dft.VALUE_BF16, torch.float16: dft.VALUE_F16, torch.float32: dft.VALUE_F32}


@pytest.fixture(scope="module", autouse=True)
def gpu(gemm_lib):
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def taken(rows, cols, dtype):
    """Rows of a workgroup's turns; 1: none takes a second."""
    a = dft.LayerNormGradArgs(value_type=KINDS[dtype], p=P, rows=rows, cols=cols, dY=1 << 40, ldy=cols, total=1 << 42, ldt=cols,
                              mean=1 << 44, rstd=1 << 45, dtotal=1 << 46, lddt=cols, dweight=1 << 48)
    need = dft.gemm_layer_norm_grad_workspace_bytes(a, torch.cuda.get_device_properties(0).multi_processor_count)
    places = need // (8 * cols)
    rows_at_once = 4 if cols <= 512 else 1  # (a workgroup of four waves has a row in each)
    return -(-rows // (places * rows_at_once))


def within(got, want, what):
    value, tol = want
    bad = ~((got.double() - value).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[0].tolist())


def normal(gen, *shape, dtype, mean=0.0):
    return (torch.randn(*shape, generator=gen, device="cuda") + mean).to(dtype)


# rows, cols: whole and ragged rows of each shape, up to five rows of a workgroup
SIZES = [(9000, 24), (9001, 511), (2600, 1536), (2100, 2047), (1700, 4095), (1030, 4096), (600, 8200), (700, 16384), (600, 16383)]


@pytest.mark.parametrize("joined", [False, True], ids=["alone", "joined"])
@pytest.mark.parametrize("kind", list(ref.TYPES))
@pytest.mark.parametrize("rows,cols", SIZES)
def test_rows_taken_one_after_another(rows, cols, kind, joined):
    dtype = ref.TYPES[kind]
    if cols <= 8192 or dtype != torch.float32:  # (wider rows in 32 bits go to the kernels that read a row again)
        assert taken(rows, cols, dtype) >= 2
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x, w, b, dy = normal(gen, rows, cols, dtype=dtype, mean=0.5), *(normal(gen, cols, dtype=dtype, mean=m) for m in (1, 0)), normal(gen, rows, cols, dtype=dtype)
    other = normal(gen, rows, cols, dtype=dtype) if joined else None
    factors = mask_reference.keep(rows, cols, P, SEED, OFFSET, "cuda")
    y, state = dft.layer_norm(x, w, b, eps=EPS, residual=other, p=P, seed=SEED, offset=OFFSET)
    within(state.total, ref.dropped(x, factors, other, dtype), "total")
    want = ref.normed(state.total, w, b, EPS)
    for got, name in ((state.mean, "mean"), (state.rstd, "rstd"), (y, "y")):
        within(got, want[name], name)
    g = dft.layer_norm_grad(dy, state, w, dtotal=other, p=P, seed=SEED, offset=OFFSET)
    want = ref.gradients(dy, state.total, state.mean, state.rstd, w, other, factors)
    for name in ("residual", "x", "weight", "bias"):
        within(getattr(g, name), want[name], name)
    # the mask of both passes is the same one, and of the definition
    kept = factors != 0
    assert float(g.x[~kept].abs().max()) == 0 and bool((g.x != 0)[kept & (g.residual != 0)].all())
