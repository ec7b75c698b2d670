"""Refusals of the layer norm, its gradients and dropout (CPU only: every bad
call is refused on the host, before anything is launched), and the generator's
published numbers."""

from __future__ import annotations

import ctypes
import math
import re
from pathlib import Path

import pytest
import torch

import dense_fp32_tiled_amd as dft
import norm_reference as ref

X, R, T, Y, D, E, S, W = (0x1000000000 * i for i in range(1, 9))  # far apart, never dereferenced


def norm_args(rows=64, cols=32, **kw):
    fields = dict(value_type=dft.VALUE_BF16, eps=1e-5, p=0.0, rows=rows, cols=cols, x=X, ldx=cols, y=Y, ldy=cols)
    fields.update(kw)
    return dft.LayerNormArgs(**fields)


def grad_args(rows=64, cols=32, **kw):
    fields = dict(value_type=dft.VALUE_BF16, p=0.0, rows=rows, cols=cols, dY=Y, ldy=cols, total=T, ldt=cols, mean=S,
                  rstd=S + 4096, dtotal=D, lddt=cols)
    fields.update(kw)
    return dft.LayerNormGradArgs(**fields)


def test_generator_gives_the_published_numbers():
    """The known answers that the generator's authors publish for Philox4x32-10."""
    ones = (1 << 128) - 1
    assert ref.philox(0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox((1 << 64) - 1, ones) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    counter = 0x243F6A88 | 0x85A308D3 << 32 | 0x13198A2E << 64 | 0x03707344 << 96
    assert ref.philox(0xA4093822 | 0x299F31D0 << 32, counter) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


@pytest.mark.parametrize("kw,status", [
    (dict(value_type=3), "UNSUPPORTED"), (dict(value_type=-1), "UNSUPPORTED"), (dict(eps=-1e-5), "UNSUPPORTED"),
    (dict(eps=math.nan), "UNSUPPORTED"), (dict(eps=math.inf), "UNSUPPORTED"), (dict(p=-0.1), "UNSUPPORTED"),
    (dict(p=1.01), "UNSUPPORTED"), (dict(p=math.nan), "UNSUPPORTED"), (dict(rows=-1), "INVALID_DIM"),
    (dict(cols=0, ldx=1, ldy=1), "INVALID_DIM"), (dict(rows=1 << 41), "INVALID_DIM"),
    (dict(cols=(1 << 31) + 1), "TOO_LARGE"), (dict(rows=1 << 30, cols=1 << 21), "TOO_LARGE"),
    (dict(ldx=31), "INVALID_LD"), (dict(ldy=31), "INVALID_LD"), (dict(residual=R, ldr=31, total=T, ldt=32), "INVALID_LD"),
    (dict(residual=R, ldr=32, total=T, ldt=31), "INVALID_LD"), (dict(x=None), "NULL"), (dict(y=None), "NULL"),
    (dict(residual=R, ldr=32, ldt=32), "NULL"), (dict(p=0.5, ldt=32), "NULL"), (dict(p=1e-9, ldt=32), "NULL"),
    (dict(y=X), "ALIAS"), (dict(y=X + 2), "ALIAS"), (dict(weight=Y), "ALIAS"), (dict(bias=Y + 2), "ALIAS"),
    (dict(mean=X), "ALIAS"), (dict(rstd=Y), "ALIAS"), (dict(mean=S, rstd=S + 4), "ALIAS"),
    (dict(residual=R, ldr=32, total=Y, ldt=32), "ALIAS"), (dict(residual=R, ldr=32, total=X + 2, ldt=32), "ALIAS"),
    (dict(residual=R, ldr=32, total=R, ldt=40), "ALIAS"), (dict(residual=R, ldr=32, total=R, ldt=32, y=R), "ALIAS"),
    (dict(residual=X, ldr=32, total=X, ldt=40), "ALIAS"), (dict(p=0.5, total=T, ldt=32, step=T), "ALIAS"),
    (dict(ldx=1 << 60), "TOO_LARGE"),
])
def test_norm_refusals(kw, status, gemm_lib):
    assert dft.gemm_layer_norm(norm_args(**kw)) == getattr(dft, "GEMM_ERR_" + status)


def test_norm_of_no_rows_needs_nothing(gemm_lib):
    assert dft.gemm_layer_norm(norm_args(rows=0, x=None, y=None)) == dft.GEMM_OK
    # total over x or over the residual passes the checks and asks for a device, which is not here
    refused = (dft.GEMM_ERR_ALIAS, dft.GEMM_ERR_NULL, dft.GEMM_ERR_INVALID_LD)
    for kw in (dict(total=X, ldt=32), dict(total=R, ldt=32), dict(residual=X, total=X, ldt=32)):
        assert dft.gemm_layer_norm(norm_args(**{**dict(residual=R, ldr=32), **kw, "rows": 0})) == dft.GEMM_OK
        if not torch.cuda.is_available():
            assert dft.gemm_layer_norm(norm_args(**{**dict(residual=R, ldr=32), **kw})) not in refused


@pytest.mark.parametrize("kw,status", [
    (dict(value_type=3), "UNSUPPORTED"), (dict(p=1.5), "UNSUPPORTED"), (dict(rows=-1), "INVALID_DIM"),
    (dict(cols=0, ldy=1, ldt=1, lddt=1), "INVALID_DIM"), (dict(ldy=31), "INVALID_LD"), (dict(ldt=31), "INVALID_LD"),
    (dict(lddt=31), "INVALID_LD"), (dict(dx=E, lddx=31), "INVALID_LD"), (dict(dstream=R, lds=31), "INVALID_LD"),
    (dict(dY=None), "NULL"), (dict(total=None), "NULL"), (dict(mean=None), "NULL"), (dict(rstd=None), "NULL"),
    (dict(dtotal=Y), "ALIAS"), (dict(dtotal=T), "ALIAS"), (dict(dx=D, lddx=32), "ALIAS"),
    (dict(dstream=D, lds=32), "ALIAS"), (dict(dweight=S), "ALIAS"), (dict(dweight=W, dbias=W + 4), "ALIAS"),
    (dict(dweight=D), "ALIAS"), (dict(workspace=W, workspace_bytes=-1), "WORKSPACE"),
    (dict(workspace=D, workspace_bytes=16), "ALIAS"), (dict(p=0.5, dx=E, lddx=32, step=E), "ALIAS"),
    (dict(cols=65535 * 2048 + 1), "TOO_LARGE"),
])
def test_grad_refusals(kw, status, gemm_lib):
    want = getattr(dft, "GEMM_ERR_" + status)
    assert dft.gemm_layer_norm_grad(grad_args(**kw)) == want
    if "workspace" not in kw:
        assert dft.gemm_layer_norm_grad_workspace_bytes(grad_args(**kw), 256) == want


def test_grad_workspace(gemm_lib):
    need = dft.gemm_layer_norm_grad_workspace_bytes
    assert need(grad_args(), 256) == 0
    assert need(grad_args(dweight=W), 0) == dft.GEMM_ERR_INVALID_DIM
    for cols in (1, 512, 513, 4096, 16384, 16385, 100000):
        for rows in (0, 1, 5, 5000):
            n = need(grad_args(rows, cols, dweight=1 << 50), 256)
            assert n % (8 * cols) == 0 and n // (8 * cols) <= min(rows, 1024) and (n > 0) == (rows > 0)
            if n and not torch.cuda.is_available():  # (the device comes before the workspace)
                assert dft.gemm_layer_norm_grad(grad_args(rows, cols, dweight=1 << 50)) < 0
    assert dft.gemm_layer_norm_grad(grad_args(dtotal=None)) == dft.GEMM_OK  # nothing wanted
    assert gemm_lib.gemm_layer_norm(None, None) == dft.GEMM_ERR_NULL
    assert gemm_lib.gemm_layer_norm_grad(None, None) == dft.GEMM_ERR_NULL
    assert gemm_lib.gemm_layer_norm_grad_workspace_bytes(None, 256) == dft.GEMM_ERR_NULL


def test_dropout_refusals(gemm_lib):
    def drop(kind=0, rows=8, cols=16, p=0.5, seed=1, offset=2, step=None, x=X, ldx=16, r=None, ldr=0, y=Y, ldy=16):
        return dft.gemm_dropout(kind, rows, cols, p, seed, offset, step, x, ldx, r, ldr, y, ldy)

    assert drop(kind=3) == drop(p=-1.0) == drop(p=2.0) == drop(p=math.nan) == dft.GEMM_ERR_UNSUPPORTED
    assert drop(rows=-1) == drop(cols=-1) == dft.GEMM_ERR_INVALID_DIM
    assert drop(ldx=15) == drop(ldy=15) == drop(r=R, ldr=15) == dft.GEMM_ERR_INVALID_LD
    assert drop(x=None) == drop(y=None) == dft.GEMM_ERR_NULL
    assert drop(y=X + 2) == drop(y=X, ldy=17) == drop(r=Y + 2, ldr=16) == drop(step=Y) == dft.GEMM_ERR_ALIAS
    assert drop(y=X, r=X + 2, ldr=16) == dft.GEMM_ERR_ALIAS  # in place, with the residual across it
    assert drop(rows=1 << 40, cols=1 << 20, ldx=1 << 20, ldy=1 << 20) == dft.GEMM_ERR_TOO_LARGE
    assert drop(rows=0, x=None, y=None) == drop(cols=0, x=None, y=None) == dft.GEMM_OK
    if not torch.cuda.is_available():
        assert drop(y=X) not in (dft.GEMM_OK, dft.GEMM_ERR_ALIAS) and drop(r=Y, ldr=16) != dft.GEMM_ERR_ALIAS


def test_torch_refusals(gemm_lib):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: dft.layer_norm(x), lambda: dft.dropout(x, 0.5, 1),
                 lambda: dft.layer_norm_grad(x, dft.NormState(x, x, x))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: dft.layer_norm(x.double()), lambda: dft.dropout(x.int(), 0.5, 1), lambda: dft.dropout([1], 0.5, 1),
                 lambda: dft.layer_norm_grad(x.long(), dft.NormState(x, x, x))):
        with pytest.raises(TypeError):
            call()


def test_structures_match_the_header(gemm_lib):
    text = (Path(__file__).resolve().parent.parent / "include" / "dense_fp32_tiled.h").read_text()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    kinds = {ctypes.c_void_p: "p", ctypes.c_int64: "int64_t", ctypes.c_int32: "int32_t", ctypes.c_uint64: "uint64_t",
             ctypes.c_float: "float", ctypes.c_double: "double"}
    for name, struct in (("gemm_layer_norm_args", dft.LayerNormArgs), ("gemm_layer_norm_grad_args", dft.LayerNormGradArgs)):
        body = re.search(r"typedef struct \{([^}]*)\}\s*" + name + ";", text).group(1)
        fields = []
        for line in filter(None, map(str.strip, body.split(";"))):
            kind = "p" if "*" in line else re.match(r"(const )?(\w+)", line).group(2)
            for part in re.sub(r"\b(const|void|float|double|u?int\d+_t)\b|\*", " ", line).split(","):
                fields.append((part.strip(), kind))
        assert fields == [(f, kinds[t]) for f, t in struct._fields_]
