"""Refusals and workspaces of the cross entropy over a vocabulary and its
gradients: every bad call is refused on the host, before anything is launched
(CPU only: the addresses are never read)."""

from __future__ import annotations

import ctypes
import re
from pathlib import Path

import pytest
import torch

import dense_fp32_tiled_amd as dft

A, B, T, L, S, G, D, E, W = (0x1000000000 * i for i in range(1, 10))  # far apart, never dereferenced


def loss_args(M=64, N=320, K=48, **kw):
    fields = dict(input_type=dft.INPUT_BF16, M=M, N=N, K=K, A=A, lda=max(K, 1), B=B,
                  ldb=max(K if kw.get("b_transposed") else N, 1), targets=T, loss=L, lse=S)
    fields.update(kw)
    return dft.CrossEntropyArgs(**fields)


def grad_args(M=64, N=320, K=48, **kw):
    ld = max(K if kw.get("b_transposed") else N, 1)
    fields = dict(input_type=dft.INPUT_BF16, M=M, N=N, K=K, A=A, lda=max(K, 1), B=B, ldb=ld, targets=T, lse=S, dloss=G,
                  dA=D, ldda=max(K, 1), dB=E, lddb=ld)
    fields.update(kw)
    return dft.CrossEntropyGradArgs(**fields)


COMMON = [
    (dict(input_type=2), "UNSUPPORTED"), (dict(target_type=2), "UNSUPPORTED"), (dict(target_type=-1), "UNSUPPORTED"),
    (dict(b_transposed=2, ldb=320), "UNSUPPORTED"), (dict(variant=dft.LINEAR_COUNT), "UNSUPPORTED"),
    (dict(variant=-1), "UNSUPPORTED"), (dict(M=-1), "INVALID_DIM"), (dict(N=0), "INVALID_DIM"), (dict(N=-5), "INVALID_DIM"),
    (dict(K=-1), "INVALID_DIM"), (dict(piece=-256), "INVALID_DIM"), (dict(piece=100), "INVALID_DIM"),
    (dict(N=1 << 31), "TOO_LARGE"), (dict(M=1 << 31), "TOO_LARGE"), (dict(M=1 << 30, K=1 << 21), "TOO_LARGE"),
    (dict(M=1 << 41), "INVALID_DIM"), (dict(lda=47), "INVALID_LD"), (dict(ldb=319), "INVALID_LD"),
    (dict(b_transposed=1, ldb=47), "INVALID_LD"), (dict(A=None), "NULL"), (dict(B=None), "NULL"), (dict(targets=None), "NULL"),
    (dict(lda=(1 << 21)), "TOO_LARGE"), (dict(b_transposed=1, ldb=1 << 21), "TOO_LARGE"),
    (dict(workspace=W, workspace_bytes=-1), "WORKSPACE"), (dict(workspace=A, workspace_bytes=64), "ALIAS"),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(lse=None), "NULL"), (dict(loss=S), "ALIAS"), (dict(loss=A), "ALIAS"), (dict(lse=T), "ALIAS"), (dict(lse=B + 4), "ALIAS"),
    (dict(workspace=S, workspace_bytes=64), "ALIAS"),
])
def test_forward_refusals(kw, status, gemm_lib):
    want = getattr(dft, "GEMM_ERR_" + status)
    args = loss_args(**kw)
    if status == "TOO_LARGE" and not torch.cuda.is_available():  # (some are found when the plan is made, for a device)
        assert dft.gemm_cross_entropy(args) < 0
    elif status != "TOO_LARGE":
        assert dft.gemm_cross_entropy(args) == want
    if "workspace" not in kw:
        assert dft.gemm_cross_entropy_workspace_bytes(args, 256) == want


@pytest.mark.parametrize("kw,status", COMMON[:-5] + COMMON[-2:] + [
    (dict(b_transposed=1, ldb=1 << 21, lddb=48), "TOO_LARGE"),
    (dict(a_grad_type=2), "UNSUPPORTED"), (dict(b_grad_type=-1), "UNSUPPORTED"), (dict(ldda=47), "INVALID_LD"),
    (dict(lddb=319), "INVALID_LD"), (dict(lse=None), "NULL"), (dict(dloss=None), "NULL"), (dict(targets=None), "NULL"),
    (dict(dA=A), "ALIAS"), (dict(dB=B), "ALIAS"), (dict(dA=E), "ALIAS"), (dict(dB=G), "ALIAS"), (dict(dA=S), "ALIAS"),
    (dict(dB=T - 4), "ALIAS"), (dict(workspace=D, workspace_bytes=64), "ALIAS"), (dict(ldda=(1 << 26) + 1), "TOO_LARGE"),
    (dict(lddb=(1 << 26) + 1), "TOO_LARGE"),
])
def test_grad_refusals(kw, status, gemm_lib):
    want = getattr(dft, "GEMM_ERR_" + status)
    args = grad_args(**kw)
    if status == "TOO_LARGE" and not torch.cuda.is_available():
        assert dft.gemm_cross_entropy_grad(args) < 0
    elif status != "TOO_LARGE":
        assert dft.gemm_cross_entropy_grad(args) == want
    if "workspace" not in kw:
        assert dft.gemm_cross_entropy_grad_workspace_bytes(args, 256) == want


def test_null_and_nothing(gemm_lib):
    assert gemm_lib.gemm_cross_entropy(None, None) == dft.GEMM_ERR_NULL
    assert gemm_lib.gemm_cross_entropy_grad(None, None) == dft.GEMM_ERR_NULL
    assert gemm_lib.gemm_cross_entropy_workspace_bytes(None, 256) == dft.GEMM_ERR_NULL
    assert gemm_lib.gemm_cross_entropy_grad_workspace_bytes(None, 256) == dft.GEMM_ERR_NULL
    assert dft.gemm_cross_entropy_workspace_bytes(loss_args(), 0) == dft.GEMM_ERR_INVALID_DIM
    assert dft.gemm_cross_entropy_grad_workspace_bytes(grad_args(), 0) == dft.GEMM_ERR_INVALID_DIM
    # no tokens, and no gradients wanted
    assert dft.gemm_cross_entropy(loss_args(M=0, A=None, B=None, targets=None, loss=None, lse=None)) == dft.GEMM_OK
    assert dft.gemm_cross_entropy_grad(grad_args(M=0, dB=None, A=None, targets=None, lse=None, dloss=None, dA=None)) == dft.GEMM_OK
    assert dft.gemm_cross_entropy_grad(grad_args(dA=None, dB=None)) == dft.GEMM_OK
    # lse alone asks for no targets
    assert dft.gemm_cross_entropy_workspace_bytes(loss_args(loss=None, targets=None), 256) > 0


def test_workspace(gemm_lib):
    """Not the logits: two floats for every 32 or 64 words, or a piece's dZ; pieces are as wide as asked."""
    need = dft.gemm_cross_entropy_workspace_bytes
    M, N, K = 8192, 131072, 4096
    far = dict(B=1 << 50, dB=1 << 52, dA=1 << 53)  # (matrices of a gigabyte)
    assert need(loss_args(M, N, K, b_transposed=1, B=1 << 50), 256) == M * (N // 64) * 8 + M * 4
    back = dft.gemm_cross_entropy_grad_workspace_bytes
    whole = back(grad_args(M, N, K, b_transposed=1, **far), 256)
    assert whole < M * N * 2  # (less than the logits in 16 bits)
    least = M * 16 + 256 + M * K * 2 + M * K * 4
    for piece in (256, 1024, 16384):
        got = back(grad_args(M, N, K, b_transposed=1, piece=piece, **far), 256)
        assert got >= least + M * piece * 2 and got < whole
    # an unaligned vocabulary is packed a piece at a time
    assert need(loss_args(24, N + 1, K, B=1 << 50), 256) < (1 << 27) + 24 * 4200 * 8 + 1024
    for M in (0, 1, 7, 100, 5000):
        for N in (1, 8, 99, 1000, 50001):
            for K in (0, 1, 64, 100, 1000):
                for t in (0, 1):
                    assert need(loss_args(M, N, K, b_transposed=t), 256) >= (8 * M if M else 0)
                    assert back(grad_args(M, N, K, b_transposed=t), 256) >= (2 * M * K if M else 0)


def test_torch_refusals(gemm_lib):
    a, b, t = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        dft.linear_cross_entropy(a, b, t)
    with pytest.raises(ValueError, match="GPU"):
        dft.linear_cross_entropy_grad(torch.zeros(4), a, b, t, torch.zeros(4))
    for bad in (a.float(), a.double(), [1.0]):
        with pytest.raises(TypeError):
            dft.linear_cross_entropy(bad, b, t)
        with pytest.raises(TypeError):
            dft.linear_cross_entropy_grad(torch.zeros(4), bad, b, t, torch.zeros(4))


def test_structures_match_the_header(gemm_lib):
    text = (Path(__file__).resolve().parent.parent / "include" / "dense_fp32_tiled.h").read_text()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    kinds = {ctypes.c_void_p: "p", ctypes.c_int64: "int64_t", ctypes.c_int32: "int32_t"}
    for name, struct in (("gemm_cross_entropy_args", dft.CrossEntropyArgs), ("gemm_cross_entropy_grad_args", dft.CrossEntropyGradArgs)):
        body = re.search(r"typedef struct \{([^}]*)\}\s*" + name + ";", text).group(1)
        fields = []
        for line in filter(None, map(str.strip, body.split(";"))):
            kind = "p" if "*" in line else re.match(r"(const )?(\w+)", line).group(2)
            for part in re.sub(r"\b(const|void|float|int\d+_t)\b|\*", " ", line).split(","):
                fields.append((part.strip(), kind))
        assert fields == [(f, kinds[t]) for f, t in struct._fields_]
