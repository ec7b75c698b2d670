"""Refusals and choices of the products with an epilogue and of the token
sort: every bad call is refused on the host, before anything is launched (CPU
only: the addresses are never read)."""

from __future__ import annotations

import ctypes

import pytest
import torch

import dense_fp32_tiled_amd as dft

A, B, D, P, R, Z, W = (0x1000000000 * i for i in range(1, 8))  # far apart, never dereferenced


def linear_args(M=64, N=32, K=48, **kw):
    fields = dict(input_type=dft.INPUT_BF16, output_type=dft.OUTPUT_SAME, activation=dft.ACT_SILU, M=M, N=N, K=K, A=A,
                  lda=max(K, 1), B=B, ldb=max(N, 1), D=D, ldd=max(N, 1))
    fields.update(kw)
    return dft.LinearArgs(**fields)


def grad_args(M=64, N=32, K=48, **kw):
    fields = dict(input_type=dft.INPUT_BF16, activation=dft.ACT_SILU, M=M, N=N, K=K, dY=D, ldy=max(N, 1), Z=Z,
                  ldz=max(N, 1), A=A, lda=max(K, 1), B=B, ldb=max(N, 1), dZ=P, lddz=max(N, 1), dA=R, ldda=max(K, 1),
                  dB=W, lddb=max(N, 1), db_stride=max(K * N, 1))
    fields.update(kw)
    return dft.LinearGradArgs(**fields)


@pytest.mark.parametrize("kw,status", [
    (dict(input_type=2), "UNSUPPORTED"), (dict(input_type=-1), "UNSUPPORTED"), (dict(output_type=2), "UNSUPPORTED"),
    (dict(activation=5), "UNSUPPORTED"), (dict(activation=-1), "UNSUPPORTED"),
    (dict(variant=dft.LINEAR_COUNT), "UNSUPPORTED"), (dict(variant=-1), "UNSUPPORTED"),
    (dict(M=-1), "INVALID_DIM"), (dict(N=-1, ldb=1, ldd=1), "INVALID_DIM"), (dict(K=-1, lda=1), "INVALID_DIM"),
    (dict(splits=33), "INVALID_DIM"), (dict(splits=-1), "INVALID_DIM"), (dict(groups=-1), "INVALID_DIM"),
    (dict(groups=65536, offsets=R, b_stride=48 * 32), "INVALID_DIM"),
    (dict(lda=47), "INVALID_LD"), (dict(ldb=31), "INVALID_LD"), (dict(ldd=31), "INVALID_LD"),
    (dict(residual=R, ldr=31), "INVALID_LD"), (dict(preact=P, ldp=0), "INVALID_LD"),
    (dict(groups=2, offsets=R, b_stride=48 * 32 - 1), "INVALID_LD"),
    (dict(groups=2, offsets=R, b_stride=48 * 32, bias=Z, bias_stride=31), "INVALID_LD"),
    (dict(A=None), "NULL"), (dict(B=None), "NULL"), (dict(D=None), "NULL"),
    (dict(groups=2, b_stride=48 * 32), "NULL"),
    (dict(D=A), "ALIAS"), (dict(D=B + 2 * 48 * 32 - 2), "ALIAS"), (dict(D=A - 2), "ALIAS"),
    (dict(preact=D, ldp=32), "ALIAS"), (dict(preact=A, ldp=32), "ALIAS"), (dict(bias=D + 2), "ALIAS"),
    (dict(residual=D + 2, ldr=32), "ALIAS"), (dict(residual=D, ldr=40), "ALIAS"),
    (dict(residual=P, ldr=32, preact=P, ldp=32), "ALIAS"),
    (dict(workspace=D, workspace_bytes=4), "ALIAS"), (dict(workspace=W, workspace_bytes=-1), "WORKSPACE"),
    (dict(lda=1 << 60), "TOO_LARGE"), (dict(M=1 << 41), "INVALID_DIM"),
    (dict(M=1 << 31, groups=1, offsets=R), "TOO_LARGE"),
    (dict(ldd=(1 << 26) + 1), "TOO_LARGE"), (dict(residual=R, ldr=(1 << 26) + 1), "TOO_LARGE"),
    (dict(preact=P, ldp=(1 << 26) + 1), "TOO_LARGE"),
])
def test_linear_refusals(kw, status, gemm_lib):
    want = getattr(dft, "GEMM_ERR_" + status)
    args = linear_args(**kw)
    assert dft.gemm_linear(args) == want
    if status not in ("WORKSPACE",) and "workspace" not in kw:
        assert dft.gemm_linear_workspace_bytes(args, 256) == want


def test_sizes_without_a_place_in_64_bits(gemm_lib):
    """Products of sizes that the byte counts could not hold are refused, by the queries too."""
    big = 1 << 26
    g = linear_args(M=big, N=big, K=8, lda=8, ldb=big, ldd=big)
    assert dft.gemm_linear_workspace_bytes(g, 256) == dft.GEMM_ERR_TOO_LARGE
    assert dft.gemm_linear(g) == dft.GEMM_ERR_TOO_LARGE
    d = grad_args(M=big, N=big, K=8, ldy=big, lda=8, ldb=big, ldda=8, lddb=big)
    assert dft.gemm_linear_grad_workspace_bytes(d, 256) == dft.GEMM_ERR_TOO_LARGE
    # (matrices so far apart that their rows' elements cannot be counted)
    assert dft.gemm_linear(linear_args(groups=2, offsets=R, ldb=1 << 60, b_stride=1)) == dft.GEMM_ERR_TOO_LARGE


def test_null_arguments(gemm_lib):
    assert gemm_lib.gemm_linear(None, None) == dft.GEMM_ERR_NULL
    assert gemm_lib.gemm_linear_grad(None, None) == dft.GEMM_ERR_NULL
    assert gemm_lib.gemm_linear_workspace_bytes(None, 256) == dft.GEMM_ERR_NULL
    assert gemm_lib.gemm_linear_grad_workspace_bytes(None, 256) == dft.GEMM_ERR_NULL
    assert gemm_lib.gemm_linear_choice(linear_args(), 256, None, None) == dft.GEMM_ERR_NULL
    assert dft.gemm_linear_workspace_bytes(linear_args(), 0) == dft.GEMM_ERR_INVALID_DIM
    assert dft.gemm_linear_grad_workspace_bytes(grad_args(), 0) == dft.GEMM_ERR_INVALID_DIM


def test_empty_outputs_need_nothing(gemm_lib):
    assert dft.gemm_linear(linear_args(M=0, A=None, B=None, D=None)) == dft.GEMM_OK
    assert dft.gemm_linear(linear_args(N=0, A=None, B=None, D=None)) == dft.GEMM_OK


@pytest.mark.parametrize("kw,status", [
    (dict(input_type=7), "UNSUPPORTED"), (dict(activation=9), "UNSUPPORTED"), (dict(a_grad_type=2), "UNSUPPORTED"),
    (dict(b_grad_type=-1), "UNSUPPORTED"), (dict(M=-1), "INVALID_DIM"), (dict(groups=-2), "INVALID_DIM"),
    (dict(ldy=31), "INVALID_LD"), (dict(ldz=31), "INVALID_LD"), (dict(lddz=31), "INVALID_LD"),
    (dict(ldda=47), "INVALID_LD"), (dict(lddb=31), "INVALID_LD"), (dict(lda=1), "INVALID_LD"),
    (dict(groups=2, offsets=0x123000, b_stride=48 * 32, db_stride=5), "INVALID_LD"),
    (dict(dY=None), "NULL"), (dict(Z=None), "NULL"), (dict(dZ=None), "NULL"), (dict(A=None), "NULL"),
    (dict(B=None), "NULL"), (dict(groups=2, b_stride=48 * 32), "NULL"),
    (dict(dA=A), "ALIAS"), (dict(dB=B), "ALIAS"), (dict(dZ=Z), "ALIAS"), (dict(dZ=D + 2), "ALIAS"),
    (dict(dbias=R + 4), "ALIAS"), (dict(workspace=A, workspace_bytes=64), "ALIAS"),
    (dict(workspace_bytes=-4), "WORKSPACE"),
])
def test_grad_refusals(kw, status, gemm_lib):
    assert dft.gemm_linear_grad(grad_args(**kw)) == getattr(dft, "GEMM_ERR_" + status)


def test_grad_ignores_what_it_does_not_read(gemm_lib):
    # (past the checks the call asks for a device, which is not here: anything but these statuses)
    refused = (dft.GEMM_ERR_NULL, dft.GEMM_ERR_INVALID_LD, dft.GEMM_ERR_ALIAS)
    assert dft.gemm_linear_grad_workspace_bytes(grad_args(dB=None, A=None, lda=0), 256) not in refused
    assert dft.gemm_linear_grad_workspace_bytes(grad_args(dA=None, B=None, ldb=0), 256) not in refused
    assert dft.gemm_linear_grad_workspace_bytes(grad_args(activation=0, Z=None, dZ=None, ldz=0, lddz=0), 256) not in refused


def choice(M, N, K, **kw):
    st, variant, splits = dft.gemm_linear_choice(linear_args(M, N, K, **kw), 256)
    assert st == dft.GEMM_OK
    return variant, splits


def test_choice(gemm_lib):
    assert choice(8192, 8192, 8192)[0] == dft.LINEAR_256x256
    assert choice(8192, 8192, 8192)[1] == 1
    assert choice(1000, 999, 513, lda=513)[0] != dft.LINEAR_256x256  # rows of odd width go through registers
    variant, splits = choice(1, 4096, 4096)
    assert variant == dft.LINEAR_32x128 and splits > 1
    assert choice(1, 4096, 0)[1] == 1
    assert choice(64, 2048, 4096, groups=32, offsets=R, b_stride=4096 * 2048)[1] == 1
    for v in range(1, dft.LINEAR_COUNT):
        assert choice(512, 512, 512, variant=v)[0] == v
        assert choice(512, 512, 512, variant=v, splits=4) == (v, 4)
    # no slice is empty: 2 tiles of K cannot be cut into 32
    assert choice(64, 64, 128, splits=32)[1] == 2
    # the workspace holds the slices' partial products
    assert dft.gemm_linear_workspace_bytes(linear_args(512, 512, 512, splits=4), 256) == 4 * 512 * 512 * 4
    assert dft.gemm_linear_workspace_bytes(linear_args(512, 512, 512, splits=1), 256) == 0


def test_every_choice_is_launchable(gemm_lib):
    """Over many sizes: a known tile, whole slices, none empty."""
    for M in (1, 7, 33, 100, 1000, 5000, 100000):
        for N in (1, 8, 99, 1024, 20000):
            for K in (0, 1, 64, 100, 1000, 30000):
                variant, splits = choice(M, N, K)
                assert 1 <= variant < dft.LINEAR_COUNT and 1 <= splits <= 32
                tiles = -(-K // 64)
                if splits > 1:
                    each = -(-tiles // splits)
                    assert (splits - 1) * each < tiles


def test_sort_refusals(gemm_lib):
    def sort(tokens=8, top_k=2, num=4, experts=A, offsets=B, order=D, position=P, ws=None, nbytes=0):
        return dft.gemm_expert_sort(tokens, top_k, num, experts, offsets, order, position, ws, nbytes)

    assert sort(tokens=-1) == dft.GEMM_ERR_INVALID_DIM
    assert sort(top_k=0) == dft.GEMM_ERR_INVALID_DIM
    assert sort(top_k=65) == dft.GEMM_ERR_INVALID_DIM
    assert sort(num=0) == dft.GEMM_ERR_INVALID_DIM
    assert sort(num=1025) == dft.GEMM_ERR_INVALID_DIM
    assert sort(tokens=1 << 31) == dft.GEMM_ERR_TOO_LARGE
    assert sort(experts=None) == dft.GEMM_ERR_NULL
    assert sort(offsets=None) == dft.GEMM_ERR_NULL
    assert sort(order=None) == dft.GEMM_ERR_NULL
    assert sort(position=None) == dft.GEMM_ERR_NULL
    assert sort(order=A) == dft.GEMM_ERR_ALIAS
    assert sort(order=P + 4) == dft.GEMM_ERR_ALIAS
    assert sort(tokens=5000) == dft.GEMM_ERR_WORKSPACE
    assert sort(tokens=5000, ws=W, nbytes=8) == dft.GEMM_ERR_WORKSPACE
    assert sort(tokens=5000, ws=W + 2, nbytes=1 << 20) == dft.GEMM_ERR_WORKSPACE
    assert sort(tokens=5000, ws=A, nbytes=1 << 20) == dft.GEMM_ERR_ALIAS
    assert sort(ws=W, nbytes=-1) == dft.GEMM_ERR_WORKSPACE
    assert dft.gemm_expert_sort_workspace_bytes(2048, 2, 64) == 0
    assert dft.gemm_expert_sort_workspace_bytes(2049, 2, 64) == 2 * 64 * 4
    assert dft.gemm_expert_sort_workspace_bytes(-1, 2, 64) == dft.GEMM_ERR_INVALID_DIM


def test_row_refusals(gemm_lib):
    def gather(kind=0, tokens=4, rows=8, top_k=2, cols=16, X=A, ldx=16, pos=B, out=D, lds=16):
        return dft.gemm_expert_gather(kind, tokens, rows, top_k, cols, X, ldx, pos, out, lds)

    def combine(kind=0, tokens=4, rows=8, top_k=2, cols=16, Y=A, ldy=16, pos=B, w=P, out=D, ldo=16):
        return dft.gemm_expert_combine(kind, tokens, rows, top_k, cols, Y, ldy, pos, w, out, ldo)

    def back(kind=0, tokens=4, rows=8, top_k=2, cols=16, d=A, ldd=16, Y=B, ldy=16, pos=D, w=P, dY=R, lddy=16, dw=W):
        return dft.gemm_expert_combine_grad(kind, tokens, rows, top_k, cols, d, ldd, Y, ldy, pos, w, dY, lddy, dw)

    for call in (gather, combine, back):
        assert call(kind=2) == dft.GEMM_ERR_UNSUPPORTED
        assert call(tokens=-1) == dft.GEMM_ERR_INVALID_DIM
        assert call(rows=-1) == dft.GEMM_ERR_INVALID_DIM
        assert call(top_k=0) == dft.GEMM_ERR_INVALID_DIM
        assert call(top_k=65) == dft.GEMM_ERR_INVALID_DIM
        assert call(cols=-1) == dft.GEMM_ERR_INVALID_DIM
        assert call(rows=1 << 32) == dft.GEMM_ERR_TOO_LARGE
        assert call(pos=None) == dft.GEMM_ERR_NULL
        assert call(tokens=0, pos=None) == dft.GEMM_OK
    assert gather(ldx=15) == gather(lds=15) == combine(ldy=15) == combine(ldo=15) == dft.GEMM_ERR_INVALID_LD
    assert back(ldd=15) == back(ldy=15) == back(lddy=15) == dft.GEMM_ERR_INVALID_LD
    assert gather(X=None) == gather(out=None) == combine(Y=None) == combine(out=None) == dft.GEMM_ERR_NULL
    assert back(d=None) == back(Y=None) == dft.GEMM_ERR_NULL
    assert gather(out=A) == combine(out=A) == combine(out=P) == back(dY=A) == back(dY=B) == back(dw=P) == dft.GEMM_ERR_ALIAS
    assert back(dY=None, dw=None) == dft.GEMM_OK  # nothing wanted


def test_torch_refusals(gemm_lib):
    """The torch functions refuse tensors that are not on a GPU, of other types, shapes or layouts."""
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        dft.linear(x, w)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        dft.linear(x.float(), w)
    with pytest.raises(TypeError):
        dft.linear([1.0], w)
    with pytest.raises(ValueError, match="GPU"):
        dft.linear_grad(torch.zeros(4, 16, dtype=torch.bfloat16), x, w)
    with pytest.raises(TypeError):
        dft.grouped_linear(x, w, None)
    with pytest.raises(TypeError):
        dft.grouped_linear_grad(x, x, w, None)
    with pytest.raises(ValueError, match="GPU"):
        dft.expert_sort(torch.zeros(4, 2, dtype=torch.int32), 4)
    with pytest.raises(TypeError):
        dft.expert_sort(torch.zeros(4, dtype=torch.int32), 4)
    position = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: dft.expert_gather(x, position), lambda: dft.expert_combine(x, position),
                 lambda: dft.expert_combine_grad(x, x, position)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        dft.expert_mlp(x, position, None, w, w)


def test_structures_match_the_header(gemm_lib):
    """Field names and order of the ctypes structures against the header's."""
    import re
    from pathlib import Path

    text = (Path(__file__).resolve().parent.parent / "include" / "dense_fp32_tiled.h").read_text()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, struct in (("gemm_linear_args", dft.LinearArgs), ("gemm_linear_grad_args", dft.LinearGradArgs)):
        body = re.search(r"typedef struct \{([^}]*)\}\s*" + name + ";", text).group(1)
        fields = []
        for line in body.split(";"):
            line = line.strip()
            if not line:
                continue
            kind = "p" if "*" in line else "i64" if "int64_t" in line else "i32"
            for part in re.sub(r"(const|void|float|int32_t|int64_t|\*)", " ", line).split(","):
                fields.append((part.strip(), kind))
        kinds = {ctypes.c_void_p: "p", ctypes.c_int64: "i64", ctypes.c_int32: "i32"}
        assert fields == [(f, kinds[t]) for f, t in struct._fields_]


@pytest.mark.parametrize("kw", [
    dict(A=D), dict(A=D + 2), dict(B=D), dict(B=D + 2), dict(Z=D), dict(Z=D + 2), dict(dA=D + 4), dict(dbias=D),
    dict(groups=2, offsets=D, b_stride=48 * 32, db_stride=48 * 32), dict(workspace=D + 16, workspace_bytes=64),
], ids=lambda kw: "-".join(kw))
def test_grad_in_place_overlaps_nothing_else(kw, gemm_lib):
    """dZ over dY is written like any other output: what else the call reads or writes may not lie there."""
    in_place = grad_args(dZ=D)
    assert dft.gemm_linear_grad_workspace_bytes(in_place, 256) >= 0
    args = grad_args(dZ=D, **kw)
    assert dft.gemm_linear_grad(args) == dft.GEMM_ERR_ALIAS
    if "workspace" not in kw:
        assert dft.gemm_linear_grad_workspace_bytes(args, 256) == dft.GEMM_ERR_ALIAS


MOST_TILES = 2 ** 22 - 1  # workgroups of a launch
SIZES = {dft.LINEAR_256x256: (256, 256), dft.LINEAR_128x128: (128, 128), dft.LINEAR_64x64: (64, 64), dft.LINEAR_32x128: (32, 128)}


@pytest.mark.parametrize("M,N,K", [(1 << 28, 8, 8), (300_000_000, 8, 8), (300_000_000, 64, 64), ((1 << 28) + 5, 9, 7),
                                   (1, 1 << 26, 8), (1 << 29, 30, 1), (1000, 60_000_000, 16)])
def test_large_sizes_take_a_tile_that_a_launch_holds(M, N, K, gemm_lib):
    variant, splits = choice(M, N, K)
    bm, bn = SIZES[variant]
    assert -(-M // bm) * -(-N // bn) * splits <= MOST_TILES
    assert dft.gemm_linear_workspace_bytes(linear_args(M, N, K), 256) >= 0
    assert dft.gemm_linear_grad_workspace_bytes(grad_args(M, N, K, activation=0, Z=None, dZ=None), 256) >= 0


def test_sizes_that_no_launch_holds(gemm_lib):
    """Refused by the queries as by the calls."""
    for kw in (dict(M=1 << 31, N=1, K=1), dict(M=1 << 28, N=64, K=64, variant=dft.LINEAR_64x64),
               dict(M=1 << 28, N=64, K=64, variant=dft.LINEAR_64x64, splits=2)):
        assert dft.gemm_linear_workspace_bytes(linear_args(**kw), 256) == dft.GEMM_ERR_TOO_LARGE
        assert dft.gemm_linear_choice(linear_args(**kw), 256)[0] == dft.GEMM_ERR_TOO_LARGE

    def grouped(n):  # the weights' gradient: the groups' tiles together
        return grad_args(M=64, N=n, K=n, groups=65535, offsets=0x123000, b_stride=n * n, db_stride=n * n, A=1 << 60,
                         B=1 << 61, dB=1 << 62, activation=0, Z=None, dZ=None)

    assert dft.gemm_linear_grad_workspace_bytes(grouped(1792), 256) >= 0  # 49 tiles of 256x256 each
    assert dft.gemm_linear_grad_workspace_bytes(grouped(2304), 256) == dft.GEMM_ERR_TOO_LARGE


def test_gradient_sizes_that_the_slopes_take(gemm_lib):
    def need(M, N, K=1, **kw):
        return dft.gemm_linear_grad_workspace_bytes(grad_args(M, N, K, dA=None, B=None, **kw), 256)

    plain = dict(activation=0, Z=None, dZ=None)
    assert need(2, 5_000_000) >= 0
    assert need(2, 65535 * 256) >= 0
    assert need(2, 65535 * 256 + 1) == dft.GEMM_ERR_TOO_LARGE
    assert need(2, 65535 * 256 + 1, **plain) >= 0
    assert need(2, 65535 * 256 + 1, dbias=0x123000, **plain) == dft.GEMM_ERR_TOO_LARGE
    assert need((1 << 29) - 64, 1) >= 0
    assert need((1 << 29) - 63, 1) == dft.GEMM_ERR_TOO_LARGE
    assert need((1 << 29) - 63, 1, **plain) >= 0
    assert need((1 << 29), 0) == 0


def test_few_rows_of_many_groups_need_little(gemm_lib):
    """Only as many groups have rows as there are rows: what a call takes of the workspace and of a launch goes by
    those."""
    def forward(M, groups, N, K, **kw):
        return linear_args(M, N, K, groups=groups, offsets=0x123000, b_stride=K * N, A=1 << 58, B=1 << 60, D=1 << 59, **kw)

    # one row: one tile row, with a whole round of 256x256 tiles or without
    assert dft.gemm_linear_workspace_bytes(forward(1, 65535, 8192, 4096, variant=dft.LINEAR_256x256), 256) == 0
    assert dft.gemm_linear_choice(forward(1, 65535, 65536, 64), 256)[0] == dft.GEMM_OK
    assert dft.gemm_linear_workspace_bytes(forward(1, 65535, 65536, 64), 256) == 0
    # the bias's gradient: one chunk of sums a row
    for M in (1, 5, 300):
        g = grad_args(M=M, N=8192, K=64, groups=65535, offsets=0x123000, b_stride=64 * 8192, A=1 << 58, B=1 << 60,
                      dA=None, dB=None, dbias=1 << 59)
        assert dft.gemm_linear_grad_workspace_bytes(g, 256) == M * 8192 * 4
