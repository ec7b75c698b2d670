"""gemm_linear and gemm_linear_grad on the GPU against float64: every tile,
type, activation and alignment, ragged sizes, slices of K, groups with empty
and uncovered rows, values that are not finite.  Integer-valued operands must
match bit for bit, and run through the LDS-poison build as well; every buffer
is NaN outside the matrices.  The bounds are derived in linear_reference."""

from __future__ import annotations

import math
import threading

import pytest
import torch

import dense_fp32_tiled_amd as dft
import linear_reference as ref
from dense_fp32_tiled_amd import build

pytestmark = pytest.mark.gpu

TILES = [dft.LINEAR_256x256, dft.LINEAR_128x128, dft.LINEAR_64x64, dft.LINEAR_32x128]
TILE_IDS = [dft.LINEAR_NAMES[v] for v in TILES]


@pytest.fixture(scope="module")
def libs(gemm_lib):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return {"plain": gemm_lib, "poison": dft.library(build.POISON_LIB)}


# (M, N, K, pads of A, B, D and Z, first element's offset): 16-byte rows with ragged tile edges and K tails, then
# widths, pitches and addresses that are not multiples of 16 bytes
SHAPES = [
    (1, 8, 8, (0, 0, 0, 0), 0),
    (1, 264, 72, (0, 8, 0, 0), 0),
    (33, 136, 200, (8, 0, 8, 8), 0),
    (257, 264, 64, (0, 0, 0, 0), 0),
    (300, 520, 328, (8, 8, 3, 1), 8),
    (130, 1, 5, (0, 0, 0, 0), 0),
    (67, 129, 65, (1, 2, 3, 4), 0),
    (259, 131, 130, (0, 3, 0, 0), 1),
    (5, 40, 16, (4, 0, 0, 0), 0),
    (70, 300, 0, (0, 0, 0, 0), 0),
]


@pytest.mark.parametrize("which", ["plain", "poison"])
@pytest.mark.parametrize("kind", list(ref.TYPES))
@pytest.mark.parametrize("tile", TILES, ids=TILE_IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:3])))
def test_forward_integers_are_exact(shape, tile, kind, which, libs):
    M, N, K, pad, offset = shape
    gen = torch.Generator().manual_seed(M * 7 + N * 3 + K)
    dtype = ref.TYPES[kind]
    a, b = ref.draw(gen, (M, K), dtype, True), ref.draw(gen, (1, K, N), dtype, True)
    bias, residual = ref.draw(gen, (1, N), dtype, True), ref.draw(gen, (M, N), torch.float32, True)
    d, _ = ref.run_forward(libs[which], a, b, bias=bias, residual=residual, kind="relu", out_dtype=torch.float32,
                           variant=tile, splits=1, pad=pad, offset=offset)
    want = ref.act(a.double() @ b[0].double() + bias[0].double(), "relu") + residual.double()
    assert torch.equal(d.double(), want)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("kind", list(ref.TYPES))
@pytest.mark.parametrize("out32", [False, True], ids=["same", "f32"])
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[4], SHAPES[6]], ids=lambda s: "x".join(map(str, s[:3])))
def test_forward_epilogue(shape, out32, kind, act, libs):
    M, N, K, pad, offset = shape
    gen = torch.Generator().manual_seed(11)
    dtype = ref.TYPES[kind]
    out = torch.float32 if out32 else dtype
    a, b = ref.draw(gen, (M, K), dtype), ref.draw(gen, (1, K, N), dtype, scale=2 * K ** -0.5)
    bias, residual = ref.draw(gen, (1, N), dtype), ref.draw(gen, (M, N), out)
    d, z = ref.run_forward(libs["plain"], a, b, bias=bias, residual=residual, kind=act, out_dtype=out, keep=True,
                           pad=pad, offset=offset)
    want_d, want_z = ref.forward(a, b, bias=bias, residual=residual, kind=act, out_dtype=out)
    ref.assert_within(d, want_d, "D")
    ref.assert_within(z, want_z, "Z")
    # no bias, no residual, D alone
    d, _ = ref.run_forward(libs["plain"], a, b, kind=act, out_dtype=out, pad=pad, offset=offset)
    ref.assert_within(d, ref.forward(a, b, kind=act, out_dtype=out)[0], "D alone")


@pytest.mark.parametrize("which", ["plain", "poison"])
@pytest.mark.parametrize("splits", [2, 3, 8, 32])
@pytest.mark.parametrize("tile", TILES, ids=TILE_IDS)
def test_forward_slices(tile, splits, which, libs):
    gen = torch.Generator().manual_seed(12)
    for M, N, K, pad in [(3, 264, 1000, (0, 0, 0, 0)), (130, 75, 705, (1, 0, 2, 0)), (65, 128, 64, (0, 0, 0, 0))]:
        a, b = ref.draw(gen, (M, K), torch.bfloat16, True), ref.draw(gen, (1, K, N), torch.bfloat16, True)
        bias, residual = ref.draw(gen, (1, N), torch.bfloat16, True), ref.draw(gen, (M, N), torch.float32, True)
        d, z = ref.run_forward(libs[which], a, b, bias=bias, residual=residual, kind="relu", out_dtype=torch.float32,
                               variant=tile, splits=splits, pad=pad, keep=True)
        zw = a.double() @ b[0].double() + bias[0].double()
        assert torch.equal(d.double(), zw.clamp(min=0) + residual.double())
        assert torch.equal(z, zw.to(torch.bfloat16))


def test_forward_residual_in_place(libs):
    gen = torch.Generator().manual_seed(13)
    for splits in (1, 4):
        a, b = ref.draw(gen, (37, 512), torch.bfloat16), ref.draw(gen, (1, 512, 200), torch.bfloat16, scale=0.05)
        r = ref.draw(gen, (37, 200), torch.bfloat16)
        d, _ = ref.run_forward(libs["plain"], a, b, residual=r, kind="silu", splits=splits, in_place=True)
        ref.assert_within(d, ref.forward(a, b, residual=r, kind="silu")[0], "D over its residual")


# rows per group (uncovered rows first and last are added), K, N, pads
GROUPS = [
    ([5, 0, 1, 40, 0, 0, 7], 64, 128, (0, 0, 0, 0)),
    ([300, 1, 257, 64], 72, 136, (8, 8, 0, 0)),
    ([0, 0, 0], 32, 40, (0, 0, 0, 0)),
    ([33, 31, 2], 37, 45, (1, 2, 3, 0)),
    ([1] * 130, 40, 24, (0, 0, 0, 0)),
]


def group_case(gen, counts, K, N, dtype, integer):
    offsets = [3]
    for c in counts:
        offsets.append(offsets[-1] + c)
    M = offsets[-1] + 6
    a, b = ref.draw(gen, (M, K), dtype, integer), ref.draw(gen, (len(counts), K, N), dtype, integer, K ** -0.5)
    # rows in no group hold NaN: they may not reach any result
    a[:3], a[M - 6:] = math.nan, math.nan
    return offsets, M, a, b


@pytest.mark.parametrize("which", ["plain", "poison"])
@pytest.mark.parametrize("tile", [0, *TILES], ids=["auto", *TILE_IDS])
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_grouped_forward(case, tile, which, libs):
    counts, K, N, pad = GROUPS[case]
    gen = torch.Generator().manual_seed(20 + case)
    for integer in (True, False):
        offsets, M, a, b = group_case(gen, counts, K, N, torch.bfloat16, integer)
        bias = ref.draw(gen, (len(counts), N), torch.bfloat16, integer)
        d, z = ref.run_forward(libs[which], a, b, offsets=offsets, bias=bias, kind="relu" if integer else "gelu",
                               out_dtype=torch.float32 if integer else None, variant=tile, pad=pad, keep=True)
        want_d, want_z = ref.forward(a, b, offsets, bias, kind="relu" if integer else "gelu",
                                     out_dtype=torch.float32 if integer else None)
        if integer:
            known = ~torch.isnan(want_d[0])
            assert torch.equal(d.double()[known], want_d[0][known])
        ref.assert_within(d, want_d, "D")
        ref.assert_within(z, want_z, "Z")


@pytest.mark.parametrize("offsets", [[-5, 4, 2, 90], [0, 100, 1000, 2000], [70, 80, 60, 64], [2 ** 31 - 1, -2 ** 31, 5, 9]])
def test_offsets_outside_the_rows_are_clamped(offsets, libs):
    gen = torch.Generator().manual_seed(30)
    a, b = ref.draw(gen, (64, 48), torch.bfloat16, True), ref.draw(gen, (3, 48, 72), torch.bfloat16, True)
    d, _ = ref.run_forward(libs["plain"], a, b, offsets=offsets, out_dtype=torch.float32)
    want = ref.forward(a, b, offsets, out_dtype=torch.float32)[0][0]
    # two groups that claim one row: either may write it
    claims = sum((torch.arange(64) >= lo) & (torch.arange(64) < hi) for _, lo, hi in ref.ranges(offsets, 3, 64))
    once = (claims == 1) if torch.is_tensor(claims) else torch.zeros(64, dtype=torch.bool)
    assert torch.equal(d.double()[once], want[once])


GRAD_SHAPES = [
    (1, 8, 8, (0, 0, 0, 0), 0),
    (70, 136, 200, (8, 8, 8, 0), 0),
    (300, 264, 328, (0, 0, 0, 0), 8),
    (67, 129, 65, (1, 2, 3, 4), 0),
    (513, 75, 33, (0, 0, 0, 0), 1),
]


@pytest.mark.parametrize("which", ["plain", "poison"])
@pytest.mark.parametrize("kind", list(ref.TYPES))
@pytest.mark.parametrize("shape", GRAD_SHAPES, ids=lambda s: "x".join(map(str, s[:3])))
def test_grad_integers_are_exact(shape, kind, which, libs):
    M, N, K, pad, offset = shape
    gen = torch.Generator().manual_seed(40 + M)
    dtype = ref.TYPES[kind]
    a, b, dy = (ref.draw(gen, s, dtype, True) for s in ((M, K), (1, K, N), (M, N)))
    z = ref.draw(gen, (M, N), dtype, True)
    for act in ("none", "relu"):
        g = ref.run_grad(libs[which], dy, a, b, preact=z, kind=act, a_dtype=torch.float32, b_dtype=torch.float32,
                         pad=pad, offset=offset)
        dz = dy.double() * ref.slope(z.double(), act)
        if act != "none":
            assert torch.equal(g["dz"].double(), dz)
        assert torch.equal(g["a"].double(), dz @ b[0].double().t())
        assert torch.equal(g["b"][0].double(), a.double().t() @ dz)
        assert torch.equal(g["bias"][0].double(), dz.sum(0))


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("kind", list(ref.TYPES))
@pytest.mark.parametrize("shape", GRAD_SHAPES, ids=lambda s: "x".join(map(str, s[:3])))
def test_grad(shape, kind, act, libs):
    M, N, K, pad, offset = shape
    gen = torch.Generator().manual_seed(50 + M)
    dtype = ref.TYPES[kind]
    a, b = ref.draw(gen, (M, K), dtype), ref.draw(gen, (1, K, N), dtype, scale=K ** -0.5)
    dy, z = ref.draw(gen, (M, N), dtype), ref.draw(gen, (M, N), dtype, scale=2.0)
    want = ref.grad(dy, a, b, preact=z, kind=act)
    g = ref.run_grad(libs["plain"], dy, a, b, preact=z, kind=act, pad=pad, offset=offset)
    for name in g:
        ref.assert_within(g[name], want[name], name)
    if act != "none":  # dZ over dY, and each gradient by itself
        g = ref.run_grad(libs["plain"], dy, a, b, preact=z, kind=act, pad=pad, offset=offset, in_place=True)
        for name in g:
            ref.assert_within(g[name], want[name], f"{name} (in place)")
    for one in ("a", "b", "bias"):
        g = ref.run_grad(libs["plain"], dy, a, b, preact=z, kind=act, want=(one,), pad=pad, offset=offset)
        ref.assert_within(g[one], want[one], f"{one} alone")


@pytest.mark.parametrize("which", ["plain", "poison"])
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_grouped_grad(case, which, libs):
    counts, K, N, pad = GROUPS[case]
    gen = torch.Generator().manual_seed(60 + case)
    for act in ("none", "silu"):
        offsets, M, a, b = group_case(gen, counts, K, N, torch.bfloat16, False)
        dy, z = ref.draw(gen, (M, N), torch.bfloat16), ref.draw(gen, (M, N), torch.bfloat16)
        dy[:3], dy[M - 6:] = math.nan, math.nan
        g = ref.run_grad(libs[which], dy, a, b, offsets=offsets, preact=z, kind=act, pad=pad, b_dtype=torch.float32)
        want = ref.grad(dy, a, b, offsets, z, act, b_dtype=torch.float32)
        for name in g:
            ref.assert_within(g[name], want[name], name)


def test_many_rows_per_group_sum_in_slices(libs):
    """Few outputs and a long contraction: dB of one matrix is sliced along M."""
    gen = torch.Generator().manual_seed(70)
    M, N, K = 5000, 72, 64
    a, b, dy = (ref.draw(gen, s, torch.bfloat16, True) for s in ((M, K), (1, K, N), (M, N)))
    g = ref.run_grad(libs["plain"], dy, a, b, b_dtype=torch.float32, a_dtype=torch.float32)
    assert torch.equal(g["b"][0].double(), a.double().t() @ dy.double())
    assert torch.equal(g["bias"][0].double(), dy.double().sum(0))


@pytest.mark.parametrize("M", [2, 16, 17, 32, 33, 64, 65])
@pytest.mark.parametrize("N", [8, 300])
def test_bias_of_few_rows(M, N, libs):
    """dbias of one chunk of rows and of a few, with and without an activation: whole numbers, exact."""
    gen = torch.Generator().manual_seed(77 + M)
    a, b, dy = (ref.draw(gen, s, torch.bfloat16, True) for s in ((M, 16), (1, 16, N), (M, N)))
    z = ref.draw(gen, (M, N), torch.bfloat16, True)
    for which in ("plain", "poison"):
        for act in ("none", "relu"):
            g = ref.run_grad(libs[which], dy, a, b, preact=z, kind=act, want=("bias",))
            assert torch.equal(g["bias"][0].double(), (dy.double() * ref.slope(z.double(), act)).sum(0)), (which, act)


def test_last_round_in_slices(libs):
    """More 256x256 tiles than CUs and a deep contraction: the tiles of the last round are cut along it and joined.
    Integer values, against float64 on the GPU (exact): forward, dA and dB, dense and grouped."""
    torch.manual_seed(74)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    N, K = 4096, 2112
    M = 256 * (cus // 16) + 200  # a row of 16 tiles past whole rounds, its rows ragged

    def ints(*shape):
        return torch.randint(-3, 4, shape, device="cuda").to(torch.bfloat16)

    a, b, bias, r = ints(M, K), ints(K, N), ints(N), ints(M, N).float()
    z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    d = dft.linear(a, b, bias=bias, residual=r, activation="relu", out_dtype=torch.float32, preact=z,
                   variant=dft.LINEAR_256x256, splits=1)
    want = a.double() @ b.double() + bias.double()
    assert torch.equal(d.double(), want.clamp(min=0) + r.double())
    assert torch.equal(z, want.to(torch.bfloat16))
    # groups: rows in none first and last, an empty one, one of a single row
    counts = [700, 0, 1, 1500, 257, 300]
    counts.append(M - 13 - sum(counts))
    offsets = torch.tensor([5, *[5 + sum(counts[: i + 1]) for i in range(len(counts))]], dtype=torch.int32, device="cuda")
    bg, biasg = ints(len(counts), K, N), ints(len(counts), N)
    out = torch.full((M, N), 7.0, device="cuda")
    dft.grouped_linear(a, bg, offsets, bias=biasg, activation="relu", out=out, variant=dft.LINEAR_256x256)
    lo = 5
    for g, c in enumerate(counts):
        want = (a[lo:lo + c].double() @ bg[g].double() + biasg[g].double()).clamp(min=0)
        assert torch.equal(out[lo:lo + c].double(), want), g
        lo += c
    assert bool((out[:5] == 7).all()) and bool((out[lo:] == 7).all())
    # the gradients' products: dA is M x K from N columns, dB (of transposed sizes) from M rows
    dy = ints(M, N)
    b2 = ints(4096, N)
    g = dft.linear_grad(dy, ints(M, 4096), b2, want=("a",), a_dtype=torch.float32)
    assert torch.equal(g.a.double(), dy.double() @ b2.double().t())
    x = ints(2112, M)
    dy2 = ints(2112, 4096)
    g = dft.linear_grad(dy2, x, ints(M, 4096), want=("b",), b_dtype=torch.float32)
    assert torch.equal(g.b.double(), x.double().t() @ dy2.double())


def test_slices_when_groups_fill_less_than_a_round(libs):
    """Rows counted for more 256x256 tiles than CUs, but in few groups (or none): every tile there is gets cut."""
    torch.manual_seed(76)
    M, N, K, groups = 600, 1024, 2112, 80
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert (M + groups * 255) // 256 * (N // 256) > cus
    a = torch.randint(-3, 4, (M, K), device="cuda").to(torch.bfloat16)
    b = torch.randint(-3, 4, (groups, K, N), device="cuda").to(torch.bfloat16)
    for first, second in ((300, 290), (1, 0), (0, 0), (0, 600)):
        offsets = torch.full((groups + 1,), first, dtype=torch.int32, device="cuda")
        offsets[0], offsets[groups] = 0, first + second
        out = torch.full((M, N), 5.0, device="cuda")
        dft.grouped_linear(a, b, offsets, out=out, variant=dft.LINEAR_256x256)
        for g, lo, hi in ((0, 0, first), (groups - 1, first, first + second)):
            assert torch.equal(out[lo:hi].double(), a[lo:hi].double() @ b[g].double())
        assert bool((out[first + second:] == 5).all())


@pytest.mark.parametrize("grouped", [False, True], ids=["one", "grouped"])
def test_odd_widths_are_packed(grouped, libs):
    """Products large enough that operands of odd widths are copied to rows of whole 16 bytes first (which takes
    workspace), forward and gradients, B's matrices apart: integer values, exact."""
    torch.manual_seed(75)
    counts = [300, 0, 1, 517] if grouped else [818]
    M, N, K, E = sum(counts) + 7, 777, 1001, len(counts)

    def ints(*shape):
        return torch.randint(-2, 3, shape, device="cuda").to(torch.float16)

    a, dy = ints(M, K + 1)[:, 1:], ints(M, N)
    b, bias = ints(E, K + 2, N)[:, :K], ints(E, N)
    lo, hi = (3, M - 4) if grouped else (0, M)
    offsets = torch.tensor([3 + sum(counts[:i]) for i in range(E + 1)], dtype=torch.int32, device="cuda")
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    g = dft.LinearArgs(input_type=dft.INPUT_F16, splits=1, groups=E if grouped else 0, M=M, N=N, K=K, A=a.data_ptr(),
                       lda=K + 1, B=b.data_ptr(), ldb=N, b_stride=(K + 2) * N, offsets=offsets.data_ptr(), D=1 << 46,
                       ldd=N)
    assert dft.gemm_linear_workspace_bytes(g, cus) >= 2 * M * (K + 7)
    if grouped:
        out = torch.full((M, N), 9.0, device="cuda")
        dft.grouped_linear(a, b, offsets, bias=bias, out=out)
        grads = dft.grouped_linear_grad(dy, a, b, offsets, a_dtype=torch.float32, b_dtype=torch.float32)
        assert bool((out[:lo] == 9).all()) and bool((out[hi:] == 9).all())
    else:
        out = dft.linear(a, b[0], bias=bias[0], out_dtype=torch.float32)
        grads = dft.linear_grad(dy, a, b[0], a_dtype=torch.float32, b_dtype=torch.float32)
        grads = grads._replace(b=grads.b[None], bias=grads.bias[None])
        counts[0] = M
    for e, c in enumerate(counts):
        A, D = a[lo:lo + c].double(), dy[lo:lo + c].double()
        assert torch.equal(out[lo:lo + c].double(), A @ b[e].double() + bias[e].double()), e
        assert torch.equal(grads.a[lo:lo + c].double(), D @ b[e].double().t()), e
        assert torch.equal(grads.b[e].double(), A.t() @ D), e
        assert torch.equal(grads.bias[e].double(), D.sum(0)), e
        lo += c


def test_empty_sizes(libs):
    gen = torch.Generator().manual_seed(71)
    lib = libs["plain"]
    for M, N, K in [(0, 16, 8), (4, 0, 8), (4, 16, 0), (0, 0, 0)]:
        a, b, dy = (ref.draw(gen, s, torch.bfloat16) for s in ((M, K), (1, K, N), (M, N)))
        ref.run_forward(lib, a, b)
        g = ref.run_grad(lib, dy, a, b)
        want = ref.grad(dy, a, b)
        for name in g:
            assert torch.equal(g[name].double(), want[name][0]), (M, N, K, name)


def test_values_that_are_not_finite(libs):
    """A NaN or infinity in one row of A (one column of B) reaches that row (column) alone, at every tile."""
    gen = torch.Generator().manual_seed(72)
    a, b = ref.draw(gen, (70, 72), torch.bfloat16), ref.draw(gen, (1, 72, 136), torch.bfloat16)
    a[31, 5], a[64, 70] = math.nan, math.inf
    b[0, 9, 130] = math.nan
    for tile in TILES:
        d, _ = ref.run_forward(libs["plain"], a, b, variant=tile, splits=1)
        want = a.double() @ b[0].double()
        assert torch.equal(torch.isnan(d), torch.isnan(want))
        assert torch.equal(torch.isinf(d), torch.isinf(want))
        fine = torch.isfinite(want)
        a2, b2 = torch.nan_to_num(a, 0, 0, 0), torch.nan_to_num(b, 0, 0, 0)
        value, tol = ref.forward(a2, b2)[0]
        assert bool(((d.double() - value).abs()[fine] <= tol[fine]).all())


def test_activations_far_out(libs):
    """Large pre-activations: act and its slope keep their limits."""
    z = torch.tensor([-3e38, -1e20, -200.0, -120.0, -30.0, -0.0, 0.0, 30.0, 120.0, 200.0, 1e20, 3e38])
    n = z.numel()
    b = torch.zeros(1, 8, n, dtype=torch.bfloat16)
    a = torch.zeros(2, 8, dtype=torch.bfloat16)
    bias = z.to(torch.bfloat16).reshape(1, n)
    dy = torch.ones(2, n, dtype=torch.bfloat16)
    zz = bias.expand(2, n).contiguous()
    for act in ref.ACTS:
        d, _ = ref.run_forward(libs["plain"], a, b, bias=bias, kind=act, out_dtype=torch.float32)
        ref.assert_within(d, ref.forward(a, b, bias=bias, kind=act, out_dtype=torch.float32)[0], act)
        g = ref.run_grad(libs["plain"], dy, a, b, preact=zz, kind=act, want=("bias",))
        if act != "none":
            assert bool(torch.isfinite(g["dz"]).all()), act
            want = torch.where(z.double().abs() < 100, ref.slope(bias[0].double().clamp(-100, 100), act),
                               (bias[0].double() > 0).double())
            assert bool(((g["dz"][0].double() - want).abs() <= 2.0 ** -8).all()), act


def test_gradients_against_differences(libs):
    """The GPU's gradients of sum(G * D) against central differences of the float64 definition.  With step h the
    difference is off by at most h^2 / 6 times the third derivative along the step (below 60 here: 1e-6 of it) and
    2^-53 / h times the sum's size; 1e-4 covers both beside the fp32 gradients' own 1e-5."""
    gen = torch.Generator().manual_seed(73)
    M, N, K = 9, 24, 16
    a, b = ref.draw(gen, (M, K), torch.bfloat16), ref.draw(gen, (1, K, N), torch.bfloat16, scale=0.25)
    bias, dy = ref.draw(gen, (1, N), torch.bfloat16), ref.draw(gen, (M, N), torch.bfloat16)
    for act in ("gelu", "gelu_tanh", "silu"):
        def loss(A, B, c):
            return (dy.double() * ref.act(A @ B + c, act)).sum()

        A, B, c = a.double(), b[0].double(), bias[0].double()
        # preact in 16 bits would move the slopes: take a bias that makes it exact
        zb = (A @ B + c).to(torch.bfloat16)
        shift = zb.double() - A @ B  # one bias per element: the loss below uses it, the gradients read zb

        def shifted(A_, B_):
            return (dy.double() * ref.act(A_ @ B_ + shift, act)).sum()

        g = ref.run_grad(libs["plain"], dy, a, b, preact=zb, kind=act, a_dtype=torch.float32, b_dtype=torch.float32)
        dz_round = (2.0 ** -8) * (dy.double().abs() * 1.13)  # dZ's rounding, through the products
        h = 1e-4
        for i, j in [(0, 0), (3, 7), (8, 15)]:
            up, down = A.clone(), A.clone()
            up[i, j] += h
            down[i, j] -= h
            slope = (shifted(up, B) - shifted(down, B)) / (2 * h)
            tol = float((dz_round[i] * B[j].abs()).sum()) + 1e-4
            assert abs(float(g["a"][i, j]) - float(slope)) <= tol
        for i, j in [(0, 0), (5, 9), (15, 23)]:
            up, down = B.clone(), B.clone()
            up[i, j] += h
            down[i, j] -= h
            slope = (shifted(A, up) - shifted(A, down)) / (2 * h)
            tol = float((dz_round[:, j] * A[:, i].abs()).sum()) + 1e-4
            assert abs(float(g["b"][0, i, j]) - float(slope)) <= tol
        assert float(loss(A, B, c)) == float(loss(A, B, c))


def test_offsets_past_31_bits(libs):
    """A pitch that puts a tile's rows beyond 2^31 bytes (loads through registers), and an output of more than 2^31
    elements."""
    dev = "cuda"
    M, N, K, ld = 300, 64, 64, 8_000_008
    big = torch.empty(M * ld, dtype=torch.bfloat16, device=dev)
    a = big.as_strided((M, K), (ld, 1))
    a.copy_(torch.randint(-3, 4, (M, K), device=dev))
    b = torch.randint(-3, 4, (K, N), device=dev).to(torch.bfloat16)
    d = dft.linear(a, b, out_dtype=torch.float32)
    assert torch.equal(d.cpu().double(), a.cpu().double() @ b.cpu().double())
    del big, a
    M, N, K = 66000, 33000, 64
    a = torch.randint(-3, 4, (M, K), device=dev).to(torch.bfloat16)
    b = torch.randint(-3, 4, (K, N), device=dev).to(torch.bfloat16)
    d = dft.linear(a, b)  # sums of 64 products of at most 9: 576, exact in fp32 and rounded once
    rows = torch.tensor([0, 1, 255, 256, 40000, M - 2, M - 1], device=dev)
    want = (a[rows].double().cpu() @ b.double().cpu()).to(torch.bfloat16)
    assert torch.equal(d[rows].cpu(), want)


@pytest.mark.parametrize("M", [1, 2, 24, 200])
def test_serving_sizes(M, libs):
    """Few rows, wide weights, the automatic tile and slices: against float64."""
    gen = torch.Generator().manual_seed(80 + M)
    a, b = ref.draw(gen, (M, 2048), torch.bfloat16), ref.draw(gen, (1, 2048, 1024), torch.bfloat16, scale=0.03)
    bias, r = ref.draw(gen, (1, 1024), torch.bfloat16), ref.draw(gen, (M, 1024), torch.bfloat16)
    d, _ = ref.run_forward(libs["plain"], a, b, bias=bias, residual=r, kind="silu")
    ref.assert_within(d, ref.forward(a, b, bias=bias, residual=r, kind="silu")[0], "D")


def test_python_entry_points_match_float64(libs):
    gen = torch.Generator().manual_seed(81)
    x, w = ref.draw(gen, (50, 96), torch.float16), ref.draw(gen, (96, 200), torch.float16, scale=0.1)
    bias, r, dy = ref.draw(gen, (200,), torch.float16), ref.draw(gen, (50, 200), torch.float16), \
        ref.draw(gen, (50, 200), torch.float16)
    X, W, B, R, DY = (t.cuda() for t in (x, w, bias, r, dy))
    z = torch.empty_like(R)
    y = dft.linear(X, W, bias=B, residual=R, activation="gelu", preact=z)
    want_y, want_z = ref.forward(x, w[None], bias=bias[None], residual=r, kind="gelu")
    ref.assert_within(y, want_y, "y")
    ref.assert_within(z, want_z, "z")
    g = dft.linear_grad(DY, X, W, preact=z, activation="gelu", b_dtype=torch.float32)
    want = ref.grad(dy, x, w[None], preact=z.cpu(), kind="gelu", b_dtype=torch.float32)
    assert g.b.dtype is torch.float32 and g.a.dtype is torch.float16
    for got, name in ((g.preact, "dz"), (g.a, "a"), (g.b[None], "b"), (g.bias[None], "bias")):
        ref.assert_within(got, want[name], name)
    # strided views, an output given, no activation
    wide = torch.zeros(50, 400, dtype=torch.float16, device="cuda")
    out = dft.linear(X[::2], W[:, :120], out=wide[::2, 100:220])
    ref.assert_within(out, ref.forward(x[::2], w[None, :, :120])[0], "strided")
    assert int((wide != 0).sum()) <= 25 * 120
    g = dft.linear_grad(DY, X, W, want=("a",))
    assert g.preact is DY and g.b is None and g.bias is None


def test_workspaces_belong_to_the_stream_of_the_call(libs):
    """With `stream` given, memory that the caller's own stream allocates while the call is queued is none of the
    call's: the caller overwrites it at once, long before the call's turn."""
    gen = torch.Generator().manual_seed(83)
    x, w = ref.draw(gen, (16, 4096), torch.bfloat16).cuda(), ref.draw(gen, (4096, 1024), torch.bfloat16, scale=0.02).cuda()
    dy, z = ref.draw(gen, (16, 1024), torch.bfloat16).cuda(), ref.draw(gen, (16, 1024), torch.bfloat16).cuda()
    big = torch.randn(4096, 4096, device="cuda")
    eager = dft.linear(x, w, splits=8)
    grads = dft.linear_grad(dy, x, w, preact=z, activation="silu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            for _ in range(20):
                big @ big
        got = dft.linear(x, w, splits=8, stream=stream)
        got_grads = dft.linear_grad(dy, x, w, preact=z, activation="silu", stream=stream)
        spoiled = [torch.full((16 * 1024 * splits,), float("nan"), device="cuda") for splits in (1, 2, 4, 8, 16, 32, 8, 4)]
        torch.cuda.synchronize()
        assert torch.equal(got, eager)
        assert all(torch.equal(p, q) for p, q in zip(got_grads, grads))
        del spoiled


def test_largest_output_pitch(libs):
    """Rows 2^26 elements apart: the epilogue's offsets within 16 rows reach their largest."""
    gen = torch.Generator().manual_seed(84)
    x, w = ref.draw(gen, (17, 72), torch.bfloat16), ref.draw(gen, (72, 40), torch.bfloat16)
    pitch = 1 << 26
    wide = torch.empty(16 * pitch + 40, dtype=torch.float32, device="cuda")
    out = wide.as_strided((17, 40), (pitch, 1))
    dft.linear(x.cuda(), w.cuda(), out=out)
    ref.assert_within(out, ref.forward(x, w[None], out_dtype=torch.float32)[0], "pitch 2^26")
    with pytest.raises(dft.GemmError):
        dft.linear(x[:2].cuda(), w.cuda(), out=wide.as_strided((2, 40), (pitch + 1, 1)))


def test_descending_offsets_stay_inside(libs):
    """Groups that overlap have more chunks of rows than there are places for their sums: none outside is read."""
    M, N, K, groups = 64, 8, 16, 5
    gen = torch.Generator().manual_seed(85)
    dy = ref.draw(gen, (M, N), torch.bfloat16).cuda()
    offsets = torch.tensor([0, 64, 0, 64, 0, 64], dtype=torch.int32, device="cuda")
    dbias = torch.empty(groups, N, device="cuda")
    g = dft.LinearGradArgs(groups=groups, M=M, N=N, K=K, offsets=offsets.data_ptr(), dY=dy.data_ptr(), ldy=N,
                           dbias=dbias.data_ptr())
    need = dft.gemm_linear_grad_workspace_bytes(g, torch.cuda.get_device_properties(0).multi_processor_count)
    assert 0 < need < 64 * N * 4
    space = torch.full((64 * N,), float("nan"), device="cuda")
    g.workspace, g.workspace_bytes = space.data_ptr(), need
    assert dft.gemm_linear_grad(g, torch.cuda.current_stream().cuda_stream) == dft.GEMM_OK
    assert bool(torch.isfinite(dbias).all())
    assert bool(space[need // 4:].isnan().all())


@pytest.mark.parametrize("tile", TILES, ids=TILE_IDS)
def test_overlapping_groups_do_no_more_work(tile, libs):
    """Offsets that go back and forth over all rows, 2000 times: no more tiles than a division of the rows needs."""
    M, K, groups = 4096, 2112, 2000
    a, b = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(groups, K, 8, dtype=torch.bfloat16, device="cuda")
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    offsets[1::2] = M
    wide = torch.full((M + 2, 8), 3.0, device="cuda")
    dft.grouped_linear(a, b, offsets, out=wide[1:M + 1], variant=tile)
    torch.cuda.synchronize()
    assert bool((wide[0] == 3).all()) and bool((wide[M + 1] == 3).all())
    assert bool(((wide == 0) | (wide == 3)).all())


def test_streams_and_graphs(libs):
    """Two calls at once on two streams, and a captured call replayed between eager ones."""
    gen = torch.Generator().manual_seed(82)
    x, w = ref.draw(gen, (16, 4096), torch.bfloat16).cuda(), ref.draw(gen, (4096, 1024), torch.bfloat16, scale=0.02).cuda()
    dy = ref.draw(gen, (16, 1024), torch.bfloat16).cuda()
    z = ref.draw(gen, (16, 1024), torch.bfloat16).cuda()
    eager = dft.linear(x, w, activation="silu")
    grads = dft.linear_grad(dy, x, w, preact=z, activation="silu")
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            one = dft.linear(x, w, activation="silu")
        with torch.cuda.stream(s2):
            two = dft.linear_grad(dy, x, w, preact=z, activation="silu")
        torch.cuda.synchronize()
        assert torch.equal(one, eager)
        assert all(torch.equal(p, q) for p, q in zip(two, grads))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = dft.linear(x, w, activation="silu")
        g = dft.linear_grad(dy, x, w, preact=z, activation="silu")
    for _ in range(4):
        y.zero_()
        for t in g:
            t.zero_()
        other = dft.linear(x, w, activation="gelu")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
        assert all(torch.equal(p, q) for p, q in zip(g, grads))
        del other


def test_packed_and_sliced_calls_captured(libs):
    """Odd widths (packed) and a last round in slices in one graph, replayed with other inputs between eager calls."""
    torch.manual_seed(78)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    M, N, K = 256 * (cus // 16) + 100, 4096, 2113
    x, w, dy = (torch.randn(*s, device="cuda").to(torch.bfloat16) for s in ((M, K), (K, N), (M, N)))

    def step():
        z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        y = dft.linear(x, w, activation="gelu", preact=z, variant=dft.LINEAR_256x256, splits=1)
        return [y, z, *dft.linear_grad(dy, x, w, preact=z, activation="gelu")]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for k in range(3):
        x.normal_()
        eager = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b), k
        del eager


def test_calls_from_several_threads(libs):
    """Each thread on a stream of its own: forward with slices, gradients with every output."""
    gen = torch.Generator().manual_seed(86)
    x, w = ref.draw(gen, (16, 2048), torch.bfloat16).cuda(), ref.draw(gen, (2048, 640), torch.bfloat16, scale=0.02).cuda()
    dy = ref.draw(gen, (16, 640), torch.bfloat16).cuda()
    want = [dft.linear(x, w, splits=4), *dft.linear_grad(dy, x, w)[:3]]
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        for _ in range(20):
            got = [dft.linear(x, w, splits=4, stream=stream), *dft.linear_grad(dy, x, w, stream=stream)[:3]]
            stream.synchronize()
            wrong.extend(k for k, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_gradient_of_the_pre_activation_alone(libs):
    gen = torch.Generator().manual_seed(87)
    x, w, dy, z = (ref.draw(gen, s, torch.bfloat16) for s in ((40, 24), (24, 56), (40, 56), (40, 56)))
    g = dft.linear_grad(dy.cuda(), x.cuda(), w.cuda(), preact=z.cuda(), activation="silu", want=())
    assert g.a is None and g.b is None and g.bias is None
    exact = dy.double() * ref.slope(z.double(), "silu")
    # the slope is off by at most 16 u (1 + |z|), the product by u of itself, then one rounding
    off = 20 * ref.U * (1 + z.double().abs()) * dy.double().abs()
    assert bool(((g.preact.cpu().double() - exact).abs() <= off + ref.half_step(exact.abs() + off, torch.bfloat16)).all())


@pytest.mark.parametrize("act", ("none", "gelu", "gelu_tanh", "silu"))
@pytest.mark.parametrize("counts", [None, [5, 0, 1, 33]], ids=["one", "grouped"])
def test_bias_gradient_against_differences(counts, act, libs):
    """Every column of dbias against the central difference of sum(G * D) over that column's bias, in float64.  With
    step h the difference is off by at most h^2 / 6 times the sum of |G| times the third derivative (below 1 for these
    activations), and by two roundings of the sums that are subtracted, 2^-52 of their size over 2 h; dbias itself by
    the bound of linear_reference."""
    gen = torch.Generator().manual_seed(74)
    offsets, M, groups = None, 39, 1
    if counts is not None:
        offsets, groups = [0], len(counts)
        for c in counts:
            offsets.append(offsets[-1] + c)
    N, K, h = 24, 16, 1e-4
    a, b = ref.draw(gen, (M, K), torch.bfloat16), ref.draw(gen, (groups, K, N), torch.bfloat16, scale=0.25)
    dy, z = ref.draw(gen, (M, N), torch.bfloat16), ref.draw(gen, (M, N), torch.bfloat16)
    got = ref.run_grad(libs["plain"], dy, a, b, offsets, preact=z, kind=act, want=("bias",))["bias"]
    _, bound = ref.grad(dy, a, b, offsets, preact=z, kind=act)["bias"]
    G, Z = dy.double(), z.double()
    for g, lo, hi in ref.ranges(offsets, groups, M):
        # (each column's bias enters that column's values alone, so all columns are moved at once)
        up, down = ((G[lo:hi] * ref.act(Z[lo:hi] + s, act)).sum(0) for s in (h, -h))
        size = (G[lo:hi].abs() * (ref.act(Z[lo:hi], act).abs() + 1)).sum(0)
        tol = bound[g] + G[lo:hi].abs().sum(0) * h * h / 6 + (hi - lo + 2) * 2.0 ** -52 * size / h
        assert bool(((got[g].double() - (up - down) / (2 * h)).abs() <= tol).all()), (g, act)
