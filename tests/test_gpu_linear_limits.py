"""The products with an epilogue at the sizes where a launch, a count or a
placement ends: outputs of more small tiles than a launch holds, more columns
than one dimension of a grid has tiles of 64, and few rows among many groups."""

from __future__ import annotations

import pytest
import torch

import dense_fp32_tiled_amd as dft

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu(gemm_lib):
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def whole(gen, *shape, most=3):
    return torch.randint(-most, most + 1, shape, generator=gen, device="cuda").to(torch.bfloat16)


def test_more_rows_than_small_tiles_have_a_launch_for():
    """2^28 rows are 2^22 tiles of 64 rows, one more than a launch holds."""
    gen = torch.Generator(device="cuda").manual_seed(91)
    M, N, K = (1 << 28) + 5, 8, 8
    rows = torch.tensor([0, 1, 127, 128, 1 << 20, (1 << 27) + 3, (1 << 28) - 1, 1 << 28, M - 1], device="cuda")
    a = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    a[rows] = whole(gen, len(rows), K)
    b, bias = whole(gen, K, N), whole(gen, N)
    d = dft.linear(a, b, bias=bias)
    want = (a[rows].cpu().double() @ b.cpu().double() + bias.cpu().double()).to(torch.bfloat16)
    assert torch.equal(d[rows].cpu(), want)
    d[rows] = bias  # every other row is the bias alone
    assert bool((d == bias).all())


def test_more_columns_than_a_grid_has_tiles_of_64():
    """Values of -1, 0 and 1: sums of 2^22 products stay exact in fp32 in any order."""
    gen = torch.Generator(device="cuda").manual_seed(92)
    M, N, K = 3, 65535 * 64 + 77, 8
    a, b, dy, z = (whole(gen, *shape, most=1) for shape in ((M, K), (K, N), (M, N), (M, N)))
    g = dft.linear_grad(dy, a, b, preact=z, activation="relu", a_dtype=torch.float32, b_dtype=torch.float32)
    dz = torch.where(z > 0, dy, torch.zeros_like(dy))
    assert torch.equal(g.preact, dz)
    assert torch.equal(g.bias, dz.float().sum(0))
    assert torch.equal(g.b.cpu(), a.cpu().float().t() @ dz.cpu().float())
    assert torch.equal(g.a.cpu().double(), dz.cpu().double() @ b.cpu().double().t())


@pytest.mark.parametrize("rows", [1, 5])
def test_few_rows_of_as_many_groups_as_there_may_be(rows):
    gen = torch.Generator(device="cuda").manual_seed(93)
    groups, N, K = 65535, 8456, 8
    used = sorted([0, groups - 1, 1, 30000, 64][:rows])
    offsets = torch.searchsorted(torch.tensor(used), torch.arange(groups + 1)).to(torch.int32).cuda()
    a, dy, z = whole(gen, rows, K), whole(gen, rows, N), whole(gen, rows, N)
    b = torch.full((groups, K, N), float("nan"), dtype=torch.bfloat16, device="cuda")  # (groups without rows: not read)
    b[used] = whole(gen, rows, K, N)
    d = dft.grouped_linear(a, b, offsets, out_dtype=torch.float32)
    want = torch.stack([a[r].cpu().double() @ b[used[r]].cpu().double() for r in range(rows)])
    assert torch.equal(d.cpu().double(), want)
    g = dft.grouped_linear_grad(dy, a, b, offsets, preact=z, activation="relu", a_dtype=torch.float32)
    dz = torch.where(z > 0, dy, torch.zeros_like(dy))
    assert torch.equal(g.preact, dz)
    want = torch.stack([b[used[r]].cpu().double() @ dz[r].cpu().double() for r in range(rows)])
    assert torch.equal(g.a.cpu().double(), want)
    for r in range(rows):
        assert torch.equal(g.b[used[r]].cpu().float(), torch.outer(a[r], dz[r]).cpu().float())
        assert torch.equal(g.bias[used[r]], dz[r].float())
        g.b[used[r]], g.bias[used[r]] = 0, 0
    assert not bool(g.bias.any()) and all(not bool(part.any()) for part in g.b.split(8192))
