"""The vocabulary's loss and its gradients on inputs in which every word and
every token counts (loss_counted.py): at the widest vocabularies, in pieces, with
joins of many slots to a thread and products cut into slices, a lost tile, slice,
piece or token shows."""

from __future__ import annotations

import pytest
import torch

import dense_fp32_tiled_amd as dft
import loss_counted as counted

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu(gemm_lib):
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def check(c, dtype, transposed, piece=0, variant=0, types=(None, None)):
    a, b = counted.operands(c, dtype, transposed)
    loss, lse = dft.linear_cross_entropy(a, b, c.targets, piece=piece, variant=variant)
    want = counted.forward(c)
    counted.assert_tokens(lse, want["lse"], "lse")
    counted.assert_tokens(loss, want["loss"], "loss")
    grads = dft.linear_cross_entropy_grad(c.g, a, b, c.targets, lse, a_dtype=types[0], b_dtype=types[1], piece=piece,
                                          variant=variant)
    want = counted.gradients(c, lse, dtype, *types, pieces=-(-c.N // (piece or 4096)))
    counted.assert_tokens(grads.a, want["a"], "a")
    counted.assert_words(c, grads.b, want["b"])


# few tokens over wide vocabularies (a row's join by one workgroup or with others, dA in many slices, dZ in two parts and,
# from 33 tokens, in one), more tokens than CUs, all sizes odd, many rounds of the largest tiles
SIZES = [(2, 150000, 512), (4, 40000, 1000), (24, 131072, 512), (32, 131071, 520), (33, 131072, 512), (200, 100001, 264),
         (300, 40000, 136), (1500, 40001, 520), (5000, 33000, 1024), (520, 14003, 200)]


@pytest.mark.parametrize("piece", [0, 4096])
@pytest.mark.parametrize("transposed", [False, True], ids=["columns", "rows"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_every_word_and_token(size, dtype, transposed, piece):
    c = counted.make(*size, device="cuda")
    check(c, dtype, transposed, piece)
    check(c, dtype, transposed, piece, types=(torch.float32, torch.float32))


@pytest.mark.parametrize("variant", range(1, dft.LINEAR_COUNT), ids=list(dft.LINEAR_NAMES.values())[1:])
@pytest.mark.parametrize("size", [(24, 20000, 192), (130, 9001, 72), (300, 5000, 40)], ids=lambda s: "x".join(map(str, s)))
def test_every_tile(size, variant):
    c = counted.make(*size, device="cuda")
    for piece in (0, 1024):
        for transposed in (False, True):
            check(c, torch.bfloat16, transposed, piece, variant)


@pytest.mark.parametrize("transposed", [False, True], ids=["columns", "rows"])
def test_places_past_32_bits(transposed):
    """A matrix of more than 2^32 bytes and 2^31 values: every word's part of the loss and of both gradients."""
    check(counted.make(3, 540_000, 4096, device="cuda"), torch.bfloat16, transposed)
