"""What the GPU's counted results are held to sees lost work: closed forms
against the definition, results rounded as they may be accepted, results without
one tile of words, one slice or one tile of tokens rejected (float64, CPU)."""

from __future__ import annotations

import pytest
import torch

import loss_counted as counted

SIZES = [(2, 150000, 512), (4, 40000, 1000), (24, 20000, 192), (33, 9000, 64), (300, 5000, 40), (1500, 8001, 130)]


def definition(c, dtype):
    a, b = (x.double() for x in counted.operands(c, dtype, False))
    z = a @ b
    lse = torch.logsumexp(z, 1)
    valid = c.targets >= 0
    goal = torch.where(valid, c.targets, 0)
    loss = torch.where(valid, lse - z.gather(1, goal[:, None])[:, 0], 0.0)
    dz = torch.exp(z - lse.float().double()[:, None])
    dz[valid.nonzero()[:, 0], goal[valid]] -= 1
    dz *= torch.where(valid, c.g.double(), 0.0)[:, None]
    return lse, loss, dz @ b.t(), a.t() @ dz


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("size", SIZES[2:], ids=lambda s: "x".join(map(str, s)))
def test_closed_forms(size, dtype):
    c = counted.make(*size)
    lse, loss, da, db = definition(c, dtype)
    want = counted.forward(c)
    assert float((want["lse"][0] - lse).abs().max()) < 1e-12 and float((want["loss"][0] - loss).abs().max()) < 1e-12
    counted.assert_tokens(lse.float(), want["lse"], "lse")
    counted.assert_tokens(loss.float(), want["loss"], "loss")
    for types in ((None, None), (torch.float32, torch.float32)):
        want = counted.gradients(c, lse.float(), dtype, *types)
        assert float((want["a"][0] - da).abs().max()) < 1e-13
        counted.assert_tokens(da.to(types[0] or dtype), want["a"], "a")
        counted.assert_words(c, db.to(types[1] or dtype), want["b"])


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_lost_slot_of_a_row_is_seen(size):
    c = counted.make(*size)
    want = counted.forward(c)
    for width in (32, 64):
        for first in range(0, c.N - width + 1, width if c.M * c.N < 1 << 20 else 7 * width):
            wrong = counted.forward(c, slice(first, first + width))["lse"][0]
            assert bool(((wrong - want["lse"][0]).abs() > want["lse"][1]).all()), (width, first)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_lost_words_and_tokens_are_seen(size, dtype):
    c = counted.make(*size)
    lse = counted.forward(c)["lse"][0].float()
    want = counted.gradients(c, lse, dtype)
    # one contraction tile of words, at both ends, between them, and each of 32 slices
    tiles = c.N // 64
    lost = [slice(64 * k, 64 * k + 64) for k in {0, 1, tiles // 3, tiles - 2, tiles - 1}]
    lost += [slice(c.N * s // 32, c.N * (s + 1) // 32) for s in range(32)]
    for words in lost:
        wrong = counted.gradients(c, lse, dtype, lost_words=words)["a"][0]
        seen = (wrong - want["a"][0]).abs() > want["a"][1]
        # (of every token that counts; a feature that holds its own target is off by the target's rounding)
        assert bool(seen.any(1)[c.targets >= 0].float().mean() > 0.9), words
    for first in range(0, c.M, max(1, c.M // 8)):
        while int(c.targets[first]) < 0:
            first += 1
        wrong = counted.gradients(c, lse, dtype, lost_tokens=slice(first, first + 1))["b"][0]
        row = int(c.token[first])
        assert bool(((wrong - want["b"][0]).abs()[row] > want["b"][1][row] + 2.0 ** -8 * want["b"][0].abs()[row]).all()), first
