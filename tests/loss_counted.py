"""Inputs of the vocabulary's loss in which every word and every token counts,
their exact results in closed form, and bounds that a lost tile, slice, piece or
token cannot pass.

Row t of A is 1 at feature t mod K and else 0, word w of B is 1 at feature
(w / 64) mod K, so that a logit is 1 where the two agree and else 0, exactly.
With N_k words and the weights of T_k, tokens of feature k:

  lse[t]   = log(N - N_k + e N_k),  k = t mod K
  dA[t][k] = g_t (N_k p(t, k) - [the target's feature is k])
  dB[k][w] = sum over the tokens of feature k of g_t (p(t, w's feature) - [w is the target])

64 words lost from any place change lse by 64 / (N e) or more, and some features'
dA by their part of at most N / K + 64 words; a lost token changes dB by its
part of at most M / K + 1 tokens.

Bounds.  u = 2^-24.  exp is relative 3u |z - m| + 4u.  lse: a lane adds 16 words
in at most 6 steps, a wave 2 more, a thread its pieces (of 32 words or more, by
1024 threads for up to 256 tokens, else 32), halvings 6, waves 16; each step has
an addition, two products and an exponential whose rounding 8u covers.  dZ is
rounded to 16 bits once (eps / 2; twice where it is held in two parts, up to 32
tokens), in fp16 also by half a least step of a scale of at least 2^13 / max g.
The sums have as many terms as words, or tokens, of a feature (what else is
added is zero), each addition off by 2u of the sum of magnitudes; a piece or a
slice is one more."""

from __future__ import annotations

import math
from typing import NamedTuple

import torch

from linear_reference import SMALLEST, U, half_step

TILE = 64


class Counted(NamedTuple):
    M: int
    N: int
    K: int
    targets: torch.Tensor
    g: torch.Tensor
    token: torch.Tensor  # the tokens' features
    word: torch.Tensor   # the words'


def make(M: int, N: int, K: int, device="cpu") -> Counted:
    t = torch.arange(M, device=device)
    targets = (t * 7919 + 13) % N
    targets[M // 2] = N - 1
    targets[-1] = 0
    targets[5::11] = -1
    g = (0.5 + 0.5 * ((t * 37) % 101).double() / 101).float() / M
    return Counted(M, N, K, targets, g, t % K, torch.arange(N, device=device) // TILE % K)


def operands(c: Counted, dtype, transposed: bool):
    a = torch.zeros(c.M, c.K, dtype=dtype, device=c.token.device)
    a[torch.arange(c.M, device=a.device), c.token] = 1
    b = torch.zeros((c.N, c.K) if transposed else (c.K, c.N), dtype=dtype, device=a.device)
    words = torch.arange(c.N, device=a.device)
    if transposed:
        b[words, c.word] = 1
        return a, b.t()
    b[c.word, words] = 1
    return a, b


def _sizes(c: Counted, words: torch.Tensor):
    """Words of each feature, of those with weight `words` (1, or 0 where they are lost)."""
    return torch.zeros(c.K, dtype=torch.float64, device=c.word.device).index_add_(0, c.word, words)


def forward(c: Counted, lost_words: slice | None = None):
    """{lse, loss}: (value, bound); `lost_words` are left out of the value."""
    words = torch.ones(c.N, dtype=torch.float64, device=c.word.device)
    if lost_words is not None:
        words[lost_words] = 0
    n = _sizes(c, words)
    lse = torch.log(n.sum() - n[c.token] + math.e * n[c.token])
    valid = c.targets >= 0
    goal = (c.word[c.targets.clamp(min=0)] == c.token).double()
    chain = 6 + 2 + -(-c.N // (32 * (1024 if c.M <= 256 else 32))) + 6 + 16
    rest = 8 * U * chain + 3 * U * 2
    return {"lse": (lse, rest + 4 * U * lse.abs()), "loss": (torch.where(valid, lse - goal, 0.0), rest + 4 * U * (1 + lse.abs()))}


def gradients(c: Counted, lse, dtype, a_dtype=None, b_dtype=None, pieces=1, lost_words: slice | None = None,
              lost_tokens: slice | None = None):
    """{a: (value, bound), b: (per feature and word's feature, its bound, targets' entries)} for the given lse."""
    device = c.word.device
    valid = c.targets >= 0
    g = torch.where(valid, c.g.double(), 0.0)
    L = lse.double()
    features = torch.arange(c.K, device=device)
    match = (c.token[:, None] == features[None]).double()
    p = torch.exp(match - L[:, None])  # of a word of each feature
    n = _sizes(c, torch.ones(c.N, dtype=torch.float64, device=device))
    held = n.clone()
    hot = torch.zeros(c.M, c.K, dtype=torch.float64, device=device)
    goal = torch.where(valid, c.targets, 0)
    here = valid.clone()
    if lost_words is not None:
        words = torch.ones(c.N, dtype=torch.float64, device=device)
        words[lost_words] = 0
        held = _sizes(c, words)
        here &= words[goal] > 0
    hot[torch.arange(c.M, device=device), c.word[goal]] = here.double()
    da = g[:, None] * (held * p - hot)
    step = (torch.finfo(dtype).eps / 2) ** (2 if c.M <= 32 else 1)
    least = SMALLEST[dtype] * float(g.max()) / 2 ** 13
    rel = 3 * U * (L.max() + 1) + 8 * U + step
    size = g[:, None] * (n * p + (c.word[goal][:, None] == features[None]).double())
    slices = 32 + pieces
    da_off = size * (rel + (n[None] + slices) * 2 * U) + least * n[None]
    out = {"a": (da, da_off + half_step(da.abs() + da_off, a_dtype or dtype))}
    weights = g.clone()
    if lost_tokens is not None:
        weights[lost_tokens] = 0
    # the tokens of a feature: sums over them of g p, for every word's feature
    def over_tokens(x):
        return torch.zeros(c.K, c.K, dtype=torch.float64, device=device).index_add_(0, c.token, x)

    tokens = torch.zeros(c.K, dtype=torch.float64, device=device).index_add_(0, c.token, torch.ones_like(g))
    db, size = over_tokens(weights[:, None] * p), over_tokens(g[:, None] * p)
    per = rel + (tokens[:, None] + 3 + slices) * 2 * U
    db_off = size * per + least * tokens[:, None]
    targets = (c.token[valid], c.targets[valid], weights[valid], g[valid] * float(per.max()))
    return {**out, "b": (db, db_off, targets, b_dtype or dtype)}


def assert_tokens(got: torch.Tensor, want, what):
    value, tol = want
    bad = ~((got.double() - value).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[0].tolist())


def assert_words(c: Counted, got: torch.Tensor, want, what="b", each=1 << 16):
    """dB (K x N), some words at a time."""
    db, off, (features, words, weights, more), dtype = want
    for first in range(0, c.N, each):
        part = slice(first, min(first + each, c.N))
        value, tol = db[:, c.word[part]], off[:, c.word[part]]
        inside = (words >= part.start) & (words < part.stop)
        at = (features[inside], words[inside] - first)
        value = value.index_put(at, -weights[inside], accumulate=True)
        tol = tol.index_put(at, more[inside], accumulate=True)
        bad = ~((got[:, part].double() - value).abs() <= tol + half_step(value.abs() + tol, dtype))
        assert not bool(bad.any()), (what, int(bad.sum()), first, bad.nonzero()[0].tolist())
