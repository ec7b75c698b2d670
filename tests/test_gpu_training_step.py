"""The operators together, as a training step runs them: a pre-normed block with
a residual stream, experts or a plain layer, dropout and the vocabulary's loss,
forward and backward, against float64's automatic gradients."""

from __future__ import annotations

import pytest
import torch

import dense_fp32_tiled_amd as dft
import norm_reference

pytestmark = pytest.mark.gpu

EPS, P, SEED = 1e-5, 0.2, 99


@pytest.fixture(scope="module", autouse=True)
def gpu(gemm_lib):
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def norm(t, w, b):
    m = t.mean(1, keepdim=True)
    return (t - m) * ((t - m).square().mean(1, keepdim=True) + EPS).rsqrt() * w + b


def step(s, n):
    """One step through the framework's operators: the loss of each token and every leaf's gradient."""
    y1, k1 = dft.layer_norm(s["x"], s["g1"], s["c1"])
    if "chosen" in s:
        mixed, kept = dft.expert_mlp(y1, s["chosen"], s["weights"], s["w1"], s["w2"], activation="silu")
    else:
        z = torch.empty(y1.shape[0], s["w1"].shape[1], dtype=y1.dtype, device="cuda")
        hidden = dft.linear(y1, s["w1"], activation="silu", preact=z)
        hidden_kept = dft.dropout(hidden, P, SEED, offset=2 * n + 1)
        mixed = dft.linear(hidden_kept, s["w2"])
    y2, k2 = dft.layer_norm(mixed, s["g2"], s["c2"], residual=s["x"], p=P, seed=SEED, offset=2 * n)
    loss, lse = dft.linear_cross_entropy(y2, s["words"].t(), s["targets"])
    head = dft.linear_cross_entropy_grad(s["dloss"], y2, s["words"].t(), s["targets"], lse)
    g2 = dft.layer_norm_grad(head.a, k2, s["g2"], p=P, seed=SEED, offset=2 * n)
    out = {"words": head.b.t(), "g2": g2.weight, "c2": g2.bias}
    if "chosen" in s:
        e = dft.expert_mlp_grad(g2.x, kept, s["weights"], s["w1"], s["w2"], activation="silu")
        out.update(w1=e.w1, w2=e.w2, weights=e.weights)
        dy1 = e.x
    else:
        b = dft.linear_grad(g2.x, hidden_kept, s["w2"])
        a = dft.linear_grad(dft.dropout(b.a, P, SEED, offset=2 * n + 1), y1, s["w1"], preact=z, activation="silu")
        out.update(w1=a.b, w2=b.b)
        dy1 = a.a
    g1 = dft.layer_norm_grad(dy1, k1, s["g1"], dtotal=g2.residual)
    out.update(x=g1.x, g1=g1.weight, c1=g1.bias)
    return loss, out


def reference(s, n):
    leaf = {k: v.detach().cpu().double().requires_grad_() for k, v in s.items() if v.is_floating_point() and k != "dloss"}
    x, (rows, width) = leaf["x"], s["x"].shape
    y1 = norm(x, leaf["g1"], leaf["c1"])
    if "chosen" in s:
        chosen = s["chosen"].cpu().tolist()
        mixed = torch.stack([sum(leaf["weights"][t, j] * (torch.nn.functional.silu(y1[t] @ leaf["w1"][e]) @ leaf["w2"][e])
                                 for j, e in enumerate(chosen[t])) for t in range(rows)])
    else:
        hidden = torch.nn.functional.silu(y1 @ leaf["w1"])
        mixed = (hidden * norm_reference.keep(rows, hidden.shape[1], P, SEED, 2 * n + 1)) @ leaf["w2"]
    y2 = norm(mixed * norm_reference.keep(rows, width, P, SEED, 2 * n) + x, leaf["g2"], leaf["c2"])
    loss = torch.nn.functional.cross_entropy(y2 @ leaf["words"].t(), s["targets"].cpu(), reduction="none", ignore_index=-100)
    loss.backward(s["dloss"].cpu().double())
    return loss.detach(), {k: v.grad for k, v in leaf.items()}


def inputs(experts, rows=50, width=72, hidden=104, words=301):
    gen = torch.Generator().manual_seed(5 + experts)

    def normal(*shape, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen) * scale + mean).half().cuda()

    s = {"x": normal(rows, width), "words": normal(words, width, scale=width ** -0.5)}
    for k in ("1", "2"):
        s["g" + k], s["c" + k] = normal(width, scale=0.1, mean=1.0), normal(width, scale=0.1)
    lead = (experts,) if experts else ()
    s["w1"], s["w2"] = normal(*lead, width, hidden, scale=width ** -0.5), normal(*lead, hidden, width, scale=hidden ** -0.5)
    if experts:
        s["chosen"] = torch.randint(0, experts, (rows, 2), generator=gen, dtype=torch.int32).cuda()
        s["weights"] = torch.softmax(torch.randn(rows, 2, generator=gen), 1).cuda()
    t = torch.randint(0, words, (rows,), generator=gen)
    t[::9] = -100
    s["targets"], s["dloss"] = t.cuda(), (torch.rand(rows, generator=gen) / rows).cuda()
    return s


def close(got, want):
    """In the 2-norm.  A value that a step keeps in fp16 is off by at most 2^-11 of itself; a gradient's path has at most 24
    such values (12 forward, 12 back), and the maps between them, of weights of norm about 2 for random matrices of
    these shapes and norms of rows whose factors are near 1, pass a relative error on about once: 24 * 2^-11."""
    loss, grads = got
    want_loss, want_grads = want
    assert float((loss.cpu().double() - want_loss).norm() / want_loss.norm()) <= 24 * 2.0 ** -11
    assert set(grads) == set(want_grads)
    for name, g in grads.items():
        w = want_grads[name]
        assert g.shape == w.shape, name
        off = float((g.cpu().double() - w).norm() / w.norm())
        assert off <= 24 * 2.0 ** -11, (name, off)


@pytest.mark.parametrize("experts", [0, 4], ids=["layer", "experts"])
def test_step(experts):
    s = inputs(experts)
    for n in range(2):
        close(step(s, n), reference(s, n))


@pytest.mark.parametrize("experts", [0, 4], ids=["layer", "experts"])
def test_captured_step(experts):
    """The whole step in a graph, replayed with new inputs among eager steps, bit for bit the eager one."""
    s = inputs(experts)
    step(s, 0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grads = step(s, 0)
    for n in range(3):
        s["x"].mul_(0.9)
        s["targets"].copy_((s["targets"] + n) % 301)
        graph.replay()
        torch.cuda.synchronize()
        want_loss, want = step(s, 0)
        assert torch.equal(loss, want_loss) and all(torch.equal(grads[k], want[k]) for k in want), n
