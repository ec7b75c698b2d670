"""The token sort, the rows it moves and the routed block on the GPU: against
plain Python and float64, with dropped pairs, experts without tokens, one
token to several workgroups of them, widths and pitches aligned to nothing.

Bounds (u = 2^-24): a weighted sum of k rows is off by at most 2 k u times the
sum of |w y|, a dot product of n exact products by at most n u sum |y d|, and
each result's rounding is finfo.eps / 2."""

from __future__ import annotations

import math

import pytest
import torch

import dense_fp32_tiled_amd as dft
import linear_reference as ref
from linear_reference import U, Guarded, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu(gemm_lib):
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def plain_sort(experts, num_experts):
    pairs = experts.flatten().tolist()
    slots = [p for e in range(num_experts) for p in ()]
    by = [[] for _ in range(num_experts)]
    for p, e in enumerate(pairs):
        if 0 <= e < num_experts:
            by[e].append(p)
    slots = [p for group in by for p in group]
    offsets = [0]
    for group in by:
        offsets.append(offsets[-1] + len(group))
    position = [-1] * len(pairs)
    for s, p in enumerate(slots):
        position[p] = s
    order = slots + [-1] * (len(pairs) - len(slots))
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor(order, dtype=i32),
            torch.tensor(position, dtype=i32).view(experts.shape))


SORTS = [(0, 2, 4), (1, 1, 1), (1, 64, 3), (16, 4, 32), (63, 1, 2), (300, 3, 1000), (1024, 4, 1024), (1025, 4, 64),
         (4097, 1, 7), (20000, 8, 128), (70000, 2, 1024)]


@pytest.mark.parametrize("drop", [False, True], ids=["all", "dropped"])
@pytest.mark.parametrize("size", SORTS, ids=lambda s: "x".join(map(str, s)))
def test_sort(size, drop):
    tokens, top_k, num = size
    gen = torch.Generator().manual_seed(tokens + num)
    experts = torch.randint(0, num, (tokens, top_k), generator=gen, dtype=torch.int32)
    if drop:
        gone = torch.rand(tokens, top_k, generator=gen) < 0.3
        odd = torch.tensor([-1, num, num + 5, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)
        experts = torch.where(gone, odd[torch.randint(0, 5, (tokens, top_k), generator=gen)], experts)
    got = dft.expert_sort(experts.cuda(), num)
    for g, w, name in zip(got, plain_sort(experts, num), ("offsets", "order", "position")):
        assert torch.equal(g.cpu(), w), name


def test_sort_of_one_expert_and_of_none():
    experts = torch.full((5000, 2), 3, dtype=torch.int32)
    for num in (8, 2):  # all to expert 3; all dropped
        got = dft.expert_sort(experts.cuda(), num)
        for g, w in zip(got, plain_sort(experts, num)):
            assert torch.equal(g.cpu(), w)


def test_sort_writes_only_its_arrays():
    """Through the C ABI: results and workspace with guard words around them."""
    tokens, top_k, num = 3000, 2, 40
    gen = torch.Generator().manual_seed(5)
    experts = torch.randint(-2, num + 2, (tokens, top_k), generator=gen, dtype=torch.int32)
    pairs, guard, mark = tokens * top_k, 16, 0x5A5A5A5
    need = dft.gemm_expert_sort_workspace_bytes(tokens, top_k, num) // 4
    assert need > 0
    sizes = [num + 1, pairs, pairs, need]
    bufs = [torch.full((n + 2 * guard,), mark, dtype=torch.int32, device="cuda") for n in sizes]
    e = experts.cuda()
    at = [b.data_ptr() + 4 * guard for b in bufs]
    st = dft.gemm_expert_sort(tokens, top_k, num, e.data_ptr(), at[0], at[1], at[2], at[3], need * 4,
                              torch.cuda.current_stream().cuda_stream)
    assert st == dft.GEMM_OK
    for b, n, w in zip(bufs, sizes, [*plain_sort(experts, num), None]):
        b = b.cpu()
        assert bool((b[:guard] == mark).all()) and bool((b[guard + n:] == mark).all())
        if w is not None:
            assert torch.equal(b[guard:guard + n], w.flatten())


ROWS = [(1, 1, 8, 0, 0), (5, 2, 1, 2, 1), (33, 4, 512, 0, 0), (70, 3, 520, 8, 8), (64, 2, 1237, 3, 1), (9, 8, 4096, 0, 0)]


def routed(gen, tokens, top_k, num=6, drop=0.25):
    experts = torch.randint(0, num, (tokens, top_k), generator=gen, dtype=torch.int32)
    experts[torch.rand(tokens, top_k, generator=gen) < drop] = -1
    return experts, plain_sort(experts, num)


@pytest.mark.parametrize("kind", list(ref.TYPES))
@pytest.mark.parametrize("case", ROWS, ids=lambda c: "x".join(map(str, c[:3])))
def test_rows_there_and_back(case, kind):
    tokens, top_k, cols, pad, offset = case
    dtype, code = ref.TYPES[kind], ref.KINDS[ref.TYPES[kind]]
    gen = torch.Generator().manual_seed(cols)
    _, (_, _, position) = routed(gen, tokens, top_k)
    rows = tokens * top_k
    pos = position.cuda()
    stream = torch.cuda.current_stream().cuda_stream
    flat = position.flatten().long()
    live = flat >= 0
    taken = torch.zeros(rows, dtype=torch.bool)
    taken[flat[live]] = True
    # there
    x = ref.draw(gen, (tokens, cols), dtype)
    gx, out = Guarded(x, pad, offset), ref.empty((rows, cols), dtype, pad=pad, offset=offset)
    st = dft.gemm_expert_gather(code, tokens, rows, top_k, cols, gx.ptr, gx.ld, pos.data_ptr(), out.ptr, out.ld, stream)
    assert st == dft.GEMM_OK
    torch.cuda.synchronize()
    token = torch.arange(rows) // top_k
    assert torch.equal(out.value()[flat[live]], x[token[live]])
    out.assert_rest_untouched("sorted", taken)
    # back, weighted and not; unused sorted rows hold NaN and may not be read
    y = ref.draw(gen, (rows, cols), dtype)
    y[~taken] = math.nan
    weights = torch.randn(tokens, top_k, generator=gen)
    for w in (weights, None):
        gy, out = Guarded(y, pad, offset), ref.empty((tokens, cols), dtype, pad=pad, offset=offset)
        dw = None if w is None else w.cuda()
        st = dft.gemm_expert_combine(code, tokens, rows, top_k, cols, gy.ptr, gy.ld, pos.data_ptr(),
                                     None if w is None else dw.data_ptr(), out.ptr, out.ld, stream)
        assert st == dft.GEMM_OK
        torch.cuda.synchronize()
        picked = torch.where(live[:, None], y.double()[flat.clamp(min=0)], 0.0).view(tokens, top_k, cols)
        terms = picked * (torch.ones(tokens, top_k) if w is None else w).double()[:, :, None]
        want, size = terms.sum(1), terms.abs().sum(1)
        ref.assert_within(out.value(), (want, 2 * top_k * U * size + half_step(want, dtype)), "out")
        out.assert_rest_untouched("out")
    # gradients
    d = ref.draw(gen, (tokens, cols), dtype)
    gd, gy = Guarded(d, pad, offset), Guarded(y, pad, offset)
    dy = ref.empty((rows, cols), dtype, pad=pad, offset=offset)
    dweights = torch.full((tokens * top_k + 2,), math.nan, device="cuda")
    dw = weights.cuda()
    st = dft.gemm_expert_combine_grad(code, tokens, rows, top_k, cols, gd.ptr, gd.ld, gy.ptr, gy.ld, pos.data_ptr(),
                                      dw.data_ptr(), dy.ptr, dy.ld, dweights.data_ptr() + 4, stream)
    assert st == dft.GEMM_OK
    torch.cuda.synchronize()
    want = torch.full((rows, cols), math.nan, dtype=torch.float64)
    want[flat[live]] = weights.flatten().double()[live, None] * d.double()[token[live]]
    ref.assert_within(dy.value(), (want, 2 * U * want.abs() + half_step(want, dtype)), "dy")
    dy.assert_rest_untouched("dy", taken)
    products = picked * d.double()[:, None, :]
    got = dweights.cpu()
    assert bool(torch.isnan(got[0])) and bool(torch.isnan(got[-1]))
    ref.assert_within(got[1:-1].view(tokens, top_k), (products.sum(2), 2 * cols * U * products.abs().sum(2)), "dweights")
    assert bool((got[1:-1][~live] == 0).all())


def test_more_tokens_than_one_launch_holds():
    """2^24 tokens and a few more: a launch's threads are fewer than 2^32, so the row kernels take several steps."""
    tokens = (1 << 24) + 5
    x = torch.randint(-8, 9, (tokens, 1), device="cuda").to(torch.bfloat16)
    position = torch.arange(tokens - 1, -1, -1, device="cuda", dtype=torch.int32).view(tokens, 1)
    weights = torch.randint(1, 5, (tokens, 1), device="cuda").float()
    rows = dft.expert_gather(x, position)
    assert torch.equal(rows, x.flip(0))
    assert torch.equal(dft.expert_combine(rows, position, weights), (x.float() * weights).to(torch.bfloat16))
    dy, dw = dft.expert_combine_grad(x, rows, position, weights)
    assert torch.equal(dy, (x.float() * weights).to(torch.bfloat16).flip(0))
    assert torch.equal(dw, x.float() * x.float())


def test_positions_outside_the_rows_are_dropped():
    x = torch.ones(4, 16, dtype=torch.bfloat16, device="cuda")
    position = torch.tensor([[-7], [3], [4], [2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    out = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    dft.expert_gather(x, position, out=out)
    assert out.sum(1).tolist() == [0, 0, 0, 16]
    assert dft.expert_combine(x, position).sum(1).tolist() == [0, 16, 0, 0]
    dy, dw = dft.expert_combine_grad(x, x, position, torch.ones(4, 1, device="cuda"), dy=torch.zeros_like(x))
    assert dy.sum(1).tolist() == [0, 0, 0, 16] and dw.flatten().tolist() == [0, 16, 0, 0]


def mlp_case(gen, tokens, top_k, E, D, H, dtype=torch.bfloat16, drop=0.0):
    experts, _ = routed(gen, tokens, top_k, E, drop)
    d = lambda *s, scale=1.0: ref.draw(gen, s, dtype, scale=scale)  # noqa: E731
    return dict(x=d(tokens, D), experts=experts, weights=torch.rand(tokens, top_k, generator=gen),
                w1=d(E, D, H, scale=D ** -0.5), b1=d(E, H), w2=d(E, H, D, scale=H ** -0.5), b2=d(E, D),
                dout=d(tokens, D))


def mlp_float64(c, activation):
    """The routed block and its gradients by autograd in float64, nothing rounded between."""
    t = {k: v.double().requires_grad_(k != "dout") for k, v in c.items() if k != "experts"}
    out = torch.zeros_like(t["x"])
    tokens, top_k = c["experts"].shape
    rows = []
    for i in range(tokens):
        total = 0
        for j in range(top_k):
            e = int(c["experts"][i, j])
            if e < 0:
                continue
            h = ref.act(t["x"][i] @ t["w1"][e] + t["b1"][e], activation)
            total = total + t["weights"][i, j] * (h @ t["w2"][e] + t["b2"][e])
        rows.append(total if torch.is_tensor(total) else out[i])
    out = torch.stack(rows)
    out.backward(t["dout"])
    return out.detach(), {k: v.grad for k, v in t.items() if k != "dout"}


@pytest.mark.parametrize("activation", ["silu", "gelu", "none"])
@pytest.mark.parametrize("size", [(1, 2, 4, 64, 96), (37, 2, 5, 72, 40), (64, 1, 3, 33, 45)], ids=lambda s: "x".join(map(str, s)))
def test_routed_block(size, activation):
    """The whole path together.  Between its steps values are rounded to bf16: hidden, back, dback, dhidden, dz and
    the rows' gradients.  Each is off by 2^-8 of itself at most, so a result that passes through n of them (five at
    most, for dw1 and dx: back's, dback's, dz's, dhidden's and its own) is off by about n 2^-8 of its typical size;
    errors of single terms add up at random, so 6 * 2^-8 of the result's root mean square bounds the error's."""
    tokens, top_k, E, D, H = size
    gen = torch.Generator().manual_seed(90 + tokens)
    c = mlp_case(gen, tokens, top_k, E, D, H, drop=0.2 if tokens > 1 else 0.0)
    want, grads = mlp_float64(c, activation)
    g = {k: v.cuda() for k, v in c.items()}
    out, state = dft.expert_mlp(g["x"], g["experts"], g["weights"], g["w1"], g["w2"], g["b1"], g["b2"],
                                activation=activation)
    got = dft.expert_mlp_grad(g["dout"], state, g["weights"], g["w1"], g["w2"], activation=activation)

    def rel(a, b):
        a = a.double().cpu()
        assert bool(torch.isfinite(a).all())
        return float((a - b).norm() / b.norm().clamp(min=1e-30))

    assert rel(out, want) <= 6 * 2.0 ** -8
    for name, value in got._asdict().items():
        assert rel(value, grads[name]) <= 6 * 2.0 ** -8, name


@pytest.mark.parametrize("tokens,top_k,D", [(0, 2, 16), (3, 1, 0)], ids=["no tokens", "no columns"])
def test_empty_rows(tokens, top_k, D):
    experts = torch.zeros(tokens, top_k, dtype=torch.int32, device="cuda")
    x = torch.zeros(tokens, D, dtype=torch.bfloat16, device="cuda")
    weights = torch.ones(tokens, top_k, device="cuda")
    offsets, order, position = dft.expert_sort(experts, 2)
    assert offsets.tolist() == [0, tokens * top_k, tokens * top_k] and order.numel() == tokens * top_k
    rows = dft.expert_gather(x, position)
    assert rows.shape == (tokens * top_k, D)
    assert torch.equal(dft.expert_combine(rows, position, weights), x)
    dy, dw = dft.expert_combine_grad(x, rows, position, weights)
    assert dy.shape == rows.shape and bool((dw == 0).all())


def test_routed_block_without_tokens():
    w1, w2 = (torch.ones(3, *s, dtype=torch.bfloat16, device="cuda") for s in ((16, 24), (24, 16)))
    b1 = torch.ones(3, 24, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda")
    weights = torch.zeros(0, 2, device="cuda")
    out, state = dft.expert_mlp(x, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), weights, w1, w2, b1)
    grads = dft.expert_mlp_grad(out, state, weights, w1, w2)
    assert out.shape == x.shape == grads.x.shape
    for g, shape in ((grads.w1, w1.shape), (grads.b1, b1.shape), (grads.w2, w2.shape), (grads.b2, (3, 16))):
        assert g.shape == shape and bool((g == 0).all())


def test_one_expert_chosen_by_every_choice():
    """The same expert in each of a token's choices: as many rows of its own."""
    gen = torch.Generator().manual_seed(97)
    x = ref.draw(gen, (5, 40), torch.float16)
    y = ref.draw(gen, (15, 40), torch.float16, True)
    experts = torch.full((5, 3), 2, dtype=torch.int32, device="cuda")
    _, order, position = dft.expert_sort(experts, 4)
    assert torch.equal(position.cpu(), torch.arange(15, dtype=torch.int32).view(5, 3))
    assert torch.equal(dft.expert_gather(x.cuda(), position).cpu(), x.repeat_interleave(3, 0))
    weights = torch.tensor([1.0, 2.0, 4.0], device="cuda").repeat(5, 1)
    want = (y.double().view(5, 3, 40) * weights.cpu().double()[..., None]).sum(1)  # small whole numbers: exact
    assert torch.equal(dft.expert_combine(y.cuda(), position, weights).cpu().double(), want)


def test_routed_block_captured():
    """Forward and backward of the routed block in a graph, replayed with new routes between eager calls."""
    gen = torch.Generator().manual_seed(99)
    c = {k: v.cuda() for k, v in mlp_case(gen, 48, 2, 6, 64, 128).items()}

    def step():
        out, state = dft.expert_mlp(c["x"], c["experts"], c["weights"], c["w1"], c["w2"], c["b1"], c["b2"])
        return [out, *dft.expert_mlp_grad(c["dout"], state, c["weights"], c["w1"], c["w2"])]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for k in range(4):
        c["experts"].copy_(torch.randint(0, 6, (48, 2), generator=gen, dtype=torch.int32))
        eager = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b), k
