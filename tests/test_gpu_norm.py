"""Layer norm, its gradients and dropout on the GPU against float64, with the
bounds of norm_reference.py: widths on both sides of every shape's limit,
pitches and addresses aligned to nothing, all three types, with and without the
residual stream, dropout and its mask, captured graphs, other streams."""

from __future__ import annotations

import math

import pytest
import torch

import dense_fp32_tiled_amd as dft
import norm_reference as ref
from linear_reference import Guarded, assert_within, empty

pytestmark = pytest.mark.gpu

EPS = 1e-5
KINDS = {torch.bfloat16: dft.VALUE_BF16, torch.float16: dft.VALUE_F16, torch.float32: dft.VALUE_F32}


@pytest.fixture(scope="module", autouse=True)
def gpu(gemm_lib):
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def normal(gen, *shape, dtype, mean=0.0, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale + mean).to(dtype)


def stream():
    return torch.cuda.current_stream().cuda_stream


# rows, cols, pitch beyond the width, first element's place
SIZES = [(1, 1, 0, 0), (3, 7, 2, 1), (5, 64, 0, 0), (17, 512, 8, 8), (16, 513, 0, 1), (9, 1024, 0, 0), (6, 1025, 1, 0),
         (7, 2048, 0, 3), (5, 2056, 0, 0), (12, 4096, 0, 0), (4, 4099, 3, 1), (3, 8192, 0, 0), (2, 8193, 0, 0),
         (4, 16384, 16, 0), (3, 16385, 0, 1), (2, 40000, 0, 0), (1200, 24, 0, 0), (1100, 1536, 0, 0), (6, 8, 0, 0),
         (9, 9, 0, 1), (5, 15, 2, 0), (3, 2049, 0, 0), (600, 8200, 0, 0), (3, 16383, 0, 1), (700, 4095, 1, 0)]
IDS = ["x".join(map(str, s)) for s in SIZES]


@pytest.mark.parametrize("joined", ["plain", "residual", "dropout", "both"])
@pytest.mark.parametrize("kind", list(ref.TYPES))
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_norm(size, kind, joined):
    (rows, cols, pad, offset), dtype = size, ref.TYPES[kind]
    gen = torch.Generator().manual_seed(rows * 7 + cols)
    x, w, b = normal(gen, rows, cols, dtype=dtype, mean=0.5), normal(gen, cols, dtype=dtype, mean=1), normal(gen, cols, dtype=dtype)
    residual = normal(gen, rows, cols, dtype=dtype) if joined in ("residual", "both") else None
    p = 0.3 if joined in ("dropout", "both") and rows * cols < 200000 else 0.0
    seed, counter = 0xFEDCBA9876543210, 5 << 33
    gx, gy, gt = Guarded(x, pad, offset), empty((rows, cols), dtype, pad=pad, offset=offset), empty((rows, cols), dtype, pad=pad)
    gw, gb = Guarded(w[None], 0, 1), Guarded(b[None], 0, 3)
    gm, gs = empty((1, rows), torch.float32, offset=1), empty((1, rows), torch.float32, offset=2)
    a = dft.LayerNormArgs(value_type=KINDS[dtype], eps=EPS, p=p, seed=seed, offset=counter, rows=rows, cols=cols,
                          x=gx.ptr, ldx=gx.ld, weight=gw.ptr, bias=gb.ptr, total=gt.ptr, ldt=gt.ld, y=gy.ptr, ldy=gy.ld,
                          mean=gm.ptr, rstd=gs.ptr)
    if residual is not None:
        gr = Guarded(residual, pad, offset)
        a.residual, a.ldr = gr.ptr, gr.ld
    assert dft.gemm_layer_norm(a, stream()) == dft.GEMM_OK
    torch.cuda.synchronize()
    for g, name in ((gy, "y"), (gm, "mean"), (gs, "rstd")):
        g.assert_rest_untouched(name)
    written = residual is not None or p > 0
    gt.assert_rest_untouched("total", None if written else torch.zeros(rows, dtype=torch.bool))
    total = x
    if written:
        total = gt.value()
        assert_within(total, ref.dropped(x, ref.keep(rows, cols, p, seed, counter), residual, dtype), "total")
    want = ref.normed(total, w, b, EPS)
    assert_within(gm.value()[0], want["mean"], "mean")
    assert_within(gs.value()[0], want["rstd"], "rstd")
    assert_within(gy.value(), want["y"], "y")


@pytest.mark.parametrize("joined", ["plain", "stream", "dropout", "both"])
@pytest.mark.parametrize("kind", list(ref.TYPES))
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_norm_grad(size, kind, joined):
    (rows, cols, pad, offset), dtype = size, ref.TYPES[kind]
    gen = torch.Generator().manual_seed(rows * 5 + cols)
    total, dy, w = normal(gen, rows, cols, dtype=dtype, mean=0.5), normal(gen, rows, cols, dtype=dtype), normal(gen, cols, dtype=dtype, mean=1)
    dstream = normal(gen, rows, cols, dtype=dtype) if joined in ("stream", "both") else None
    p = 0.3 if joined in ("dropout", "both") and rows * cols < 200000 else 0.0
    seed, counter = 77, 3
    mean = total.double().mean(1).float()
    rstd = (total.double().var(1, correction=0) + EPS).rsqrt().float()
    gy, gt, gw = Guarded(dy, pad, offset), Guarded(total, pad, offset), Guarded(w[None], 0, 1)
    gm, gs = Guarded(mean[None], 0, 1), Guarded(rstd[None], 0, 2)
    gd, gx = empty((rows, cols), dtype, pad=pad, offset=offset), empty((rows, cols), dtype, pad=pad)
    dw, db = empty((1, cols), torch.float32, offset=1), empty((1, cols), torch.float32, offset=3)
    a = dft.LayerNormGradArgs(value_type=KINDS[dtype], p=p, seed=seed, offset=counter, rows=rows, cols=cols, dY=gy.ptr,
                              ldy=gy.ld, total=gt.ptr, ldt=gt.ld, mean=gm.ptr, rstd=gs.ptr, weight=gw.ptr, dtotal=gd.ptr,
                              lddt=gd.ld, dx=gx.ptr, lddx=gx.ld, dweight=dw.ptr, dbias=db.ptr)
    if dstream is not None:
        gr = Guarded(dstream, pad, offset)
        a.dstream, a.lds = gr.ptr, gr.ld
    need = dft.gemm_layer_norm_grad_workspace_bytes(a, torch.cuda.get_device_properties(0).multi_processor_count)
    ws = empty((1, need // 4), torch.float32, offset=4)
    a.workspace, a.workspace_bytes = ws.ptr, need
    assert dft.gemm_layer_norm_grad(a, stream()) == dft.GEMM_OK
    torch.cuda.synchronize()
    for g, name in ((gd, "dtotal"), (gx, "dx"), (dw, "dweight"), (db, "dbias"), (ws, "workspace")):
        g.assert_rest_untouched(name)
    want = ref.gradients(dy, total, mean, rstd, w, dstream, ref.keep(rows, cols, p, seed, counter))
    for g, name in ((gd, "residual"), (gx, "x"), (dw, "weight"), (db, "bias")):
        value = g.value()
        assert_within(value[0] if name in ("weight", "bias") else value, want[name], name)


@pytest.mark.parametrize("kind", list(ref.TYPES))
@pytest.mark.parametrize("size", [(1, 1, 0, 0), (3, 7, 2, 1), (40, 64, 0, 0), (64, 513, 1, 1), (9, 4096, 8, 8), (2, 16385, 0, 3)],
                         ids=lambda s: "x".join(map(str, s)))
def test_dropout(size, kind):
    (rows, cols, pad, offset), dtype = size, ref.TYPES[kind]
    gen = torch.Generator().manual_seed(cols)
    x, r = normal(gen, rows, cols, dtype=dtype), normal(gen, rows, cols, dtype=dtype)
    for p, residual, place in ((0.1, None, "new"), (0.5, r, "new"), (0.0, r, "new"), (1.0, r, "x"), (0.25, None, "x"),
                               (0.75, r, "residual"), (1.0, None, "new")):
        gx, gy, gr = Guarded(x, pad, offset), empty((rows, cols), dtype, pad=pad, offset=offset), Guarded(r, pad, offset)
        out = {"new": gy, "x": gx, "residual": gr}[place]
        st = dft.gemm_dropout(KINDS[dtype], rows, cols, p, 9, 1 << 63, None, gx.ptr, gx.ld,
                              None if residual is None else gr.ptr, gr.ld, out.ptr, out.ld, stream())
        assert st == dft.GEMM_OK
        torch.cuda.synchronize()
        for g in (gx, gy, gr):
            g.assert_rest_untouched("y", None if g is not gy or place == "new" else torch.zeros(rows, dtype=torch.bool))
        factors = ref.keep(rows, cols, p, 9, 1 << 63) if p < 1 else torch.zeros(rows, cols, dtype=torch.float64)
        assert_within(out.value(), ref.dropped(x, factors, residual, dtype), (p, place))


def test_dropout_share_and_independence():
    """The share that is kept, and of pairs that differ by row, column, offset and seed: each count of n draws is within
    six standard deviations, sqrt(n q (1 - q)), of n q."""
    rows, cols, p = 512, 1024, 0.3
    x = torch.ones(rows, cols, device="cuda")
    q = 1 - ref.drop_count(p) / 65536
    a, b, c = (dft.dropout(x, p, *k) != 0 for k in ((1, 0), (1, 1), (2, 0)))
    assert not torch.equal(a, b) and not torch.equal(a, c)
    pairs = {"all": a, "offset": a & b, "seed": a & c, "row": a[1:] & a[:-1], "column": a[:, 1:] & a[:, :-1],
             "block": a[:, 8:] & a[:, :-8]}
    for name, kept in pairs.items():
        share, n = q if name == "all" else q * q, kept.numel()
        # (neighbours overlap: up to three times the variance of independent pairs)
        assert abs(float(kept.sum()) - n * share) <= 6 * math.sqrt(3 * n * share * (1 - share)), name


def test_masked_values_do_not_matter():
    """Whatever a dropped element holds, its result is the residual's; its gradient is zero."""
    x = torch.randn(8, 100, device="cuda")
    kept = dft.dropout(torch.ones_like(x), 0.4, 5) != 0
    bad = torch.where(kept, x, torch.tensor([math.nan, math.inf] * 50, device="cuda"))
    r = torch.randn_like(x)
    assert torch.equal(dft.dropout(bad, 0.4, 5, residual=r), dft.dropout(x, 0.4, 5, residual=r))
    y, state = dft.layer_norm(x, residual=r, p=0.4, seed=5)
    y2, state2 = dft.layer_norm(bad, residual=r, p=0.4, seed=5)
    assert torch.equal(y, y2) and all(torch.equal(s, t) for s, t in zip(state, state2))
    g = dft.layer_norm_grad(torch.randn_like(x), state, p=0.4, seed=5)
    assert bool(((g.x == 0) == ~kept).all())


def test_rows_of_one_value_and_without_weight():
    """A constant row: y is the bias, rstd eps^-1/2; a NaN or infinity stays in its row."""
    x = torch.full((4, 1000), 3.0, device="cuda")
    bias = torch.randn(1000, device="cuda")
    y, state = dft.layer_norm(x, None, bias)
    assert torch.equal(y, bias.expand(4, 1000)) and torch.equal(state.mean, x[:, 0])
    assert_within(state.rstd.cpu(), (torch.full((4,), EPS ** -0.5, dtype=torch.float64), torch.full((4,), 316.3 * 2e-7, dtype=torch.float64)), "rstd")
    assert state.total is x
    x = torch.randn(4, 1000, device="cuda")
    clean = dft.layer_norm(x)[0]
    x[1, 17], x[2, 999] = math.nan, math.inf
    y, _ = dft.layer_norm(x)
    assert bool(y[1:3].isnan().all()) and torch.equal(y[[0, 3]], clean[[0, 3]])


def test_far_mean_keeps_its_digits():
    """Deviations of 1 around 4096: the two-pass variance."""
    gen = torch.Generator().manual_seed(3)
    x = (torch.randn(6, 3000, generator=gen) + 4096).float()
    y, state = dft.layer_norm(x.cuda())
    want = ref.normed(x, None, None, EPS)
    for got, name in ((state.mean, "mean"), (state.rstd, "rstd"), (y, "y")):
        assert_within(got.cpu(), want[name], name)
    # (whatever the bound: the mean squared deviation is right to a millionth part)
    var = x.double().var(1, correction=0)
    assert bool((((state.rstd.cpu().double() ** -2 - EPS) / var - 1).abs() < 1e-4).all())


def test_gradient_against_differences():
    """The whole block's loss along a random direction, in float32 against central differences of float64."""
    gen = torch.Generator().manual_seed(11)
    rows, cols, p, seed = 6, 70, 0.2, 123
    x, r, w, b, dy, ds = (torch.randn(*s, generator=gen) for s in ((rows, cols),) * 2 + ((cols,),) * 2 + ((rows, cols),) * 2)
    factors = ref.keep(rows, cols, p, seed, 0)

    def loss(x, r, w, b):
        t = x * factors + r
        m = t.mean(1, keepdim=True)
        y = (t - m) * ((t - m).square().mean(1, keepdim=True) + EPS).rsqrt() * w + b
        return (y * dy.double()).sum() + (t * ds.double()).sum()

    y, state = dft.layer_norm(x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), p=p, seed=seed)
    g = dft.layer_norm_grad(dy.cuda(), state, w.cuda(), dtotal=ds.cuda(), p=p, seed=seed)
    leaves = [t.double() for t in (x, r, w, b)]
    for i, got in enumerate((g.x, g.residual, g.weight, g.bias)):
        way = torch.randn(leaves[i].shape, generator=gen, dtype=torch.float64)
        h = 1e-4
        up, down = list(leaves), list(leaves)
        up[i], down[i] = leaves[i] + h * way, leaves[i] - h * way
        slope = float(loss(*up) - loss(*down)) / (2 * h)
        mine = float((got.cpu().double() * way).sum())
        # third derivatives of the block are of order 10^2 here: h^2 / 6 of them, and fp32's roundings of the sums
        assert abs(mine - slope) <= 1e-5 * (1 + float((got.cpu().double() * way).abs().sum())), (i, mine, slope)


def test_no_rows_and_what_is_wanted():
    x, w = torch.zeros(0, 40, device="cuda"), torch.ones(40, device="cuda")
    y, state = dft.layer_norm(x, w, w, residual=x, p=0.5, seed=1)
    assert y.shape == (0, 40) and state.mean.shape == (0,)
    g = dft.layer_norm_grad(x, state, w, p=0.5, seed=1)
    assert float(g.weight.abs().sum()) == 0 == float(g.bias.abs().sum()) and g.x.shape == (0, 40)
    assert dft.dropout(x, 0.5, 1).shape == (0, 40)
    x = torch.randn(6, 40, device="cuda")
    _, state = dft.layer_norm(x, w, p=0.5, seed=1)
    every = dft.layer_norm_grad(x, state, w, p=0.5, seed=1)
    for names in (("x",), ("residual",), ("weight",), ("bias",), ("x", "bias"), ("weight", "residual"), ()):
        some = dft.layer_norm_grad(x, state, w, p=0.5, seed=1, want=names)
        for n in ("x", "residual", "weight", "bias"):
            assert torch.equal(getattr(some, n), getattr(every, n)) if n in names else getattr(some, n) is None
    plain = dft.layer_norm_grad(x, state, w)
    assert plain.x is plain.residual
    with pytest.raises(ValueError, match="want"):
        dft.layer_norm_grad(x, state, w, want=("y",))


def test_refused_tensors():
    x = torch.randn(4, 16, device="cuda")
    for kw in (dict(weight=x[0, :8]), dict(weight=x[0].half()), dict(residual=x[:3]), dict(residual=x.half()),
               dict(residual=x.t()), dict(p=1.5), dict(p=0.5, seed=-1), dict(p=0.5, seed=1 << 64),
               dict(p=0.5, step=torch.zeros(1, device="cuda")), dict(total=torch.empty_like(x)), dict(out=x[:, :8]),
               dict(bias=x[0].cpu())):
        with pytest.raises((TypeError, ValueError)):
            dft.layer_norm(x, **kw)
    for bad in (x[0], x[None], x.t()[::2], x.expand(4, 16)[:, ::2]):
        with pytest.raises((TypeError, ValueError)):
            dft.dropout(bad, 0.5, 1)
    with pytest.raises(dft.GemmError):
        dft.layer_norm(x, out=x)
    with pytest.raises(dft.GemmError):
        dft.layer_norm(x, eps=-1.0)
    with pytest.raises(dft.GemmError):
        dft.layer_norm(x, residual=x, total=x, out=x)


def test_total_in_place():
    gen = torch.Generator().manual_seed(2)
    for cols in (64, 4096, 20000):
        x, r = normal(gen, 5, cols, dtype=torch.bfloat16).cuda(), normal(gen, 5, cols, dtype=torch.bfloat16).cuda()
        y, state = dft.layer_norm(x, residual=r, p=0.1, seed=4)
        for over in ("x", "residual"):
            a, b = x.clone(), r.clone()
            y2, state2 = dft.layer_norm(a, residual=b, p=0.1, seed=4, total=a if over == "x" else b)
            assert torch.equal(y, y2) and torch.equal(state2.total, state.total)
            assert state2.total is (a if over == "x" else b)
        both, _ = dft.layer_norm(x, residual=x)
        a = x.clone()
        assert torch.equal(dft.layer_norm(a, residual=a, total=a)[0], both)


def test_streams_and_graphs():
    """Another stream's results, and a captured pass whose mask follows a counter on the device, replayed among eager
    work."""
    gen = torch.Generator().manual_seed(8)
    x, r, w = (normal(gen, *s, dtype=torch.bfloat16).cuda() for s in ((300, 520), (300, 520), (520,)))
    dy = normal(gen, 300, 520, dtype=torch.bfloat16).cuda()

    def step_of(n, step=None):
        y, state = dft.layer_norm(x, w, residual=r, p=0.2, seed=3, offset=n, step=step)
        g = dft.layer_norm_grad(dy, state, w, p=0.2, seed=3, offset=n, step=step)
        z = dft.dropout(y, 0.2, 3, offset=n, step=step)
        return [y, *state, *g, z]

    want = [step_of(100 + n) for n in range(4)]
    assert not torch.equal(want[0][-1], want[1][-1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, state = dft.layer_norm(x, w, residual=r, p=0.2, seed=3, offset=100, stream=side)
    g = dft.layer_norm_grad(dy, state, w, p=0.2, seed=3, offset=100, stream=side)
    z = dft.dropout(y, 0.2, 3, offset=100, stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([y, *state, *g, z], want[0]))
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step_of(100, step)
        step += 1
    for n in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want[n])), n
        step_of(7)  # eager work between the replays
    step.fill_(-100)  # (a counter may run below its start)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(held, step_of(0)))


def test_places_past_32_bits():
    """More than 2^32 elements: the last rows against the definition."""
    rows, cols = 66000, 65544
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    y = dft.dropout(x, 0.5, 21, out=x)
    for row in (0, 65535, rows - 1):
        assert torch.equal(y[row].double().cpu(), ref.keep_row(row, cols, 0.5, 21, 0)), row
    del x, y
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")  # (a pitch: the chunks are found by division)
    view = x[:, :65536]
    y, state = dft.layer_norm(view, p=0.5, seed=21, total=view, out=torch.empty(rows, 65536, dtype=torch.bfloat16, device="cuda"))
    row = rows - 1
    assert torch.equal(state.total[row].double().cpu(), ref.keep_row(row, 65536, 0.5, 21, 0))
    want = ref.normed(state.total[row:].cpu(), None, None, EPS)
    assert_within(y[row:].cpu(), want["y"], "y")
