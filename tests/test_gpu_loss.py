"""The cross entropy over a vocabulary and its gradients on the GPU against
float64, with the bounds of loss_reference.py: every tile, both layouts of the
vocabulary's matrix, one piece and many, odd sizes and pitches, rows without a
target, captured graphs, other streams."""

from __future__ import annotations

import math

import pytest
import torch

import dense_fp32_tiled_amd as dft
import loss_reference as ref
from linear_reference import KINDS, TYPES, Guarded, assert_within, empty

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu(gemm_lib):
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def stream():
    return torch.cuda.current_stream().cuda_stream


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def problem(M, N, K, dtype, seed, scale=2.0, none=0.15):
    gen = torch.Generator().manual_seed(seed)
    a = torch.randn(M, K, generator=gen).to(dtype)
    b = (torch.randn(K, N, generator=gen) * scale * max(K, 1) ** -0.5).to(dtype)
    t = torch.randint(0, N, (M,), generator=gen)
    odd = torch.tensor([-1, -100, N, N + 7, -2 ** 31, 2 ** 31 - 1])
    t = torch.where(torch.rand(M, generator=gen) < none, odd[torch.randint(0, 6, (M,), generator=gen)], t)
    g = torch.rand(M, generator=gen) / max(M, 1)
    return a, b, t, g


def run_forward(a, b, targets, transposed=False, pad=(0, 0), offset=0, piece=0, variant=0, wide=False):
    (M, K), N = a.shape, b.shape[1]
    ga, gb = Guarded(a, pad[0], offset), Guarded(b.t() if transposed else b, pad[1], offset)
    t = targets.to(torch.int64 if wide else torch.int32).cuda()
    loss, lse = empty((1, M), torch.float32, offset=1), empty((1, M), torch.float32, offset=3)
    c = dft.CrossEntropyArgs(input_type=KINDS[a.dtype], target_type=int(wide), b_transposed=int(transposed), variant=variant,
                             M=M, N=N, K=K, piece=piece, A=ga.ptr, lda=ga.ld, B=gb.ptr, ldb=gb.ld, targets=t.data_ptr(),
                             loss=loss.ptr, lse=lse.ptr)
    need = dft.gemm_cross_entropy_workspace_bytes(c, cus())
    assert need >= 0, need
    ws = empty((1, -(-need // 4)), torch.float32, offset=4)
    c.workspace, c.workspace_bytes = ws.ptr, need
    assert dft.gemm_cross_entropy(c, stream()) == dft.GEMM_OK
    torch.cuda.synchronize()
    for g, name in ((loss, "loss"), (lse, "lse"), (ws, "workspace")):
        g.assert_rest_untouched(name)
    return loss.value()[0], lse.value()[0]


def run_grad(g, a, b, targets, lse, transposed=False, pad=(0, 0), offset=0, piece=0, variant=0, wide=False, a_dtype=None,
             b_dtype=None, want="ab"):
    (M, K), N, dtype = a.shape, b.shape[1], a.dtype
    a_dtype, b_dtype = a_dtype or dtype, b_dtype or dtype
    ga, gb = Guarded(a, pad[0], offset), Guarded(b.t() if transposed else b, pad[1], offset)
    t = targets.to(torch.int64 if wide else torch.int32).cuda()
    gl, gg = Guarded(lse[None].float(), 0, 1), Guarded(g[None], 0, 2)
    da, db = empty((M, K), a_dtype, pad=pad[0], offset=offset), empty((N, K) if transposed else (K, N), b_dtype, pad=pad[1], offset=offset)
    c = dft.CrossEntropyGradArgs(input_type=KINDS[dtype], target_type=int(wide), b_transposed=int(transposed), variant=variant,
                                 a_grad_type=int(a_dtype == torch.float32), b_grad_type=int(b_dtype == torch.float32), M=M,
                                 N=N, K=K, piece=piece, A=ga.ptr, lda=ga.ld, B=gb.ptr, ldb=gb.ld, targets=t.data_ptr(),
                                 lse=gl.ptr, dloss=gg.ptr)
    if "a" in want:
        c.dA, c.ldda = da.ptr, da.ld
    if "b" in want:
        c.dB, c.lddb = db.ptr, db.ld
    need = dft.gemm_cross_entropy_grad_workspace_bytes(c, cus())
    assert need >= 0, need
    ws = empty((1, -(-need // 4)), torch.float32, offset=4)
    c.workspace, c.workspace_bytes = ws.ptr, need
    assert dft.gemm_cross_entropy_grad(c, stream()) == dft.GEMM_OK
    torch.cuda.synchronize()
    nothing = torch.zeros(1, dtype=torch.bool)
    da.assert_rest_untouched("dA", None if "a" in want else nothing.expand(M))
    db.assert_rest_untouched("dB", None if "b" in want else nothing.expand(db.rows))
    ws.assert_rest_untouched("workspace")
    return da.value(), db.value().t() if transposed else db.value()


# tokens, words, width, pitches beyond the widths, first element's place
SIZES = [(1, 1, 1, (0, 0), 0), (3, 5, 7, (1, 2), 1), (5, 1000, 64, (0, 0), 0), (33, 300, 40, (0, 4), 0), (64, 256, 64, (0, 0), 0),
         (130, 520, 72, (8, 8), 8), (257, 513, 129, (0, 0), 0), (24, 4000, 128, (0, 0), 0), (300, 1001, 200, (8, 7), 0),
         (7, 777, 1030, (2, 0), 3)]
IDS = ["x".join(map(str, s[:3])) for s in SIZES]


@pytest.mark.parametrize("variant", range(dft.LINEAR_COUNT), ids=list(dft.LINEAR_NAMES.values()))
@pytest.mark.parametrize("transposed", [False, True], ids=["columns", "rows"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_loss_and_gradients(size, kind, transposed, variant):
    M, N, K, pad, offset = size
    a, b, t, g = problem(M, N, K, TYPES[kind], M + N + K)
    for piece in (0, 256):
        kw = dict(transposed=transposed, pad=pad, offset=offset, piece=piece, variant=variant, wide=piece > 0)
        loss, lse = run_forward(a, b, t, **kw)
        want = ref.forward(a, b, t)
        assert_within(lse, want["lse"], "lse")
        assert_within(loss, want["loss"], "loss")
        da, db = run_grad(g, a, b, t, lse, **kw)
        want = ref.gradients(g, a, b, t, lse, pieces=-(-N // 256))
        assert_within(da, want["a"], "da")
        assert_within(db, want["b"], "db")


@pytest.mark.parametrize("types", [(torch.float32, None), (None, torch.float32), (torch.float32, torch.float32)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_fp32_gradients_and_one_alone(kind, types):
    a, b, t, g = problem(70, 600, 90, TYPES[kind], 4)
    lse = ref.forward(a, b, t)["lse"][0].float()
    want = ref.gradients(g, a, b, t, lse, *types, pieces=3)
    for piece in (0, 256):
        da, db = run_grad(g, a, b, t, lse, a_dtype=types[0], b_dtype=types[1], piece=piece)
        assert_within(da, want["a"], "da")
        assert_within(db, want["b"], "db")
        assert torch.equal(run_grad(g, a, b, t, lse, a_dtype=types[0], piece=piece, want="a")[0], da)
        assert torch.equal(run_grad(g, a, b, t, lse, b_dtype=types[1], piece=piece, want="b")[1], db)


# sizes of whole rounds of the largest tiles: many per workgroup, a last round that is cut along the contraction, several
# pieces, and rows longer than one step of the join
LARGE = [(4096, 8192, 128, False, 0), (5000, 8192, 4096, True, 0), (5000, 8192, 4096, False, 2048), (2, 150000, 512, True, 0),
         (1500, 40001, 520, False, 8192),
         # short contractions of many tiles: of the logits, of dB, of both; one contraction tile
         (130, 70001, 72, False, 0), (300, 40000, 136, True, 0), (520, 14003, 200, False, 0), (520, 14000, 712, True, 0),
         (66, 3000, 64, True, 256), (100, 900, 63, False, 0), (4, 40000, 1000, False, 0)]


@pytest.mark.parametrize("size", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_large(size):
    M, N, K, transposed, piece = size
    a, b, t, g = (x.cuda() for x in problem(M, N, K, torch.bfloat16, N))
    laid = b.t().contiguous().t() if transposed else b
    loss, lse = dft.linear_cross_entropy(a, laid, t, piece=piece)
    want = ref.forward(a, b, t)
    assert_within(lse.cpu(), [x.cpu() for x in want["lse"]], "lse")
    assert_within(loss.cpu(), [x.cpu() for x in want["loss"]], "loss")
    grads = dft.linear_cross_entropy_grad(g, a, laid, t, lse, piece=piece)
    want = ref.gradients(g, a, b, t, lse, pieces=-(-N // (piece or N)))
    for got, name in ((grads.a, "a"), (grads.b, "b")):
        value, tol = want[name]
        bad = ~((got.double() - value).abs() <= tol)
        assert not bool(bad.any()), (name, int(bad.sum()), bad.nonzero()[0].tolist())
    assert grads.b.stride() == laid.stride()


def test_small_probabilities_in_fp16():
    """A mean over many tokens of a flat distribution: dZ of 1e-9, held scaled; whole rows without target weigh nothing."""
    a, b, t, _ = problem(600, 3000, 64, torch.float16, 9, scale=0.1)
    for weight in (1e-7, 1.0 / 600, 3e4, 1e-30, 0.0):
        g = torch.full((600,), weight)
        g[::7] *= 0.01
        lse = ref.forward(a, b, t)["lse"][0].float()
        da, db = run_grad(g, a, b, t, lse, a_dtype=torch.float32, b_dtype=torch.float32)
        want = ref.gradients(g, a, b, t, lse, torch.float32, torch.float32)
        assert_within(da, want["a"], weight)
        assert_within(db, want["b"], weight)


def test_confident_rows_keep_their_digits():
    """A target far above every other word: the loss is the others' small share, not zero."""
    a = torch.eye(8, 64).to(torch.bfloat16)
    b = torch.zeros(64, 500, dtype=torch.bfloat16)
    t = torch.arange(8) * 60
    for i in range(8):
        b[i, t[i]] = 8.0 + 2 * i
    loss, lse = run_forward(a, b, t)
    exact = torch.log1p(499 * torch.exp(-(8.0 + 2 * torch.arange(8).double())))
    # The sum 1 + x is rounded at each addition to what already holds the 1, by u (1 + x) with x < 0.17: at most 15 in a
    # lane's 16 words, 2 over the wave's lanes and one for each other of the row's at most 16 pieces (500 words, 32 or
    # more in each): 32 of them, 38u.  (The logarithm's and the final sum's roundings are relative to the loss, as the
    # exponentials' 1e-5.)
    assert bool(((loss.double() - exact).abs() <= 38 * 2.0 ** -24 + 1e-5 * exact).all())


def test_rows_without_target_hold_anything():
    a, b, t, g = problem(40, 700, 64, torch.bfloat16, 3, none=0.4)
    gone = (t < 0) | (t >= 700)
    assert 5 < int(gone.sum()) < 35
    lse = ref.forward(a, b, t)["lse"][0].float()
    da, db = run_grad(g, a, b, t, lse)
    bad = a.clone()
    bad[gone] = math.nan
    bad_lse, bad_g = torch.where(gone, math.nan, lse), torch.where(gone, math.inf, g)
    loss, _ = run_forward(bad, b, t)
    assert bool((loss[gone] == 0).all()) and not bool(loss.isnan().any())
    da2, db2 = run_grad(bad_g, bad, b, t, bad_lse)
    assert torch.equal(da, da2) and torch.equal(db, db2) and float(da2[gone].abs().max()) == 0
    # no row has one
    none = torch.full_like(t, -1)
    loss, _ = run_forward(a, b, none)
    da, db = run_grad(g, a, b, none, lse)
    assert float(loss.abs().max()) == 0 == float(da.float().abs().max()) == float(db.float().abs().max())


def test_infinite_logits():
    """-infinity takes a word out of its row; a NaN or +infinity spoils its row alone."""
    a, b, t, g = problem(6, 300, 32, torch.bfloat16, 5, none=0.0)
    a = a.abs()
    b[:, 100] = -math.inf
    t = torch.tensor([1, 2, 3, 200, 299, 0])
    loss, lse = run_forward(a, b, t)
    keep = torch.ones(300, dtype=torch.bool)
    keep[100] = False
    want = ref.forward(a, b[:, keep], torch.where(t > 100, t - 1, t))
    assert_within(lse, want["lse"], "lse")
    assert_within(loss, want["loss"], "loss")
    b[:, 100] = 0
    clean = run_forward(a, b, t)
    a[2], a[4] = math.nan, math.inf
    got = run_forward(a, b, t)
    for x, y in zip(got, clean):
        assert bool(x[[2, 4]].isnan().all()) and torch.equal(x[[0, 1, 3, 5]], y[[0, 1, 3, 5]])


def test_gradient_against_differences():
    """The mean loss along random directions of a and b against central differences in float64."""
    a, b, t, g = problem(20, 90, 24, torch.bfloat16, 13)
    loss, lse = run_forward(a, b, t)
    da, db = run_grad(g, a, b, t, lse, a_dtype=torch.float32, b_dtype=torch.float32)
    gen = torch.Generator().manual_seed(1)

    def total(A, B):
        valid = (t >= 0) & (t < 90)
        z = A @ B
        each = torch.logsumexp(z, 1) - z.gather(1, torch.where(valid, t, 0)[:, None])[:, 0]
        return float((torch.where(valid, each, 0.0) * g.double()).sum())

    A, B, h = a.double(), b.double(), 1e-5
    for way_a, way_b, grad in ((torch.randn(A.shape, generator=gen).double(), 0, da), (0, torch.randn(B.shape, generator=gen).double(), db)):
        slope = (total(A + h * way_a, B + h * way_b) - total(A - h * way_a, B - h * way_b)) / (2 * h)
        way = way_a if torch.is_tensor(way_a) else way_b
        terms = grad.double() * way
        # dZ has 8 bits: each term's error is at most 2^-8 of the sums of |dZ| behind it, far less than |terms| / 50 here
        assert abs(float(terms.sum()) - slope) <= 0.02 * float(terms.square().sum().sqrt()) + 1e-6, (float(terms.sum()), slope)


@pytest.mark.parametrize("transposed", [False, True], ids=["columns", "rows"])
@pytest.mark.parametrize("size", [SIZES[k] for k in (1, 5, 6, 9)], ids=lambda s: "x".join(map(str, s[:3])))
def test_reads_only_what_was_copied(size, transposed, monkeypatch):
    """The debug build, whose LDS holds NaN before the first copy: the same results, every tile."""
    from dense_fp32_tiled_amd import build

    M, N, K, pad, offset = size
    a, b, t, g = problem(M, N, K, torch.bfloat16, M + N)
    poison = dft.library(build.POISON_LIB)
    for variant in range(dft.LINEAR_COUNT):
        kw = dict(transposed=transposed, pad=pad, offset=offset, variant=variant)
        clean = run_forward(a, b, t, **kw)
        clean += run_grad(g, a, b, t, clean[1], **kw)
        with monkeypatch.context() as patch:
            patch.setattr(dft, "library", lambda path=None: poison)
            dirty = run_forward(a, b, t, **kw)
            dirty += run_grad(g, a, b, t, dirty[1], **kw)
        assert all(torch.equal(x, y) for x, y in zip(clean, dirty)), variant


def test_no_tokens_no_width_and_lse_alone():
    b = torch.randn(16, 50, device="cuda").bfloat16()
    a, t = torch.zeros(0, 16, device="cuda").bfloat16(), torch.zeros(0, dtype=torch.int64, device="cuda")
    loss, lse = dft.linear_cross_entropy(a, b, t)
    assert loss.shape == lse.shape == (0,)
    g = dft.linear_cross_entropy_grad(lse, a, b, t, lse)
    assert g.a.shape == (0, 16) and g.b.shape == (16, 50) and float(g.b.float().abs().max()) == 0
    a, b, t = torch.zeros(4, 0, device="cuda").half(), torch.zeros(0, 50, device="cuda").half(), torch.arange(4, device="cuda")
    loss, lse = dft.linear_cross_entropy(a, b, t)
    assert bool(((loss - math.log(50)).abs() < 1e-6).all()) and torch.equal(loss, lse)
    g = dft.linear_cross_entropy_grad(loss, a, b, t, lse)
    assert g.a.shape == (4, 0) and g.b.shape == (0, 50)
    a, b = torch.randn(4, 24, device="cuda").half(), torch.randn(24, 50, device="cuda").half()
    none, lse = dft.linear_cross_entropy(a, b)
    assert none is None and torch.equal(lse, dft.linear_cross_entropy(a, b, t)[1])
    g = dft.linear_cross_entropy_grad(loss, a, b, t, lse, want=())
    assert g.a is None and g.b is None


def test_refused_tensors():
    a, b = torch.randn(4, 16, device="cuda").bfloat16(), torch.randn(16, 40, device="cuda").bfloat16()
    t, f = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    bad = [dict(b=b.half()), dict(b=b[:8]), dict(b=b[0]), dict(b=b.cpu()), dict(targets=t.float()), dict(targets=t[:3]),
           dict(targets=t.cpu()), dict(targets=t.short()), dict(a=a[0]), dict(a=a.t()), dict(b=b.expand(2, 16, 40)[0][:, ::2])]
    for kw in bad:
        with pytest.raises((TypeError, ValueError)):
            dft.linear_cross_entropy(**{**dict(a=a, b=b, targets=t), **kw})
        with pytest.raises((TypeError, ValueError)):
            dft.linear_cross_entropy_grad(**{**dict(dloss=f, a=a, b=b, targets=t, lse=f), **kw})
    for kw in (dict(lse=f[:2]), dict(dloss=f.double()), dict(targets=None), dict(a_dtype=torch.float16), dict(want=("c",))):
        with pytest.raises((TypeError, ValueError)):
            dft.linear_cross_entropy_grad(**{**dict(dloss=f, a=a, b=b, targets=t, lse=f), **kw})
    for kw in (dict(piece=100), dict(variant=99), dict(workspace=torch.empty(16, device="cuda"))):
        with pytest.raises(dft.GemmError):
            dft.linear_cross_entropy(a, b, t, **kw)
        with pytest.raises(dft.GemmError):
            dft.linear_cross_entropy_grad(f, a, b, t, f, **kw)


def test_streams_and_graphs():
    """Another stream's results, and both passes captured and replayed with new inputs among eager work; two captured
    graphs have a workspace each."""
    a, b, t, g = (x.cuda() for x in problem(300, 2100, 136, torch.bfloat16, 21))

    def both(**kw):
        loss, lse = dft.linear_cross_entropy(a, b, t, piece=1024, **kw)
        grads = dft.linear_cross_entropy_grad(g, a, b, t, lse, piece=1024, **kw)
        return [loss, lse, *grads]

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = both()
        graphs.append((graph, held))
    for n in range(4):
        t.copy_((t + 17 * n) % 2100)
        a.mul_(0.9)
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = both()
        for _, held in graphs:
            assert all(torch.equal(x, y) for x, y in zip(held, want)), n


@pytest.mark.parametrize("size", [(40000, 300, 24), (33000, 301, 25), (65536 + 3, 1000, 8)], ids=lambda s: "x".join(map(str, s)))
def test_more_tokens_than_are_taken_at_once(size):
    M, N, K = size
    a, b, t, g = (x.cuda() for x in problem(M, N, K, torch.float16, 8))
    for piece in (0, 256):
        loss, lse = dft.linear_cross_entropy(a, b, t, piece=piece)
        want = ref.forward(a, b, t)
        assert_within(lse, [x.cpu() for x in want["lse"]], "lse")
        assert_within(loss, [x.cpu() for x in want["loss"]], "loss")
        grads = dft.linear_cross_entropy_grad(g, a, b, t, lse, piece=piece)
        want = ref.gradients(g, a, b, t, lse, pieces=4)
        for got, name in ((grads.a, "a"), (grads.b, "b")):
            assert bool(((got.double() - want[name][0]).abs() <= want[name][1]).all()), name


@pytest.mark.parametrize("transposed", [False, True], ids=["columns", "rows"])
def test_places_past_32_bits(transposed):
    """A vocabulary's matrix of more than 2^32 bytes and 2^31 values: the loss, the tokens' gradient, and the words' at both ends."""
    M, N, K = 3, 540_000, 4096
    gen = torch.Generator(device="cuda").manual_seed(2)
    a = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    b = torch.empty((N, K) if transposed else (K, N), device="cuda", dtype=torch.bfloat16)
    for part in b.chunk(16):
        part.copy_(torch.randn(part.shape, device="cuda", generator=gen) * K ** -0.5)
    b = b.t() if transposed else b
    t = torch.tensor([0, N - 1, 300_000], device="cuda")
    g = torch.tensor([0.5, 0.25, 1.0], device="cuda")
    loss, lse = dft.linear_cross_entropy(a, b, t)
    grads = dft.linear_cross_entropy_grad(g, a, b, t, lse)
    pieces = [slice(i, min(i + 60_000, N)) for i in range(0, N, 60_000)]
    wide = a.double()
    z = torch.cat([wide @ b[:, p].double() for p in pieces], 1)
    e = (K + 2) * 2 * 2.0 ** -24 * float((wide.abs() @ b[:, pieces[0]].double().abs()).max()) * 1.5  # (any other word's, at most)
    exact = torch.logsumexp(z, 1)
    tol = 2 * e + 8 * 2.0 ** -24 * (N / 32 + 100)
    assert bool(((lse - exact).abs() <= tol).all())
    assert bool(((loss - (exact - z[torch.arange(M), t])).abs() <= tol).all())
    dz = torch.exp(z - lse.double()[:, None])
    dz[torch.arange(M), t] -= 1
    dz *= g.double()[:, None]
    da = sum(dz[:, p] @ b[:, p].double().t() for p in pieces)
    # dZ in two parts is exact beside its logits' e; da sums N products of it, and both are rounded once
    size = sum(dz[:, p].abs() @ b[:, p].double().abs().t() for p in pieces)
    assert bool(((grads.a.double() - da).abs() <= 2 * (e + N * 2.0 ** -23) * size + da.abs() * 2.0 ** -8 + 2.0 ** -30).all())
    for p in (pieces[0], slice(299_990, 300_010), pieces[-1]):
        want, size = wide.t() @ dz[:, p], wide.abs().t() @ dz[:, p].abs()
        assert bool(((grads.b[:, p].double() - want).abs() <= 2 * e * size + want.abs() * 2.0 ** -8 + 2.0 ** -30).all()), p
