"""Measured cases of the layer norm and its gradients, dropout, and the vocabulary's cross entropy with its gradients.

Each case is one pass through one operator, as a training or scoring step calls it:

  norm       total = dropout(x) + residual, y = (total - mean) rstd weight + bias over each row, with total, mean and
             rstd kept for the backward pass
  norm_grad  the gradients of x, residual, weight and bias for those of y and of total
  dropout    x keep / (1 - p) + residual, the keep bits drawn from a counter, never stored
  loss       each token's cross entropy of softmax(a b) with its target, the logits never stored
  loss_grad  the gradients of a and b

With ``own`` false they are computed from elementary torch operations in 32 bits.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # a serving step's tokens between two blocks: the call's latency
        {"name": "norm_step", "op": "norm", "type": "bf16", "rows": 16, "cols": 4096, "residual": True, "p": 0.0},
        # rows aligned to nothing
        {"name": "norm_ragged", "op": "norm", "type": "f16", "rows": 1000, "cols": 999, "residual": False, "p": 0.0},
        # a training step's tokens: the residual stream joined, with dropout: the rows' bytes
        {"name": "norm_large", "op": "norm", "type": "bf16", "rows": 16384, "cols": 4096, "residual": True, "p": 0.1},
        # gradients of a small batch held in 32 bits, odd width
        {"name": "norm_grad_ragged", "op": "norm_grad", "type": "f32", "rows": 1000, "cols": 513, "joined": False,
         "p": 0.0},
        # gradients of a training step's tokens, the residual stream's own gradient joined
        {"name": "norm_grad_large", "op": "norm_grad", "type": "bf16", "rows": 16384, "cols": 4096, "joined": True,
         "p": 0.1},
        # a small activation held in 32 bits, odd width
        {"name": "dropout_ragged", "op": "dropout", "type": "f32", "rows": 1000, "cols": 999, "residual": False,
         "p": 0.25},
        # a training step's widened activation: the rows' bytes
        {"name": "dropout_large", "op": "dropout", "type": "bf16", "rows": 8192, "cols": 16384, "residual": False,
         "p": 0.1},
        # a few tokens scored against a vocabulary that the embedding shares: the weights' bytes
        {"name": "loss_step", "op": "loss", "type": "bf16", "tokens": 24, "vocab": 131072, "width": 4096,
         "tied": True},
        # every size odd, the weights' rows aligned to nothing
        {"name": "loss_ragged", "op": "loss", "type": "f16", "tokens": 1000, "vocab": 32001, "width": 513,
         "tied": False},
        # a training step's loss: the matrix cores' rate
        {"name": "loss_large", "op": "loss", "type": "bf16", "tokens": 8192, "vocab": 131072, "width": 4096,
         "tied": True},
        # gradients of a fine-tuning batch over an odd vocabulary
        {"name": "loss_grad_ragged", "op": "loss_grad", "type": "f16", "tokens": 1000, "vocab": 32001, "width": 1000,
         "tied": False},
        # gradients of a training step's loss
        {"name": "loss_grad_large", "op": "loss_grad", "type": "bf16", "tokens": 8192, "vocab": 131072,
         "width": 4096, "tied": True},
    ]


def _log_size(rng, low, high):
    """A whole number of [low, high], even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A matrix width: three in four are multiples of 8, as models have them, the others any number."""
    w = _log_size(rng, low, high)
    return w if rng.random() < 0.25 else max(low, w - w % 8)


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "dropout", "loss", "loss_grad"))
    if op in ("loss", "loss_grad"):
        return {"op": op, "type": rng.choice(("bf16", "f16")), "tokens": _log_size(rng, 1, 8192),
                "vocab": _width(rng, 1000, 131072), "width": _width(rng, 64, 4096), "tied": rng.random() < 0.5}
    cols = _width(rng, 64, 16384)
    case = {"op": op, "type": rng.choice(("bf16", "f16", "f32")), "rows": _log_size(rng, 1, min(16384, (1 << 26) // cols)),
            "cols": cols, "p": rng.choice((0.0, 0.1, round(rng.uniform(0.01, 0.9), 3)))}
    case["joined" if op == "norm_grad" else "residual"] = rng.random() < 0.5
    if op == "dropout" and case["p"] == 0.0:
        case["p"] = 0.5
    return case


# ---- inputs ---------------------------------------------------------------------------
class _Inputs:
    """Draws of one seed on the GPU."""

    def __init__(self, seed, dtype):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        self.dtype = dtype

    def normal(self, *shape, scale=1.0, mean=0.0):
        x = torch.randn(*shape, device="cuda", generator=self.gen, dtype=torch.float32)
        return x.mul_(scale).add_(mean).to(self.dtype)

    def uniform(self, *shape):
        return torch.rand(*shape, device="cuda", generator=self.gen)

    def whole(self, low, high, *shape):
        return torch.randint(low, high, shape, device="cuda", generator=self.gen)


def _row_statistics(total):
    wide = total.float()
    mean = wide.mean(1)
    return mean, torch.rsqrt((wide - mean[:, None]).square().mean(1) + EPS)


def prepare(case, seed):
    draws = _Inputs(seed, TYPES[case["type"]])
    s = dict(case)
    if case["op"] in ("loss", "loss_grad"):
        t, v, d = case["tokens"], case["vocab"], case["width"]
        s["a"] = draws.normal(t, d)
        # logits of a few units, as a model's are
        w = draws.normal(*((v, d) if case["tied"] else (d, v)), scale=2.5 * d ** -0.5)
        s["b"] = w.t() if case["tied"] else w
        targets = draws.whole(0, v, t)
        s["targets"] = torch.where(draws.uniform(t) < 0.05, -100, targets)  # padding among the tokens
        if case["op"] == "loss_grad":
            logits = s["a"].float() @ s["b"].float()
            s["lse"] = torch.logsumexp(logits, 1)
            s["dloss"] = draws.uniform(t) / t  # a mean over tokens of different weights
        return s
    rows, cols = case["rows"], case["cols"]
    # the counter's start is the program's: a seed for the run, an offset for the place in it
    s["seed"], s["offset"] = 0x9E3779B97F4A7C15 ^ seed, 1000003 * seed + 17
    if case["op"] == "norm_grad":
        s["total"], s["dy"] = draws.normal(rows, cols, mean=0.3), draws.normal(rows, cols)
        s["mean"], s["rstd"] = _row_statistics(s["total"])
        s["weight"] = draws.normal(cols, scale=0.2, mean=1.0)
        s["dtotal"] = draws.normal(rows, cols) if case["joined"] else None
        return s
    s["x"] = draws.normal(rows, cols, mean=0.3)
    s["addend"] = draws.normal(rows, cols) if case["residual"] else None
    if case["op"] == "norm":
        s["weight"], s["bias"] = draws.normal(cols, scale=0.2, mean=1.0), draws.normal(cols, scale=0.2)
    return s


# ---- the plain forms ------------------------------------------------------------------
LOW = 0xFFFFFFFF


def _philox(seed, offset, blocks):
    """Philox4x32-10 (Salmon et al., 2011) with the seed as key and (block, offset) as counter: blocks x 4 words."""
    c0, c1 = blocks & LOW, blocks >> 32
    c2, c3 = torch.full_like(blocks, offset & LOW), torch.full_like(blocks, offset >> 32 & LOW)
    k0, k1 = seed & LOW, seed >> 32 & LOW
    for _ in range(10):
        m0, m1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # modulo 2^64
        c0, c1, c2, c3 = (m1 >> 32 & LOW) ^ c1 ^ k0, m1 & LOW, (m0 >> 32 & LOW) ^ c3 ^ k1, m0 & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    return torch.stack([c0, c1, c2, c3], 1)


def _drop_count(p):
    """Of 65536 equally likely 16-bit numbers, how many drop an element."""
    return int(math.floor(p * 65536 + 0.5))


def _kept(s, x):
    """dropout(x), x in 32 bits: a row's elements 8 i to 8 i + 7 take one block's eight 16-bit halves, low one first."""
    if s["p"] == 0.0:
        return x
    rows, cols = x.shape
    each = (cols + 7) // 8
    words = _philox(s["seed"], s["offset"], torch.arange(rows * each, device=x.device))
    halves = torch.stack([words & 0xFFFF, words >> 16], 2).view(rows, each * 8)[:, :cols]
    drop = _drop_count(s["p"])
    return torch.where(halves < drop, 0.0, x * (65536 / (65536 - drop)))


def _plain_dropout(s):
    y = _kept(s, s["x"].float())
    if s["addend"] is not None:
        y = y + s["addend"].float()
    return {"y": y.to(s["x"].dtype)}


def _plain_norm(s):
    dtype = s["x"].dtype
    out = {}
    total = s["x"]
    if s["p"] > 0 or s["addend"] is not None:
        total = out["total"] = _plain_dropout(s)["y"]
    out["mean"], out["rstd"] = _row_statistics(total)
    unit = (total.float() - out["mean"][:, None]) * out["rstd"][:, None]
    out["y"] = (unit * s["weight"].float() + s["bias"].float()).to(dtype)
    return out


def _plain_norm_grad(s):
    dtype, dy = s["dy"].dtype, s["dy"].float()
    unit = (s["total"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dunit = dy * s["weight"].float()
    dtotal = (dunit - dunit.mean(1, keepdim=True) - unit * (dunit * unit).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dtotal"] is not None:
        dtotal = dtotal + s["dtotal"].float()
    out = {"dresidual": dtotal.to(dtype), "dweight": (dy * unit).sum(0), "dbias": dy.sum(0)}
    if s["p"] > 0:
        out["dx"] = _kept(s, dtotal).to(dtype)
    return out


def _plain_logits(s):
    return s["a"].float() @ s["b"].float()


def _plain_loss(s):
    logits = _plain_logits(s)
    most = logits.amax(1, keepdim=True)
    lse = most[:, 0] + torch.log(torch.exp(logits - most).sum(1))
    valid = (s["targets"] >= 0) & (s["targets"] < s["vocab"])
    at = torch.where(valid, s["targets"], 0)
    loss = torch.where(valid, lse - logits.gather(1, at[:, None])[:, 0], 0.0)
    return {"loss": loss, "lse": lse}


def _plain_loss_grad(s):
    dtype = s["a"].dtype
    dz = torch.exp(_plain_logits(s) - s["lse"][:, None])
    valid = (s["targets"] >= 0) & (s["targets"] < s["vocab"])
    at = torch.where(valid, s["targets"], 0)
    dz[torch.arange(s["tokens"], device=dz.device), at] -= 1.0
    dz *= torch.where(valid, s["dloss"], 0.0)[:, None]
    return {"da": (dz @ s["b"].float().t()).to(dtype), "db": (s["a"].float().t() @ dz).to(dtype)}


# ---- the framework's calls --------------------------------------------------------------
def _own_norm(s):
    import dense_fp32_tiled_amd as dft

    y, kept = dft.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, residual=s["addend"], p=s["p"], seed=s["seed"],
                             offset=s["offset"])
    out = {"mean": kept.mean, "rstd": kept.rstd, "y": y}
    if s["p"] > 0 or s["addend"] is not None:
        out = {"total": kept.total, **out}
    return out


def _own_norm_grad(s):
    import dense_fp32_tiled_amd as dft

    kept = dft.NormState(s["total"], s["mean"], s["rstd"])
    g = dft.layer_norm_grad(s["dy"], kept, s["weight"], dtotal=s["dtotal"], p=s["p"], seed=s["seed"],
                            offset=s["offset"])
    out = {"dresidual": g.residual, "dweight": g.weight, "dbias": g.bias}
    if s["p"] > 0:
        out["dx"] = g.x
    return out


def _own_dropout(s):
    import dense_fp32_tiled_amd as dft

    return {"y": dft.dropout(s["x"], s["p"], s["seed"], s["offset"], residual=s["addend"])}


def _own_loss(s):
    import dense_fp32_tiled_amd as dft

    loss, lse = dft.linear_cross_entropy(s["a"], s["b"], s["targets"])
    return {"loss": loss, "lse": lse}


def _own_loss_grad(s):
    import dense_fp32_tiled_amd as dft

    g = dft.linear_cross_entropy_grad(s["dloss"], s["a"], s["b"], s["targets"], s["lse"])
    return {"da": g.a, "db": g.b}


def run(state):
    op = state["op"]
    if op == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    if op == "norm_grad":
        return _own_norm_grad(state) if own else _plain_norm_grad(state)
    if op == "dropout":
        return _own_dropout(state) if own else _plain_dropout(state)
    if op == "loss":
        return _own_loss(state) if own else _plain_loss(state)
    return _own_loss_grad(state) if own else _plain_loss_grad(state)


# ---- what a pass cannot do without ---------------------------------------------------------
def work(case):
    op, size = case["op"], 4 if case["type"] == "f32" else 2
    if op in ("loss", "loss_grad"):
        t, v, d = case["tokens"], case["vocab"], case["width"]
        once = size * (t * d + d * v)
        if op == "loss":
            return {"bytes": once + 16 * t, "flops": 2 * t * v * d + 4 * t * v}
        # the logits again, and the two gradients' products
        return {"bytes": 2 * once + 16 * t, "flops": 6 * t * v * d + 4 * t * v}
    rows, cols = case["rows"], case["cols"]
    each, drop = rows * cols, case["p"] > 0
    if op == "dropout":
        return {"bytes": size * each * (2 + case["residual"]), "flops": 2 * each}
    if op == "norm":
        # x and residual read; y and, where it is not x itself, total written
        passes = 2 + case["residual"] + (case["residual"] or drop)
        return {"bytes": size * (each * passes + 2 * cols) + 8 * rows, "flops": 8 * each}
    # dy, total and the stream's gradient read; the gradients of total and, with dropout, of x written
    return {"bytes": size * (each * (3 + case["joined"] + drop) + cols) + 8 * rows + 8 * cols, "flops": 14 * each}


# ---- the definitions in 64 bits --------------------------------------------------------------
def _wide_product(x, m):
    """The high and low 32 bits of x m for 32-bit x and m, from 16-bit digits."""
    x0, x1, m0, m1 = x % 65536, x // 65536, m % 65536, m // 65536
    middle = x1 * m0 + x0 * m0 // 65536
    other = x0 * m1 + middle % 65536
    return x1 * m1 + middle // 65536 + other // 65536, other % 65536 * 65536 + x0 * m0 % 65536


def _exact_keep(case, s, device):
    """The keep mask as factors: 0 or 1 / (1 - p), p the share of the 65536 numbers that drop."""
    rows, cols = case["rows"], case["cols"]
    if case["p"] == 0.0:
        return torch.ones(1, 1, dtype=torch.float64, device=device)
    each = -(-cols // 8)
    index = torch.arange(rows * each, device=device)
    counter = [index % 2 ** 32, index // 2 ** 32, index * 0 + s["offset"] % 2 ** 32, index * 0 + s["offset"] // 2 ** 32]
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32 % 2 ** 32]
    for turn in range(10):
        (h0, l0), (h1, l1) = _wide_product(counter[0], 0xD2511F53), _wide_product(counter[2], 0xCD9E8D57)
        ka, kb = (key[0] + turn * 0x9E3779B9) % 2 ** 32, (key[1] + turn * 0xBB67AE85) % 2 ** 32
        counter = [h1 ^ counter[1] ^ ka, l1, h0 ^ counter[3] ^ kb, l0]
    draws = torch.empty(rows, each, 4, 2, dtype=torch.int64, device=device)
    for word in range(4):
        draws[:, :, word, 0] = (counter[word] % 65536).view(rows, each)
        draws[:, :, word, 1] = (counter[word] // 65536).view(rows, each)
    drop = int(np.rint(case["p"] * 65536))
    keep = draws.view(rows, -1)[:, :cols] >= drop
    return keep.double() * (65536 / (65536 - drop))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("loss", "loss_grad"):
        a, b, targets = s["a"].double(), s["b"].double(), s["targets"].tolist()
        z = a @ b
        hit = [t for t, y in enumerate(targets) if 0 <= y < case["vocab"]]
        goal = [targets[t] for t in hit]
        if op == "loss":
            lse = torch.logsumexp(z, dim=1)
            loss = torch.zeros_like(lse)
            loss[hit] = lse[hit] - z[hit, goal]
            return {"loss": loss, "lse": lse}
        z = z.sub_(s["lse"].double()[:, None]).exp_()
        z[hit, goal] -= 1
        scale = torch.zeros(len(targets), dtype=torch.float64, device=z.device)
        scale[hit] = s["dloss"].double()[hit]
        z.mul_(scale[:, None])
        return {"da": torch.matmul(z, b.t()), "db": torch.matmul(a.t(), z)}
    device = (s["dy"] if op == "norm_grad" else s["x"]).device
    keep = _exact_keep(case, s, device)
    if op == "norm_grad":
        dy, gain, rstd = s["dy"].double(), s["weight"].double(), s["rstd"].double().unsqueeze(1)
        unit = (s["total"].double() - s["mean"].double().unsqueeze(1)) * rstd
        g = dy * gain
        n = case["cols"]
        dtotal = rstd / n * (n * g - g.sum(1, True) - unit * torch.linalg.vecdot(g, unit).unsqueeze(1))
        if case["joined"]:
            dtotal = dtotal + s["dtotal"].double()
        out = {"dresidual": dtotal, "dweight": torch.einsum("rc,rc->c", dy, unit), "dbias": dy.sum(0)}
        if case["p"] > 0:
            out["dx"] = dtotal * keep
        return out
    total = s["x"].double() * keep
    if case["residual"]:
        total = total + s["addend"].double()
    if op == "dropout":
        return {"y": total}
    out = {"total": total} if case["residual"] or case["p"] > 0 else {}
    held = total.to(s["x"].dtype).double()  # the rows are normalised as they are kept
    var, mean = torch.var_mean(held, 1, correction=0)
    out.update(mean=mean, rstd=(var + EPS) ** -0.5)
    out["y"] = (held - mean[:, None]) / (var + EPS).sqrt()[:, None] * s["weight"].double() + s["bias"].double()
    return out
