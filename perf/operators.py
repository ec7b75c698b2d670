"""Measured cases of the products with an epilogue, their gradients, the experts' products and the token sort.

Each case is one pass through one operator, as a training or serving step calls it:

  linear        y = act(x w + bias) + residual, with z = x w + bias kept for the backward pass
  linear_grad   dz = dy act'(z), dx = dz w^T, dw = x^T dz, dbias = sum of dz over the tokens
  experts       linear with one weight per expert, over rows sorted by expert
  experts_grad  its gradients
  tokens        (token, choice) pairs sorted by expert, the rows gathered, and back: the experts' rows summed
                with the router's weights, and the gradients of both

With ``own`` false they are computed from elementary torch operations in 32 bits.
"""

import math

import torch

own = False

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one token of a serving step through a square projection: the call's latency
        {"name": "linear_token", "op": "linear", "type": "bf16", "m": 1, "n": 4096, "k": 4096, "act": "silu",
         "residual": True, "keep": False},
        # a batch of single tokens through the widening half of a block: the weights' bytes
        {"name": "linear_step", "op": "linear", "type": "bf16", "m": 24, "n": 16384, "k": 4096, "act": "gelu",
         "residual": False, "keep": False},
        # every dimension odd, rows aligned to nothing: the ragged shape of the plain products
        {"name": "linear_ragged", "op": "linear", "type": "f16", "m": 1000, "n": 999, "k": 513, "act": "gelu",
         "residual": True, "keep": True},
        # a training step's largest product: the matrix cores' rate
        {"name": "linear_large", "op": "linear", "type": "bf16", "m": 8192, "n": 8192, "k": 8192, "act": "silu",
         "residual": True, "keep": True},
        # gradients of the ragged shape
        {"name": "linear_grad_ragged", "op": "linear_grad", "type": "f16", "m": 1000, "n": 999, "k": 513,
         "act": "gelu"},
        # gradients of a training step's widening product
        {"name": "linear_grad_large", "op": "linear_grad", "type": "bf16", "m": 8192, "n": 8192, "k": 4096,
         "act": "silu"},
        # sixteen tokens of a serving step, four experts each: a few rows per expert, the weights' bytes
        {"name": "experts_step", "op": "experts", "type": "bf16", "tokens": 16, "top_k": 4, "experts": 32, "n": 2048,
         "k": 4096, "act": "silu", "keep": False},
        # a training step's experts, two per token
        {"name": "experts_large", "op": "experts", "type": "bf16", "tokens": 8192, "top_k": 2, "experts": 8,
         "n": 4096, "k": 4096, "act": "silu", "keep": True},
        # gradients of a small fine-tuning batch: few rows per expert, sizes that end inside tiles
        {"name": "experts_grad_small", "op": "experts_grad", "type": "f16", "tokens": 250, "top_k": 2, "experts": 16,
         "n": 1496, "k": 1000, "act": "gelu"},
        # gradients of a training step's experts
        {"name": "experts_grad_large", "op": "experts_grad", "type": "bf16", "tokens": 4096, "top_k": 2,
         "experts": 8, "n": 4096, "k": 4096, "act": "silu"},
        # the router's answer for a serving step: the calls' latency
        {"name": "tokens_step", "op": "tokens", "type": "bf16", "tokens": 16, "top_k": 4, "experts": 32, "n": 4096},
        # a training step's tokens: the rows' bytes
        {"name": "tokens_large", "op": "tokens", "type": "bf16", "tokens": 16384, "top_k": 4, "experts": 64,
         "n": 4096},
    ]


def _log_size(rng, low, high):
    """A whole number of [low, high], even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A matrix width: three in four are multiples of 8, as models have them, the others any number."""
    w = _log_size(rng, low, high)
    return w if rng.random() < 0.25 else max(low, w - w % 8)


def draw(rng):
    op = rng.choice(("linear", "linear_grad", "experts", "experts_grad", "tokens"))
    case = {"op": op, "type": rng.choice(("bf16", "f16"))}
    if op in ("linear", "linear_grad"):
        case.update(m=_log_size(rng, 1, 8192), n=_width(rng, 64, 8192),
                    k=_width(rng, 64, 8192 if op == "linear" else 4096), act=rng.choice(ACTIVATIONS))
        if op == "linear":
            case.update(residual=rng.random() < 0.5, keep=rng.random() < 0.5)
    elif op in ("experts", "experts_grad"):
        case.update(tokens=_log_size(rng, 1, 8192 if op == "experts" else 4096), top_k=rng.choice((1, 2)),
                    experts=_log_size(rng, 2, 32), n=_width(rng, 64, 4096), k=_width(rng, 64, 4096),
                    act=rng.choice(ACTIVATIONS))
        if op == "experts":
            case.update(keep=rng.random() < 0.5)
    else:
        case.update(tokens=_log_size(rng, 1, 16384), top_k=rng.choice((1, 2, 3, 4)), experts=_log_size(rng, 2, 64),
                    n=_width(rng, 64, 4096))
    return case


# ---- inputs ---------------------------------------------------------------------------
class _Inputs:
    """Draws of one seed on the GPU."""

    def __init__(self, seed, dtype):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        self.dtype = dtype

    def normal(self, *shape, scale=1.0):
        x = torch.randn(*shape, device="cuda", generator=self.gen, dtype=torch.float32)
        return x.mul_(scale).to(self.dtype)

    def route(self, tokens, top_k, experts):
        """Each token's top_k different experts (fewer experts than that: any), some liked better than others, and
        the router's weights, which sum to one over a token's choices."""
        liked = torch.randn(experts, device="cuda", generator=self.gen)
        score = torch.randn(tokens, experts, device="cuda", generator=self.gen) + 0.5 * liked
        best, chosen = score.topk(min(top_k, experts), dim=1)
        turn = torch.arange(top_k, device="cuda") % chosen.shape[1]
        chosen, best = chosen[:, turn], best[:, turn]
        return chosen.to(torch.int32).contiguous(), torch.softmax(best, dim=1).contiguous()


def prepare(case, seed):
    dtype, op = TYPES[case["type"]], case["op"]
    draws = _Inputs(seed, dtype)
    s = dict(case)
    if op == "tokens":
        t, k, n = case["tokens"], case["top_k"], case["n"]
        s["chosen"], s["weights"] = draws.route(t, k, case["experts"])
        s["x"], s["y"], s["dout"] = draws.normal(t, n), draws.normal(t * k, n), draws.normal(t, n)
        return s
    n, k = case["n"], case["k"]
    if op.startswith("experts"):
        e, m = case["experts"], case["tokens"] * case["top_k"]
        chosen, _ = draws.route(case["tokens"], case["top_k"], e)
        counts = torch.bincount(chosen.flatten().long(), minlength=e)
        s["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
        s["most"] = int(counts.max())  # rows of the fullest expert: the plain form's padding
        s["w"], s["bias"] = draws.normal(e, k, n, scale=k ** -0.5), draws.normal(e, n)
    else:
        m = case["m"]
        s["w"], s["bias"] = draws.normal(k, n, scale=k ** -0.5), draws.normal(n)
    s["x"] = draws.normal(m, k)
    if op.endswith("_grad"):
        s["dy"], s["z"] = draws.normal(m, n), draws.normal(m, n)
        del s["bias"]
    elif case.get("residual"):
        s["residual"] = draws.normal(m, n)
    return s


# ---- the plain forms ------------------------------------------------------------------
def _act(z, kind):
    if kind == "relu":
        return torch.where(z > 0, z, 0.0)
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if kind == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    return torch.ones_like(z)


def _place(s):
    """Where each sorted row goes when every expert's rows are padded to the fullest expert's."""
    offsets = s["offsets"].long()
    row = torch.arange(s["x"].shape[0], device=offsets.device)
    expert = torch.searchsorted(offsets[1:], row, right=True)
    return expert, expert * s["most"] + row - offsets[expert]


def _padded(s, place, rows):
    out = rows.new_zeros(s["experts"] * s["most"], rows.shape[1])
    out[place] = rows
    return out.view(s["experts"], s["most"], rows.shape[1])


def _plain_linear(s):
    if s["op"] == "experts":
        expert, place = _place(s)
        z = torch.bmm(_padded(s, place, s["x"].float()), s["w"].float()).flatten(0, 1)[place]
        z = z + s["bias"].float()[expert]
    else:
        z = s["x"].float() @ s["w"].float() + s["bias"].float()
    y = _act(z, s["act"])
    if s.get("residual") is not None and s["residual"] is not False:
        y = y + s["residual"].float()
    dtype = s["x"].dtype
    return {"y": y.to(dtype), "z": z.to(dtype)} if s["keep"] else {"y": y.to(dtype)}


def _plain_linear_grad(s):
    dtype = s["x"].dtype
    slope = s["dy"].float() * _act_slope(s["z"].float(), s["act"])
    dz = slope.to(dtype)  # what the two products read
    if s["op"] == "experts_grad":
        expert, place = _place(s)
        pz, px = _padded(s, place, dz.float()), _padded(s, place, s["x"].float())
        dx = torch.bmm(pz, s["w"].float().transpose(1, 2).contiguous()).flatten(0, 1)[place]
        dw = torch.bmm(px.transpose(1, 2).contiguous(), pz)
        dbias = _padded(s, place, slope).sum(1)
    else:
        dx, dw, dbias = dz.float() @ s["w"].float().t(), s["x"].float().t() @ dz.float(), slope.sum(0)
    return {"dz": dz, "dx": dx.to(dtype), "dw": dw.to(dtype), "dbias": dbias}


def _plain_tokens(s):
    t, k, n = s["tokens"], s["top_k"], s["n"]
    dtype = s["x"].dtype
    pairs = s["chosen"].flatten().long()
    order = torch.argsort(pairs, stable=True)
    counts = (pairs[:, None] == torch.arange(s["experts"], device=pairs.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    position = torch.empty_like(order)
    position[order] = torch.arange(t * k, device=order.device)
    rows = s["x"][order // k]
    back = s["y"].float()[position].view(t, k, n)
    out = (s["weights"][:, :, None] * back).sum(1)
    dout = s["dout"].float()
    dy = (s["weights"].flatten()[order][:, None] * dout[order // k]).to(dtype)
    dweights = (back * dout[:, None, :]).sum(2)
    dx = s["y"].float()[position].view(t, k, n).sum(1)  # the gather's gradient, of rows that are y's here
    return {"offsets": offsets.int(), "order": order.int(), "position": position.int().view(t, k), "rows": rows,
            "out": out.to(dtype), "dy": dy, "dweights": dweights, "dx": dx.to(dtype)}


# ---- the framework's calls --------------------------------------------------------------
def _own_linear(s):
    import dense_fp32_tiled_amd as dft

    z = torch.empty(s["x"].shape[0], s["n"], dtype=s["x"].dtype, device=s["x"].device) if s["keep"] else None
    if s["op"] == "experts":
        y = dft.grouped_linear(s["x"], s["w"], s["offsets"], bias=s["bias"], activation=s["act"], preact=z)
    else:
        residual = s["residual"] if torch.is_tensor(s["residual"]) else None
        y = dft.linear(s["x"], s["w"], bias=s["bias"], residual=residual, activation=s["act"], preact=z)
    return {"y": y, "z": z} if s["keep"] else {"y": y}


def _own_linear_grad(s):
    import dense_fp32_tiled_amd as dft

    if s["op"] == "experts_grad":
        g = dft.grouped_linear_grad(s["dy"], s["x"], s["w"], s["offsets"], preact=s["z"], activation=s["act"])
    else:
        g = dft.linear_grad(s["dy"], s["x"], s["w"], preact=s["z"], activation=s["act"])
    return {"dz": g.preact, "dx": g.a, "dw": g.b, "dbias": g.bias}


def _own_tokens(s):
    import dense_fp32_tiled_amd as dft

    offsets, order, position = dft.expert_sort(s["chosen"], s["experts"])
    rows = dft.expert_gather(s["x"], position)
    out = dft.expert_combine(s["y"], position, s["weights"])
    dy, dweights = dft.expert_combine_grad(s["dout"], s["y"], position, s["weights"])
    dx = dft.expert_combine(s["y"], position)
    return {"offsets": offsets, "order": order, "position": position, "rows": rows, "out": out, "dy": dy,
            "dweights": dweights, "dx": dx}


def run(state):
    if state["op"] == "tokens":
        return _own_tokens(state) if own else _plain_tokens(state)
    if state["op"].endswith("_grad"):
        return _own_linear_grad(state) if own else _plain_linear_grad(state)
    return _own_linear(state) if own else _plain_linear(state)


# ---- what a pass cannot do without ---------------------------------------------------------
def _busy_experts(case):
    """Experts that at least one row goes to, when rows choose evenly."""
    rows, e = case["tokens"] * case["top_k"], case["experts"]
    return e * (1 - (1 - 1 / e) ** rows)


def work(case):
    op, n = case["op"], case["n"]
    if op == "tokens":
        t, k = case["tokens"], case["top_k"]
        pair = t * k
        # each of x, y and dout read once; rows and dy written; out and dx written; ids, weights and their gradient
        rows = 2 * n * (t + pair + t + 2 * pair + 2 * t)
        return {"bytes": rows + pair * (4 + 4 + 4 + 4 + 4) + 4 * (case["experts"] + 1), "flops": 6 * pair * n}
    k = case["k"]
    m = case["tokens"] * case["top_k"] if op.startswith("experts") else case["m"]
    e = _busy_experts(case) if op.startswith("experts") else 1
    if op.endswith("_grad"):
        # dy, z, x and w read; dz, dx, dw and dbias written (dw and dbias for every expert)
        every = case.get("experts", 1)
        size = 2 * (3 * m * n + 2 * m * k + e * k * n + every * k * n) + 4 * every * n
        return {"bytes": size, "flops": 4 * m * n * k + 10 * m * n}
    size = 2 * (m * k + e * k * n + e * n + m * n * (1 + int(case.get("residual", False)) + int(case["keep"])))
    return {"bytes": size, "flops": 2 * m * n * k + 10 * m * n}


# ---- the definitions in 64 bits --------------------------------------------------------------
def _exact_act(z, kind):
    """The activation and its slope, from the normal distribution's integral and the logistic function."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        up = (z > 0).double()
        return z * up, up
    if kind == "gelu":
        below = torch.special.ndtr(z)
        return z * below, below + z * torch.exp(z.square() / -2) / (2 * math.pi) ** 0.5
    inner, slope = (z, torch.ones_like(z)) if kind == "silu" else (
        (8 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3), (8 / math.pi) ** 0.5 * (1 + 0.134145 * z ** 2))
    gate = torch.special.expit(inner)  # (1 + tanh(u)) / 2 is the logistic function of 2 u
    return z * gate, gate + z * gate * (1 - gate) * slope


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tokens":
        t, k = case["tokens"], case["top_k"]
        y, dout, weights = s["y"].double(), s["dout"].double(), s["weights"].double()
        member = s["chosen"].flatten()
        slots = [torch.nonzero(member == e).flatten() for e in range(case["experts"])]
        order = torch.cat(slots)
        sizes = torch.tensor([0] + [x.numel() for x in slots], device=member.device)
        position = torch.sort(order).indices.view(t, k)
        out, dx, dweights = torch.zeros_like(dout), torch.zeros_like(dout), torch.zeros_like(weights)
        dy = torch.zeros_like(y)
        for j in range(k):
            chosen = y[position[:, j]]
            out += weights[:, j, None] * chosen
            dx += chosen
            dweights[:, j] = torch.linalg.vecdot(chosen, dout)
            dy[position[:, j]] = weights[:, j, None] * dout
        return {"offsets": sizes.cumsum(0).int(), "order": order.int(), "position": position.int(),
                "rows": s["x"].double()[torch.div(order, k, rounding_mode="floor")], "out": out, "dy": dy,
                "dweights": dweights, "dx": dx}
    x, w = s["x"].double(), s["w"]
    m, n = x.shape[0], case["n"]
    if op.startswith("experts"):
        ends = s["offsets"].tolist()
        parts = [(slice(ends[e], ends[e + 1]), e) for e in range(case["experts"])]
    else:
        parts, w = [(slice(0, m), 0)], w[None]
    if op.endswith("_grad"):
        dz = s["dy"].double() * _exact_act(s["z"].double(), case["act"])[1]
        dx, dw = torch.empty_like(x), torch.zeros(len(parts), case["k"], n, dtype=torch.float64, device=x.device)
        dbias = torch.zeros(len(parts), n, dtype=torch.float64, device=x.device)
        for rows, e in parts:
            dx[rows] = dz[rows] @ w[e].double().t()
            dw[e] = x[rows].t() @ dz[rows]
            dbias[e] = dz[rows].sum(0)
        if op == "linear_grad":
            dw, dbias = dw[0], dbias[0]
        return {"dz": dz, "dx": dx, "dw": dw, "dbias": dbias}
    z = torch.empty(m, n, dtype=torch.float64, device=x.device)
    bias = s["bias"].double().view(len(parts), n)
    for rows, e in parts:
        z[rows] = torch.addmm(bias[e], x[rows], w[e].double())
    y = _exact_act(z, case["act"])[0]
    if case.get("residual"):
        y = y + s["residual"].double()
    return {"y": y, "z": z} if case["keep"] else {"y": y}
