"""A linear layer from its forward pass to the update of its weight, as timed cases.

Three operators, each in its plain form (elementary torch operations) and as the
call a user of the library makes:

* ``linear``: ``act(x w^T + bias) + residual``, for training with the sum before the
  activation beside it;
* ``gradients``: the gradients of that layer's input, weight and bias;
* ``orthogonalize``: the nearest orthogonal matrix, about, of a weight's update, by
  Newton-Schulz steps.

``own`` selects the side: False for the plain forms, True for the library's.
"""
import math

import torch

own = False

DEVICE = "cuda:0"
ACTIVATIONS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
QUINTIC = (3.4445, -4.7750, 2.0315)  # p(s) = a s + b s^3 + c s^5 takes (0, 1] towards 1
NORM_EPS = 1e-7


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a serving step: the weight read once, a launch's latency beside it
        {"name": "linear one token", "op": "linear", "m": 1, "n": 4096, "k": 4096, "act": "silu", "bias": True,
         "residual": False, "out": "bf16", "save": False},
        # a step of a few sequences through a narrow layer: little to spread over the card but the long rows
        {"name": "linear few tokens narrow", "op": "linear", "m": 24, "n": 1000, "k": 8192, "act": "none", "bias": True,
         "residual": True, "out": "bf16", "save": False},
        # a chunk of a prompt
        {"name": "linear prompt chunk", "op": "linear", "m": 512, "n": 4096, "k": 4096, "act": "gelu_tanh",
         "bias": False, "residual": False, "out": "bf16", "save": False},
        # training, every edge ragged, fp32 out with the sum before the activation
        {"name": "linear ragged training", "op": "linear", "m": 5000, "n": 7000, "k": 3000, "act": "gelu", "bias": True,
         "residual": False, "out": "f32", "save": True},
        # the large square product of training and prefill, with all of the epilogue
        {"name": "linear large", "op": "linear", "m": 8192, "n": 8192, "k": 8192, "act": "gelu_tanh", "bias": True,
         "residual": True, "out": "bf16", "save": False},
        # one short sequence's gradients: latency, and the weight's gradient to write
        {"name": "gradients one sequence", "op": "gradients", "m": 129, "n": 2048, "k": 1024, "act": "silu",
         "dw": "bf16"},
        # many tokens against a small weight: the long axis is summed over; fp32 gradient for an accumulating optimiser
        {"name": "gradients long batch", "op": "gradients", "m": 32768, "n": 1024, "k": 1024, "act": "none",
         "dw": "f32"},
        # training, every edge ragged
        {"name": "gradients ragged", "op": "gradients", "m": 5000, "n": 7000, "k": 3000, "act": "gelu", "dw": "bf16"},
        # a large layer in training
        {"name": "gradients large", "op": "gradients", "m": 8192, "n": 8192, "k": 8192, "act": "silu", "dw": "bf16"},
        # the smallest weights: latency of a chain of products
        {"name": "orthogonalize small", "op": "orthogonalize", "stack": 1, "rows": 256, "cols": 256, "dtype": "bf16"},
        # a tall ragged weight, its update in fp32
        {"name": "orthogonalize tall ragged", "op": "orthogonalize", "stack": 1, "rows": 7000, "cols": 3000,
         "dtype": "f32"},
        # one shape's weights of several layers at once
        {"name": "orthogonalize stack", "op": "orthogonalize", "stack": 12, "rows": 1024, "cols": 4096,
         "dtype": "bf16"},
    ]


def _between(rng, low, high):
    """A whole number whose logarithm is spread evenly over [low, high]."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "gradients", "gradients", "orthogonalize"])
    if op == "linear":
        act = rng.choice(ACTIVATIONS)
        return {"op": op, "m": _between(rng, 1, 8192), "n": _between(rng, 16, 8192), "k": _between(rng, 16, 8192),
                "act": act, "bias": rng.random() < 0.6, "residual": rng.random() < 0.4,
                "out": rng.choice(["bf16", "bf16", "f32"]), "save": rng.random() < 0.4}
    if op == "gradients":
        act = rng.choice(ACTIVATIONS)
        # a gradient of the weight in fp32 is asked for where no activation's gradient is rounded on the way
        return {"op": op, "m": _between(rng, 1, 16384), "n": _between(rng, 16, 5000), "k": _between(rng, 16, 5000),
                "act": act, "dw": rng.choice(["bf16", "f32"]) if act == "none" else "bf16"}
    rows, cols = _between(rng, 1, 5000), _between(rng, 1, 5000)
    return {"op": op, "stack": _between(rng, 1, max(1, min(32, (1 << 24) // (rows * cols)))), "rows": rows,
            "cols": cols, "dtype": rng.choice(["bf16", "f32"])}


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
STEPS = 5


def work(case):
    if case["op"] == "orthogonalize":
        short, long, e = min(case["rows"], case["cols"]), max(case["rows"], case["cols"]), case["rows"] * case["cols"]
        # a step's products: the Gram matrix and its square, both symmetric, and the product with the matrix
        step = short * short * long + short ** 3 + 2 * short * short * long
        return {"bytes": case["stack"] * e * (SIZE[case["dtype"]] + 2), "flops": case["stack"] * STEPS * step}
    m, n, k = case["m"], case["n"], case["k"]
    if case["op"] == "linear":
        out = m * n * (SIZE[case["out"]] * (2 if case["residual"] else 1) + (2 if case["save"] else 0))
        return {"bytes": 2 * (m * k + n * k) + out + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    return {"bytes": m * n * (2 if case["act"] == "none" else 4) + 4 * m * k + 2 * n * k + n * k * SIZE[case["dw"]] + 4 * n,
            "flops": 4 * m * n * k}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _rows(m, n, g, scale=1.0, loud=0.0, dtype=torch.bfloat16):
    """An m x n matrix whose rows start at whole 16 bytes, as the library's own results do: normal values, a share
    `loud` of the columns ten times larger, as activations have them."""
    x = torch.randn((m, 8 * ((n + 7) // 8)), generator=g, device=DEVICE).mul_(scale)
    if loud:
        x *= torch.where(torch.rand(x.shape[1], generator=g, device=DEVICE) < loud, 10.0, 1.0)
    return x.to(dtype)[:, :n]


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "orthogonalize":
        # an update as momentum leaves it: some strong directions over a floor, rows and columns of unlike size
        b, r, c = case["stack"], case["rows"], case["cols"]
        q = max(1, min(r, c) // 8)
        x = torch.randn((b, r, c), generator=g, device=DEVICE)
        u = torch.randn((b, r, q), generator=g, device=DEVICE)
        v = torch.randn((b, q, c), generator=g, device=DEVICE) / math.sqrt(q)
        x = 0.3 * x + torch.stack([u[i] @ v[i] for i in range(b)])
        x *= torch.exp(0.5 * torch.randn((b, r, 1), generator=g, device=DEVICE))
        x *= torch.exp(0.5 * torch.randn((b, 1, c), generator=g, device=DEVICE))
        x = (1e-3 * x).to(TYPES[case["dtype"]])
        s["x"] = x[0] if b == 1 else x
        return s
    m, n, k = case["m"], case["n"], case["k"]
    s["x"] = _rows(m, k, g, loud=0.01)
    s["w"] = _rows(n, k, g, scale=k ** -0.5)
    if case["op"] == "linear":
        s["bias"] = (0.1 * torch.randn(n, generator=g, device=DEVICE)).bfloat16() if case["bias"] else None
        s["residual"] = _rows(m, n, g, dtype=TYPES[case["out"]]) if case["residual"] else None
    else:
        s["dy"] = _rows(m, n, g, scale=1e-2)
        s["z"] = None if case["act"] == "none" else _rows(m, n, g, scale=1.4)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _activation(case):
    return None if case["act"] == "none" else case["act"]


def _own_linear(s):
    import persistent_tile_scheduling_amd as pts
    c = s["case"]
    out = pts.linear(s["x"], s["w"], s["bias"], activation=_activation(c), residual=s["residual"],
                     out_dtype=TYPES[c["out"]], preactivation=c["save"])
    return out if c["save"] else (out,)


def _own_gradients(s):
    import persistent_tile_scheduling_amd as pts
    c = s["case"]
    return tuple(pts.linear_backward(s["dy"], s["x"], s["w"], s["z"], activation=_activation(c),
                                     dw_dtype=TYPES[c["dw"]]))


def _own_orthogonalize(s):
    import persistent_tile_scheduling_amd as pts
    return (pts.orthogonalize(s["x"], STEPS, QUINTIC, NORM_EPS),)


_own = {"linear": _own_linear, "gradients": _own_gradients, "orthogonalize": _own_orthogonalize}


def _act(z, kind):
    if kind == "relu":
        return torch.where(z < 0, 0.0, z)
    if kind == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if kind == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _slope(z, kind):
    if kind == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if kind == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        p = 1.0 / (1.0 + torch.exp(-2.0 * c * (z + 0.044715 * z * z * z)))
        return p + z * p * (1.0 - p) * 2.0 * c * (1.0 + 3.0 * 0.044715 * z * z)
    p = 1.0 / (1.0 + torch.exp(-z))
    return p + z * p * (1.0 - p)


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if c["bias"]:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if c["residual"]:
        y = y + s["residual"].float()
    y = y.to(TYPES[c["out"]])
    return (y, z.bfloat16()) if c["save"] else (y,)


def _plain_gradients(s):
    c = s["case"]
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _slope(s["z"].float(), c["act"])
    dx = dz @ s["w"].float()
    dw = dz.t() @ s["x"].float()
    return dx.bfloat16(), dw.to(TYPES[c["dw"]]), dz.sum(0)


def _plain_orthogonalize(s):
    x = s["x"].float() if s["x"].dim() == 3 else s["x"].float().unsqueeze(0)
    wide = x.shape[1] <= x.shape[2]
    if not wide:
        x = x.transpose(1, 2).contiguous()
    x = x / ((x * x).sum((1, 2), keepdim=True).sqrt() + NORM_EPS)
    a, b, c = QUINTIC
    for _ in range(STEPS):
        gram = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    if not wide:
        x = x.transpose(1, 2)
    return (x.bfloat16().view(s["x"].shape) if wide else x.bfloat16().contiguous().view(s["x"].shape),)


_plain = {"linear": _plain_linear, "gradients": _plain_gradients, "orthogonalize": _plain_orthogonalize}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_parts(z, kind):
    """act(z) and act'(z) in 64 bits."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0), (z > 0).double()
    if kind == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z.square() / 2) * 0.3989422804014327
    if kind == "gelu_tanh":
        u = 0.7978845608028654 * (z + 0.044715 * z ** 3)
        t = torch.tanh(u)
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * 0.7978845608028654 * (1 + 0.134145 * z * z)
    p = torch.sigmoid(z)
    return z * p, p * (1 + z * (1 - p))


def _exact_linear(s):
    c, y, zs = s["case"], [], []
    w = s["w"].double()
    for x in s["x"].double().split(2048):
        z = torch.mm(x, w.t())
        zs.append(z + s["bias"].double() if c["bias"] else z)
        y.append(_exact_parts(zs[-1], c["act"])[0])
    y, z = torch.cat(y), torch.cat(zs)
    if c["residual"]:
        y += s["residual"].double()
    return (y, z) if c["save"] else (y,)


def _exact_gradients(s):
    c, dx = s["case"], []
    x, w, dw, db = s["x"], s["w"].double(), 0.0, 0.0
    for lo in range(0, c["m"], 4096):
        dz = s["dy"][lo:lo + 4096].double()
        if c["act"] != "none":
            dz = dz * _exact_parts(s["z"][lo:lo + 4096].double(), c["act"])[1]
        dx.append(torch.mm(dz, w))
        dw = dw + torch.mm(dz.t(), x[lo:lo + 4096].double())
        db = db + dz.sum(0)
    return torch.cat(dx), dw, db


def _exact_orthogonalize(s):
    out = []
    for x in (s["x"] if s["x"].dim() == 3 else [s["x"]]):
        y = x.double()
        y = y / (torch.linalg.norm(y) + NORM_EPS)
        a, b, c = QUINTIC
        for _ in range(STEPS):      # on the shorter side, from the left or the right
            if y.shape[0] <= y.shape[1]:
                g = torch.mm(y, y.t())
                y = a * y + b * torch.mm(g, y) + c * torch.mm(g, torch.mm(g, y))
            else:
                g = torch.mm(y.t(), y)
                y = a * y + b * torch.mm(y, g) + c * torch.mm(torch.mm(y, g), g)
        out.append(y)
    return (torch.stack(out) if s["x"].dim() == 3 else out[0],)


def exact(case, seed):
    return {"linear": _exact_linear, "gradients": _exact_gradients,
            "orthogonalize": _exact_orthogonalize}[case["op"]](prepare(case, seed))
