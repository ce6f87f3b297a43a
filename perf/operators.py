"""The operators of a layer of routed experts in 8-bit floating point, as timed cases.

Five operators, each in its plain form (elementary torch operations) and as the
calls a user of the library makes:

* ``quantize``: a matrix, or the gated activation of one, to e4m3 with an fp32
  scale for each block of 128 (of a row, or 128 x 128);
* ``product``: ``D = A . B`` of two such matrices;
* ``experts``: one such product per expert, over rows ordered by expert whose
  offsets are in device memory;
* ``route``: scores, choice and weights of each token's experts, the order of the
  rows by expert, and for training the gradient of the logits;
* ``combine``: the weighted sum of each token's expert outputs, and its gradients.

``own`` selects the side: False for the plain forms, True for the library's.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda:0"
BLOCK = 128          # elements that share a scale, along k (and along n for weights)
E4M3_MAX = 448.0     # largest finite e4m3 value
TINY_SCALE = 2.0 ** -126
WEIGHT_EPS = 1e-20   # keeps a renormalised weight finite when every chosen score underflows


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token's activations before a product: a launch's latency
        {"name": "quantize one token", "op": "quantize", "m": 1, "k": 4096, "dtype": "bf16", "gated": False,
         "across": False, "square": False},
        # the activations of a large batch between two products, with the gate applied on the way; odd width
        {"name": "quantize gated batch", "op": "quantize", "m": 8192, "k": 7000, "dtype": "bf16", "gated": True,
         "across": False, "square": False},
        # a gradient read down its columns, for the product that gives the weights' gradient
        {"name": "quantize across rows", "op": "quantize", "m": 5000, "k": 7000, "dtype": "f32", "gated": False,
         "across": True, "square": False},
        # one step of serving: a handful of sequences against a square weight
        {"name": "product few rows", "op": "product", "m": 8, "n": 4096, "k": 4096, "out": "bf16", "rows": False},
        # the large square product of training and prefill
        {"name": "product large", "op": "product", "m": 8192, "n": 8192, "k": 8192, "out": "bf16", "rows": False},
        # the gradient of a weight: both operands scaled along the tokens, fp32 out, every edge ragged
        {"name": "product weight gradient", "op": "product", "m": 5000, "n": 7000, "k": 3000, "out": "f32",
         "rows": True},
        # one step of serving 16 tokens: 128 rows over 64 experts, most with one to four rows
        {"name": "experts few rows", "op": "experts", "experts": 64, "active": 55, "m": 128, "tokens": 16, "n": 4096,
         "k": 4096, "gather": True, "out": "bf16"},
        # prefill of 4096 tokens, 8 experts each, loads as uneven as a trained router leaves them
        {"name": "experts prefill", "op": "experts", "experts": 64, "active": 64, "m": 32768, "tokens": 4096,
         "n": 4096, "k": 4096, "gather": True, "out": "bf16"},
        # one token's router: sigmoid scores, a balancing bias, 4 of 8 groups
        {"name": "route one token", "op": "route", "m": 1, "experts": 256, "top": 8, "dtype": "f32",
         "score": "sigmoid", "bias": True, "groups": 8, "keep": 4, "pair": True, "norm": True, "train": False,
         "padded": False},
        # a training batch's router: softmax scores, with the gradient of the logits
        {"name": "route training batch", "op": "route", "m": 16384, "experts": 128, "top": 8, "dtype": "f32",
         "score": "softmax", "bias": False, "groups": 1, "keep": 1, "pair": False, "norm": True, "train": True,
         "padded": False},
        # the end of a serving step: 16 tokens
        {"name": "combine few tokens", "op": "combine", "m": 16, "n": 4096, "top": 8, "dtype": "bf16",
         "train": False, "padded": False},
        # a training batch's combination with both gradients
        {"name": "combine training batch", "op": "combine", "m": 8192, "n": 4096, "top": 8, "dtype": "bf16",
         "train": True, "padded": False},
    ]


def _between(rng, low, high):
    """A whole number whose logarithm is spread evenly over [low, high]."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "experts", "experts", "route", "combine"])
    if op == "quantize":
        form = rng.choice(["rows", "rows", "gated", "across", "square"])
        return {"op": op, "m": _between(rng, 1, 8192), "k": _between(rng, 32, 8192),
                "dtype": rng.choice(["bf16", "f32"]), "gated": form == "gated",
                "across": form == "across" or (form == "square" and rng.random() < 0.5), "square": form == "square"}
    if op == "product":
        return {"op": op, "m": _between(rng, 1, 8192), "n": _between(rng, 32, 8192), "k": _between(rng, 32, 8192),
                "out": rng.choice(["bf16", "f32"]), "rows": rng.random() < 0.3}
    if op == "experts":
        experts = _between(rng, 2, 64)
        tokens, top = _between(rng, 1, 4096), rng.randint(1, min(8, experts))
        m = tokens * top
        return {"op": op, "experts": experts, "active": min(m, rng.randint((experts + 1) // 2, experts)), "m": m,
                "tokens": tokens, "n": _between(rng, 64, 4096), "k": _between(rng, 64, 4096),
                "gather": rng.random() < 0.5,
                "out": rng.choice(["bf16", "f32"])}
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * rng.randint(2, 512 // groups)
        keep = rng.randint(1, groups)
        return {"op": op, "m": _between(rng, 1, 16384), "experts": experts,
                "top": rng.randint(1, min(16, keep * (experts // groups))), "dtype": rng.choice(["bf16", "f32"]),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "keep": keep, "pair": rng.random() < 0.5, "norm": rng.random() < 0.7, "train": rng.random() < 0.5,
                "padded": rng.random() < 0.3}
    return {"op": op, "m": _between(rng, 1, 8192), "n": _between(rng, 64, 4096), "top": rng.randint(1, 8),
            "dtype": rng.choice(["bf16", "bf16", "f32"]),
            "train": rng.random() < 0.5, "padded": rng.random() < 0.3}


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    op = case["op"]
    if op == "quantize":
        m, k = case["m"], case["k"]
        scales = _blocks(m) * _blocks(k) if case["square"] else m * _blocks(k)
        return {"bytes": m * k * (SIZE[case["dtype"]] * (2 if case["gated"] else 1) + 1) + 4 * scales,
                "flops": m * k * (8 if case["gated"] else 3)}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        scales = m * _blocks(k) + (n if case["rows"] else _blocks(n)) * _blocks(k)
        return {"bytes": m * k + n * k + 4 * scales + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}
    if op == "experts":
        m, n, k, a = case["m"], case["n"], case["k"], case["active"]
        read = case["tokens"] if case["gather"] else m
        return {"bytes": read * (k + 4 * _blocks(k)) + a * (n * k + 4 * _blocks(n) * _blocks(k)) +
                m * n * SIZE[case["out"]] + (4 * m if case["gather"] else 0) + 4 * (case["experts"] + 1),
                "flops": 2 * m * n * k}
    if op == "route":
        m, e, t = case["m"], case["experts"], case["top"]
        once = m * e * SIZE[case["dtype"]] + 16 * m * t + 4 * (e + 1) + (4 * e if case["bias"] else 0)
        more = m * e * SIZE[case["dtype"]] + 4 * m * t if case["train"] else 0
        return {"bytes": once + more, "flops": m * e * (8 if case["train"] else 4)}
    m, n, t, s = case["m"], case["n"], case["top"], SIZE[case["dtype"]]
    once = m * t * n * s + m * n * s + 8 * m * t
    more = m * n * s + m * t * n * s + 4 * m * t if case["train"] else 0
    return {"bytes": once + more, "flops": 2 * m * t * n * (3 if case["train"] else 1)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _matrix(shape, g, dtype):
    """Activations as they occur: normal values, a few channels ten times larger."""
    x = torch.randn(shape, generator=g, device=DEVICE)
    loud = torch.rand(shape[-1], generator=g, device=DEVICE) < 0.01
    return (x * torch.where(loud, 10.0, 1.0)).to(dtype)


def _codes(shape, g, k):
    """e4m3 values as a quantiser leaves them (normal values whose block maximum is
    near 448), rows padded to a multiple of 16."""
    wide = torch.randn((*shape, 16 * ((k + 15) // 16)), generator=g, device=DEVICE).mul_(128.0).clamp_(-448.0, 448.0)
    return wide.to(torch.float8_e4m3fn)[..., :k]


def _scales(shape, g, low):
    return low * (0.5 + torch.rand(shape, generator=g, device=DEVICE))


def _sizes(case, seed):
    """Rows of each expert: `active` of them, chosen and weighted at random."""
    rng = np.random.default_rng(seed)
    e, a, m = case["experts"], case["active"], case["m"]
    sizes = np.zeros(e, dtype=np.int64)
    at = rng.permutation(e)[:a]
    p = np.exp(0.5 * rng.standard_normal(a))
    sizes[at] = 1 + rng.multinomial(m - a, p / p.sum())
    return sizes


def _order(case, g):
    """Experts of each token at random, without repeats, and the rows ordered by expert:
    (positions of each token's rows, number of rows); a padded batch's last tokens have none."""
    m, t = case["m"], case["top"]
    e = max(16, 2 * t)
    ids = torch.rand((m, e), generator=g, device=DEVICE).argsort(dim=1)[:, :t]
    if case["padded"]:
        ids[m - m // 4:] = e
    flat = ids.reshape(-1)
    order = flat.sort(stable=True).indices
    positions = torch.empty_like(order)
    positions[order] = torch.arange(m * t, device=DEVICE)
    positions = torch.where(flat == e, -2 - positions, positions)
    return positions.view(m, t).to(torch.int32)


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = {"case": case}
    if op == "quantize":
        m, k = case["m"], case["k"]
        if case["across"]:
            s["x"] = _matrix((k, m), g, TYPES[case["dtype"]]).t()
        else:
            s["x"] = _matrix((m, 2 * k if case["gated"] else k), g, TYPES[case["dtype"]])
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        kb = _blocks(k)
        s["a"], s["a_scale"] = _codes((m,), g, k), _scales((kb, m), g, 0.008).t()
        s["b"] = _codes((n,), g, k)
        s["b_scale"] = _scales((kb, n), g, 0.0004).t() if case["rows"] else _scales((_blocks(n), kb), g, 0.0004)
    elif op == "experts":
        m, n, k, e = case["m"], case["n"], case["k"], case["experts"]
        kb, have = _blocks(k), case["tokens"] if case["gather"] else m
        s["a"], s["a_scale"] = _codes((have,), g, k), _scales((kb, have), g, 0.008).t()
        s["b"], s["b_scale"] = _codes((e, n), g, k), _scales((e, _blocks(n), kb), g, 0.0004)
        sizes = _sizes(case, seed)
        s["most"] = int(sizes.max())
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).to(DEVICE)
        s["rows"] = torch.randint(0, have, (m,), generator=g, device=DEVICE, dtype=torch.int32) if case["gather"] else None
    elif op == "route":
        m, e = case["m"], case["experts"]
        x = torch.randn((m, e), generator=g, device=DEVICE) + 0.5 * torch.randn((1, e), generator=g, device=DEVICE)
        if case["padded"]:
            x[m - m // 4:] = float("-inf")
        s["logits"] = x.to(TYPES[case["dtype"]])
        s["bias"] = 0.05 * torch.randn(e, generator=g, device=DEVICE) if case["bias"] else None
        s["dweights"] = torch.randn((m, case["top"]), generator=g, device=DEVICE) if case["train"] else None
    else:
        m, n, t = case["m"], case["n"], case["top"]
        s["y"] = _matrix((m * t, n), g, TYPES[case["dtype"]])
        s["positions"] = _order(case, g)
        w = torch.rand((m, t), generator=g, device=DEVICE) + 0.05
        s["weights"] = torch.where(s["positions"] >= 0, w / w.sum(1, keepdim=True), 0.0)
        s["dout"] = torch.randn((m, n), generator=g, device=DEVICE).to(TYPES[case["dtype"]]) if case["train"] else None
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_quantize(s):
    import persistent_tile_scheduling_amd as pts
    c = s["case"]
    return pts.quantize_fp8(s["x"], block=(BLOCK, BLOCK) if c["square"] else (1, BLOCK), swiglu=c["gated"])


def _own_product(s):
    import persistent_tile_scheduling_amd as pts
    return pts.gemm_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"], TYPES[s["case"]["out"]])


def _own_experts(s):
    import persistent_tile_scheduling_amd as pts
    return pts.gemm_fp8_experts(s["a"], s["a_scale"], s["b"], s["b_scale"], s["offsets"], s["rows"],
                                TYPES[s["case"]["out"]])


def _own_route(s):
    import persistent_tile_scheduling_amd as pts
    c = s["case"]
    r = pts.moe_route(s["logits"], c["top"], score=c["score"], bias=s["bias"], groups=c["groups"],
                      topk_groups=c["keep"], group_score="top2_sum" if c["pair"] else "max", renormalize=c["norm"])
    if not c["train"]:
        return tuple(r)
    d = pts.moe_route_backward(s["dweights"], s["logits"], r.ids, score=c["score"], renormalize=c["norm"])
    return (*r, d)


def _own_combine(s):
    import persistent_tile_scheduling_amd as pts
    out = pts.moe_combine(s["y"], s["weights"], s["positions"])
    if not s["case"]["train"]:
        return (out,)
    return (out, *pts.moe_combine_backward(s["dout"], s["y"], s["weights"], s["positions"]))


_own = {"quantize": _own_quantize, "product": _own_product, "experts": _own_experts, "route": _own_route,
        "combine": _own_combine}


def _plain_quantize(s):
    c, x = s["case"], s["x"].float()
    m, k = c["m"], c["k"]
    if c["gated"]:
        gate, up = x[:, :k], x[:, k:]
        x = gate / (1.0 + torch.exp(-gate)) * up
    tall = BLOCK if c["square"] else 1
    mb, kb = (m + tall - 1) // tall, _blocks(k)
    full = x.new_zeros((mb * tall, kb * BLOCK))
    full[:m, :k] = x
    full = full.view(mb, tall, kb, BLOCK)
    most = full.abs().amax(dim=(1, 3))
    scale = most / torch.full_like(most, E4M3_MAX)      # by a tensor: a division by a number becomes a product
    scale = torch.where(torch.isfinite(most), scale.clamp(min=TINY_SCALE), float("nan"))
    q = (full / scale[:, None, :, None]).view(mb * tall, kb * BLOCK)[:m, :k]
    return q.to(torch.float8_e4m3fn), scale


def _values(codes, scale, n, k):
    """What codes and block scales stand for, in 32 bits; scale has a row per row of `codes`, or per 128 rows."""
    if scale.shape[-2] != n:
        scale = scale.repeat_interleave(BLOCK, -2)[..., :n, :]
    return codes.float() * scale.repeat_interleave(BLOCK, -1)[..., :k]


def _plain_product(s):
    c = s["case"]
    a = _values(s["a"], s["a_scale"], c["m"], c["k"])
    b = _values(s["b"], s["b_scale"], c["n"], c["k"])
    return (a @ b.t()).to(TYPES[c["out"]])


def _plain_experts(s):
    c = s["case"]
    have = c["tokens"] if c["gather"] else c["m"]
    a = _values(s["a"], s["a_scale"], have, c["k"])
    b = _values(s["b"], s["b_scale"], c["n"], c["k"])
    row = torch.arange(c["m"], device=DEVICE)
    expert = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    rank = row - s["offsets"].long()[expert]
    if c["gather"]:
        a = a[s["rows"].long()]
    x = a.new_zeros((c["experts"], s["most"], c["k"]))
    x[expert, rank] = a
    y = torch.matmul(x, b.transpose(1, 2).contiguous())
    return y[expert, rank].to(TYPES[c["out"]])


def _plain_route(s):
    c = s["case"]
    m, e, t = c["m"], c["experts"], c["top"]
    x = s["logits"].double()                       # 64 bits: the choice goes by differences of scores
    open_ = x > float("-inf")
    if c["score"] == "softmax":
        top = x.amax(1, keepdim=True)
        p = torch.exp(x - torch.where(torch.isfinite(top), top, 0.0))
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    choice = p + s["bias"].double() if c["bias"] else p
    by = torch.where(open_, choice if c["bias"] else x, float("-inf"))
    if c["groups"] > 1:
        of = torch.where(open_, choice, float("-inf")).view(m, c["groups"], -1).sort(dim=2, descending=True).values
        # without a bias the largest scores are compared by their logits
        group = by.view(m, c["groups"], -1).amax(2) if not c["pair"] else of[:, :, 0] + torch.where(of[:, :, 1] > float("-inf"), of[:, :, 1], 0.0)
        kept = group.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        keep = torch.zeros((m, c["groups"]), dtype=torch.bool, device=DEVICE).scatter_(1, kept, True)
        by = torch.where(keep.repeat_interleave(e // c["groups"], 1), by, float("-inf"))
    best = by.sort(dim=1, descending=True, stable=True)
    have = best.values[:, :t] > float("-inf")
    ids = torch.where(have, best.indices[:, :t], -1)
    chosen = torch.where(have, p.gather(1, ids.clamp(min=0)), 0.0)
    total = chosen.sum(1, keepdim=True) + WEIGHT_EPS
    weights = chosen / total if c["norm"] else chosen
    flat = torch.where(ids < 0, e, ids).reshape(-1)
    order = flat.sort(stable=True).indices
    offsets = torch.searchsorted(flat[order], torch.arange(e + 1, device=DEVICE))
    positions = torch.empty_like(order)
    positions[order] = torch.arange(m * t, device=DEVICE)
    positions = torch.where(flat == e, -2 - positions, positions).view(m, t)
    out = (ids.int(), weights.float(), offsets.int(), (order // t).int(), positions.int())
    if not c["train"]:
        return out
    dw = s["dweights"].double()
    if c["norm"]:
        dw = (dw - (dw * weights).sum(1, keepdim=True)) / total
    dp = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0), torch.where(have, dw, 0.0))
    if c["score"] == "softmax":
        dx = p * (dp - (dp * p).sum(1, keepdim=True))
    else:
        dx = dp * p * (1.0 - p)
    return (*out, dx.to(s["logits"].dtype))


def _plain_combine(s):
    c = s["case"]
    at = s["positions"].long()
    have = (at >= 0).unsqueeze(2)
    y = torch.where(have, s["y"].float()[at.clamp(min=0)], 0.0)
    w = torch.where(have, s["weights"].unsqueeze(2), 0.0)
    out = (w * y).sum(1).to(s["y"].dtype)
    if not c["train"]:
        return (out,)
    dout = s["dout"].float().unsqueeze(1)
    place = torch.where(at >= 0, at, -2 - at).reshape(-1)
    dy = torch.empty_like(s["y"])
    dy[place] = (w * dout).to(dy.dtype).view(-1, c["n"])
    return out, dy, (y * dout).sum(2)


_plain = {"quantize": _plain_quantize, "product": _plain_product, "experts": _plain_experts, "route": _plain_route,
          "combine": _plain_combine}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _nearest_e4m3(v):
    """v rounded to the nearest e4m3 value, ties to the even one: three fraction bits above 2^-6, steps of 2^-9 below."""
    exponent = torch.frexp(v).exponent - 1
    step = torch.ldexp(torch.ones_like(v), exponent.clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_quantize(s):
    c, x = s["case"], s["x"].double()
    k = c["k"]
    if c["gated"]:
        x = x[:, :k] * torch.sigmoid(x[:, :k]) * x[:, k:]
    scale = []
    for lo in range(0, k, BLOCK):
        most = x[:, lo:lo + BLOCK].abs().amax(1)
        if c["square"]:
            most = torch.stack([part.max() for part in most.split(BLOCK)])
        scale.append((most / E4M3_MAX).float().double())
    scale = torch.stack(scale, 1)
    wide = scale.repeat_interleave(BLOCK, 0)[:c["m"]] if c["square"] else scale
    q = torch.empty_like(x)
    for b, lo in enumerate(range(0, k, BLOCK)):
        q[:, lo:lo + BLOCK] = _nearest_e4m3(x[:, lo:lo + BLOCK] / wide[:, b:b + 1])
    return q, scale


def _exact_rows(a, a_scale, b, b_scale):
    """Sum over blocks of scale . scale . (sum of the block's products); every term in 64 bits."""
    m, n, k = a.shape[0], b.shape[0], a.shape[1]
    out = torch.zeros((m, n), dtype=torch.float64, device=DEVICE)
    column = b_scale.double()
    if b_scale.shape[0] != n:
        column = column[torch.arange(n, device=DEVICE) // BLOCK]
    for i, lo in enumerate(range(0, k, BLOCK)):
        part = a[:, lo:lo + BLOCK].double() * a_scale[:, i:i + 1].double()
        out += part @ (b[:, lo:lo + BLOCK].double() * column[:, i:i + 1]).t()
    return out


def _exact_product(s):
    return _exact_rows(s["a"], s["a_scale"], s["b"], s["b_scale"])


def _exact_experts(s):
    c, at = s["case"], s["offsets"].tolist()
    out = torch.zeros((c["m"], c["n"]), dtype=torch.float64, device=DEVICE)
    for e in range(c["experts"]):
        lo, hi = at[e], at[e + 1]
        if lo == hi:
            continue
        pick = s["rows"][lo:hi].long() if c["gather"] else slice(lo, hi)
        out[lo:hi] = _exact_rows(s["a"].view(torch.uint8)[pick].view(torch.float8_e4m3fn), s["a_scale"][pick],
                                 s["b"][e], s["b_scale"][e])
    return out


def _exact_route(s):
    c = s["case"]
    m, e, t = c["m"], c["experts"], c["top"]
    x = s["logits"].double().cpu().numpy()
    live = np.isfinite(x).any(axis=1)
    z = np.where(live[:, None], x, 0.0)
    if c["score"] == "softmax":
        p = np.exp(z - z.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
    else:
        p = np.where(z >= 0, 1.0, np.exp(-np.abs(z))) / (1.0 + np.exp(-np.abs(z)))
    add = s["bias"].double().cpu().numpy() if c["bias"] else np.zeros(e)
    chosen, size = np.full((m, t), -1), e // c["groups"]
    for i in np.flatnonzero(live):
        by = p[i] + add if c["bias"] else z[i]
        pool = np.arange(e)
        if c["groups"] > 1:
            if c["pair"]:
                rank = [np.sort((p[i] + add)[j * size:(j + 1) * size])[-2:].sum() for j in range(c["groups"])]
            else:
                rank = [by[j * size:(j + 1) * size].max() for j in range(c["groups"])]
            best = sorted(range(c["groups"]), key=lambda j: (-rank[j], j))[:c["keep"]]
            pool = np.concatenate([np.arange(j * size, (j + 1) * size) for j in sorted(best)])
        chosen[i] = pool[np.lexsort((pool, -by[pool]))[:t]]
    rows = np.arange(m)[:, None]
    got = np.where(chosen >= 0, p[rows, chosen], 0.0)
    total = got.sum(axis=1, keepdims=True) + WEIGHT_EPS
    weights = got / total if c["norm"] else got
    out = (None, torch.from_numpy(weights), None, None, None)
    if not c["train"]:
        return out
    dw = s["dweights"].double().cpu().numpy()
    dx = np.zeros((m, e))
    for j in range(t):          # the derivative of each weight by each score, by the quotient rule
        for i in range(t if c["norm"] else 1):
            at = i if c["norm"] else j
            by_score = dw[:, j] * ((i == j) / total[:, 0] - got[:, j] / total[:, 0] ** 2) if c["norm"] else dw[:, j]
            ok = chosen[:, at] >= 0
            score = got[:, at]
            if c["score"] == "softmax":
                np.add.at(dx, (np.flatnonzero(ok), chosen[ok, at]), (by_score * score)[ok])
                dx[ok] -= (by_score * score)[ok, None] * p[ok]
            else:
                np.add.at(dx, (np.flatnonzero(ok), chosen[ok, at]), (by_score * score * (1.0 - score))[ok])
    return (*out, torch.from_numpy(dx))


def _exact_combine(s):
    c = s["case"]
    m, t, n = c["m"], c["top"], c["n"]
    out = torch.zeros((m, n), dtype=torch.float64, device=DEVICE)
    dy = torch.zeros((m * t, n), dtype=torch.float64, device=DEVICE) if c["train"] else None
    dw = torch.zeros((m, t), dtype=torch.float64, device=DEVICE)
    for j in range(t):
        token = torch.nonzero(s["positions"][:, j] >= 0)[:, 0]
        at, w = s["positions"][token, j].long(), s["weights"][token, j].double().unsqueeze(1)
        y = s["y"][at].double()
        out[token] += w * y
        if c["train"]:
            d = s["dout"][token].double()
            dy[at] = w * d
            dw[token, j] = (y * d).sum(1)
    return (out, dy, dw) if c["train"] else (out,)


def exact(case, seed):
    if case["op"] == "route" and case["m"] * case["experts"] > 1 << 23:
        return None             # the choice is made token by token on the host
    return {"quantize": _exact_quantize, "product": _exact_product, "experts": _exact_experts,
            "route": _exact_route, "combine": _exact_combine}[case["op"]](prepare(case, seed))
