"""The operators of a transformer block among candidates, as cases to be measured and checked.

Around the attention weights by relative position that the library has, such a
block needs three more:

  linear    y = act(x weight^T + bias) + residual, and its gradient to x, the
            weight and the bias: every projection and both halves of a
            feed-forward part;
  layer     layer normalisation of rows with its affine map, the residual
            stream added before it and returned, and its gradient;
  rotary    queries and keys turned by their positions on several axes (time,
            row, column), whole numbers or fractions; the gradient is the turn
            backwards.

`own` says which form run() takes: elementary torch operations in 32 bits
(angles in 64), or the library's entry points.  exact() restates each operator
in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


# --------------------------------------------------------------------- cases

def listed():
    return [
        # One new entry for each of 16 live streams through a wide projection:
        # the weights are read for sixteen rows, latency counts.
        dict(name="linear-16-rows", op="linear", rows=16, inner=1024, outer=4096, type="bf16", act="none",
             residual=False, train=False),
        # The feed-forward part of one image's 300 candidates, inference.
        dict(name="linear-300", op="linear", rows=300, inner=256, outer=1024, type="bf16", act="gelu",
             residual=False, train=False),
        # A full-precision projection with nothing even about it.
        dict(name="linear-odd", op="linear", rows=1517, inner=333, outer=251, type="f32", act="relu",
             residual=True, train=True),
        # A wide model over every cell of 16 images' 32 x 32 maps: the largest,
        # bound by the tensor cores.
        dict(name="linear-16384", op="linear", rows=16384, inner=4096, outer=4096, type="f16", act="gelu",
             residual=True, train=False),
        # The training step of the feed-forward part of 16 images' 300 candidates.
        dict(name="linear-grad-4800", op="linear_grad", rows=4800, inner=1024, outer=4096, type="bf16", act="silu"),
        # 300 candidates of one image, the residual added on the way: latency counts.
        dict(name="layer-300", op="layer", rows=300, width=256, type="bf16", residual=True, train=False),
        # The finest level's cells (80 x 80) of a training batch of 16, with the
        # statistics that the gradient reads.
        dict(name="layer-102400", op="layer", rows=102400, width=1024, type="bf16", residual=True, train=True),
        # Its gradient, the residual stream's own added in.
        dict(name="layer-grad-102400", op="layer_grad", rows=102400, width=1024, type="bf16", residual=True),
        # Odd rows in full precision.
        dict(name="layer-grad-odd", op="layer_grad", rows=1517, width=999, type="f32", residual=False),
        # One new query and key for each of 16 streams, far into their history.
        dict(name="rotary-step", op="rotary", batch=16, tokens=1, heads=16, beside=8, dim=64, pairs="32", type="bf16",
             place="far", halves=True, shared=False),
        # Queries and keys of four clips of 16 frames of 40 x 40 cells, a slice
        # of the packed projection, on three axes.
        dict(name="rotary-clips", op="rotary", batch=4, tokens=25600, heads=16, beside=8, dim=64, pairs="8 12 12",
             type="bf16", place="cells", halves=True, shared=True),
        # The gradient for candidates at the centres of their boxes, neighbouring
        # elements paired, the last ones not turned.
        dict(name="rotary-grad-centres", op="rotary_grad", batch=3, tokens=517, heads=5, beside=0, dim=46,
             pairs="11 10", type="f32", place="centres", halves=False, shared=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear_grad", "layer", "layer_grad", "rotary", "rotary_grad"])
    kind = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op in ("linear", "linear_grad"):
        step = rng.choice([1, 8, 64])  # most widths are round, some are not
        inner, outer = (max(1, _log(rng, 8, 4096) // step) * step for _ in range(2))
        most = (4_000_000_000 if kind == "f32" else 64_000_000_000) // (inner * outer)
        rows = _log(rng, 1, max(1, min(20_000, most)))
        case = dict(op=op, rows=rows, inner=inner, outer=outer, type=kind,
                    act=rng.choice(["none", "relu", "silu", "gelu"]))
        if op == "linear":
            case.update(residual=rng.random() < 0.5, train=rng.random() < 0.5)
        return case
    if op in ("layer", "layer_grad"):
        step = rng.choice([1, 8, 64])
        width = max(8, _log(rng, 8, 16_384) // step * step)  # fewer leave a gradient of rounding alone
        rows = _log(rng, 1, max(1, min(100_000, 50_000_000 // width)))
        case = dict(op=op, rows=rows, width=width, type=kind, residual=rng.random() < 0.6)
        if op == "layer":
            case["train"] = rng.random() < 0.5
        return case
    axes = rng.randint(1, 3)
    pairs = [rng.randint(1, 128 // axes // rng.choice([1, 2, 4])) for _ in range(axes)]
    dim = 2 * sum(pairs) + rng.choice([0, 0, rng.randint(1, 16)])
    heads, beside = _log(rng, 1, 32), rng.choice([0, 0, 1, 4])
    batch = _log(rng, 1, 16)
    tokens = _log(rng, 1, max(1, min(8192, 50_000_000 // (batch * (heads + beside) * dim))))
    return dict(op=op, batch=batch, tokens=tokens, heads=heads, beside=beside, dim=dim,
                pairs=" ".join(str(n) for n in pairs), type=kind,
                place=rng.choice(["far", "cells", "centres"]), halves=rng.random() < 0.6, shared=rng.random() < 0.3)


def _pairs(case):
    """Pairs of elements turned by each axis."""
    return [int(n) for n in case["pairs"].split()]


# -------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    t = TYPES[case["type"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = dict(case=case)
    if case["op"] in ("linear", "linear_grad"):
        M, K, N = case["rows"], case["inner"], case["outer"]
        # Rows as a normalisation leaves them; weights that keep their size.
        s.update(x=normal(M, K).to(t), weight=(normal(N, K) / math.sqrt(K)).to(t), bias=0.2 * normal(N))
        if case["op"] == "linear":
            s["residual"] = normal(M, N).to(t) if case["residual"] else None
        else:
            s["dy"] = normal(M, N).to(t)
            s["pre"] = None if case["act"] == "none" else _plain_pre(s).to(t)
        return s
    if case["op"] in ("layer", "layer_grad"):
        M, C = case["rows"], case["width"]
        x = normal(M, C)
        x.mul_(0.5 + normal(C).abs()).add_(normal(C))  # a stream's features differ in spread and offset
        s.update(x=x.to(t), weight=1 + 0.2 * normal(C), bias=0.2 * normal(C))
        second = normal(M, C).to(t) if case["residual"] else None
        if case["op"] == "layer":
            s["residual"] = second
        else:
            s.update(dy=normal(M, C).to(t), dsum=second)
            v = s["x"].float()
            s["mean"] = v.mean(1)
            s["rstd"] = ((v - s["mean"][:, None]).square().mean(1) + EPS).rsqrt()
        return s
    B, n, H, D, axes = case["batch"], case["tokens"], case["heads"], case["dim"], len(_pairs(case))
    s["x"] = normal(B, n, H + case["beside"], D).to(t)[:, :, :H]
    sets = 1 if case["shared"] else B
    if case["place"] == "centres":  # of boxes in pixels
        s["positions"] = 1280 * torch.rand(sets, n, axes, generator=gen, device=dev)
    elif case["place"] == "cells":  # counted through from the last axis on, 40 cells an axis
        at = torch.arange(n, device=dev)[None] + torch.randint(0, 40, (sets, 1), generator=gen, device=dev)
        parts = [at // 40 ** a % (40 if a < axes - 1 else 1 << 30) for a in range(axes)]
        s["positions"] = torch.stack(parts[::-1], -1).to(torch.int32)
    else:  # somewhere in a long history
        first = torch.randint(0, 1_000_000, (sets, 1, axes), generator=gen, device=dev)
        s["positions"] = (first + torch.arange(n, device=dev)[None, :, None]).to(torch.int32)
    s["lut"] = _library().rotary_lut(*_pairs(case), base=10000.0).to(dev) if own else None
    return s


# ---------------------------------------------------------------- plain form

def _plain_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _plain_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        r = 1 / (1 + torch.exp(-z))
        return r * (1 + z * (1 - r))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _plain_pre(s):
    return s["x"].float() @ s["weight"].float().T + s["bias"]


def _plain_linear(s):
    c, t = s["case"], s["x"].dtype
    z = _plain_pre(s)
    y = _plain_act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return (y.to(t), z.to(t)) if c["train"] else y.to(t)


def _plain_linear_grad(s):
    c, t = s["case"], s["x"].dtype
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _plain_slope(s["pre"].float(), c["act"])
    return (dz @ s["weight"].float()).to(t), (dz.T @ s["x"].float()).to(t), dz.sum(0)


def _plain_layer(s):
    c, x = s["case"], s["x"]
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(x.dtype)  # the stream, an output: the norm is of what it holds
    v = x.float()
    mean = v.mean(1)
    d = v - mean[:, None]
    rstd = 1 / torch.sqrt(d.square().mean(1) + EPS)
    y = (d * rstd[:, None] * s["weight"] + s["bias"]).to(x.dtype)
    out = (y,) if s["residual"] is None else (y, x)
    return out + (mean, rstd) if c["train"] else out


def _plain_layer_grad(s):
    rstd, dy = s["rstd"][:, None], s["dy"].float()
    u = (s["x"].float() - s["mean"][:, None]) * rstd
    du = dy * s["weight"]
    dx = rstd * (du - du.mean(1, keepdim=True) - u * (du * u).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return dx.to(s["x"].dtype), (dy * u).sum(0), dy.sum(0)


def _plain_rotary(s, sign):
    c, x = s["case"], s["x"].float()
    angle = []
    for a, n in enumerate(_pairs(c)):
        frequency = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / n)
        angle.append(s["positions"][..., a, None].double() * frequency)
    angle = torch.cat(angle, -1)[:, :, None]  # [sets, tokens, 1, pairs]
    cos, sin = torch.cos(angle).float(), sign * torch.sin(angle).float()
    P = sum(_pairs(c))
    if c["halves"]:
        a, b = x[..., :P], x[..., P:2 * P]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * P:]], -1).to(s["x"].dtype)


# ----------------------------------------------------------------------- run

def _library():
    import greedy_iou_nms_gb300 as g
    return g


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op in ("rotary", "rotary_grad"):
            return _plain_rotary(s, 1.0 if op == "rotary" else -1.0)
        return {"linear": _plain_linear, "linear_grad": _plain_linear_grad, "layer": _plain_layer,
                "layer_grad": _plain_layer_grad}[op](s)
    g = _library()
    if op == "linear":
        return g.linear_act(s["x"], s["weight"], s["bias"], act=c["act"], residual=s["residual"],
                            return_pre=c["train"])
    if op == "linear_grad":
        return g.linear_act_grad(s["dy"], s["x"], s["weight"], s["pre"], act=c["act"])
    if op == "layer":
        out = g.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, residual=s["residual"], return_stats=c["train"])
        return out if isinstance(out, tuple) else (out,)
    if op == "layer_grad":
        return g.layer_norm_grad(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"], dsum=s["dsum"])
    turn = g.rotary if op == "rotary" else g.rotary_grad
    return turn(s["x"], s["positions"], s["lut"], halves=c["halves"])


def work(case):
    c = case
    e = 4 if c["type"] == "f32" else 2
    if c["op"] in ("linear", "linear_grad"):
        M, K, N = c["rows"], c["inner"], c["outer"]
        if c["op"] == "linear":
            outs = 1 + c["residual"] + c["train"]
            return {"bytes": e * (M * K + N * K + outs * M * N) + 4 * N, "flops": 2 * M * N * K}
        ins = 1 if c["act"] == "none" else 2  # dy, pre
        return {"bytes": e * (2 * M * K + 2 * N * K + ins * M * N) + 4 * N, "flops": 4 * M * N * K}
    if c["op"] == "layer":
        M, n = c["rows"], c["rows"] * c["width"]
        return {"bytes": (4 if c["residual"] else 2) * e * n + 8 * c["width"] + (8 * M if c["train"] else 0),
                "flops": 8 * n}
    if c["op"] == "layer_grad":
        M, n = c["rows"], c["rows"] * c["width"]
        return {"bytes": (4 if c["residual"] else 3) * e * n + 12 * c["width"] + 8 * M, "flops": 14 * n}
    n = c["batch"] * c["tokens"] * c["heads"] * c["dim"]
    sets = 1 if c["shared"] else c["batch"]
    return {"bytes": 2 * e * n + 4 * sets * c["tokens"] * len(_pairs(c)) + 8 * sum(_pairs(c)), "flops": 3 * n}


# ------------------------------------------------------- the same in 64 bits

def _exact_act(z, act):
    """The activation and its derivative."""
    if act == "relu":
        return z.clamp(min=0), torch.sign(z.clamp(min=0))
    if act == "silu":
        r = torch.sigmoid(z)
        return z * r, r + z * r * torch.sigmoid(-z)
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    op, x = case["op"], s["x"].double()
    if op == "linear":
        z = torch.addmm(s["bias"].double(), x, s["weight"].double().T)
        y = _exact_act(z, case["act"])[0]
        if s["residual"] is not None:
            y = s["residual"].double() + y
        return (y, z) if case["train"] else y
    if op == "linear_grad":
        dz = s["dy"].double()
        if s["pre"] is not None:
            dz = _exact_act(s["pre"].double(), case["act"])[1] * dz
        ones = torch.ones(1, dz.shape[0], dtype=torch.float64, device="cuda")
        return torch.mm(dz, s["weight"].double()), torch.mm(x.T, dz).T, torch.mm(ones, dz)[0]
    if op == "layer":
        out = ()
        if s["residual"] is not None:
            # The stream's rounding is part of the definition; a sum of two 16-bit values is exact in 64 bits.
            whole = s["residual"].double() + x
            x = whole.to(s["x"].dtype).double()
            out = (whole,)
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(s["bias"].double(), (x - mean) * rstd, s["weight"].double())
        return (y,) + out + ((mean[:, 0], rstd[:, 0]) if case["train"] else ())
    if op == "layer_grad":
        C = case["width"]
        rstd = s["rstd"].double().unsqueeze(1)
        u = torch.sub(x, s["mean"].double().unsqueeze(1)).mul_(rstd)
        dy = s["dy"].double()
        dbias, dweight = torch.einsum("mc->c", dy), torch.einsum("mc,mc->c", dy, u)
        du = s["weight"].double() * dy
        along = torch.einsum("mc,mc->m", du, u).unsqueeze(1) / C
        dx = (du - du.sum(1, keepdim=True) / C - along * u) * rstd
        return dx if s["dsum"] is None else dx + s["dsum"].double(), dweight, dbias
    # As complex numbers: first and second element of each pair, times e^(i angle).
    P, first = sum(_pairs(case)), 0
    out = x.clone()
    for axis, n in enumerate(_pairs(case)):
        j = torch.arange(n, device="cuda", dtype=torch.float64)
        angle = s["positions"][:, :, axis].double()[:, :, None, None] * torch.exp(-j / n * math.log(10000.0))
        turn = torch.polar(torch.ones_like(angle), angle if op == "rotary" else -angle)
        i = torch.arange(first, first + n, device="cuda")
        at, behind = (i, i + P) if case["halves"] else (2 * i, 2 * i + 1)
        z = torch.complex(x[..., at], x[..., behind]) * turn
        out[..., at], out[..., behind] = z.real, z.imag
        first += n
    return out
