"""The operators of a trainable detection head, as cases to be measured and checked.

Three operators sit around the decode and the suppression of this library:

  norm      group normalisation of a channels-last feature map with its
            affine map, activation and dropout, and its gradient;
  dropout   x -> mask * x / keep (+ residual) with the mask drawn from a
            counter-based generator and never stored; the gradient is the
            same map of the incoming gradient;
  relation  attention weights among candidates or window cells: softmax over
            the keys of scale * score + table[bucket of the relative
            position], its gradient to the scores and to the table, and the
            bucket map itself.

`own` says which form run() takes: elementary torch operations in 32 bits, or
the library's entry points.  exact() restates each operator in 64 bits.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # One image's coarsest level (20 x 20 of a 640 input), inference: what
        # a live camera waits for, so latency counts.
        dict(name="norm-20x20", op="norm", batch=1, pixels=400, channels=256, groups=32, type="bf16", act="silu",
             p=0.0, train=False),
        # The finest level (80 x 80) of a training batch of 16, statistics
        # returned for the backward pass.
        dict(name="norm-80x80", op="norm", batch=16, pixels=6400, channels=256, groups=32, type="bf16", act="silu",
             p=0.0, train=True),
        # A ragged full-precision map: 37 x 41 pixels, 90 channels in groups of 15.
        dict(name="norm-odd", op="norm", batch=3, pixels=1517, channels=90, groups=6, type="f32", act="relu",
             p=0.0, train=True),
        # The middle level's gradient in the same training step.
        dict(name="norm-grad-40x40", op="norm_grad", batch=16, pixels=1600, channels=256, groups=32, type="bf16",
             act="silu", p=0.0),
        # A mask branch's 160 x 160 map with dropout, the gradient: the
        # largest of the norms, beyond what one cluster of SMs holds.
        dict(name="norm-grad-160x160", op="norm_grad", batch=8, pixels=25600, channels=128, groups=32, type="f16",
             act="gelu", p=0.1),
        # 300 candidates an image, features added back after dropout: a small call.
        dict(name="dropout-300", op="dropout", shape0=16 * 300, shape1=256, type="bf16", p=0.1, residual=True,
             grad=False),
        # The attention weights of 1000 candidates, 8 heads, 16 images: the
        # gradient through their dropout, a pure stream.
        dict(name="dropout-weights", op="dropout", shape0=16 * 8 * 1000, shape1=1000, type="bf16", p=0.2,
             residual=False, grad=True),
        # One new query per image against 8192 earlier entries, distances in 32
        # logarithmic buckets, later entries masked: serving, latency counts.
        dict(name="relation-one-query", op="relation", batch=16, heads=8, queries=1, keys=8192, type="f32",
             layout="log", buckets=32, keep=1.0),
        # Candidates kept by the suppression (300 an image, some images fewer),
        # positions by grid cell, 15 x 15 buckets, map computed per call.
        dict(name="relation-300", op="relation", batch=16, heads=8, queries=300, keys=300, type="bf16",
             layout="cells", buckets=225, keep=0.7),
        # 7 x 7 windows over the 80 x 80 level of 16 images: one map for all.
        dict(name="relation-windows", op="relation", batch=2304, heads=8, queries=49, keys=49, type="f16",
             layout="window", buckets=169, keep=1.0),
        # The gradient of 8 x 8 windows, shared map.
        dict(name="relation-grad-windows", op="relation_grad", batch=1600, heads=8, queries=64, keys=64, type="f16",
             layout="window", buckets=225, keep=1.0),
        # The gradient among 1000 candidates of each of 16 images, a map per image.
        dict(name="relation-grad-1000", op="relation_grad", batch=16, heads=8, queries=1000, keys=1000, type="bf16",
             layout="cells", buckets=225, keep=0.9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "dropout", "relation", "relation_grad"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op in ("norm", "norm_grad"):
        groups = rng.choice([1, 2, 4, 5, 8, 16, 32, 32])
        channels = groups * rng.choice([1, 2, 3, 4, 8, 8, 15, 16])
        batch = _log(rng, 1, 32)
        most = (13_000_000 if kind == "f32" else 26_000_000) // (batch * channels)
        pixels = _log(rng, 1, max(1, min(102_400, most)))
        pixels = max(pixels, -(-8 // (channels // groups)))  # two values in a group leave a gradient of rounding alone
        case = dict(op=op, batch=batch, pixels=pixels, channels=channels, groups=groups, type=kind,
                    act=rng.choice(["none", "relu", "silu", "gelu"]), p=rng.choice([0.0, 0.0, 0.1, 0.5]))
        if op == "norm":
            case["train"] = rng.random() < 0.5
        return case
    if op == "dropout":
        rows, cols = _log(rng, 1, 64_000), _log(rng, 1, 1000)
        return dict(op=op, shape0=rows, shape1=cols, type=kind, p=rng.choice([0.05, 0.1, 0.3, 0.5]),
                    residual=rng.random() < 0.4, grad=False) | ({"grad": True, "residual": False}
                                                                if rng.random() < 0.4 else {})
    layout = rng.choice(["log", "cells", "window"])
    if layout == "window":
        side = rng.randint(3, 16)
        queries = keys = side * side
        buckets = (2 * side - 1) ** 2
        heads = rng.choice([1, 3, 4, 8])
        batch = _log(rng, 1, max(1, min(2000, 50_000_000 // (heads * queries * keys))))
    else:
        batch, heads = _log(rng, 1, 16), rng.choice([1, 3, 4, 8])
        keys = _log(rng, 8, 4000)  # one key's weight is 1 and its gradient 0, whatever the input
        queries = keys if rng.random() < 0.6 else _log(rng, 1, 300)
        queries = max(1, min(queries, 50_000_000 // (batch * heads * keys)))
        buckets = rng.choice([16, 32, 48]) if layout == "log" else rng.choice([9, 81, 225])
    return dict(op=op, batch=batch, heads=heads, queries=queries, keys=keys, type=kind, layout=layout,
                buckets=buckets, keep=rng.choice([1.0, 0.8, 0.5]))


# -------------------------------------------------------------------- inputs

def _lut(case):
    """The table of bucket parts by clamped relative position: [axes, 2 * reach + 1]."""
    n = case["buckets"]
    if case["layout"] == "log":
        # Distances back: exact below n/2, then logarithmic up to 1024; an
        # entry that lies ahead of the query is masked.
        exact, reach = n // 2, 1024
        part = np.full((1, 2 * reach + 1), -1, np.int32)
        for d in range(reach + 1):
            b = d if d < exact else min(n - 1, exact + int(math.log(d / exact) / math.log(reach / exact)
                                                           * (n - exact) + 1e-9))
            part[0, reach - d] = b
        return part
    reach = (math.isqrt(n) - 1) // 2  # 2 * reach + 1 buckets an axis
    step = np.arange(2 * reach + 1, dtype=np.int32)
    return np.stack([step * (2 * reach + 1), step])


def _positions(case, gen):
    """Query and key positions, [sets, length, axes] int32."""
    B, Q, K = case["batch"], case["queries"], case["keys"]
    if case["layout"] == "log":
        # Queries are the last ones of a history of keys; each image stands elsewhere in it.
        last = torch.randint(max(0, K - max(1, K // 8)), K, (B, 1, 1), generator=gen)
        q = (last - torch.arange(Q - 1, -1, -1)[None, :, None]).to(torch.int32)
        return q, torch.arange(K, dtype=torch.int32)[None, :, None]
    if case["layout"] == "window":
        side = math.isqrt(Q)
        at = torch.arange(Q)
        cell = torch.stack([at // side, at % side], -1).to(torch.int32)[None]
        return cell, cell
    centre = torch.randint(0, 80, (B, 20, 2), generator=gen)  # candidates stand in clusters on the 80 x 80 grid
    pick = torch.randint(0, 20, (B, K), generator=gen)
    cell = torch.gather(centre, 1, pick[..., None].expand(-1, -1, 2)) + torch.randint(-6, 7, (B, K, 2), generator=gen)
    cell = cell.to(torch.int32)
    at = torch.arange(Q) % K
    return cell[:, at].contiguous(), cell


def prepare(case, seed):
    dev = torch.device("cuda")
    t = TYPES[case["type"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    key = int(torch.randint(0, 1 << 62, (1,), generator=host))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = dict(case=case, seed=key, offset=seed & 0xFFFF)
    if case["op"] in ("norm", "norm_grad"):
        N, S, C, G = case["batch"], case["pixels"], case["channels"], case["groups"]
        x = normal(N, S, C)
        x.mul_(0.5 + normal(C).abs()).add_(normal(C))  # channels of a convolution differ in spread and offset
        s.update(x=x.to(t), weight=1 + 0.2 * normal(C), bias=0.2 * normal(C), eps=1e-5)
        if case["op"] == "norm_grad":
            s["dy"] = normal(N, S, C).to(t)
            v = s["x"].float().view(N, S, G, C // G)
            mean = v.mean((1, 3))
            var = (v - mean[:, None, :, None]).square().mean((1, 3))
            s.update(mean=mean, rstd=(var + s["eps"]).rsqrt())
        return s
    if case["op"] == "dropout":
        s["x"] = normal(case["shape0"], case["shape1"]).to(t)
        s["residual"] = normal(case["shape0"], case["shape1"]).to(t) if case["residual"] else None
        return s
    B, H, Q, K = case["batch"], case["heads"], case["queries"], case["keys"]
    q, k = _positions(case, host)
    s.update(q_pos=q.to(dev), k_pos=k.to(dev), lut=torch.from_numpy(_lut(case)).to(dev))
    s["table"] = 0.5 * normal(case["buckets"], H)
    s["scale"] = 1.0 / math.sqrt(32.0)
    s["mask"] = None
    if case["keep"] < 1.0:
        # Valid entries come first, as the suppression returns them; counts differ by image and one image has none.
        least = int(case["keep"] * K)
        count = torch.randint(least, K + 1, (B,), generator=host)
        if B > 2:
            count[1] = 0
        s["mask"] = (torch.arange(K)[None] < count[:, None]).to(dev)
    # Windows have one map that the model keeps; the others' positions are new with each call.
    s["map"] = _plain_buckets(s) if case["layout"] == "window" else None
    scores = 4.0 * normal(B, H, Q, K)
    if case["op"] == "relation":
        s["scores"] = scores.to(t)
    else:
        buckets = s["map"] if s["map"] is not None else _plain_buckets(s)
        s["map"] = buckets
        s["probs"] = _plain_softmax(scores, s, buckets).to(t)
        s["dprobs"] = normal(B, H, Q, K).to(t)
    return s


# ---------------------------------------------------------------- plain form

def _plain_kept(n, s, p):
    """Which of n elements are kept, and the factor of the kept: 16-bit fields
    of Philox 4x32-10 words (Salmon et al., "Parallel random numbers: as easy
    as 1, 2, 3", 2011), eight elements a block; counter (block, offset), key seed."""
    low = 0xFFFFFFFF
    block = torch.arange((n + 7) // 8, device="cuda")
    c = [block & low, block >> 32, torch.full_like(block, s["offset"] & low), torch.full_like(block, s["offset"] >> 32)]
    k0, k1 = s["seed"] & low, s["seed"] >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # 64-bit products; the sign bit is data
        c = [((b >> 32) & low) ^ c[1] ^ k0, b & low, ((a >> 32) & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(c, 1)
    field = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n]
    limit = _limit(p)
    return field < limit, (65536.0 / limit if limit else 0.0)


def _limit(p):
    """A field below this is kept: the keep probability in 65536ths, rounded to nearest."""
    return int(math.floor((1.0 - p) * 65536.0 + 0.5))


def _plain_drop(x, s, p):
    if p == 0.0:
        return x
    kept, factor = _plain_kept(x.numel(), s, p)
    return torch.where(kept.view(x.shape), x * factor, torch.zeros_like(x))


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


def _plain_norm(s):
    c, x = s["case"], s["x"].float()
    N, S, C, G = c["batch"], c["pixels"], c["channels"], c["groups"]
    v = x.view(N, S, G, C // G)
    mean = v.mean((1, 3))
    d = v - mean[:, None, :, None]
    rstd = 1 / torch.sqrt(d.square().mean((1, 3)) + s["eps"])
    z = (d * rstd[:, None, :, None]).view(N, S, C) * s["weight"] + s["bias"]
    y = _plain_drop(_plain_act(z, c["act"]), s, c["p"]).to(s["x"].dtype)
    return (y, mean, rstd) if c["train"] else y


def _plain_norm_grad(s):
    c, x = s["case"], s["x"].float()
    N, S, C, G = c["batch"], c["pixels"], c["channels"], c["groups"]
    wide = (N, S, G, C // G)
    unit = ((x.view(wide) - s["mean"][:, None, :, None]) * s["rstd"][:, None, :, None]).view(N, S, C)
    dz = _plain_drop(s["dy"].float(), s, c["p"]) * _plain_slope(unit * s["weight"] + s["bias"], c["act"])
    dweight, dbias = (dz * unit).sum((0, 1)), dz.sum((0, 1))
    du = (dz * s["weight"]).view(wide)
    unit = unit.view(wide)
    m1, m2 = du.mean((1, 3), keepdim=True), (du * unit).mean((1, 3), keepdim=True)
    dx = s["rstd"][:, None, :, None] * (du - m1 - unit * m2)
    return dx.view(N, S, C).to(s["x"].dtype), dweight, dbias


def _plain_buckets(s):
    lut, q, k = s["lut"], s["q_pos"].long(), s["k_pos"].long()
    reach = (lut.shape[1] - 1) // 2
    rel = (k[:, None] - q[:, :, None]).clamp(-reach, reach) + reach  # [sets, queries, keys, axes]
    part = lut.long()[torch.arange(lut.shape[0], device="cuda"), rel]
    return torch.where((part < 0).any(-1), -1, part.sum(-1)).to(torch.int16)


def _plain_valid(s, buckets):
    valid = (buckets >= 0)[:, None]
    return valid if s["mask"] is None else valid & s["mask"][:, None, None, :]


def _plain_softmax(scores, s, buckets):
    bias = s["table"].float()[buckets.clamp(min=0).long()].permute(0, 3, 1, 2)
    valid = _plain_valid(s, buckets)
    low = torch.full((), -math.inf, device="cuda")
    a = torch.where(valid, scores.float() * s["scale"] + bias, low)
    top = a.amax(-1, keepdim=True)
    e = torch.where(valid, torch.exp(a - torch.where(top == -math.inf, torch.zeros_like(top), top)), 0.0)
    total = e.sum(-1, keepdim=True)
    return torch.where(total == 0, torch.zeros_like(e), e / total)


def _plain_relation(s):
    buckets = s["map"] if s["map"] is not None else _plain_buckets(s)
    probs = _plain_softmax(s["scores"], s, buckets).to(s["scores"].dtype)
    return probs if s["map"] is not None else (probs, buckets)


def _plain_relation_grad(s):
    p, dp = s["probs"].float(), s["dprobs"].float()
    valid = _plain_valid(s, s["map"])
    da = torch.where(valid, p * (dp - torch.where(valid, p * dp, 0.0).sum(-1, keepdim=True)), 0.0)
    B, H, Q, _ = p.shape
    n, sets = s["case"]["buckets"], s["map"].shape[0]
    per = (da.sum(0, keepdim=True) if sets == 1 else da).permute(0, 2, 3, 1).reshape(-1, H)
    # Each query's sums first, then over the queries: short chains of additions.
    row = torch.arange(sets * Q, device="cuda").view(sets, Q, 1) * (n + 1)
    at = row + torch.where(s["map"] < 0, n, s["map"].long())
    dtable = torch.zeros(sets * Q * (n + 1), H, device="cuda").index_add_(0, at.reshape(-1), per)
    dtable = dtable.view(sets * Q, n + 1, H).sum(0)[:n]
    return (da * s["scale"]).to(s["probs"].dtype), dtable


# ----------------------------------------------------------------------- run

def _library():
    import greedy_iou_nms_gb300 as g
    return g


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "dropout":
            y = _plain_drop(s["x"].float(), s, c["p"])
            return (y if s["residual"] is None else y + s["residual"].float()).to(s["x"].dtype)
        return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "relation": _plain_relation,
                "relation_grad": _plain_relation_grad}[op](s)
    g = _library()
    if op == "norm":
        return g.group_norm_act(s["x"], c["groups"], s["weight"], s["bias"], eps=s["eps"], act=c["act"], p=c["p"],
                                seed=s["seed"], offset=s["offset"], return_stats=c["train"])
    if op == "norm_grad":
        return g.group_norm_act_grad(s["dy"], s["x"], s["mean"], s["rstd"], c["groups"], s["weight"], s["bias"],
                                     act=c["act"], p=c["p"], seed=s["seed"], offset=s["offset"])
    if op == "dropout":
        if c["grad"]:
            return g.dropout_grad(s["x"], c["p"], s["seed"], s["offset"])
        return g.dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s["residual"])
    if op == "relation":
        if s["map"] is not None:
            return g.relation_softmax(s["scores"], s["table"], s["map"], scale=s["scale"], key_mask=s["mask"])
        buckets = g.relation_buckets(s["q_pos"], s["k_pos"], s["lut"])
        return g.relation_softmax(s["scores"], s["table"], buckets, scale=s["scale"], key_mask=s["mask"]), buckets
    return g.relation_softmax_grad(s["dprobs"], s["probs"], s["map"], c["buckets"], scale=s["scale"],
                                   key_mask=s["mask"])


def work(case):
    c = case
    e = 4 if c["type"] == "f32" else 2
    if c["op"] in ("norm", "norm_grad"):
        n = c["batch"] * c["pixels"] * c["channels"]
        few = 8 * c["channels"] + 8 * c["batch"] * c["groups"]  # weight and bias; mean and rstd
        if c["op"] == "norm":
            return {"bytes": 2 * e * n + few - (0 if c["train"] else 8 * c["batch"] * c["groups"]), "flops": 12 * n}
        return {"bytes": 3 * e * n + few + 8 * c["channels"], "flops": 30 * n}
    if c["op"] == "dropout":
        n = c["shape0"] * c["shape1"]
        return {"bytes": (3 if c["residual"] else 2) * e * n, "flops": 2 * n}
    B, H, Q, K = c["batch"], c["heads"], c["queries"], c["keys"]
    n, sets = B * H * Q * K, 1 if c["layout"] == "window" else B
    few = 4 * c["buckets"] * H + (B * K if c["keep"] < 1.0 else 0)
    if c["op"] == "relation":
        # The map is an input where the model keeps one, an output where the call makes it.
        axes = 1 if c["layout"] == "log" else 2
        pos = 0 if c["layout"] == "window" else 4 * axes * (B * Q + (K if c["layout"] == "log" else B * K))
        return {"bytes": 2 * e * n + 2 * sets * Q * K + pos + few, "flops": 6 * n}
    return {"bytes": 3 * e * n + 2 * sets * Q * K + few, "flops": 7 * n}


# ------------------------------------------------------- the same in 64 bits

def _exact_kept(n, seed, offset, p):
    """The generator again, on the host in unsigned 64-bit words."""
    u = np.uint64
    low, half = u(0xFFFFFFFF), u(32)
    limit = _limit(p)
    got = np.empty((n + 7) // 8 * 8, np.bool_)
    for at in range(0, (n + 7) // 8, 1 << 20):
        ctr = np.arange(at, min(at + (1 << 20), (n + 7) // 8), dtype=np.uint64)
        x0, x1 = ctr & low, ctr >> half
        x2, x3 = np.full_like(ctr, offset & 0xFFFFFFFF), np.full_like(ctr, offset >> 32)
        for r in range(10):
            k0 = u(((seed & 0xFFFFFFFF) + r * 0x9E3779B9) & 0xFFFFFFFF)
            k1 = u(((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
            left, right = x0 * u(0xD2511F53), x2 * u(0xCD9E8D57)
            x0, x1, x2, x3 = (right >> half) ^ x1 ^ k0, right & low, (left >> half) ^ x3 ^ k1, left & low
        for w, x in enumerate((x0, x1, x2, x3)):
            got[8 * at + 2 * w:8 * (at + len(ctr)):8] = (x & u(0xFFFF)) < u(limit)
            got[8 * at + 2 * w + 1:8 * (at + len(ctr)):8] = (x >> u(16)) < u(limit)
    return torch.from_numpy(got[:n]).to("cuda"), (65536.0 / limit if limit else 0.0)


def _exact_drop(x, s, p):
    if p == 0.0:
        return x
    kept, factor = _exact_kept(x.numel(), s["seed"], s["offset"], p)
    return (x * factor).masked_fill_(~kept.view(x.shape), 0.0)


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
    op = case["op"]
    if op == "dropout":
        y = _exact_drop(s["x"].double(), s, case["p"])
        return y if s["residual"] is None else s["residual"].double() + y
    if op in ("norm", "norm_grad"):
        N, S, C, G = case["batch"], case["pixels"], case["channels"], case["groups"]
        x = s["x"].double().view(N, S, G, -1).permute(0, 2, 1, 3).reshape(N, G, -1)  # a group's values in one row

        def back(v):
            return v.view(N, G, S, C // G).permute(0, 2, 1, 3).reshape(N, S, C)

        weight, bias = s["weight"].double(), s["bias"].double()
        if op == "norm":
            var, mean = torch.var_mean(x, dim=2, correction=0)
            rstd = (var + s["eps"]) ** -0.5
            unit = back((x - mean[..., None]) * rstd[..., None])
            y = _exact_drop(_exact_act(unit * weight + bias, case["act"])[0], s, case["p"])
            return (y, mean, rstd) if case["train"] else y
        mean, rstd = s["mean"].double(), s["rstd"].double()
        unit = back((x - mean[..., None]) * rstd[..., None])
        dz = _exact_act(unit * weight + bias, case["act"])[1] * _exact_drop(s["dy"].double(), s, case["p"])
        flat = dz.view(N * S, C)
        dbias, dweight = flat.sum(0), (flat * unit.view(N * S, C)).sum(0)
        du = (dz * weight).view(N, S, G, -1).permute(0, 2, 1, 3).reshape(N, G, -1)
        unit = unit.view(N, S, G, -1).permute(0, 2, 1, 3).reshape(N, G, -1)
        m = du.shape[2]
        dx = (du - du.sum(2, keepdim=True) / m - unit * ((du * unit).sum(2, keepdim=True) / m)) * rstd[..., None]
        return back(dx), dweight, dbias
    buckets = s["map"]
    if buckets is None:
        buckets = torch.zeros((), dtype=torch.int64, device="cuda")
        reach = s["lut"].shape[1] // 2
        for axis, part in enumerate(s["lut"].long()):
            apart = s["k_pos"].long()[:, None, :, axis] - s["q_pos"].long()[:, :, None, axis]
            buckets = buckets + part[reach + torch.clamp(apart, -reach, reach)]
    masked = (buckets < 0).unsqueeze(1)
    if s["mask"] is not None:
        masked = masked | ~s["mask"].view(case["batch"], 1, 1, -1)
    if op == "relation":
        a = s["scores"].double() * s["scale"]
        a += s["table"].double().T[:, buckets.clamp(min=0).long()].transpose(0, 1)
        a.masked_fill_(masked, -math.inf)
        probs = torch.nan_to_num_(torch.softmax(a, -1), nan=0.0)  # a row with nothing to attend to is zero
        return probs if s["map"] is not None else (probs, None)
    p, dp = s["probs"].double().masked_fill(masked, 0.0), s["dprobs"].double().masked_fill(masked, 0.0)
    da = p * dp - p * (p * dp).sum(-1, keepdim=True)
    n, B, H = case["buckets"], case["batch"], case["heads"]
    at = buckets.long().masked_fill(buckets < 0, n).unsqueeze(1).expand(B, H, -1, -1)
    at = at + torch.arange(H, device="cuda").view(1, H, 1, 1) * (n + 1)
    dtable = torch.zeros(H * (n + 1), dtype=torch.float64, device="cuda").index_add_(0, at.reshape(-1), da.reshape(-1))
    return da * s["scale"], dtable.view(H, n + 1)[:, :n].T
