"""The operators of a transformer block in 64 bits, in elementary torch
operations (differentiable), and the bounds that their tests hold results to."""
import math

import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24  # half a step of binary32


def half_step(t):
    return torch.finfo(t).eps / 2


def act(z, kind):
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    return z


def slope(z, kind):
    if kind == "relu":
        return (z > 0).double()
    if kind == "silu":
        r = torch.sigmoid(z)
        return r * (1 + z * (1 - r))
    if kind == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def act_error(t):
    """Of act(z) relative to max(|z|, 1), of act'(z) to 1: the sigmoid is right
    to 2^-22 (1 + |z|) of itself, the normal distribution function to 2^-24 (20
    + 2 z^2) of its smaller tail (2^-21 in 16 bits); act' multiplies either by
    up to |z| once more, where the tails are below e^-|z|: 2^-19 covers both."""
    return 2.0 ** -19


def linear(x, w, bias, kind, residual=None):
    z = x.double() @ w.double().T
    if bias is not None:
        z = z + bias.double()
    y = act(z, kind)
    return (y if residual is None else y + residual.double()), z


def product_bound(a, b, t):
    """Of a binary32 sum of a @ b: an addition is off by half a step (a whole
    one on the tensor cores, which may cut) of the terms' sizes so far."""
    k = a.shape[-1]
    return (k + 2) * (U if t is torch.float32 else 2 * U) * (a.double().abs() @ b.double().abs())


def layer(x, w, b, eps, residual=None):
    t = x.dtype
    s = x if residual is None else (x.float() + residual.float()).to(t)
    v = s.double()
    var, mean = torch.var_mean(v, dim=-1, correction=0, keepdim=True)
    rstd = (var + eps) ** -0.5
    u = (v - mean) * rstd
    y = u if w is None else u * w.double()
    if b is not None:
        y = y + b.double()
    return y, s, mean[..., 0], rstd[..., 0]


def layer_grad(dy, x, mean, rstd, w, dsum=None):
    g, m, r = dy.double(), mean.double()[..., None], rstd.double()[..., None]
    u = (x.double() - m) * r
    du = g if w is None else g * w.double()
    dx = r * (du - du.mean(-1, keepdim=True) - u * (du * u).mean(-1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.double()
    flat = (g * u).flatten(0, -2) if g.dim() > 1 else (g * u)[None]
    return dx, flat.sum(0), g.reshape(-1, g.shape[-1]).sum(0)


def rotary(x, positions, pairs, halves, base=10000.0, sign=1.0):
    P, v = sum(pairs), x.double()
    angle = torch.cat([positions[..., a, None].double() * base ** (-torch.arange(n, dtype=torch.float64) / n)
                       for a, n in enumerate(pairs)], -1)[:, :, None]
    c, s = torch.cos(angle), sign * torch.sin(angle)
    out = v.clone()
    first, second = (slice(0, P), slice(P, 2 * P)) if halves else (slice(0, 2 * P, 2), slice(1, 2 * P, 2))
    out[..., first] = v[..., first] * c - v[..., second] * s
    out[..., second] = v[..., second] * c + v[..., first] * s
    return out
