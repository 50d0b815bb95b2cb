"""The detection-head operators restated in 64 bits (torch on the CPU), from
their formulas in include/gbnms.h; shares no code with the library."""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step above 1
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}  # half a step of the smallest numbers
EPS = 2.0 ** -24


def philox(block, offset, seed):
    """The four words of Philox 4x32-10, in Python integers."""
    m = 0xFFFFFFFF
    c = [block & m, block >> 32, offset & m, offset >> 32]
    k = [seed & m, seed >> 32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & m, (a >> 32) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def limit(p):
    return int(math.floor((1.0 - p) * 65536.0 + 0.5))


def kept(n, p, seed, offset, start=0):
    """Keep flags of elements start .. start + n - 1 (start a multiple of 8)."""
    flags = []
    for b in range((n + 7) // 8):
        for w in philox(start // 8 + b, offset, seed):
            flags += [(w & 0xFFFF) < limit(p), (w >> 16) < limit(p)]
    return torch.tensor(flags[:n], dtype=torch.bool)


def drop(x, p, seed, offset):
    if p == 0:
        return x
    k = kept(x.numel(), p, seed, offset).view(x.shape)
    return torch.where(k, x * (65536.0 / max(limit(p), 1)), torch.zeros_like(x))


def act(z, name):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.special.erf(z / math.sqrt(2)))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if name == "gelu":
        return 0.5 * (1 + torch.special.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def norm(x, groups, weight, bias, eps, name, p=0.0, seed=0, offset=0):
    """(y, mean, rstd, z) of x [batch, pixels, channels] (float64)."""
    N, S, C = x.shape
    v = x.view(N, S, groups, C // groups)
    mean = v.mean((1, 3))
    rstd = 1 / torch.sqrt((v - mean[:, None, :, None]).square().mean((1, 3)) + eps)
    z = ((v - mean[:, None, :, None]) * rstd[:, None, :, None]).view(N, S, C) * weight + bias
    return drop(act(z, name), p, seed, offset), mean, rstd, z


def norm_grad(dy, x, mean, rstd, groups, weight, bias, name, p=0.0, seed=0, offset=0):
    """(dx, dweight, dbias) and the sums of the terms' sizes behind the last
    two, and per image and group the size of dx's terms."""
    N, S, C = x.shape
    D = C // groups
    u = ((x.view(N, S, groups, D) - mean[:, None, :, None]) * rstd[:, None, :, None]).view(N, S, C)
    dz = drop(dy, p, seed, offset) * slope(u * weight + bias, name)
    du, uv = (dz * weight).view(N, S, groups, D), u.view(N, S, groups, D)
    m1, m2 = du.mean((1, 3), keepdim=True), (du * uv).mean((1, 3), keepdim=True)
    r = rstd[:, None, :, None]
    dx = (r * (du - m1 - uv * m2)).view(N, S, C)
    size = (r * (du.abs() + m1.abs() + (uv * m2).abs() + du.abs().mean((1, 3), keepdim=True)
                 + uv.abs() * (du * uv).abs().mean((1, 3), keepdim=True))).view(N, S, C)
    return (dx, (dz * u).sum((0, 1)), dz.sum((0, 1))), (size, (dz * u).abs().sum((0, 1)), dz.abs().sum((0, 1)))


def buckets(q_pos, k_pos, lut):
    reach = lut.shape[1] // 2
    sets = max(q_pos.shape[0], k_pos.shape[0])
    out = torch.full((sets, q_pos.shape[1], k_pos.shape[1]), -1, dtype=torch.int16)
    q, k, lut = q_pos.tolist(), k_pos.tolist(), lut.tolist()
    for s in range(sets):
        for i, a in enumerate(q[s % len(q)]):
            for j, b in enumerate(k[s % len(k)]):
                parts = [lut[x][reach + max(-reach, min(reach, kb - qa))] for x, (qa, kb) in enumerate(zip(a, b))]
                if min(parts) >= 0 and sum(parts) <= 32767:
                    out[s, i, j] = sum(parts)
    return out


def valid_pairs(buckets, num_buckets, key_mask):
    ok = ((buckets >= 0) & (buckets < num_buckets))[:, None]
    return ok if key_mask is None else ok & key_mask.bool()[:, None, None, :]


def softmax(scores, table, buckets, scale, key_mask=None):
    """(probs, logits) in float64."""
    ok = valid_pairs(buckets, table.shape[0], key_mask)
    bias = table[buckets.long().clamp(0, table.shape[0] - 1)].permute(0, 3, 1, 2)
    a = torch.where(ok, scores * scale + bias, torch.full((), -math.inf, dtype=torch.float64))
    top = a.amax(-1, keepdim=True) if a.shape[-1] else a.sum(-1, keepdim=True)
    e = torch.where(ok.expand_as(a), torch.exp(a - torch.where(torch.isinf(top) & (top < 0), 0.0, top)), 0.0)
    total = e.sum(-1, keepdim=True)
    return torch.where(ok & (total != 0), e / total, 0.0), a


def softmax_grad(dprobs, probs, buckets, num_buckets, scale, key_mask=None):
    """(dscores, dtable), and the sizes of the terms behind them."""
    ok = valid_pairs(buckets, num_buckets, key_mask).expand_as(probs)
    p, dp = torch.where(ok, probs, 0.0), torch.where(ok, dprobs, 0.0)
    da = p * (dp - (p * dp).sum(-1, keepdim=True))
    size = p * (dp.abs() + (p * dp).abs().sum(-1, keepdim=True))
    at = torch.where(ok, buckets.long()[:, None].expand_as(probs), num_buckets)

    def by_bucket(v):
        t = torch.zeros(num_buckets + 1, probs.shape[1], dtype=torch.float64)
        for h in range(probs.shape[1]):
            t[:, h].index_add_(0, at[:, h].reshape(-1), v[:, h].reshape(-1))
        return t[:num_buckets]

    return (scale * da, by_bucket(da)), (abs(scale) * size, by_bucket(size))


def close(got, ref, slack):
    """got (any type) within one rounding of its type and slack of ref."""
    got64 = got.detach().cpu().double()
    room = U[got.dtype] * ref.abs() * (1 + 1e-6) + TINY[got.dtype] + slack
    bad = ~((got64 - ref).abs() <= room)
    assert not bad.any(), (int(bad.sum()), float((got64 - ref).abs()[bad].max()), float((got64 - ref)[bad].abs().sub(
        room.expand_as(ref)[bad] if torch.is_tensor(room) else room).max()))
