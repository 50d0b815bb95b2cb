"""Group normalisation with activation and dropout (nms_group_norm_run) and
its gradient against 64 bits.

Tolerances, fixed beforehand.  A result is rounded once to its type; before
that, with values a few spreads from their mean, u = (x - mean) * rstd is off
by a few units of 2^-24 of (|u| + |mean| / spread), so 64 * 2^-24 * (1 + the
largest magnitude of z) covers u, the affine map and the activation.  Sums of
the gradient are chains of at most some hundred additions: 256 * 2^-24 of the
sum of their terms' sizes."""
import math

import numpy as np
import pytest

import greedy_iou_nms_gb300 as g
import head_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.build()
    g.load()


def _inputs(seed, N, S, C, t, param=torch.float32):
    r = torch.Generator().manual_seed(seed)
    x = torch.randn(N, S, C, generator=r) * (0.5 + torch.rand(C, generator=r)) + torch.randn(C, generator=r)
    dy = torch.randn(N, S, C, generator=r)
    w, b = 1 + 0.3 * torch.randn(C, generator=r), 0.3 * torch.randn(C, generator=r)
    return x.to(t), dy.to(t), w.to(param), b.to(param)


def _check(x, dy, w, b, groups, act, p=0.0, seed=7, offset=3, eps=1e-5, dev=None):
    """Forward and gradient of CPU tensors (dev: what the GPU gets instead)."""
    xd, dyd = dev if dev else (x.cuda(), dy.cuda())
    wd, bd = (None if v is None else v.cuda() for v in (w, b))
    w64 = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    b64 = torch.zeros(x.shape[-1], dtype=torch.float64) if b is None else b.double()
    flat = x.reshape(x.shape[0], -1, x.shape[-1]).double()
    y, mean, rstd = g.group_norm_act(xd, groups, wd, bd, eps=eps, act=act, p=p, seed=seed, offset=offset,
                                     return_stats=True)
    ry, rmean, rrstd, z = R.norm(flat, groups, w64, b64, eps, act, p, seed, offset)
    factor = 65536 / max(R.limit(p), 1)
    spread = (flat.view(flat.shape[0], flat.shape[1], groups, -1) - rmean[:, None, :, None]).square().mean((1, 3))
    R.close(mean, rmean, 64 * R.EPS * (spread.sqrt() + rmean.abs()))
    R.close(rstd, rrstd, 64 * R.EPS * rrstd)
    assert y.shape == xd.shape and y.dtype == x.dtype
    R.close(y.reshape(ry.shape), ry, 64 * R.EPS * factor * (1 + z.abs().max()))
    assert torch.equal(y, g.group_norm_act(xd, groups, wd, bd, eps=eps, act=act, p=p, seed=seed, offset=offset))
    dx, dw, db = g.group_norm_act_grad(dyd, xd, mean, rstd, groups, wd, bd, act=act, p=p, seed=seed, offset=offset)
    (rx, rw, rb), (sx, sw, sb) = R.norm_grad(dy.reshape(flat.shape).double(), flat, mean.cpu().double(),
                                             rstd.cpu().double(), groups, w64, b64, act, p, seed, offset)
    assert dx.shape == xd.shape and dx.dtype == x.dtype
    room = 1 + z.abs().max()  # the slope is as far off as z is
    R.close(dx.reshape(rx.shape), rx, 64 * R.EPS * room * sx)
    R.close(dw, rw, 256 * R.EPS * sw + 64 * R.EPS * room * sb)
    R.close(db, rb, 256 * R.EPS * sb)
    again = g.group_norm_act_grad(dyd, xd, mean, rstd, groups, wd, bd, act=act, p=p, seed=seed, offset=offset)
    assert all(torch.equal(u, v) for u, v in zip((dx, dw, db), again))
    return y, dx


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("N,S,C,groups", [(2, 400, 64, 8), (3, 37, 90, 6)])
def test_types_and_activations(t, act, N, S, C, groups):
    _check(*_inputs(1, N, S, C, t), groups, act)


@pytest.mark.parametrize("N,S,C,groups", [
    (1, 1, 32, 4), (1, 2, 8, 1), (5, 7, 3, 1), (2, 63, 1, 1), (1, 1000, 17, 17), (2, 65, 520, 4), (1, 129, 2048, 1),
    (1, 6401, 32, 4), (2, 1600, 256, 32), (1, 40, 1024, 2), (70, 3, 24, 3), (1, 25600, 16, 2), (9, 333, 40, 5),
    (1, 100000, 8, 1), (1300, 4, 16, 4)])
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_shapes(t, N, S, C, groups):
    _check(*_inputs(N + S + C, N, S, C, t), groups, "silu")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("N,S,C,groups,p", [(2, 50, 64, 8, 0.1), (1, 33, 12, 3, 0.5), (2, 9, 7, 7, 0.9),
                                            (1, 20, 16, 2, 1.0), (1, 20, 18, 2, 0.25)])
def test_dropout_in_the_epilogue(t, N, S, C, groups, p):
    """Rows of whole, half, quarter and odd generator blocks."""
    x, dy, w, b = _inputs(5, N, S, C, t)
    _check(x, dy, w, b, groups, "silu", p=p, seed=(1 << 63) + 12345, offset=(1 << 40) + 9)


def test_epilogue_draws_the_mask_of_dropout():
    x, _, w, b = _inputs(6, 2, 100, 32, torch.float32)
    x, w, b = x.cuda(), w.cuda(), b.cuda()
    y = g.group_norm_act(x, 4, w, b, act="silu")
    assert torch.equal(g.dropout(y, 0.3, 11, 5), g.group_norm_act(x, 4, w, b, act="silu", p=0.3, seed=11, offset=5))


@pytest.mark.parametrize("which", ["none", "weight", "bias", "half", "bfloat"])
def test_parameters(which):
    t = {"half": torch.float16, "bfloat": torch.bfloat16}.get(which, torch.float32)
    x, dy, w, b = _inputs(8, 2, 60, 48, t, param=t)
    if which in ("none", "weight", "bias"):
        w, b = (w if which == "weight" else None), (b if which == "bias" else None)
    _check(x, dy, w, b, 6, "silu")


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cut", [(0, 64), (8, 40), (3, 33), (1, 2)])
def test_a_slice_of_the_channels_is_read_in_place(t, cut):
    """Channel slices of a wider map: strides, and starts that no vector meets."""
    r = torch.Generator().manual_seed(3)
    wide, dwide = (torch.randn(2, 10, 13, 96, generator=r).to(t).cuda() for _ in range(2))
    x, dy = wide[..., cut[0]:cut[1]], dwide[..., cut[0]:cut[1]]
    C = cut[1] - cut[0]
    w, b = torch.randn(C, generator=r), torch.randn(C, generator=r)
    before = wide.clone()
    _check(x.cpu().contiguous(), dy.cpu().contiguous(), w, b, 2 if C % 2 == 0 else 1, "silu", dev=(x, dy))
    assert torch.equal(wide, before)


def test_orders_and_expanded_gradients():
    r = torch.Generator().manual_seed(4)
    nchw = torch.randn(2, 24, 9, 11, generator=r).cuda()
    x = nchw.contiguous(memory_format=torch.channels_last).permute(0, 2, 3, 1)
    y = g.group_norm_act(x, 3, act="relu")
    assert torch.equal(y, g.group_norm_act(nchw.permute(0, 2, 3, 1), 3, act="relu"))
    flipped = nchw.permute(0, 3, 2, 1)  # columns before rows
    assert torch.equal(g.group_norm_act(flipped, 3), g.group_norm_act(flipped.contiguous(), 3))
    _, mean, rstd = g.group_norm_act(x, 3, act="relu", return_stats=True)
    one = torch.ones((), device="cuda").expand(x.shape)
    for u, v in zip(g.group_norm_act_grad(one, x, mean, rstd, 3, act="relu"),
                    g.group_norm_act_grad(one.contiguous(), x, mean, rstd, 3, act="relu")):
        assert torch.equal(u, v)


def test_misaligned_start():
    """A map that starts 2 or 4 bytes past a vector boundary."""
    for t in (torch.float32, torch.bfloat16):
        x, dy, w, b = _inputs(9, 2, 50, 32, t)
        base = torch.empty(x.numel() + 1, dtype=t, device="cuda")
        shifted = base[1:].view(x.shape)
        shifted.copy_(x)
        _check(x, dy, w, b, 4, "gelu", dev=(shifted, dy.cuda()))


@pytest.mark.parametrize("S", [400, 30000])
def test_mean_far_above_the_spread_and_outliers(S):
    """A mean of 2000 spreads keeps the variance to 2^-24 * 64 relative; a
    first pixel 10000 spreads out (as the deviations' origin) too."""
    r = torch.Generator().manual_seed(2)
    x = torch.randn(2, S, 16, generator=r)
    x[0] += 2000.0
    x[1, 0] = 10000.0
    y, mean, rstd = g.group_norm_act(x.cuda(), 2, return_stats=True)
    v = x.double().view(2, S, 2, 8)
    rm = v.mean((1, 3))
    rr = 1 / torch.sqrt((v - rm[:, None, :, None]).square().mean((1, 3)) + 1e-5)
    R.close(mean, rm, 64 * R.EPS * rm.abs())
    # The mean's own rounding, 2^-24 of 2000 spreads, adds its square to the variance: nothing.
    R.close(rstd, rr, 64 * R.EPS * rr)


def test_constant_groups_and_single_values():
    x = torch.full((2, 30, 8), 3.5, device="cuda")
    y, mean, rstd = g.group_norm_act(x, 2, bias=torch.full((8,), 0.25, device="cuda"), return_stats=True)
    assert (mean == 3.5).all() and torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    assert (y == 0.25).all()
    y = g.group_norm_act(torch.full((1, 1, 4), 9.0, device="cuda"), 4)
    assert (y == 0).all()


def test_not_a_number_stays_in_its_group():
    x, dy, w, b = (v.cuda() for v in _inputs(1, 2, 40, 16, torch.float32))
    clean = g.group_norm_act(x, 4, w, b, act="silu")
    x[0, 3, 5] = float("nan")
    y = g.group_norm_act(x, 4, w, b, act="silu")
    assert y[0, :, 4:8].isnan().all()
    y[0, :, 4:8] = clean[0, :, 4:8]
    assert torch.equal(y, clean)


def test_nothing_to_do():
    for shape in ((0, 5, 8), (3, 0, 8)):
        x = torch.empty(shape, device="cuda")
        y, mean, rstd = g.group_norm_act(x, 2, return_stats=True)
        assert y.shape == x.shape and (mean == 0).all() and (rstd == 0).all()
        dx, dw, db = g.group_norm_act_grad(x, x, mean, rstd, 2)
        assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_gradient_against_differences(act):
    """<dx, v> and the parameters' gradients against central differences of
    the 64-bit forward: an error of h^2 (1e-8) and of the gradient's own
    2^-24 * 256 of its terms."""
    x, dy, w, b = _inputs(12, 2, 30, 12, torch.float32)
    r = torch.Generator().manual_seed(1)
    vx, vw, vb = (torch.randn(s, generator=r, dtype=torch.float64) for s in (x.shape, w.shape, b.shape))
    args = (3, 1e-5, act, 0.2, 77, 8)

    def loss(h):
        y = R.norm(x.double() + h * vx, args[0], w.double() + h * vw, b.double() + h * vb, *args[1:])[0]
        return float((y * dy.double()).sum())

    h = 1e-5
    numeric = (loss(h) - loss(-h)) / (2 * h)
    _, mean, rstd = g.group_norm_act(x.cuda(), 3, w.cuda(), b.cuda(), act=act, p=0.2, seed=77, offset=8,
                                     return_stats=True)
    dx, dw, db = g.group_norm_act_grad(dy.cuda(), x.cuda(), mean, rstd, 3, w.cuda(), b.cuda(), act=act, p=0.2,
                                       seed=77, offset=8)
    terms = [(d.cpu().double() * v) for d, v in ((dx, vx), (dw, vw), (db, vb))]
    size = sum(float(t.abs().sum()) for t in terms)
    assert abs(sum(float(t.sum()) for t in terms) - numeric) <= 256 * R.EPS * size + 1e-6 * size


def test_another_stream():
    x, dy, w, b = (v.cuda() for v in _inputs(13, 2, 500, 64, torch.bfloat16))
    want = g.group_norm_act(x, 8, w, b, act="silu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = g.group_norm_act(x, 8, w, b, act="silu")
    s.synchronize()
    assert torch.equal(got, want)


def test_in_a_graph():
    x, dy, w, b = (v.cuda() for v in _inputs(14, 2, 700, 64, torch.bfloat16))
    y, mean, rstd = g.group_norm_act(x, 8, w, b, act="silu", return_stats=True)
    want = (y, *g.group_norm_act_grad(dy, x, mean, rstd, 8, w, b, act="silu"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, m, rs = g.group_norm_act(x, 8, w, b, act="silu", return_stats=True)
        got = (y, *g.group_norm_act_grad(dy, x, m, rs, 8, w, b, act="silu"))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_refusals():
    x = torch.randn(2, 9, 12, device="cuda")
    stats = torch.ones(2, 3, device="cuda")
    for bad in (dict(act="tanh"), dict(p=1.5), dict(p=float("nan")), dict(seed=-1), dict(offset=1 << 64)):
        with pytest.raises(ValueError):
            g.group_norm_act(x, 3, **bad)
    for bad in (dict(weight=torch.ones(11, device="cuda")), dict(weight=torch.ones(12)),
                dict(bias=torch.ones(12, device="cuda", dtype=torch.float64)),
                dict(weight=torch.ones(24, device="cuda")[::2])):
        with pytest.raises(ValueError):
            g.group_norm_act(x, 3, **bad)
    for bad in (x.cpu(), x.double(), x[0, 0]):
        with pytest.raises(ValueError):
            g.group_norm_act(bad, 3)
    for groups in (5, 0, -1):
        with pytest.raises(g.NmsError) as e:
            g.group_norm_act(x, groups)
        assert e.value.code == g.NMS_ERR_INVALID_ARG
    with pytest.raises(g.NmsError):
        g.group_norm_act(x, 3, eps=-1.0)
    with pytest.raises(ValueError):
        g.group_norm_act_grad(x[:1], x, stats, stats, 3)
    with pytest.raises(ValueError):
        g.group_norm_act_grad(x, x, stats[:1], stats, 3)


@pytest.mark.parametrize("N,S,C,groups", [(1, 4000, 16, 2), (3, 2047, 24, 3), (1, 4096, 64, 1), (2, 700, 30, 2),
                                          (1, 9000, 256, 32), (1, 30000, 36, 9), (40, 1, 64, 8)])
@pytest.mark.parametrize("t", [torch.float32, torch.float16])
def test_slabs_over_blocks_and_pieces(t, N, S, C, groups):
    """Slabs over two to eight blocks of a cluster with a short last one, and
    images of few and of many pieces."""
    _check(*_inputs(S, N, S, C, t), groups, "gelu", p=0.1)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("S,C,groups", [(40, 16, 4), (300, 90, 6), (9000, 32, 8), (700, 48, 3)])
@pytest.mark.parametrize("where", [0.0, 0.5, 1.0])
def test_infinity_leaves_no_number_in_its_group(act, S, C, groups, where):
    """inf - inf: mean and variance of such a group are no numbers, nor are
    its results and its input's gradient; other groups keep their bits."""
    x, dy, w, b = (v.cuda() for v in _inputs(1, 2, S, C, torch.bfloat16))
    clean = g.group_norm_act(x, groups, w, b, act=act, return_stats=True)
    dclean = g.group_norm_act_grad(dy, x, *clean[1:], groups, w, b, act=act)[0]
    D = C // groups
    bad = slice(D, 2 * D)
    for value in (math.inf, -math.inf):
        x[1, int(where * (S - 1)), D + int(where * (D - 1))] = value
        y, mean, rstd = g.group_norm_act(x, groups, w, b, act=act, return_stats=True)
        assert y[1, :, bad].isnan().all() and not mean[1, 1].isfinite() and rstd[1, 1].isnan()
        dx = g.group_norm_act_grad(dy, x, mean, rstd, groups, w, b, act=act)[0]
        assert dx[1, :, bad].isnan().all()
        y[1, :, bad], dx[1, :, bad] = clean[0][1, :, bad], dclean[1, :, bad]
        assert torch.equal(y, clean[0]) and torch.equal(dx, dclean)


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("spread,eps", [(1e13, 1e-5), (1e15, 1e-5), (1e16, 0.0), (1e-6, 0.0), (1e-13, 0.0),
                                        (1e-16, 0.0)])
@pytest.mark.parametrize("S,C,groups", [(40, 16, 4), (9000, 32, 8), (700, 258, 3), (30000, 20, 2)])
def test_spreads_far_from_one(t, spread, eps, S, C, groups):
    """Small maps and large ones alike; the gradient goes along with x, so
    that its projections on u count."""
    x, dy, w, b = _inputs(S, 2, S, C, torch.float32)
    _check((x * spread).to(t), (dy + 2 * x).to(t), w, b, groups, "silu", eps=eps)


@pytest.mark.parametrize("t,N,S,C,groups", [(torch.bfloat16, 16, 25600, 512, 32), (torch.bfloat16, 16, 25600, 504, 84),
                                            (torch.float32, 16, 25600, 256, 16), (torch.bfloat16, 16, 25600, 510, 17)])
@pytest.mark.parametrize("far", [1e3, 1e5])
def test_outliers_at_the_start_of_long_pieces(t, N, S, C, groups, far):
    """Pieces of about a thousand rows, 256 and 2048 values to a thread, whose
    first values stand far out; mean and rstd against 64 bits."""
    gen = torch.Generator(device="cuda").manual_seed(C)
    x = torch.randn(N, S, C, generator=gen, device="cuda").to(t)
    D = C // groups
    for k in range(groups):
        x[k % N, 0, k * D] = far
        x[k % N, S // 2 // 1024 * 1024, k * D] = -far
        x[k % N, k, k * D + D - 1] = far
    _, mean, rstd = g.group_norm_act(x, groups, return_stats=True)
    for n in range(N):
        var, m = torch.var_mean(x[n].double().view(S, groups, D), dim=(0, 2), correction=0)
        R.close(mean[n], m.cpu(), (64 * R.EPS * (var.sqrt() + m.abs())).cpu())
        R.close(rstd[n], (1 / torch.sqrt(var + 1e-5)).cpu(), (64 * R.EPS / torch.sqrt(var + 1e-5)).cpu())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("groups", [1, 512])
def test_gelu_from_tail_to_tail(t, groups):
    """z given exactly (as the bias, with weight 0), on a large and a small
    map.  The density's exponent z^2 log2(e) / 2 (+ 1.33) is off by three
    roundings (3 ln 2 of them, 1.5 z^2, in the density) and 2^x and 1/x by 2^-22.
    The distribution function: in binary32 for z < 0 within 2^-24 (20 + 2 z^2) of
    itself and beyond 0 by that of the tail and a rounding; in 16 bits within
    2^-21, and for z < 0 within 3e-5 of itself."""
    z = torch.cat([torch.linspace(-10, 10, 4001), torch.linspace(-0.1, 0.1, 95)])
    C = z.numel()
    zero = torch.zeros(C, device="cuda")
    x = torch.randn(1, 8, C, generator=torch.Generator().manual_seed(1)).to(t).cuda()
    dy = torch.zeros_like(x)
    dy[0, 0] = 1
    y, mean, rstd = g.group_norm_act(x, groups, zero, z.cuda(), act="gelu", return_stats=True)
    slope = g.group_norm_act_grad(dy, x, mean, rstd, groups, zero, z.cuda(), act="gelu")[2]  # dbias
    z = z.double()
    cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
    part = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if t == torch.float32:
        off = torch.where(z < 0, cdf, 1 - cdf) * (20 + 2 * z * z) * R.EPS + torch.where(z < 0, 0.0, R.EPS)
    else:
        off = torch.where(z < 0, torch.clamp(3e-5 * cdf, max=2.0 ** -21), torch.full_like(z, 2.0 ** -21))
    density_off = (8 + 2 * z * z) * R.EPS
    R.close(y[0, 0], z * cdf, z.abs() * off + R.EPS * (z * cdf).abs())
    R.close(slope, cdf + part, off + part.abs() * density_off + 2 * R.EPS * (cdf + part.abs()))


@pytest.mark.parametrize("N,S,C,groups", [(40000, 1, 8, 1), (300000, 1, 8, 1), (1, 3000000, 2, 1), (5000, 3, 24, 3)])
def test_parameter_gradients_of_many_images(N, S, C, groups):
    """Terms of one size and sign, whose roundings go one way: their sums are
    as right as those of a few hundred."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn(N, S, C, generator=gen, device="cuda")
    dy = torch.full_like(x, 0.1)
    _, mean, rstd = g.group_norm_act(x, groups, return_stats=True)
    dx, dw, db = g.group_norm_act_grad(dy, x, mean, rstd, groups)
    u = x.double().view(N, S, groups, -1).sub(mean.double()[:, None, :, None]).mul(rstd.double()[:, None, :, None])
    dz = dy[0, 0, 0].double() * u.view(-1, C)
    R.close(db, torch.full((C,), float(dy[0, 0, 0].double() * N * S), dtype=torch.float64),
            256 * R.EPS * float(dy[0, 0, 0]) * N * S)
    R.close(dw, dz.sum(0).cpu(), 256 * R.EPS * dz.abs().sum(0).cpu())
    dw = g.group_norm_act_grad(u.view_as(x).float(), x, mean, rstd, groups)[1]  # terms that go along with u
    square = u.view(-1, C).float().double() * u.view(-1, C)
    R.close(dw, square.sum(0).cpu(), 256 * R.EPS * square.sum(0).cpu())


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,S,C,groups", [(4, 100, 64, 8), (5, 100, 64, 8), (16, 40, 256, 32), (17, 40, 256, 32),
                                          (1, 2048, 64, 8), (1, 2049, 64, 8), (76, 4, 256, 32), (77, 4, 256, 32),
                                          (700, 3, 48, 3), (3, 400, 90, 6)])
def test_both_sides_of_the_cluster_sizes(t, N, S, C, groups):
    _check(*_inputs(N * S, N, S, C, t), groups, "silu")
