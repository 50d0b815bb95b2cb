"""Gradients of very many rows: sums that are cut into stretches, and as many
blocks as keep every chain of additions short."""
import pytest

import block_reference as R
import greedy_iou_nms_gb300 as g

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.build()
    g.load()


def _positive(r, shape, t):
    """Of one sign, so that what additions cut off mounts."""
    return (0.5 + torch.rand(shape, generator=r, device="cuda")).to(t)


def _product(a, b, step=25000):
    """a^T b in 64 bits, some rows at a time."""
    return sum(a[i:i + step].double().T @ b[i:i + step].double() for i in range(0, a.shape[0], step))


def _cut(t):
    """Relative to a sum of one sign: the tensor cores cut each product below 2^-25 of the sum so far, and that below 2^-23
    after 16 of them, as many products as they add up by themselves."""
    return (2 ** 12 if t is torch.float16 else 2 ** 15) * (2.0 ** -25 + 2.0 ** -27)


# Operands that changed places, tiles split over blocks, pairs with several tiles each.
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("rows,inner,outer", [(16, 1 << 18, 136), (16, 5000, 4096), (300, 1 << 17, 264), (20000, 1 << 16, 1032),
                                              (5000, 33000, 1600)])
def test_long_widths(rows, inner, outer, kind):
    t = R.TYPES[kind]
    r = torch.Generator("cuda").manual_seed(4)
    x, w = ((_positive(r, s, torch.float32) / 64).to(t) for s in ((rows, inner), (outer, inner)))
    b, res = _positive(r, (outer,), torch.float32), _positive(r, (rows, outer), t)
    y, pre = g.linear_act(x, w, b, act="relu", residual=res, return_pre=True)
    some = torch.arange(rows) if rows < 200 else torch.cat([torch.arange(100), torch.arange(rows - 100, rows)])
    z = x[some].double() @ w.double().T + b.double()
    near = (_cut(t) + 80 * R.U) * z
    assert bool(((pre[some].double() - z).abs() <= near + (R.half_step(t) + 2 * R.U) * z).all())
    z = z + res[some].double()
    assert bool(((y[some].double() - z).abs() <= near + (R.half_step(t) + 4 * R.U) * z).all())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("rows,inner,outer", [(40, 200, 40000), (3000, 1032, 40000)])
def test_long_gradients_to_x(rows, inner, outer, act, kind):
    t = R.TYPES[kind]
    r = torch.Generator("cuda").manual_seed(5)
    dy, w, z = ((_positive(r, s, torch.float32) / d).to(t) for s, d in (((rows, outer), 64), ((outer, inner), 64),
                                                                        ((rows, outer), 1)))
    x = torch.zeros(rows, inner, dtype=t, device="cuda")
    dx, dw, _ = g.linear_act_grad(dy, x, w, z, act=act, need=(True, True, False))
    ref = (dy.double() * R.slope(z.double(), act)) @ w.double()
    slope = 1.5 * R.act_error(t) * (act != "none")
    # In two parts: the lower one's sum is cut too.
    off = _cut(t) * (1 + 2 * R.half_step(t)) + 80 * R.U + R.half_step(t) ** 2 + slope + R.half_step(t) + 2 * R.U
    assert float((dx.double() / ref - 1).abs().max()) <= off and not bool(dw.any())


@pytest.mark.parametrize("kind,act", [("f32", "none"), ("f32", "silu"), ("bf16", "none"), ("bf16", "silu"), ("f16", "none")])
def test_linear(kind, act):
    """More tiles than the few that are cut for want of blocks."""
    rows, inner, outer = 300000, 1288, 40
    t = R.TYPES[kind]
    r = torch.Generator("cuda").manual_seed(1)
    x, dy = _positive(r, (rows, inner), t), (_positive(r, (rows, outer), t).float() / 256).to(t)
    w, z = torch.ones(outer, inner, dtype=t, device="cuda"), _positive(r, (rows, outer), t)
    _, dw, db = g.linear_act_grad(dy, x, w, z, act=act, need=(False, True, True))
    dz = dy.double() * R.slope(z.double(), act)
    slope = 1.5 * R.act_error(t) * (act != "none")  # relative to slopes of 0.7 and more
    ref = _product(dz, x)
    if t is torch.float32:
        # 2^12 sums of 64 one after another, half a step each; 24 times 16 products of the tensor cores in each of them,
        # cut as above; the products that are left out, two of 2^-25 and one of 2^-34; the slopes.
        off = (2 ** 12 + 8) * R.U + 24 * 16 * (2.0 ** -25 + 2.0 ** -27) + 2.0 ** -24 + slope
    else:
        # The stretches' cuts and their binary32 sum; the lower parts of dz; the result's rounding.
        off = _cut(t) + 80 * R.U + R.half_step(t) ** 2 + slope + (R.half_step(t) + 2 * R.U)
    assert float((dw.double() / ref - 1).abs().max()) <= off
    # A warp adds 256 rows and its block eight of those; the runs' sums are compensated.
    assert float((db.double() / dz.sum(0) - 1).abs().max()) <= (256 + 8 + 4) * R.U + slope


def test_slopes_sums_of_many_wide_rows():
    rows, outer = 300000, 2560
    r = torch.Generator("cuda").manual_seed(2)
    dy = _positive(r, (rows, outer), torch.bfloat16)
    x, w = torch.ones(rows, 8, dtype=torch.bfloat16, device="cuda"), torch.ones(outer, 8, dtype=torch.bfloat16, device="cuda")
    db = g.linear_act_grad(dy, x, w, need=(False, False, True))[2]
    ref = sum(dy[i:i + 25000].double().sum(0) for i in range(0, rows, 25000))
    assert float((db.double() / ref - 1).abs().max()) <= (256 + 8 + 4) * R.U


@pytest.mark.parametrize("rows,width,kind", [(320000, 999, "f32"), (3800000, 64, "bf16")])
def test_layer_norm(rows, width, kind):
    """Parameters' sums over more rows than one wave of blocks takes 256 at a time."""
    t = R.TYPES[kind]
    r = torch.Generator("cuda").manual_seed(3)
    x, dy = _positive(r, (rows, width), t), _positive(r, (rows, width), t)
    w = torch.ones(width, device="cuda")
    _, mean, rstd = g.layer_norm(x, w, return_stats=True)
    dx, dw, db = g.layer_norm_grad(dy, x, mean, rstd, w)
    size = ref_w = ref_b = 0.0
    for i in range(0, rows, 25000):
        s = slice(i, min(i + 25000, rows))
        ref = R.layer_grad(dy[s], x[s], mean[s], rstd[s], w)
        ref_w, ref_b = ref_w + ref[1], ref_b + ref[2]
        size = size + (dy[s].double() * (x[s].double() - mean[s].double()[:, None]) * rstd[s].double()[:, None]).abs().sum(0)
        # Moments and averages of `width` terms of a size, and the gradient's own dozen of roundings of terms up to rstd
        # times 8 (|du| up to 1.5, |u| up to 2 of a flat distribution).
        near = (width + 12) * R.U * 8 * float(rstd[s].max()) + R.half_step(t) * ref[0].abs()
        assert bool(((dx[s].double() - ref[0]).abs() <= near).all())
    # 256 rows a team and its block's teams (16 of them, or one); u itself is off by three roundings.
    assert bool(((dw.double() - ref_w).abs() <= (256 + 16 + 8) * R.U * size).all())
    assert float((db.double() / ref_b - 1).abs().max()) <= (256 + 16 + 4) * R.U


def test_same_bits_in_graphs_and_on_two_streams():
    """Calls at the same time have scratch memory of their own."""
    r = torch.Generator("cuda").manual_seed(6)
    x, w = ((_positive(r, s, torch.float32) / 64 - 1 / 64).half() for s in ((9000, 9000), (328, 9000)))

    def both():
        y, pre = g.linear_act(x, w, act="gelu", return_pre=True)
        return (y, *g.linear_act_grad(y, x, w, pre, act="gelu"))

    def same(a, b):
        return all(torch.equal(p, q) for p, q in zip(a, b))

    first = both()
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(both())
    for s in sides:
        s.synchronize()
    assert all(same(first, out) for out in outs)
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            held.append(both())
    x.copy_(x.flip(0))
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    again = both()
    assert all(same(again, out) for out in held) and not same(again, first)
