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


@pytest.mark.parametrize("kind,act", [("f32", "none"), ("f32", "silu")])
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
    # 2^12 sums of 64 one after another, half a step each; 24 steps of the tensor cores in each of them, which cut up
    # to 2^-25; the products that are left out, two of 2^-25 and one of 2^-34; the slopes.
    off = (2 ** 12 + 8) * R.U + 24 * 2.0 ** -25 + 2.0 ** -24 + slope
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
