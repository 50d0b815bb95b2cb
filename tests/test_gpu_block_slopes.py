"""What the 16-bit linear layer's gradient keeps of dz = dy act'(z): the products
take it in two parts, so that their results are off by their own rounding and not
by that of a factor too."""
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


def _inputs(rows, inner, outer, kind, seed):
    r = torch.Generator().manual_seed(seed)
    t = R.TYPES[kind]
    x = torch.randn(rows, inner, generator=r).to(t)
    w = (torch.randn(outer, inner, generator=r) / inner ** 0.5).to(t)
    return x, w, (0.7 * torch.randn(rows, outer, generator=r)).to(t), torch.randn(rows, outer, generator=r).to(t)


# Operands changed places (up to 64 rows), tiles of one block and of two, tiles split over a cluster, stretches of many
# rows, rows that are copied first.
SIZES = [(1, 8, 8), (17, 72, 200), (60, 1000, 520), (300, 256, 1024), (257, 264, 520), (1000, 136, 8), (2600, 520, 1544),
         (20000, 64, 72), (5000, 333, 14), (130, 127, 129), (9000, 24, 3000)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("rows,inner,outer", SIZES)
def test_products_take_unrounded_slopes(rows, inner, outer, kind, act):
    """Off by: the activation's error; dz in two parts (half a step of half a step, and in binary16 half of its smallest
    number, twice over for its parts); a binary32 sum that cuts; the result's rounding."""
    x, w, z, dy = _inputs(rows, inner, outer, kind, rows + inner)
    t = x.dtype
    got = g.linear_act_grad(dy.cuda(), x.cuda(), w.cuda(), z.cuda(), act=act)
    dz = dy.double() * R.slope(z.double(), act)
    least = 2.0 ** -24 if t is torch.float16 else 0.0
    off = R.act_error(t) * dy.double().abs() + (R.half_step(t) ** 2 + 2 * R.U) * dz.abs() + least
    for out, a, b, e in ((got[0], dz, w.double(), off), (got[1], dz.T, x.double(), off.T)):
        ref, size = a @ b, a.abs() @ b.abs()
        # The lower parts' sum, 2^-8 of the upper parts' at most, is cut as often.
        bound = (a.shape[1] + 2) * 2 * R.U * (1 + 2 * R.half_step(t)) * size + e @ b.abs()
        bound = bound + R.half_step(t) * (ref.abs() + bound) + least
        assert ((out.cpu().double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_errors_are_those_of_the_results_rounding(kind):
    """By size: a rounding to nearest is off by 1 / sqrt(3) of half a step of 2^e in its mean square, and the values of a
    bell curve have 1.36 times the mean square's root of their 2^e, whatever its width: 0.425 of eps / 2.  The rounding of
    a factor on top of that makes it 0.6."""
    x, w, z, dy = _inputs(1200, 512, 1024, kind, 5)
    dz = dy.double() * R.slope(z.double(), "silu")
    got = g.linear_act_grad(dy.cuda(), x.cuda(), w.cuda(), z.cuda(), act="silu")
    for out, ref in ((got[0], dz @ w.double()), (got[1], dz.T @ x.double())):
        assert float((out.cpu().double() - ref).norm() / ref.norm()) <= 0.5 * R.half_step(x.dtype)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("rows,inner,outer", [(17, 72, 200), (700, 264, 520), (5000, 333, 14)])
def test_rounded_slopes_are_the_callers_choice(rows, inner, outer, kind):
    """With round_slopes the products are those of dz rounded; ReLU passes dy on, so that nothing changes."""
    from greedy_iou_nms_gb300 import autograd as ops
    x, w, z, dy = (v.cuda() for v in _inputs(rows, inner, outer, kind, 6))
    got = g.linear_act_grad(dy, x, w, z, act="gelu", round_slopes=True)
    # dz rounded: the gradient to x by a weight that is the identity.
    one = torch.eye(outer, dtype=dy.dtype, device="cuda")
    dz = g.linear_act_grad(dy, torch.zeros_like(dy), one, z, act="gelu", round_slopes=True)[0]
    ref = g.linear_act_grad(dz, x, w)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert torch.equal(got[2], g.linear_act_grad(dy, x, w, z, act="gelu")[2])
    for p, q in zip(g.linear_act_grad(dy, x, w, z, act="relu", round_slopes=True), g.linear_act_grad(dy, x, w, z, act="relu")):
        assert torch.equal(p, q)
    leaves = [v.clone().requires_grad_() for v in (x, w)]
    y = ops.linear_act(*leaves, act="gelu", round_slopes=True)
    y.backward(dy)
    pre = g.linear_act(x, w, return_pre=True)[1]
    for p, q in zip(leaves, g.linear_act_grad(dy, x, w, pre, act="gelu", round_slopes=True)):
        assert torch.equal(p.grad, q)


def test_slopes_beyond_the_largest_binary16():
    """dz above 65504 (an activation's slope is up to 1.13) is finite in two parts."""
    dy, z = torch.full((40, 64), 65504.0).half(), torch.full((40, 64), 1.4).half()
    x, w = torch.full((40, 32), 2.0 ** -6).half(), (0.25 * torch.eye(64))[:, :32].half().contiguous()
    for act in ("gelu", "silu"):
        dz = dy.double() * R.slope(z.double(), act)
        got = g.linear_act_grad(dy.cuda(), x.cuda(), w.cuda(), z.cuda(), act=act)
        assert float(dz.min()) > 65520.0  # which rounds to an infinity
        for out, ref in ((got[0], dz @ w.double()), (got[1], dz.T @ x.double())):
            assert float((out.cpu().double() - ref).abs().max()) <= 2.0 ** -10 * float(ref.abs().max())
