"""Sums of a linear layer that leave binary32, and infinite operands: what the
definition has there, whichever kernel takes the call."""
import math

import pytest

import block_reference as R
import greedy_iou_nms_gb300 as g

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# A stream of the weight, tiles on the plain units, binary32 on the tensor cores; of 16 bits operands changed places,
# tiles of one block, of two.
SIZES = [(6, 72, 136), (200, 72, 136), (600, 72, 1600), (5000, 520, 1544)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.build()
    g.load()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,inner,outer", SIZES)
def test_activations_of_an_overflowing_sum(rows, inner, outer, kind):
    """2e38 twice is beyond binary32: z, and act(z) of every kind, is infinite."""
    t = R.TYPES[kind]
    x, w = torch.zeros(rows, inner, dtype=t), torch.ones(outer, inner, dtype=t)
    x[0], x[1, 3], x[1, 40], x[2, 5] = 1.0, 2e38, 2e38, 2e38
    for act in ("none", "relu", "silu", "gelu"):
        y, pre = g.linear_act(x.cuda(), w.cuda(), act=act, return_pre=True)
        assert (pre[1] == math.inf).all() and (y[1] == math.inf).all(), act
        assert (pre[2] == float(x[2, 5])).all() and (y[2] == float(x[2, 5])).all(), act
        assert (pre[0] == inner).all() and (y[0] == inner).all() and (y[3:] == 0).all(), act


def _infinite(x, w):
    """x w^T where some of x and w are infinite, the rest of it finite: in 64 bits, by torch."""
    return x.double() @ w.double().T


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,inner,outer", SIZES)
def test_infinite_operands(rows, inner, outer, kind):
    """An infinity times a number is one of the product's sign, times 0 a NaN, and opposite ones add up to a NaN."""
    t = R.TYPES[kind]
    r = torch.Generator().manual_seed(rows)
    # Whole numbers of 8 bits have no lower parts, fractions have them.
    x, w = torch.randint(-8, 9, (rows, inner), generator=r).to(t), torch.randn(outer, inner, generator=r).to(t)
    w[::2] = torch.randint(1, 5, w[::2].shape, generator=r).to(t)
    x[0, 1], x[1, 2], x[2, 3], x[2, 4] = math.inf, -math.inf, math.inf, -math.inf
    w[4, 1], w[5, 6], w[6, 2], w[7, 1] = math.inf, -math.inf, 0.0, 0.0
    x[rows - 1, 6] = 0.0
    ref = _infinite(x, w)
    y = g.linear_act(x.cuda(), w.cuda()).cpu()
    whole = torch.isfinite(ref)
    assert bool(whole[2:, 8:].any()) and bool(torch.isnan(ref).any()) and bool((ref == math.inf).any())
    assert torch.equal(torch.isfinite(y), whole)
    assert torch.equal(torch.isnan(y), torch.isnan(ref)) and torch.equal(y[~whole & ~torch.isnan(ref)].double(),
                                                                        ref[~whole & ~torch.isnan(ref)])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("rows,inner,outer", SIZES)
def test_infinite_operands_of_a_gradient(rows, inner, outer, act, kind):
    t = R.TYPES[kind]
    r = torch.Generator().manual_seed(outer)
    x, w, dy = (torch.randint(-4, 5, s, generator=r).to(t) for s in ((rows, inner), (outer, inner), (rows, outer)))
    x[0, 1], w[4, 2], dy[1, 3], dy[2, 0] = math.inf, -math.inf, math.inf, -math.inf
    z = torch.ones(rows, outer, dtype=t)
    got = g.linear_act_grad(dy.cuda(), x.cuda(), w.cuda(), z.cuda(), act=act)
    for out, ref in zip(got, (_infinite(dy, w.T), _infinite(dy.T, x.T), dy.double().sum(0))):
        out, odd = out.cpu().double(), ~torch.isfinite(ref)
        assert bool(odd.any()) and torch.equal(torch.isnan(out), torch.isnan(ref))
        odd &= ~torch.isnan(ref)
        assert torch.equal(out[odd], ref[odd]) and bool(torch.isfinite(out[torch.isfinite(ref)]).all())
