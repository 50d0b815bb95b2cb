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
SIZES = [(3, 72, 136), (200, 72, 136), (600, 72, 1600), (5000, 520, 1544)]


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
