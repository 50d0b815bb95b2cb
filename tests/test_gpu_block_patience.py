"""Waits of the products on the tensor cores that give up: with no patience at all
a wait for an ordinary copy runs out, the call comes back with its status set and
no wrong number among its results, and the next one is right."""
import ctypes
import math

import pytest

import greedy_iou_nms_gb300 as g

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
USUAL = 2_000_000_000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.build()
    g.load()


class _Patience:
    """Waits of this thread's launches give up after so many ns."""

    def __init__(self, ns):
        self.ns = ns

    def __enter__(self):
        g.load().gbnms_product_patience(ctypes.c_uint64(self.ns))

    def __exit__(self, *_):
        torch.cuda.synchronize()
        g.load().gbnms_product_patience(ctypes.c_uint64(USUAL))


def _given_up(call, usual):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with _Patience(0):
        out = call(status)
    assert status.item() == g.NMS_ERR_TIMEOUT
    lost = 0
    for p, q in zip(out, usual):
        nan = torch.isnan(p)
        lost += int(nan.sum())
        assert torch.equal(p[~nan], q[~nan])
    assert lost > 0
    status.zero_()
    again = call(status)
    assert status.item() == g.NMS_OK
    assert all(torch.equal(p, q) for p, q in zip(again, usual))


# 16 bits: operands changed places and four blocks to a tile, one block to a tile, tiles split over blocks, pairs with
# several tiles each.  Binary32: few tiles split, several tiles to a block.
@pytest.mark.parametrize("kind,rows,inner,outer", [
    ("bf16", 16, 1024, 4096), ("f16", 64, 4096, 128), ("bf16", 300, 256, 1024), ("bf16", 130, 4096, 136),
    ("f16", 5000, 520, 4104), ("f32", 1517, 333, 251), ("f32", 300, 4096, 264), ("f32", 3000, 264, 2056)])
def test_forward(kind, rows, inner, outer):
    r = torch.Generator().manual_seed(rows)
    t = TYPES[kind]
    x, w, res = (torch.randn(s, generator=r).to(t).cuda() for s in ((rows, inner), (outer, inner), (rows, outer)))
    usual = g.linear_act(x, w, act="silu", residual=res, return_pre=True)
    assert not any(bool(torch.isnan(v).any()) for v in usual)
    _given_up(lambda status: g.linear_act(x, w, act="silu", residual=res, return_pre=True, status=status), usual)


# Stretches of many rows whose sums a second kernel joins; dz in two parts; binary32 with stretches and without.
@pytest.mark.parametrize("kind,rows,inner,outer,act", [
    ("bf16", 20000, 64, 72, "none"), ("f16", 2600, 520, 1544, "gelu"), ("f32", 20000, 64, 72, "none"),
    ("f32", 2600, 520, 1544, "silu")])
def test_gradient(kind, rows, inner, outer, act):
    r = torch.Generator().manual_seed(rows)
    t = TYPES[kind]
    x, w, z, dy = (torch.randn(s, generator=r).to(t).cuda() for s in ((rows, inner), (outer, inner), (rows, outer),
                                                                     (rows, outer)))
    need = (True, True, False)
    usual = g.linear_act_grad(dy, x, w, z, act=act, need=need)[:2]
    _given_up(lambda status: g.linear_act_grad(dy, x, w, z, act=act, need=need, status=status)[:2], usual)


def test_a_status_word_is_left_alone():
    x, w = torch.ones(40, 64, device="cuda"), torch.ones(72, 64, device="cuda")
    status = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    assert bool((g.linear_act(x.half(), w.half(), status=status) == 64).all())
    assert math.isfinite(float(g.linear_act(x, w, status=status).sum())) and status.item() == 7
