"""The differentiable forms (greedy_iou_nms_gb300.autograd) against torch's
own autograd over elementary operations in 64 bits, and the example head."""
import importlib.util
import os

import pytest

import greedy_iou_nms_gb300 as g
import head_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.build()
    g.load()


def _leaves(*tensors):
    return [t.clone().cuda().requires_grad_() for t in tensors], [t.double().clone().requires_grad_() for t in tensors]


def _near(got, ref):
    """Within 1e-5 of the largest entry: some tens of roundings of sums whose
    terms are no larger than a few times it."""
    assert got.dtype == torch.float32
    assert float((got.cpu().double() - ref).abs().max()) <= 1e-5 * float(ref.abs().max())


def test_group_norm_act():
    from greedy_iou_nms_gb300 import autograd as ops
    r = torch.Generator().manual_seed(0)
    x, w, b, dy = (torch.randn(s, generator=r) for s in ((2, 5, 7, 24), (24,), (24,), (2, 5, 7, 24)))
    (xg, wg, bg), (x6, w6, b6) = _leaves(x, w, b)
    y = ops.group_norm_act(xg, 3, wg, bg, act="silu", p=0.2, seed=5, offset=1)
    y.backward(dy.cuda())
    ref = R.norm(x6.view(2, 35, 24), 3, w6, b6, 1e-5, "silu", 0.2, 5, 1)[0]
    ref.backward(dy.double().view(2, 35, 24))
    for got, want in ((xg.grad, x6.grad), (wg.grad, w6.grad), (bg.grad, b6.grad)):
        _near(got, want)


def test_parameter_types_and_absent_ones():
    from greedy_iou_nms_gb300 import autograd as ops
    x = torch.randn(2, 9, 16, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    w = torch.ones(16, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    ops.group_norm_act(x, 4, w, act="relu").sum().backward()
    assert w.grad.dtype == torch.bfloat16 and x.grad.dtype == torch.bfloat16
    y = torch.randn(2, 9, 16, device="cuda", requires_grad=True)
    ops.group_norm_act(y, 4).square().sum().backward()
    assert y.grad.shape == y.shape


def test_dropout():
    from greedy_iou_nms_gb300 import autograd as ops
    x = torch.randn(7, 33, device="cuda", requires_grad=True)
    res = torch.randn(7, 33, device="cuda", requires_grad=True)
    dy = torch.randn(7, 33, device="cuda")
    ops.dropout(x, 0.4, 9, 2, residual=res).backward(dy)
    assert torch.equal(x.grad, g.dropout(dy, 0.4, 9, 2)) and torch.equal(res.grad, dy)


def test_relation_softmax():
    from greedy_iou_nms_gb300 import autograd as ops
    r = torch.Generator().manual_seed(3)
    s, t, dp = (torch.randn(v, generator=r) for v in ((3, 2, 11, 17), (9, 2), (3, 2, 11, 17)))
    m = torch.randint(-1, 9, (3, 11, 17), generator=r).to(torch.int16)
    mask = torch.rand(3, 17, generator=r) < 0.8
    (sg, tg), (s6, t6) = _leaves(s, t)
    ops.relation_softmax(sg, tg, m.cuda(), scale=0.6, key_mask=mask.cuda()).backward(dp.cuda())
    R.softmax(s6, t6, m, 0.6, mask)[0].backward(dp.double())
    _near(sg.grad, s6.grad)
    _near(tg.grad, t6.grad)


def test_example_head_learns_and_suppresses():
    spec = importlib.util.spec_from_file_location("detection_head", os.path.join(ROOT, "examples", "detection_head.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, found, kept, model = example.main(steps=30)
    assert torch.isfinite(losses).all() and losses[-5:].mean() < 0.7 * losses[:5].mean()
    assert (kept >= 1).all() and (kept <= found).all()
    assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in model.parameters())
    assert float(model.table.grad.abs().sum()) > 0
