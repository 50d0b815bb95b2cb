"""The transformer block's operators for torch's autograd, one by one and run
together as a block among candidates, against torch's own autograd over
elementary operations in 64 bits."""
import pytest

import block_reference as B
import greedy_iou_nms_gb300 as g
import head_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.build()
    g.load()


def _leaves(*tensors):
    return [t.clone().cuda().requires_grad_() for t in tensors], [t.double().clone().requires_grad_() for t in tensors]


def _near(got, ref, steps=1e-5):
    """Within 1e-5 of the largest entry: some tens of roundings of sums whose
    terms are no larger than a few times it."""
    got, ref = got.detach().cpu().double(), ref.detach()
    assert float((got - ref).abs().max()) <= steps * float(ref.abs().max())


def test_linear_act():
    from greedy_iou_nms_gb300 import autograd as ops
    r = torch.Generator().manual_seed(0)
    x, w, b, res, dy = (torch.randn(s, generator=r) for s in ((2, 9, 24), (40, 24), (40,), (2, 9, 40), (2, 9, 40)))
    for act in ("none", "relu", "silu", "gelu"):
        got, ref = _leaves(x, w, b, res)
        ops.linear_act(*got[:3], act=act, residual=got[3]).backward(dy.cuda())
        B.linear(*ref[:3], act, ref[3])[0].backward(dy.double())
        for p, q in zip(got, ref):
            assert p.grad.dtype is p.dtype
            _near(p.grad, q.grad)


def test_linear_act_parts():
    from greedy_iou_nms_gb300 import autograd as ops
    x = torch.randn(5, 16, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(8, 16, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    b = torch.zeros(8, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    ops.linear_act(x, w, b, act="gelu").sum().backward()
    assert w.grad.dtype is torch.bfloat16 and b.grad.dtype is torch.bfloat16
    res = torch.randn(5, 8, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    ops.linear_act(x, w.detach(), residual=res).sum().backward()
    assert torch.equal(res.grad, torch.ones_like(res))
    with torch.no_grad():
        assert not ops.linear_act(x, w, b, act="gelu").requires_grad


def test_layer_norm():
    from greedy_iou_nms_gb300 import autograd as ops
    r = torch.Generator().manual_seed(1)
    x, w, b, res, dy, ds = (torch.randn(s, generator=r) for s in ((2, 7, 20), (20,), (20,), (2, 7, 20), (2, 7, 20),
                                                                  (2, 7, 20)))
    got, ref = _leaves(x, w, b, res)
    y, s = ops.layer_norm(*got[:3], residual=got[3])
    torch.autograd.backward([y, s], [dy.cuda(), ds.cuda()])
    s6 = ref[0] + ref[3]
    y6 = torch.nn.functional.layer_norm(s6, (20,), *ref[1:3])
    torch.autograd.backward([y6, s6], [dy.double(), ds.double()])
    for p, q in zip(got, ref):
        _near(p.grad, q.grad)
    # Without residual and parameters; only the sum used; only the norm used.
    (xg,), (x6,) = _leaves(x)
    ops.layer_norm(xg).backward(dy.cuda())
    torch.nn.functional.layer_norm(x6, (20,)).backward(dy.double())
    _near(xg.grad, x6.grad)
    (xg, rg), _ = _leaves(x, res)
    ops.layer_norm(xg, residual=rg)[1].backward(ds.cuda())
    assert torch.equal(xg.grad.cpu(), ds) and torch.equal(rg.grad.cpu(), ds)
    (xg, rg), (x6, r6) = _leaves(x, res)
    ops.layer_norm(xg, residual=rg)[0].backward(dy.cuda())
    torch.nn.functional.layer_norm(x6 + r6, (20,)).backward(dy.double())
    _near(rg.grad, r6.grad)
    _near(xg.grad, x6.grad)


def test_rotary():
    from greedy_iou_nms_gb300 import autograd as ops
    r = torch.Generator().manual_seed(2)
    x, dy = (torch.randn(2, 6, 3, 30, generator=r) for _ in range(2))
    p = torch.randint(0, 40, (2, 6, 2), generator=r).to(torch.int32)
    for halves in (True, False):
        (xg,), (x6,) = _leaves(x)
        ops.rotary(xg, p.cuda(), g.rotary_lut(8, 6).cuda(), halves=halves).backward(dy.cuda())
        B.rotary(x6, p, (8, 6), halves).backward(dy.double())
        _near(xg.grad, x6.grad)


def _block(ops, x, p, side, buckets, table, mask, lut):
    """A pre-norm block among candidates; ops: the library's operators, or None: elementary operations in 64 bits."""
    batch, n, width = x.shape
    heads, dim = table.shape[1], width // table.shape[1]
    if ops is None:
        y = torch.nn.functional.layer_norm(x, (width,), p["w1"], p["b1"])
        qkv = B.linear(y, p["qkv"], p["qkv_b"], "none")[0].view(batch, n, 3 * heads, dim)
        turned = B.rotary(qkv[:, :, :2 * heads], side, (dim // 4, dim // 4), True)
    else:
        y = ops.layer_norm(x, p["w1"], p["b1"])
        qkv = ops.linear_act(y, p["qkv"], p["qkv_b"]).view(batch, n, 3 * heads, dim)
        turned = ops.rotary(qkv[:, :, :2 * heads], side, lut)
    q, k, v = (t.transpose(1, 2) for t in (turned[:, :, :heads], turned[:, :, heads:], qkv[:, :, 2 * heads:]))
    scores = q @ k.mT
    if ops is None:
        probs = R.softmax(scores, table, buckets, dim ** -0.5, mask)[0]
        mixed = (probs @ v).transpose(1, 2).reshape(batch, n, width)
        mixed = B.linear(mixed, p["join"], None, "none")[0]
        s = x + mixed
        y = torch.nn.functional.layer_norm(s, (width,), p["w2"], p["b2"])
        hidden = B.linear(y, p["up"], p["up_b"], "gelu")[0]
        return B.linear(hidden, p["down"], p["down_b"], "none", s)[0]
    probs = ops.relation_softmax(scores, table, buckets, scale=dim ** -0.5, key_mask=mask)
    mixed = ops.linear_act((probs @ v).transpose(1, 2).reshape(batch, n, width), p["join"])
    y, s = ops.layer_norm(mixed, p["w2"], p["b2"], residual=x)
    return ops.linear_act(ops.linear_act(y, p["up"], p["up_b"], act="gelu"), p["down"], p["down_b"], residual=s)


def test_block_among_candidates():
    from greedy_iou_nms_gb300 import autograd as ops
    r = torch.Generator().manual_seed(3)
    batch, n, heads, width, wide = 2, 13, 2, 32, 72
    shapes = dict(w1=(width,), b1=(width,), qkv=(3 * width, width), qkv_b=(3 * width,), join=(width, width), w2=(width,),
                  b2=(width,), up=(wide, width), up_b=(wide,), down=(width, wide), down_b=(width,))
    p = {k: torch.randn(s, generator=r) / (s[-1] ** 0.5 if len(s) == 2 else 1.0) for k, s in shapes.items()}
    x, dy, table = (torch.randn(s, generator=r) for s in ((batch, n, width), (batch, n, width), (25, heads)))
    side = torch.randint(0, 9, (batch, n, 2), generator=r).to(torch.int32)
    mask = torch.arange(n)[None] < torch.tensor([[n], [n - 4]])
    buckets = g.relation_buckets(side.cuda(), side.cuda(), g.relation_lut_cells(2, 2).cuda())
    names = list(p)
    got, ref = _leaves(x, table, *p.values())
    y = _block(ops, got[0], dict(zip(names, got[2:])), side.cuda(), buckets, got[1], mask.cuda(),
               g.rotary_lut(width // heads // 4, width // heads // 4).cuda())
    y.backward(dy.cuda())
    y6 = _block(None, ref[0], dict(zip(names, ref[2:])), side, buckets.cpu(), ref[1], mask, None)
    y6.backward(dy.double())
    # Eight operators one after another, and their gradients, each within some 1e-6 of its sums (the two matrix
    # products of torch in binary32 among them).
    torch.backends.cuda.matmul.allow_tf32 = False
    _near(y, y6.detach(), 5e-5)
    for a, b in zip(got, ref):
        _near(a.grad, b.grad, 5e-5)


def test_backward_in_a_graph():
    """The gradients captured as one graph and replayed on other inputs."""
    from greedy_iou_nms_gb300 import autograd as ops
    x = torch.randn(40, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    w = (torch.randn(48, 64, device="cuda") / 8).to(torch.bfloat16).requires_grad_()
    nw = torch.ones(64, device="cuda", requires_grad=True)

    def step():
        y, s = ops.layer_norm(x, nw, residual=x)
        z = ops.linear_act(y, w, act="silu")
        return torch.autograd.grad([z, s], [x, w, nw], [torch.ones_like(z), torch.ones_like(s)])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    with torch.no_grad():
        x.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(held, step()):
        assert torch.equal(p, q)
