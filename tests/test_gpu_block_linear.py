"""The linear layer and its gradient against 64 bits."""
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


def _inputs(rows, inner, outer, kind, seed=0):
    r = torch.Generator().manual_seed(seed)
    t = R.TYPES[kind]
    x = torch.randn(rows, inner, generator=r).to(t)
    w = (torch.randn(outer, inner, generator=r) / inner ** 0.5).to(t)
    return x, w, 0.3 * torch.randn(outer, generator=r), torch.randn(rows, outer, generator=r).to(t)


def _same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def _check(got, ref, bound):
    assert got.shape == ref.shape
    smallest = 2.0 ** -25 if got.dtype is torch.float16 else 0.0
    bound = bound + (R.half_step(got.dtype) + 2 * R.U) * (ref.abs() + bound) + smallest
    over = (got.cpu().double() - ref).abs() - bound
    assert (over <= 0).all(), float(over.max())


def _forward(x, w, b, act, res, train=True):
    out = g.linear_act(x.cuda(), w.cuda(), None if b is None else b.cuda(), act=act,
                       residual=None if res is None else res.cuda(), return_pre=train)
    y, z = R.linear(x, w, b, act, res)
    near = R.product_bound(x, w.T, x.dtype) + 2 * R.U * z.abs()
    if train:
        _check(out[1], z, near)
    got = out[0] if train else out
    # No activation is steeper than 1.13.
    sum_error = 0 if act == "none" else R.act_error(x.dtype) * (z.abs() + 1) * (1 if act != "relu" else 0)
    _check(got, y, 1.13 * near + sum_error + R.U * (0 if res is None else res.double().abs()))


def _backward(x, w, z, dy, act, seed=0):
    t = x.dtype
    pre = None if act == "none" else z.to(t)
    out = g.linear_act_grad(dy.cuda(), x.cuda(), w.cuda(), None if pre is None else pre.cuda(), act=act)
    slope = torch.ones_like(dy, dtype=torch.float64) if pre is None else R.slope(pre.double(), act)
    dz = dy.double() * slope
    off = torch.zeros_like(dz)
    if act in ("silu", "gelu"):
        off = R.act_error(t) * dy.double().abs()
    rounded = off if act == "none" else off + (R.half_step(t) + 2 * R.U) * dz.abs()  # the products take dz rounded
    if t is torch.float16 and act != "none":
        rounded = rounded + 2.0 ** -25
    _check(out[0], dz @ w.double(), R.product_bound(dz, w, t) + rounded @ w.double().abs())
    _check(out[1], dz.T @ x.double(), R.product_bound(dz.T, x, t) + rounded.T @ x.double().abs())
    # A warp adds 256 rows, its block's and the runs' sums follow; the derivative's own roundings beside them.
    assert out[2].dtype is torch.float32
    assert ((out[2].cpu().double() - dz.sum(0)).abs() <= 300 * R.U * dz.abs().sum(0) + off.sum(0) + 1e-30).all()


SIZES = [(1, 1, 1), (1, 8, 8), (3, 5, 7), (16, 64, 128), (17, 72, 200), (5, 513, 33), (130, 127, 129), (128, 128, 256),
         (300, 256, 1024), (257, 264, 520), (64, 1000, 40), (1, 4096, 1000), (2, 48, 4096), (2000, 40, 24),
         (1000, 136, 8), (9000, 24, 40), (400, 600, 603), (70, 1030, 64), (20, 24, 1100)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,inner,outer", SIZES)
def test_forward(rows, inner, outer, kind):
    x, w, b, res = _inputs(rows, inner, outer, kind, rows + inner + outer)
    for act, bias, more, train in (("none", b, None, False), ("gelu", b, res, True), ("silu", None, res, False),
                                   ("relu", b.to(x.dtype), None, True), ("none", None, res, False)):
        _forward(x, w, bias, act, more, train)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,inner,outer", SIZES)
def test_gradient(rows, inner, outer, kind):
    x, w, b, dy = _inputs(rows, inner, outer, kind, rows + inner + outer + 1)
    z = R.linear(x, w, b, "none")[1]
    for act in ("none", "relu", "silu", "gelu"):
        _backward(x, w, z, dy, act)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_larger(kind):
    """Several tiles to an SM, a long sum for the weight's gradient."""
    x, w, b, res = _inputs(2600, 520, 1544, kind, 7)
    _forward(x, w, b, "gelu", res)
    _backward(x, w, R.linear(x, w, b, "none")[1], res, "silu")
    x, w, b, res = _inputs(20000, 64, 72, kind, 8)
    _forward(x, w, b, "none", res)
    _backward(x, w, R.linear(x, w, b, "none")[1], res, "none")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,inner,outer", [(20011, 333, 10), (9000, 64, 16), (1500, 2500, 4), (40000, 72, 1),
                                              (5000, 31, 13), (8200, 29, 17), (3000, 1200, 6), (1023, 4, 2),
                                              (140001, 6, 32), (700, 402, 33), (2000, 2050, 25)])
def test_gradient_of_few_outputs(rows, inner, outer, kind):
    """Weights of a few rows: a stream of x."""
    x, w, b, dy = _inputs(rows, inner, outer, kind, rows)
    z = R.linear(x, w, b, "none")[1]
    for act in ("none", "gelu"):
        _backward(x, w, z, dy, act)


def test_gradient_by_parts_of_rows_with_gaps():
    """dz goes to the tensor cores' parts straight from dy: rows that lie apart, start anywhere, or are one row."""
    rows, inner, outer = 900, 300, 523
    x, w, b, _ = (v.cuda() for v in _inputs(rows, inner, outer, "f32", 21))
    wide = torch.randn(rows, outer + 14, generator=torch.Generator().manual_seed(22)).cuda()
    z = g.linear_act(x, w, b)
    for dy in (wide[:, 3:3 + outer], wide[:, :outer], wide[5:6, :outer].expand(rows, outer)):
        for act in ("none", "silu"):
            for need in ((True, True, True), (True, False, False), (False, True, True), (False, False, True)):
                got = g.linear_act_grad(dy, x, w, z, act=act, need=need)
                ref = g.linear_act_grad(dy.contiguous(), x, w, z, act=act)
                for p, q, wanted in zip(got, ref, need):
                    # The columns' sums are taken in another order where a thread has another number of columns.
                    assert p is None if not wanted else \
                        torch.equal(p, q) if p.dim() > 1 else torch.allclose(p, q, rtol=0, atol=1e-3)


def test_whole_numbers_are_exact():
    """Small whole numbers have exact products and sums in every type, whatever the order."""
    r = torch.Generator().manual_seed(3)
    for kind in ("f32", "f16", "bf16"):
        for rows, inner, outer in ((1, 100, 40), (200, 136, 264), (513, 24, 1000)):
            x, w, dy = (torch.randint(-1, 2, s, generator=r).to(R.TYPES[kind])
                        for s in ((rows, inner), (outer, inner), (rows, outer)))
            y = g.linear_act(x.cuda(), w.cuda())
            assert torch.equal(y.cpu().double(), (x.double() @ w.double().T).to(x.dtype).double())
            dx, dw, db = g.linear_act_grad(dy.cuda(), x.cuda(), w.cuda())
            assert torch.equal(dx.cpu().double(), (dy.double() @ w.double()).to(x.dtype).double())
            assert torch.equal(dw.cpu().double(), (dy.double().T @ x.double()).to(x.dtype).double())
            assert torch.equal(db.cpu().double(), dy.double().sum(0))


def test_gradient_against_differences():
    x, w, b, dy = _inputs(6, 20, 9, "f32", 4)
    z = R.linear(x, w, b, "none")[1]
    for act in ("silu", "gelu"):
        dx, dw, db = (v.cpu().double() for v in
                      g.linear_act_grad(dy.cuda(), x.cuda(), w.cuda(), z.float().cuda(), act=act))

        def loss(x, w, b):
            return float((R.linear(x, w, b, act)[0] * dy).sum())

        h = 1e-5
        for grad, at in ((dx, 0), (dw, 1), (db, 2)):
            v = [x.double(), w.double(), b.double()]
            for i in (0, grad.numel() // 2, grad.numel() - 1):
                step = torch.zeros(grad.numel(), dtype=torch.float64)
                step[i] = h
                up, down = ([q + s * step.view(q.shape) if k == at else q for k, q in enumerate(v)] for s in (1, -1))
                assert abs((loss(*up) - loss(*down)) / (2 * h) - float(grad.view(-1)[i])) < 2e-5


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_strides_and_starts(kind):
    """Slices of wider tensors, odd starts and rows, repeated rows, leading axes."""
    r = torch.Generator().manual_seed(5)
    t = R.TYPES[kind]
    wide = torch.randn(4, 30, 96, generator=r).to(t).cuda()
    table = torch.randn(50, 96, generator=r).to(t).cuda()
    res = torch.randn(4, 30, 100, generator=r).to(t).cuda()
    for x, w in ((wide[..., 32:64], table[:, 32:64]), (wide[..., 3:35], table[:, 1:33]), (wide[:, ::2, :32], table[:40, :32]),
                 (wide[..., :31], table[:, :31]), (wide[:1, :, :32].expand(4, 30, 32), table[::2, :32]),
                 (wide[0, 0, :32], table[:, :32]), (wide.transpose(1, 2)[..., :24], torch.randn(24, 50, generator=r).to(t).cuda().T)):
        y = g.linear_act(x, w)
        assert y.shape == (*x.shape[:-1], w.shape[0])
        assert _same([y], [g.linear_act(x.contiguous(), w.contiguous())])
        got = g.linear_act_grad(y, x, w, y, act="silu")
        ref = g.linear_act_grad(y, x.contiguous(), w.contiguous(), y, act="silu")
        assert _same(got, ref)
    x, w = wide[..., :32], table[:, :32]
    part = res[..., 7:57]
    assert _same([g.linear_act(x, w, residual=part)], [g.linear_act(x, w, residual=part.contiguous())])
    got, ref = g.linear_act_grad(part, x, w), g.linear_act_grad(part.contiguous(), x, w)
    assert _same(got, ref)
    spread = res[:1, :1, :50].expand(4, 30, 50)
    got, ref = g.linear_act_grad(spread, x, w), g.linear_act_grad(spread.contiguous(), x, w)
    assert _same(got, ref)


def test_only_what_is_needed():
    x, w, b, dy = (v.cuda() for v in _inputs(70, 40, 56, "bf16", 6))
    whole = g.linear_act_grad(dy, x, w)
    for need in ((True, False, False), (False, True, False), (False, False, True), (True, False, True),
                 (False, False, False)):
        for got, ref, wanted in zip(g.linear_act_grad(dy, x, w, need=need), whole, need):
            assert torch.equal(got, ref) if wanted else got is None


def test_far_apart_sizes():
    """Binary32 operands whose parts differ by many powers of two, and whose results nearly cancel."""
    r = torch.Generator().manual_seed(12)
    for rows, inner, outer in ((40, 64, 48), (300, 520, 520)):
        x = torch.randn(rows, inner, generator=r) * 2.0 ** torch.randint(-30, 30, (rows, 1), generator=r)
        w = torch.randn(outer, inner, generator=r) * 2.0 ** torch.randint(-30, 30, (outer, 1), generator=r)
        x[:, 1::2] = -x[:, ::2] * (1 + 2.0 ** -12 * torch.randn(rows, inner // 2, generator=r))
        w[:, 1::2] = w[:, ::2]
        y = g.linear_act(x.cuda(), w.cuda())
        _check(y, x.double() @ w.double().T, R.product_bound(x, w.T, torch.float32))
    x = torch.full((300, 520), 3.4e38)  # rounds to an infinity in 8 bits
    y = g.linear_act(x.cuda(), torch.eye(520).mul(0.5).cuda())
    assert torch.equal(y.cpu(), x / 2)


def test_no_rows():
    for kind in ("f32", "f16"):
        x, w, dy = (torch.empty(s, dtype=R.TYPES[kind], device="cuda") for s in ((2, 0, 24), (40, 24), (2, 0, 40)))
        assert g.linear_act(x, w).shape == (2, 0, 40)
        dx, dw, db = g.linear_act_grad(dy, x, w, dy, act="gelu")
        assert dx.shape == x.shape and float(dw.abs().sum()) == 0 and float(db.abs().sum()) == 0


def test_not_finite_stays_in_its_rows():
    for kind in ("f32", "bf16"):
        for rows, outer in ((3, 136), (200, 136), (600, 1600)):  # the last one: binary32 on the tensor cores too
            x, w, b, dy = (v.cuda() for v in _inputs(rows, 72, outer, kind, 9))
            x[1, 5] = float("nan")
            x[rows - 1, 71] = float("inf")
            y = g.linear_act(x, w, b, act="silu")
            clean = [r for r in range(rows) if r not in (1, rows - 1)]
            assert torch.isfinite(y[clean]).all() and torch.isnan(y[1]).all()
            assert not torch.isfinite(g.linear_act(x, w, b)[rows - 1]).any()


def test_same_bits_graph_and_streams():
    x, w, b, res = (v.cuda() for v in _inputs(700, 200, 328, "bf16", 10))

    def both():
        y, pre = g.linear_act(x, w, b, act="gelu", residual=res, return_pre=True)
        return (y, pre, *g.linear_act_grad(y, x, w, pre, act="gelu"))

    first = both()
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(both())
    for s in sides:
        s.synchronize()
    for out in outs:
        assert _same(first, out)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    held = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            held.append(both())
    x.copy_(x.flip(0))
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    again = both()
    for out in held:
        assert _same(again, out)
