"""Layer normalisation and its gradient against 64 bits."""
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


def _inputs(rows, width, kind, residual, seed=0):
    r = torch.Generator().manual_seed(seed)
    t = R.TYPES[kind]
    x = (torch.randn(rows, width, generator=r) * (0.5 + torch.randn(width, generator=r).abs())
         + torch.randn(width, generator=r)).to(t)
    w, b = 1 + 0.2 * torch.randn(width, generator=r), 0.2 * torch.randn(width, generator=r)
    more = torch.randn(rows, width, generator=r).to(t) if residual else None
    return x, w, b, more, torch.randn(rows, width, generator=r).to(t)


def _check_forward(x, w, b, more, eps=1e-5):
    t, n = x.dtype, x.shape[-1]
    out = g.layer_norm(x.cuda(), *(None if v is None else v.cuda() for v in (w, b)), eps=eps,
                       residual=None if more is None else more.cuda(), return_stats=True)
    y, s, mean, rstd = R.layer(x, w, b, eps, more)
    got = [v.cpu().double() for v in out]
    if more is not None:
        assert torch.equal(out[1].cpu(), s)
    # A thread adds up to 32 values, its team's sums follow in 9 to 21 additions: the mean of the deviations, which
    # corrects the first mean, is off by 32 roundings of their average size, their squares' sum by 56 of itself.
    d = (s.double() - mean[..., None]).abs()
    assert ((got[-2] - mean).abs() <= 2 * R.U * mean.abs() + 32 * R.U * d.mean(-1)).all()
    assert ((got[-1] - rstd).abs() <= 64 * R.U * rstd).all()
    u = d * rstd[..., None]
    bound = R.U * (70 * u + 32) * (1 if w is None else w.double().abs())
    bound = bound + (2 * R.U + R.half_step(t)) * (y.abs() + bound)
    if t is torch.float16:
        bound = bound + 2.0 ** -25  # half a step of its smallest numbers
    assert ((got[0] - y).abs() <= bound).all()


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,width", [(1, 1), (1, 8), (3, 7), (5, 33), (300, 256), (17, 264), (9, 512), (4, 1000),
                                        (4, 1024), (3, 1025), (3, 2048), (2, 2056), (2, 4096), (2, 4104), (2, 8192),
                                        (1, 16383), (2, 16384), (3, 50), (2, 8986), (1003, 8), (37, 64), (66, 63), (33, 10), (35, 65), (21, 128)])
@pytest.mark.parametrize("residual", [False, True])
def test_forward(rows, width, kind, residual):
    x, w, b, more, _ = _inputs(rows, width, kind, residual, rows + width)
    _check_forward(x, w, b, more)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,width", [(1, 8), (3, 7), (5, 33), (301, 256), (700, 264), (2000, 12), (4, 1000),
                                        (1300, 1024), (3, 1025), (2, 2056), (700, 4096), (2, 4104), (2, 16384), (300, 50), (5, 8186), (5, 8986), (3, 12345), (20003, 8), (37, 64), (66, 63), (33, 10), (1, 64), (35, 65), (21, 128), (9999, 100)])
@pytest.mark.parametrize("more", [False, True])
def test_gradient(rows, width, kind, more):
    x, w, _, dsum, dy = _inputs(rows, width, kind, more, rows * width)
    _, _, mean, rstd = R.layer(x, None, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    out = g.layer_norm_grad(dy.cuda(), x.cuda(), mean.cuda(), rstd.cuda(), w.cuda(),
                            dsum=None if dsum is None else dsum.cuda())
    dx, dw, db = R.layer_grad(dy, x, mean, rstd, w, dsum)
    u = ((x.double() - mean.double()[:, None]) * rstd.double()[:, None]).abs()
    du = dy.double().abs() * w.double().abs()
    near = 4 * R.U * (x.double().abs() * rstd.double()[:, None]).abs()  # of u: the difference's own rounding
    size = du + du.mean(1, keepdim=True) + u * (du * u).mean(1, keepdim=True)
    bound = rstd.double()[:, None] * (64 * R.U * size + near * (du * u).mean(1, keepdim=True)
                                      + u * (du * near).mean(1, keepdim=True))
    bound = bound + (R.half_step(x.dtype) + 4 * R.U) * (dx.abs() + (0 if dsum is None else dsum.double().abs()))
    assert ((out[0].cpu().double() - dx).abs() <= bound + 2.0 ** -25).all()
    # A team adds up to 256 rows, its block and the blocks' join follow.
    terms = (dy.double().abs() * u).sum(0)
    assert ((out[1].cpu().double() - dw).abs() <= 300 * R.U * terms + (dy.double().abs() * near).sum(0) + 1e-30).all()
    assert ((out[2].cpu().double() - db).abs() <= 300 * R.U * dy.double().abs().sum(0) + 1e-30).all()


def test_gradient_against_differences():
    r = torch.Generator().manual_seed(2)
    x, dy, w = (torch.randn(s, generator=r) for s in ((3, 24), (3, 24), (24,)))
    y, _, mean, rstd = R.layer(x, w, None, 1e-5)
    dx = g.layer_norm_grad(dy.cuda(), x.cuda(), mean.float().cuda(), rstd.float().cuda(), w.cuda())[0].cpu().double()
    h = 1e-5
    for i, j in ((0, 0), (1, 7), (2, 23)):
        step = torch.zeros_like(x, dtype=torch.float64)
        step[i, j] = h
        up, down = (R.layer(x.double() + s, w, None, 1e-5)[0] for s in (step, -step))
        # A central difference is off by h^2 / 6 third derivatives; the kernel by binary32.
        assert abs(float(((up - down) * dy).sum() / (2 * h) - dx[i, j])) < 1e-5


def test_mean_far_from_zero():
    """2000 spreads off zero: what binary32 keeps of the rows decides, not the moments."""
    r = torch.Generator().manual_seed(3)
    for width in (40, 1024, 5000):
        x = (100 + 0.05 * torch.randn(6, width, generator=r))
        _, mean, rstd = (v.cpu().double() for v in g.layer_norm(x.cuda(), eps=0.0, return_stats=True))
        ref = R.layer(x, None, None, 0.0)
        assert ((rstd - ref[3]).abs() <= 64 * R.U * ref[3]).all()
        assert ((mean - ref[2]).abs() <= 2 * R.U * ref[2].abs()).all()


def _same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_strides_and_shapes():
    """A slice of wider rows, repeated rows, leading axes."""
    r = torch.Generator().manual_seed(4)
    wide = torch.randn(4, 6, 96, generator=r).cuda()
    w = torch.randn(32, generator=r).cuda()
    for x in (wide[..., 32:64], wide[:, ::2, :32], wide[:, :1, :32].expand(4, 6, 32), wide[:1, :1, :32].expand(4, 6, 32),
              wide.transpose(0, 1)[..., :32], wide[0, 0, :32]):
        c = x.contiguous()
        y = g.layer_norm(x, w)
        assert y.shape == x.shape and _same([y], [g.layer_norm(c, w)])
        mean, rstd = g.layer_norm(x, return_stats=True)[1:]
        assert _same(g.layer_norm_grad(x, x, mean, rstd, w, dsum=x), g.layer_norm_grad(c, c, mean, rstd, w, dsum=c))


def test_rows_that_start_at_an_odd_element():
    """They move element by element, other threads hold them and the sums take
    another order: as near to 64 bits as any."""
    r = torch.Generator().manual_seed(4)
    wide, w, b = torch.randn(7, 96, generator=r), torch.randn(32, generator=r), torch.randn(32, generator=r)
    for kind in ("f32", "bf16"):
        x = wide.to(R.TYPES[kind])
        y, _, mean, rstd = R.layer(x[:, 3:35], w, b, 1e-5)
        got = g.layer_norm(x.cuda()[:, 3:35], w.cuda(), b.cuda()).cpu().double()
        u = ((x[:, 3:35].double() - mean[:, None]) * rstd[:, None]).abs()
        bound = R.U * (70 * u + 32) * w.double().abs()
        assert ((got - y).abs() <= bound + (2 * R.U + R.half_step(x.dtype)) * (y.abs() + bound)).all()


def test_parameters():
    r = torch.Generator().manual_seed(5)
    x = torch.randn(3, 48, generator=r).to(torch.bfloat16)
    w, b = torch.randn(48, generator=r).to(torch.bfloat16), torch.randn(48, generator=r).to(torch.bfloat16)
    for ww, bb in ((None, None), (w, None), (None, b), (w, b), (w.float(), b.float())):
        _check_forward(x, ww, bb, None)
    # Parameters that start at an odd element.
    wide = torch.randn(49, generator=r).cuda()
    assert torch.equal(g.layer_norm(x.cuda(), wide[1:]), g.layer_norm(x.cuda(), wide[1:].clone()))


def test_empty_and_not_finite():
    for shape in ((0, 16), (2, 0, 16)):
        x = torch.empty(shape, device="cuda")
        y, s, mean, rstd = g.layer_norm(x, residual=x, return_stats=True)
        assert y.shape == x.shape and mean.shape == x.shape[:-1]
        dx, dw, db = g.layer_norm_grad(x, x, mean, rstd)
        assert dx.shape == x.shape and float(dw.abs().sum() + db.abs().sum()) == 0
    for width in (16, 2000):
        x = torch.randn(4, width, device="cuda")
        x[1, 3], x[2, 5] = float("inf"), float("nan")
        y, mean, rstd = g.layer_norm(x, return_stats=True)
        assert torch.isfinite(y[[0, 3]]).all() and torch.isnan(y[[1, 2]]).all()
        assert torch.isfinite(rstd[[0, 3]]).all() and torch.isnan(rstd[[1, 2]]).all() and torch.isnan(mean[2])
        assert torch.equal(y[[0, 3]], g.layer_norm(x[[0, 3]]))


def test_same_bits_graph_and_stream():
    x, w, b, more, dy = (v.cuda() for v in _inputs(999, 320, "bf16", True, 6))

    def both():
        y, s, mean, rstd = g.layer_norm(x, w, b, residual=more, return_stats=True)
        return (y, s, mean, rstd, *g.layer_norm_grad(dy, s, mean, rstd, w, dsum=more))

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = both()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = both()
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(third[0], both()[0]) and torch.equal(third[5], both()[5])


def test_sum_in_place():
    """The C entry's sum may be the residual itself."""
    x, w, _, more, _ = (None if v is None else v.cuda() for v in _inputs(50, 200, "f16", True, 7))
    y, total = g.layer_norm(x, w, residual=more)
    out, stream = torch.empty_like(y), more.clone()
    st = g.nms_layer_norm_run(x.data_ptr(), 200, stream.data_ptr(), 200, g.NMS_TYPE_F16, 50, 200, w.data_ptr(), 0,
                              g.NMS_TYPE_F32, 1e-5, out.data_ptr(), stream.data_ptr(), 0, 0,
                              torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == g.NMS_OK and torch.equal(out, y) and torch.equal(stream, total)
