"""The transformer block's C entries between canaries: nothing but their outputs
and the workspace that they ask for is written, and results go over the residual
where the header allows it."""
import pytest

import greedy_iou_nms_gb300 as g

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, g.NMS_TYPE_F32), "f16": (torch.float16, g.NMS_TYPE_F16),
         "bf16": (torch.bfloat16, g.NMS_TYPE_BF16)}
PAD = 4096  # bytes of canaries on either side


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.build()
    g.load()


class Guarded:
    """A buffer of so many bytes, canaries before and behind it."""

    def __init__(self, nbytes):
        self.bytes = nbytes
        self.all = torch.full((2 * PAD + nbytes,), 0xA5, dtype=torch.uint8, device="cuda")

    @property
    def at(self):
        return self.all.data_ptr() + PAD

    def view(self, dtype, shape):
        return self.all[PAD:PAD + self.bytes].view(dtype).view(shape)

    def intact(self):
        return bool((self.all[:PAD] == 0xA5).all() and (self.all[PAD + self.bytes:] == 0xA5).all())


def _stream():
    return torch.cuda.current_stream().cuda_stream


SIZES = [(1, 24, 40), (3, 33, 7), (17, 200, 72), (64, 520, 136), (130, 127, 129), (300, 1032, 250), (2100, 64, 1003),
         (9001, 24, 40), (600, 520, 520), (9001, 72, 10), (30000, 24, 4), (1500, 202, 29)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,inner,outer", SIZES)
def test_linear(rows, inner, outer, kind):
    t, code = TYPES[kind]
    r = torch.Generator().manual_seed(rows)
    x, w, dy = (torch.randn(s, generator=r).to(t).cuda() for s in ((rows, inner), (outer, inner), (rows, outer)))
    b = torch.randn(outer, generator=r).cuda()
    e = x.element_size()
    aligned = int(inner * e % 16 == 0)
    need = g.nms_linear_workspace_size(code, rows, inner, outer, aligned)
    y, pre, ws, status = Guarded(e * rows * outer), Guarded(e * rows * outer), Guarded(need), Guarded(4)
    status.view(torch.int32, (1,)).zero_()
    over = Guarded(e * rows * outer)  # the residual, which the result replaces
    over.view(t, (rows, outer)).copy_(dy)
    for out, second, residual in ((y, pre.at, dy.data_ptr()), (over, 0, over.at)):
        st = g.nms_linear_run(x.data_ptr(), inner, code, rows, inner, w.data_ptr(), inner, outer, b.data_ptr(),
                              g.NMS_TYPE_F32, g.NMS_ACT_SILU, residual, outer, out.at, second, status.at,
                              ws.at if need else 0, need, _stream())
        assert st == g.NMS_OK
    torch.cuda.synchronize()
    ref = g.linear_act(x, w, b, act="silu", residual=dy, return_pre=True)
    assert torch.equal(y.view(t, (rows, outer)), ref[0]) and torch.equal(pre.view(t, (rows, outer)), ref[1])
    assert torch.equal(over.view(t, (rows, outer)), ref[0])
    assert status.view(torch.int32, (1,)).item() == 0
    need = g.nms_linear_grad_workspace_size(code, rows, inner, outer, int(aligned and outer * e % 16 == 0))
    dx, dw, db, gws = Guarded(e * rows * inner), Guarded(e * outer * inner), Guarded(4 * outer), Guarded(need)
    for act, z in ((g.NMS_ACT_GELU, ref[1].data_ptr()), (g.NMS_ACT_NONE, 0)):
        st = g.nms_linear_grad_run(dy.data_ptr(), outer, x.data_ptr(), inner, code, rows, inner, w.data_ptr(), inner,
                                   outer, z, act, dx.at, dw.at, db.at, status.at, gws.at, need, _stream())
        assert st == g.NMS_OK
        torch.cuda.synchronize()
        got = g.linear_act_grad(dy, x, w, ref[1], act="gelu" if z else "none")
        assert torch.equal(dx.view(t, (rows, inner)), got[0]) and torch.equal(dw.view(t, (outer, inner)), got[1])
        assert torch.equal(db.view(torch.float32, (outer,)), got[2])
    assert all(v.intact() for v in (y, pre, ws, status, over, dx, dw, db, gws))
    # A byte less of workspace is refused.
    st = g.nms_linear_grad_run(dy.data_ptr(), outer, x.data_ptr(), inner, code, rows, inner, w.data_ptr(), inner, outer, 0,
                               g.NMS_ACT_NONE, dx.at, dw.at, db.at, 0, gws.at, need - 1, _stream())
    assert st == g.NMS_ERR_WORKSPACE


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,width", [(1, 1), (5, 7), (1001, 50), (33, 100), (77, 256), (300, 999), (40, 2050), (9, 5001),
                                        (3, 12345), (2, 16384)])
def test_layer_norm(rows, width, kind):
    t, code = TYPES[kind]
    r = torch.Generator().manual_seed(width)
    x, more, dy = (torch.randn(rows, width, generator=r).to(t).cuda() for _ in range(3))
    w = torch.randn(width, generator=r).cuda()
    n = x.element_size() * rows * width
    y, total, mean, rstd = Guarded(n), Guarded(n), Guarded(4 * rows), Guarded(4 * rows)
    st = g.nms_layer_norm_run(x.data_ptr(), width, more.data_ptr(), width, code, rows, width, w.data_ptr(), 0,
                              g.NMS_TYPE_F32, 1e-5, y.at, total.at, mean.at, rstd.at, _stream())
    need = g.nms_layer_norm_workspace_size(rows, width)
    dx, dw, db, ws = Guarded(n), Guarded(4 * width), Guarded(4 * width), Guarded(need)
    st |= g.nms_layer_norm_grad_run(dy.data_ptr(), width, total.at, width, more.data_ptr(), width, code, rows, width,
                                    mean.at, rstd.at, w.data_ptr(), g.NMS_TYPE_F32, dx.at, dw.at, db.at, ws.at, need,
                                    _stream())
    torch.cuda.synchronize()
    assert st == g.NMS_OK and all(v.intact() for v in (y, total, mean, rstd, dx, dw, db, ws))
    ref = g.layer_norm(x, w, residual=more, return_stats=True)
    assert torch.equal(y.view(t, x.shape), ref[0]) and torch.equal(total.view(t, x.shape), ref[1])
    got = g.layer_norm_grad(dy, ref[1], ref[2], ref[3], w, dsum=more)
    assert torch.equal(dx.view(t, x.shape), got[0]) and torch.equal(dw.view(torch.float32, (width,)), got[1])
    assert torch.equal(db.view(torch.float32, (width,)), got[2])


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,pairs", [((1, 1, 1, 2), 1), ((2, 19, 3, 64), 32), ((3, 7, 5, 43), 20), ((1, 100, 9, 80), 8),
                                         ((2, 3, 300, 16), 8)])
def test_rotary(shape, pairs, kind):
    t, code = TYPES[kind]
    r = torch.Generator().manual_seed(pairs)
    x = torch.randn(shape, generator=r).to(t).cuda()
    p = torch.randint(0, 1000, (shape[0], shape[1], 1), generator=r).to(torch.int32).cuda()
    lut = g.rotary_lut(pairs).cuda()
    s = x.stride()
    for halves in (1, 0):
        y = Guarded(x.element_size() * x.numel())
        st = g.nms_rotary_run(x.data_ptr(), *s[:3], code, *shape, p.data_ptr(), g.NMS_POSITION_I32, shape[0], 1,
                              lut.data_ptr(), pairs, halves, 0, y.at, *s[:3], _stream())
        torch.cuda.synchronize()
        assert st == g.NMS_OK and y.intact()
        assert torch.equal(y.view(t, shape), g.rotary(x, p, lut, halves=bool(halves)))
