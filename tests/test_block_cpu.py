"""The transformer block's operators without a GPU: host-side argument checks of
the C entries, workspace sizes, the table of turns and the tensor functions'
refusals."""
import math

import pytest

import greedy_iou_nms_gb300 as g

torch = pytest.importorskip("torch")

FAKE = 1 << 20  # an aligned non-null address; never dereferenced on these paths
BIG = 1 << 60
BAD, CAP, WS = g.NMS_ERR_INVALID_ARG, g.NMS_ERR_CAPACITY, g.NMS_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    g.build()
    return g.load()


def test_layer_norm_checks():
    f = dict(x=FAKE, x_row=64, residual=FAKE, residual_row=64, type=g.NMS_TYPE_F16, rows=3, width=64, weight=FAKE,
             bias=FAKE, param_type=g.NMS_TYPE_F32, eps=1e-5, y=FAKE, sum=FAKE, mean=FAKE, rstd=FAKE, stream=0)
    b = dict(dy=FAKE, dy_row=64, x=FAKE, x_row=64, dsum=FAKE, dsum_row=64, type=g.NMS_TYPE_F16, rows=3, width=64,
             mean=FAKE, rstd=FAKE, weight=FAKE, param_type=g.NMS_TYPE_F32, dx=FAKE, dweight=FAKE, dbias=FAKE,
             workspace=FAKE, workspace_bytes=BIG, stream=0)
    for run, a in ((g.nms_layer_norm_run, f), (g.nms_layer_norm_grad_run, b)):
        for bad, code in ((dict(type=3), BAD), (dict(param_type=g.NMS_TYPE_BF16), BAD), (dict(rows=-1), BAD),
                          (dict(width=0), BAD), (dict(width=16385), CAP), (dict(rows=1 << 31), CAP), (dict(x=0), BAD),
                          (dict(x=FAKE + 1), BAD), (dict(x_row=-1), BAD), (dict(x_row=1 << 60), BAD),
                          (dict(weight=FAKE + 2), BAD), (dict(mean=FAKE + 2), BAD), (dict(rstd=FAKE + 2), BAD)):
            assert run(**dict(a, **bad)) == code, (run, bad)
    for bad in (dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(y=0), dict(sum=0), dict(residual=0),
                dict(residual=FAKE + 1), dict(sum=FAKE + 1), dict(residual_row=-1), dict(bias=FAKE + 1)):
        assert g.nms_layer_norm_run(**dict(f, **bad)) == BAD, bad
    need = g.nms_layer_norm_workspace_size(3, 64)
    for bad, code in ((dict(dy=0), BAD), (dict(dx=0), BAD), (dict(dsum=FAKE + 1), BAD), (dict(dy_row=-1), BAD),
                      (dict(dsum_row=-1), BAD), (dict(mean=0), BAD), (dict(rstd=0), BAD), (dict(dweight=FAKE + 2), BAD),
                      (dict(workspace=0), WS), (dict(workspace=FAKE + 8), WS), (dict(workspace_bytes=need // 2), WS)):
        assert g.nms_layer_norm_grad_run(**dict(b, **bad)) == code, bad
    assert g.nms_layer_norm_run(**dict(f, rows=0, x=0, y=0)) == g.NMS_OK
    for bad in ((-1, 8), (1, 0), (1, 16385), (1 << 31, 8)):
        with pytest.raises(g.NmsError):
            g.nms_layer_norm_workspace_size(*bad)


def test_linear_checks():
    f = dict(x=FAKE, x_row=64, type=g.NMS_TYPE_BF16, rows=3, inner=64, weight=FAKE, weight_row=64, outer=40, bias=FAKE,
             bias_type=g.NMS_TYPE_F32, act=g.NMS_ACT_GELU, residual=FAKE, residual_row=40, y=FAKE, pre=FAKE, dev_status=0,
             workspace=FAKE, workspace_bytes=BIG, stream=0)
    b = dict(dy=FAKE, dy_row=40, x=FAKE, x_row=64, type=g.NMS_TYPE_BF16, rows=3, inner=64, weight=FAKE, weight_row=64,
             outer=40, pre=FAKE, act=g.NMS_ACT_GELU, dx=FAKE, dweight=FAKE, dbias=FAKE, dev_status=0, workspace=FAKE,
             workspace_bytes=BIG, stream=0)
    for run, a in ((g.nms_linear_run, f), (g.nms_linear_grad_run, b)):
        for bad, code in ((dict(type=3), BAD), (dict(act=4), BAD), (dict(act=-1), BAD), (dict(rows=-1), BAD),
                          (dict(inner=0), BAD), (dict(outer=0), BAD), (dict(inner=(1 << 20) + 1), CAP),
                          (dict(outer=(1 << 20) + 1), CAP), (dict(rows=1 << 31), CAP),
                          (dict(rows=1 << 30, inner=1 << 10), CAP), (dict(inner=1 << 20, outer=1 << 20), CAP),
                          (dict(x=0), BAD), (dict(x=FAKE + 1), BAD), (dict(weight=0), BAD), (dict(weight=FAKE + 1), BAD),
                          (dict(x_row=-1), BAD), (dict(x_row=1 << 60), BAD), (dict(weight_row=-1), BAD),
                          (dict(pre=FAKE + 1), BAD), (dict(dev_status=FAKE + 2), BAD)):
            assert run(**dict(a, **bad)) == code, (run, bad)
    for bad in (dict(bias_type=g.NMS_TYPE_F16), dict(bias=FAKE + 2), dict(y=0), dict(y=FAKE + 1), dict(residual=FAKE + 1),
                dict(residual_row=-1)):
        assert g.nms_linear_run(**dict(f, **bad)) == BAD, bad
    for bad, code in ((dict(dy=0), BAD), (dict(dy=FAKE + 1), BAD), (dict(dy_row=-1), BAD), (dict(pre=0), BAD),
                      (dict(dx=FAKE + 1), BAD), (dict(dweight=FAKE + 1), BAD), (dict(dbias=FAKE + 2), BAD),
                      (dict(workspace=0), WS), (dict(workspace=FAKE + 8), WS), (dict(workspace_bytes=16), WS)):
        assert g.nms_linear_grad_run(**dict(b, **bad)) == code, bad
    assert g.nms_linear_run(**dict(f, rows=0, x=0, weight=0, y=0)) == g.NMS_OK
    for size in (g.nms_linear_workspace_size, g.nms_linear_grad_workspace_size):
        for bad in ((7, 1, 1, 1, 1), (0, -1, 1, 1, 1), (0, 1, 0, 1, 1), (0, 1, 1, 0, 1), (0, 1, 1, 1 << 21, 1)):
            with pytest.raises(g.NmsError):
                size(*bad)


def test_rotary_checks():
    a = dict(x=FAKE, x_batch=640, x_token=64, x_head=32, type=g.NMS_TYPE_F16, batch=2, tokens=10, heads=2, dim=32,
             positions=FAKE, position_type=g.NMS_POSITION_I32, sets=2, axes=2, lut=FAKE, pairs=16, halves=1, inverse=0,
             y=FAKE, y_batch=640, y_token=64, y_head=32, stream=0)
    for bad, code in ((dict(type=3), BAD), (dict(position_type=1), BAD), (dict(batch=-1), BAD), (dict(tokens=-1), BAD),
                      (dict(heads=-1), BAD), (dict(dim=0), BAD), (dict(axes=0), BAD), (dict(pairs=17), BAD),
                      (dict(pairs=-1), BAD), (dict(sets=3), BAD), (dict(sets=0), BAD), (dict(axes=9), CAP),
                      (dict(dim=4097), CAP), (dict(heads=(1 << 20) + 1), CAP), (dict(tokens=1 << 31), CAP),
                      (dict(batch=1 << 20, sets=1, tokens=1 << 20), CAP), (dict(tokens=1 << 28, heads=1 << 10), CAP),
                      (dict(x=0), BAD), (dict(y=0), BAD), (dict(x=FAKE + 1), BAD), (dict(y=FAKE + 1), BAD),
                      (dict(positions=0), BAD), (dict(positions=FAKE + 2), BAD), (dict(lut=0), BAD),
                      (dict(lut=FAKE + 4), BAD), (dict(x_batch=-1), BAD), (dict(x_token=-1), BAD), (dict(x_head=-1), BAD),
                      (dict(y_batch=-1), BAD), (dict(y_token=1 << 60), BAD), (dict(y_head=-1), BAD)):
        assert g.nms_rotary_run(**dict(a, **bad)) == code, bad
    assert g.nms_rotary_run(**dict(a, tokens=0, x=0, y=0)) == g.NMS_OK


def test_table_of_turns():
    lut = g.rotary_lut(4, 0, 2, base=100.0)
    assert lut.dtype is torch.int64 and lut.shape == (2, 6) and lut[1].tolist() == [0, 0, 0, 0, 2, 2]
    for got, j, n in zip(lut[0].tolist(), (0, 1, 2, 3, 0, 1), (4, 4, 4, 4, 2, 2)):
        assert got / 2 ** 64 == pytest.approx(100.0 ** (-j / n) / (2 * math.pi), rel=1e-15)
    # A radian a position, to the last of 64 bits: 2^64 / (2 pi) from 60 digits of pi.
    assert g.rotary_lut(1)[0].item() == 2935890503282001226
    for bad in ((), (0,), (-1, 4), (1,) * 9):
        with pytest.raises(ValueError):
            g.rotary_lut(*bad)
    for base in (0.5, math.nan, math.inf):
        with pytest.raises(ValueError):
            g.rotary_lut(4, base=base)


def _z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


X, W, HALF = _z(3, 8), _z(5, 8), _z(3, 8, dtype=torch.float16)
VEC, POS, LUT, STATS = _z(2, 4, 3, 8), _z(2, 4, 2, dtype=torch.int32), _z(2, 4, dtype=torch.int64), _z(3)


# That the operands lie on a CUDA device is the last thing to be looked at, so everything before it shows here.
@pytest.mark.parametrize("message,call", [
    ("x must be a float32", lambda: g.linear_act(_z(3, 8, dtype=torch.float64), W)),
    ("x must be a tensor", lambda: g.linear_act(None, W)),
    ("rows must be", lambda: g.linear_act(_z(), W)),
    ("weight must be a tensor", lambda: g.linear_act(X, None)),
    ("weight must be .outer, inner", lambda: g.linear_act(X, _z(5, 7))),
    ("weight must be .outer, inner", lambda: g.linear_act(X, _z(5, 8, dtype=torch.float16))),
    ("weight must be .outer, inner", lambda: g.linear_act(X, W[0])),
    ("weight must be .outer, inner", lambda: g.linear_act(X, W.to("meta"))),
    ("bias must be a contiguous", lambda: g.linear_act(X, W, _z(4))),
    ("bias must be a contiguous", lambda: g.linear_act(X, W, _z(10)[::2])),
    ("bias must be a contiguous", lambda: g.linear_act(X, W, _z(1, 5))),
    ("bias must be a contiguous", lambda: g.linear_act(HALF, W.half(), _z(5, dtype=torch.bfloat16))),
    ("act must be", lambda: g.linear_act(X, W, act="tanh")),
    ("residual must be", lambda: g.linear_act(X, W, residual=X)),
    ("residual must be", lambda: g.linear_act(X, W, residual=_z(3, 5, dtype=torch.float16))),
    ("dy must be", lambda: g.linear_act_grad(X, X, W)),
    ("dy must be", lambda: g.linear_act_grad(_z(3, 5, dtype=torch.float16), X, W)),
    ("needs the forward's pre", lambda: g.linear_act_grad(_z(3, 5), X, W, act="gelu")),
    ("pre must have", lambda: g.linear_act_grad(_z(3, 5), X, W, _z(3, 4), act="gelu")),
    ("pre must have", lambda: g.linear_act_grad(_z(3, 5), X, W, _z(3, 5, dtype=torch.float16), act="gelu")),
    ("act must be", lambda: g.linear_act_grad(_z(3, 5), X, W, act=None)),
    ("rows must be", lambda: g.layer_norm(_z())),
    ("weight must be a contiguous", lambda: g.layer_norm(X, _z(7))),
    ("bias must be a contiguous", lambda: g.layer_norm(X, _z(8), _z(8, dtype=torch.float16))),
    ("all of them alike", lambda: g.layer_norm(HALF, _z(8), _z(8, dtype=torch.float16))),
    ("residual must have", lambda: g.layer_norm(X, residual=HALF)),
    ("residual must have", lambda: g.layer_norm(X, residual=_z(1, 8))),
    ("dy must have", lambda: g.layer_norm_grad(HALF, X, STATS, STATS)),
    ("mean and rstd", lambda: g.layer_norm_grad(X, X, _z(4), STATS)),
    ("mean and rstd", lambda: g.layer_norm_grad(X, X, STATS, STATS.half())),
    ("mean and rstd", lambda: g.layer_norm_grad(X, X, STATS, _z(6)[::2])),
    ("dsum must have", lambda: g.layer_norm_grad(X, X, STATS, STATS, dsum=HALF)),
    ("x must be .batch, tokens", lambda: g.rotary(VEC[0], POS, LUT)),
    ("positions must be", lambda: g.rotary(VEC, POS.long(), LUT)),
    ("positions must be", lambda: g.rotary(VEC, POS[0], LUT)),
    ("positions must be", lambda: g.rotary(VEC, _z(3, 4, 2, dtype=torch.int32), LUT)),
    ("positions must be", lambda: g.rotary_grad(VEC, POS[:, :3], LUT)),
    ("lut must be", lambda: g.rotary(VEC, POS, LUT.int())),
    ("lut must be", lambda: g.rotary(VEC, POS, _z(2, 5, dtype=torch.int64))),
    ("lut must be", lambda: g.rotary(VEC, POS, LUT[:1])),
    ("x must be a float32, float16 or bfloat16 CUDA", lambda: g.linear_act(X, W)),
    ("x must be a float32, float16 or bfloat16 CUDA", lambda: g.linear_act_grad(_z(3, 5), X, W)),
    ("x must be a float32, float16 or bfloat16 CUDA", lambda: g.layer_norm(X, residual=X)),
    ("x must be a float32, float16 or bfloat16 CUDA", lambda: g.layer_norm_grad(X, X, STATS, STATS)),
    ("x must be a float32, float16 or bfloat16 CUDA", lambda: g.rotary(VEC, POS, LUT))])
def test_tensor_functions_refuse(message, call):
    with pytest.raises(ValueError, match=message):
        call()


def test_negated_views_are_refused():
    """A view whose memory holds the values' opposites."""
    x = torch.randn(3, 1, 2).contiguous().view(3, 2).view(torch.complex64).conj().imag  # [3, 1]
    assert x.is_neg()
    w = torch.ones(4, 1)
    for call in (lambda: g.linear_act(x, w), lambda: g.linear_act(w, w, residual=x), lambda: g.layer_norm(x),
                 lambda: g.linear_act_grad(x, x, w), lambda: g.rotary(x[:, :, None, None], x, w)):
        with pytest.raises(ValueError, match="negated view"):
            call()


def test_arguments_that_are_no_numbers():
    with pytest.raises(TypeError):
        g.layer_norm(X, eps="small")
    with pytest.raises(TypeError):
        g.linear_act_grad(_z(3, 5), X, W, need=(True, True))


def test_a_missing_binding_raises(monkeypatch):
    """No other path stands in for the C++ half."""
    from greedy_iou_nms_gb300 import _build, block
    monkeypatch.setattr(block, "_native_module", None)
    monkeypatch.setattr(_build, "BINDING_LIB", _build.BINDING_LIB + ".missing")
    with pytest.raises(RuntimeError, match="not built"):
        g.layer_norm(X)
