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


class Beside(torch.Tensor):
    """A CPU tensor that says it lies on the second CUDA device."""
    is_cuda = True

    def get_device(self):
        return 1


def _on(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Beside)


def test_tensor_functions_refuse():
    cpu = torch.randn(3, 8)
    x, w, half = _on(3, 8), _on(5, 8), _on(3, 8, dtype=torch.float16)
    vec, pos, lut = _on(2, 4, 3, 8), _on(2, 4, 2, dtype=torch.int32), _on(2, 4, dtype=torch.int64)
    stats = _on(3)
    for call in (lambda: g.linear_act(cpu, cpu), lambda: g.linear_act(_on(3, 8, dtype=torch.float64), w),
                 lambda: g.linear_act(x, _on(5, 7)), lambda: g.linear_act(x, _on(5, 8, dtype=torch.float16)),
                 lambda: g.linear_act(x, w[0]), lambda: g.linear_act(x, torch.zeros(5, 8)), lambda: g.linear_act(x, w, _on(4)),
                 lambda: g.linear_act(x, w, _on(10)[::2]), lambda: g.linear_act(half, half, _on(3, dtype=torch.bfloat16)),
                 lambda: g.linear_act(x, w, act="tanh"), lambda: g.linear_act(x, w, residual=x),
                 lambda: g.linear_act(x, w, residual=_on(3, 5, dtype=torch.float16)), lambda: g.linear_act(_on(), w),
                 lambda: g.linear_act_grad(x, x, w), lambda: g.linear_act_grad(_on(3, 5), x, w, act="gelu"),
                 lambda: g.linear_act_grad(_on(3, 5), x, w, _on(3, 4), act="gelu"),
                 lambda: g.linear_act_grad(_on(3, 5, dtype=torch.float16), x, w),
                 lambda: g.layer_norm(cpu), lambda: g.layer_norm(x, _on(7)), lambda: g.layer_norm(x, residual=half),
                 lambda: g.layer_norm(x, residual=cpu), lambda: g.layer_norm(_on()),
                 lambda: g.layer_norm_grad(half, x, stats, stats), lambda: g.layer_norm_grad(x, x, _on(4), stats),
                 lambda: g.layer_norm_grad(x, x, stats, _on(3, dtype=torch.float16)),
                 lambda: g.layer_norm_grad(x, x, stats, stats, dsum=half),
                 lambda: g.rotary(vec[0], pos, lut), lambda: g.rotary(vec, pos.long(), lut), lambda: g.rotary(vec, pos[0], lut),
                 lambda: g.rotary(vec, _on(3, 4, 2, dtype=torch.int32), lut), lambda: g.rotary(vec, pos, lut.int()),
                 lambda: g.rotary(vec, pos, _on(2, 5, dtype=torch.int64)), lambda: g.rotary(vec, pos, lut[:1]),
                 lambda: g.rotary(vec, torch.zeros(2, 4, 2, dtype=torch.int32), lut),
                 lambda: g.rotary(torch.zeros(2, 4, 3, 8), pos, lut)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("current", [0, 1])
def test_launches_go_to_the_tensors_device(lib, monkeypatch, current):
    """Another device being current, each tensor function makes its operands'
    device current for the launch and hands over that device's stream."""
    from greedy_iou_nms_gb300 import head
    head._torch()
    now, calls = [current], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    class Recorder:
        def __getattr__(self, name):
            if not name.endswith("_run"):
                return getattr(lib, name)
            return lambda *args: calls.append((name, now[0], args[-1])) or 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(head, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(head, "_loaded", Recorder())
    x, w = _on(3, 8), _on(5, 8)
    g.linear_act(x, w)
    g.linear_act_grad(_on(3, 5), x, w)
    g.layer_norm(x)
    g.layer_norm_grad(x, x, _on(3), _on(3))
    g.rotary(_on(2, 4, 3, 8), _on(2, 4, 1, dtype=torch.int32), _on(2, 4, dtype=torch.int64))
    g.rotary_grad(_on(2, 4, 3, 8), _on(2, 4, 1, dtype=torch.int32), _on(2, 4, dtype=torch.int64))
    assert [c[0] for c in calls] == ["nms_linear_run", "nms_linear_grad_run", "nms_layer_norm_run",
                                     "nms_layer_norm_grad_run", "nms_rotary_run", "nms_rotary_run"]
    assert all(at == 1 and stream == 1001 for _, at, stream in calls) and now[0] == current
