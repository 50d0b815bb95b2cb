"""The detection-head operators without a GPU: the generator's published
vectors (of the tests' own restatement), host-side argument checks of the C
entries, workspace sizes and the position tables."""
import math

import pytest

import greedy_iou_nms_gb300 as g

torch = pytest.importorskip("torch")
import head_reference as R  # noqa: E402

FAKE = 1 << 20  # an aligned non-null address; never dereferenced on these paths
BIG = 1 << 40
BAD, CAP, WS = g.NMS_ERR_INVALID_ARG, g.NMS_ERR_CAPACITY, g.NMS_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    g.build()
    return g.load()


def test_philox_vectors():
    """Philox 4x32-10 known answers for all-zero and all-one counter and key."""
    assert R.philox(0, 0, 0) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    ones = (1 << 64) - 1
    assert R.philox(ones, ones, ones) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]


def test_dropout_checks():
    a = dict(x=FAKE, residual=0, type=g.NMS_TYPE_BF16, n=10, drop_p=0.5, seed=1, offset=0, y=FAKE, stream=0)
    for bad, code in ((dict(type=3), BAD), (dict(type=-1), BAD), (dict(n=-1), BAD), (dict(drop_p=-0.01), BAD),
                      (dict(drop_p=1.01), BAD), (dict(drop_p=math.nan), BAD), (dict(x=0), BAD), (dict(y=0), BAD),
                      (dict(x=FAKE + 1), BAD), (dict(y=FAKE + 1), BAD), (dict(residual=FAKE + 1), BAD),
                      (dict(type=g.NMS_TYPE_F32, x=FAKE + 2), BAD), (dict(n=(1 << 47) + 1), CAP)):
        assert g.nms_dropout_run(**dict(a, **bad)) == code, bad
    assert g.nms_dropout_run(**dict(a, n=0, x=0, y=0)) == g.NMS_OK


def _norm(**kw):
    a = dict(x=FAKE, x_image=640, x_pixel=64, type=g.NMS_TYPE_F32, batch=2, pixels=10, channels=64, groups=8,
             weight=0, bias=0, param_type=g.NMS_TYPE_F32, eps=1e-5, act=g.NMS_ACT_SILU, drop_p=0.0, seed=0, offset=0,
             y=FAKE, mean=FAKE, rstd=FAKE, workspace=FAKE, workspace_bytes=BIG, stream=0)
    a.update(kw)
    return g.nms_group_norm_run(**a)


def _norm_grad(**kw):
    a = dict(dy=FAKE, dy_image=640, dy_pixel=64, x=FAKE, x_image=640, x_pixel=64, type=g.NMS_TYPE_F32, batch=2,
             pixels=10, channels=64, groups=8, mean=FAKE, rstd=FAKE, weight=0, bias=0, param_type=g.NMS_TYPE_F32,
             act=g.NMS_ACT_SILU, drop_p=0.0, seed=0, offset=0, dx=FAKE, dweight=FAKE, dbias=FAKE, workspace=FAKE,
             workspace_bytes=BIG, stream=0)
    a.update(kw)
    return g.nms_group_norm_grad_run(**a)


def test_norm_checks():
    shared = ((dict(type=7), BAD), (dict(param_type=g.NMS_TYPE_F16), BAD), (dict(act=4), BAD), (dict(act=-1), BAD),
              (dict(drop_p=2.0), BAD), (dict(batch=-1), BAD), (dict(pixels=-1), BAD), (dict(channels=0), BAD),
              (dict(groups=0), BAD), (dict(groups=7), BAD), (dict(x_pixel=63), BAD), (dict(x_pixel=-64), BAD),
              (dict(x_image=-1), BAD), (dict(x=0), BAD), (dict(x=FAKE + 2), BAD), (dict(weight=FAKE + 2), BAD),
              (dict(mean=FAKE + 2), BAD), (dict(workspace=0), WS), (dict(workspace=FAKE + 8), WS),
              (dict(workspace_bytes=g.nms_group_norm_workspace_size(2, 10, 64, 8) - 1), WS),
              (dict(channels=16392, x_pixel=16392), CAP), (dict(batch=(1 << 20) + 1), CAP),
              (dict(pixels=(1 << 28) + 1), CAP), (dict(x_image=1 << 60), BAD), (dict(x_pixel=1 << 60), BAD),
              (dict(batch=1 << 20, channels=16384, groups=4096, x_pixel=16384), CAP))
    for run in (_norm, _norm_grad):
        for bad, code in shared:
            assert run(**bad) == code, (run, bad)
    for bad, code in ((dict(y=0), BAD), (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD), (dict(eps=math.inf), BAD)):
        assert _norm(**bad) == code, bad
    for bad, code in ((dict(dx=0), BAD), (dict(dy=0), BAD), (dict(mean=0), BAD), (dict(rstd=0), BAD),
                      (dict(dy_pixel=1), BAD), (dict(dweight=FAKE + 2), BAD)):
        assert _norm_grad(**bad) == code, bad
    assert _norm(batch=0, x=0, y=0, workspace=0) == g.NMS_OK
    with pytest.raises(g.NmsError):
        g.nms_group_norm_workspace_size(1, 1, 10, 3)


def test_relation_checks():
    f = dict(scores=FAKE, type=g.NMS_TYPE_F16, batch=2, heads=3, queries=4, keys=5, buckets=FAKE, sets=2, table=FAKE,
             num_buckets=6, key_mask=0, scale=1.0, probs=FAKE, stream=0)
    b = dict(dprobs=FAKE, probs=FAKE, type=g.NMS_TYPE_F16, batch=2, heads=3, queries=4, keys=5, buckets=FAKE, sets=2,
             num_buckets=6, key_mask=0, scale=1.0, dscores=FAKE, dtable=FAKE, workspace=FAKE, workspace_bytes=BIG,
             stream=0)
    for run, a in ((g.nms_relation_softmax_run, f), (g.nms_relation_softmax_grad_run, b)):
        for bad, code in ((dict(type=9), BAD), (dict(batch=-1), BAD), (dict(heads=0), BAD), (dict(queries=-1), BAD),
                          (dict(keys=-1), BAD), (dict(sets=3), BAD), (dict(sets=0), BAD), (dict(num_buckets=0), BAD),
                          (dict(num_buckets=1025), CAP), (dict(heads=4097), CAP), (dict(scale=math.nan), BAD),
                          (dict(probs=0), BAD), (dict(probs=FAKE + 1), BAD), (dict(buckets=0), BAD),
                          (dict(buckets=FAKE + 1), BAD), (dict(batch=1 << 30, sets=1, queries=1 << 20), CAP)):
            assert run(**dict(a, **bad)) == code, bad
    assert g.nms_relation_softmax_run(**dict(f, table=FAKE + 2)) == BAD
    for bad, code in ((dict(dtable=0), BAD), (dict(dprobs=0), BAD), (dict(dscores=FAKE + 1), BAD), (dict(workspace=0), WS),
                      (dict(workspace_bytes=g.nms_relation_grad_workspace_size(2, 3, 4, 5, 6) - 1), WS)):
        assert g.nms_relation_softmax_grad_run(**dict(b, **bad)) == code, bad
    m = dict(q_pos=FAKE, q_sets=1, k_pos=FAKE, k_sets=3, queries=4, keys=5, axes=2, lut=FAKE, reach=3, buckets=FAKE,
             stream=0)
    for bad, code in ((dict(q_sets=2), BAD), (dict(q_sets=-1), BAD), (dict(queries=-1), BAD), (dict(axes=0), BAD),
                      (dict(axes=5), CAP), (dict(reach=-1), BAD), (dict(reach=(1 << 20) + 1), CAP), (dict(lut=0), BAD),
                      (dict(q_pos=FAKE + 2), BAD), (dict(buckets=FAKE + 1), BAD), (dict(keys=1 << 48), CAP)):
        assert g.nms_relation_buckets_run(**dict(m, **bad)) == code, bad


def test_tensor_functions_refuse_cpu_tensors():
    x = torch.randn(2, 9, 12)
    m = torch.zeros(1, 4, 5, dtype=torch.int16)
    for call in (lambda: g.group_norm_act(x, 3), lambda: g.dropout(x, 0.5, 0),
                 lambda: g.relation_softmax(torch.randn(1, 2, 4, 5), torch.randn(3, 2), m),
                 lambda: g.relation_buckets(m.int(), m.int(), torch.zeros(5, 3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()


def test_logarithmic_table():
    lut = g.relation_lut_log(8, 64)[0].tolist()
    assert len(lut) == 129 and lut == lut[::-1]  # as far behind as ahead
    back = lut[64:]
    assert back[:4] == [0, 1, 2, 3] and back == sorted(back) and back[64] == 7 and set(back) == set(range(8))
    assert all(b == 4 + int(math.log(d / 4) / math.log(16) * 4 + 1e-12) for d, b in enumerate(back) if 4 < d < 64)
    own = g.relation_lut_log(8, 64, ahead="own")[0].tolist()
    assert own[:65] == lut[:65] and own[65:] == [8 + b for b in back[1:]]
    masked = g.relation_lut_log(8, 64, ahead="mask")[0].tolist()
    assert masked[:65] == lut[:65] and masked[65:] == [-1] * 64
    for bad in ((1, 64), (8, 3)):
        with pytest.raises(ValueError):
            g.relation_lut_log(*bad)
    with pytest.raises(ValueError):
        g.relation_lut_log(8, 64, ahead="none")


def test_cell_table():
    lut = g.relation_lut_cells(1, 2)
    assert lut.tolist() == [[0, 0, 5, 10, 10], [0, 1, 2, 3, 4]] and lut.dtype == torch.int32


class OnSecond(torch.Tensor):
    """A CPU tensor that says it lies on the second CUDA device."""
    is_cuda = True

    def get_device(self):
        return 1


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

    def on(v):
        return v.as_subclass(OnSecond)

    x, stats = on(torch.randn(2, 9, 12)), on(torch.ones(2, 3))
    scores, table = on(torch.randn(2, 3, 4, 5)), on(torch.randn(6, 3))
    pos, lut = on(torch.zeros(1, 4, 2, dtype=torch.int32)), on(torch.zeros(2, 5, dtype=torch.int32))
    m = on(torch.zeros(1, 4, 5, dtype=torch.int16))
    g.group_norm_act(x, 3)
    g.group_norm_act_grad(x, x, stats, stats, 3)
    g.dropout(x, 0.5, 1)
    g.relation_buckets(pos, pos, lut)
    g.relation_softmax(scores, table, m)
    g.relation_softmax_grad(scores, scores, m, 6)
    assert [c[0] for c in calls] == ["nms_group_norm_run", "nms_group_norm_grad_run", "nms_dropout_run",
                                     "nms_relation_buckets_run", "nms_relation_softmax_run",
                                     "nms_relation_softmax_grad_run"]
    assert all(at == 1 and stream == 1001 for _, at, stream in calls) and now[0] == current


@pytest.mark.parametrize("batch", [1, 2, 3, 4, 16, 64])
@pytest.mark.parametrize("heads,queries,keys,nb", [(32, 8192, 8192, 1024), (8, 1000, 1025, 225), (8, 4096, 512, 1024),
                                                   (16, 3000, 65, 1024), (1, 100, 9000, 32), (4, 5000, 1000, 32)])
def test_relation_gradient_workspace_stays_beside_the_operands(batch, heads, queries, keys, nb):
    """The tables of sums take no more than a third of what three 16-bit
    operands do, beside one wave of tables; one image, or two of long rows,
    need that wave alone (a table for each of an SM's 16 warps at most)."""
    wave = 4 * nb * (152 * 4 + heads) + 256
    room = wave + (0 if batch == 1 or batch < 4 and keys > 1024 else batch * heads * queries * keys * 6 // 3)
    assert g.nms_relation_grad_workspace_size(batch, heads, queries, keys, nb) <= room


@pytest.mark.parametrize("scale", [math.inf, -math.inf, 1e39])
def test_relation_refuses_an_infinite_scale(scale):
    """scale * 0 in a masked place has to be 0; 1e39 is infinite in binary32."""
    f = dict(scores=FAKE, type=g.NMS_TYPE_F16, batch=0, heads=3, queries=4, keys=5, buckets=FAKE, sets=1, table=FAKE,
             num_buckets=6, key_mask=0, scale=1.0, probs=FAKE, stream=0)
    assert g.nms_relation_softmax_run(**f) == g.NMS_OK  # no images: nothing is launched
    assert g.nms_relation_softmax_run(**dict(f, scale=scale)) == BAD
    b = dict(dprobs=FAKE, probs=FAKE, type=g.NMS_TYPE_F16, batch=2, heads=3, queries=4, keys=5, buckets=FAKE, sets=2,
             num_buckets=6, key_mask=0, scale=scale, dscores=FAKE, dtable=FAKE, workspace=0, workspace_bytes=0, stream=0)
    assert g.nms_relation_softmax_grad_run(**b) == BAD


@pytest.mark.parametrize("num_buckets,max_distance", [(9, 128), (10, 160), (19, 288), (39, 608), (2, 1), (3, 1),
                                                      (8, 4), (7, 50), (32, 128), (33, 1000)])
def test_logarithmic_table_on_its_boundaries(num_buckets, max_distance):
    """Against whole numbers: bucket exact + k from (d / exact)^span >= (max /
    exact)^k on, distances that meet it with equality among them."""
    exact = num_buckets // 2
    span = num_buckets - exact
    back = g.relation_lut_log(num_buckets, max_distance)[0].tolist()[max_distance:]
    for d, bucket in enumerate(back):
        if d < exact:
            assert bucket == d
            continue
        k = max(k for k in range(span) if d ** span * exact ** k >= max_distance ** k * exact ** span)
        assert bucket == exact + k, d


def test_logarithmic_table_of_the_largest_sizes():
    back = g.relation_lut_log(1024, 1 << 20)[0][1 << 20:]
    assert (back[1:] >= back[:-1]).all() and back[511] == 511 and back[-1] == 1023


def test_the_suppressions_launches_too(lib, monkeypatch):
    """The same of the tensor functions of the suppression and the decode."""
    from greedy_iou_nms_gb300 import head
    head._torch()
    now, calls = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    class Recorder:
        def __getattr__(self, name):
            if not (name.endswith("_run") or name in ("nms_iou_mask", "nms_resolve_mask", "nms_decode_boxes7")):
                return getattr(lib, name)
            return lambda *args: calls.append((name, now[0], args[-1])) or 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch, "empty", torch.zeros)  # counts and statuses that no kernel writes
    monkeypatch.setattr(head, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(g, "_lib", Recorder())

    def on(*shape):
        return torch.zeros(*shape).as_subclass(OnSecond)

    g.nms(on(8, 4), on(8), 0.5)
    g.nms(on(8, 4), on(8), 0.5, fast=True)
    g.matrix_nms(on(8, 4), on(8), 0.1)
    g.lane_nms(on(8, 77), on(8), 0.5)
    g.iou_mask(on(8, 4), 0.5)
    g.resolve_mask(torch.zeros(8, 2, dtype=torch.int64).as_subclass(OnSecond))
    g.decode_boxes7(on(2, 9, 7), 0.3, 5)
    g.boxes7_nms(on(2, 36), 2, 0.5)
    assert [c[0] for c in calls] == ["nms_run", "nms_fast_run", "nms_matrix_run", "nms_lane_run", "nms_iou_mask",
                                     "nms_resolve_mask", "nms_decode_boxes7", "nms_boxes7_run"]
    assert all(at == 1 and stream == 1001 for _, at, stream in calls) and now[0] == 0
