"""The transformer block's operators without a GPU: checks that came after the
first ones."""
import pytest

import greedy_iou_nms_gb300 as g

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def lib():
    g.build()
    return g.load()


@pytest.mark.parametrize("status", [torch.zeros(2, dtype=torch.int32), torch.zeros(1), torch.zeros(1, dtype=torch.int64),
                                    torch.zeros(1, dtype=torch.int32, device="meta")])
def test_status_is_one_int32_beside_x(status):
    x, w, dy = torch.zeros(3, 8), torch.zeros(5, 8), torch.zeros(3, 5)
    for call in (lambda s: g.linear_act(x, w, status=s), lambda s: g.linear_act_grad(dy, x, w, status=s)):
        with pytest.raises(ValueError, match="status must be one int32"):
            call(status)
        with pytest.raises(ValueError, match="status must be a tensor"):
            call(3)
        with pytest.raises(ValueError, match="CUDA"):  # the last check
            call(torch.zeros(1, dtype=torch.int32))


def test_long_sums_of_a_weights_gradient_are_cut():
    """From 2^18 rows on there is room for the sums of two stretches, whatever the type and however many the results."""
    for kind in (g.NMS_TYPE_F32, g.NMS_TYPE_F16, g.NMS_TYPE_BF16):
        for inner, outer in ((2048, 2048), (40, 4096)):
            few, more = (g.nms_linear_grad_workspace_size(kind, rows, inner, outer, 1) for rows in (1 << 18, (1 << 18) + 1))
            assert more - few >= 2 * 4 * inner * outer
    # Products on the plain units: a chain of theirs is 2^16 long at most.
    few, more = (g.nms_linear_grad_workspace_size(g.NMS_TYPE_F32, rows, 1 << 15, 32, 1) for rows in (1 << 16, (1 << 16) + 1))
    assert more - few >= 2 * 4 * 32 << 15


def test_the_binding_is_of_this_torch_and_interpreter(monkeypatch, tmp_path):
    """Another torch or interpreter means another file, and a torch without CUDA none: the library builds without it."""
    import os
    import sysconfig
    from greedy_iou_nms_gb300 import _build
    name = os.path.basename(_build.BINDING_LIB)
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name
    assert _build._with_binding() and os.path.exists(_build.BINDING_LIB) and not _build._stale()
    monkeypatch.setattr(_build, "BINDING_LIB", str(tmp_path / name.replace(torch.__version__, "0.0")))
    assert _build._stale()
    (tmp_path / "lib").mkdir()
    monkeypatch.setattr(_build, "_torch_folder", lambda: str(tmp_path))
    assert not _build._with_binding() and not _build._stale()
    assert _build._torch_version() == "none"


def test_the_largest_widths_of_a_linear_layer():
    most = g.NMS_LINEAR_MAX_WIDTH
    for size in (g.nms_linear_workspace_size, g.nms_linear_grad_workspace_size):
        for kind in (g.NMS_TYPE_F32, g.NMS_TYPE_F16, g.NMS_TYPE_BF16):
            for inner, outer in ((most, 1), (1, most), (most, most)):
                assert size(kind, 1, inner, outer, 1) >= 0
            for inner, outer in ((most + 1, 1), (1, most + 1)):
                with pytest.raises(g.NmsError) as e:
                    size(kind, 1, inner, outer, 1)
                assert e.value.code == g.NMS_ERR_CAPACITY
            assert size(kind, 1 << 20, most, 1, 1) >= 0  # 2^38 elements
            with pytest.raises(g.NmsError) as e:
                size(kind, (1 << 20) + 1, most, 1, 1)
            assert e.value.code == g.NMS_ERR_CAPACITY
