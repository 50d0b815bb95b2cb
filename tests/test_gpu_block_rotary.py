"""Rotary positions and their gradient against 64 bits."""
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


def _inputs(B, n, H, D, axes, kind, place, sets=None, seed=0):
    r = torch.Generator().manual_seed(seed)
    x = torch.randn(B, n, H, D, generator=r).to(R.TYPES[kind])
    sets = sets or B
    if place == "far":
        p = torch.randint(-(1 << 31), 1 << 31, (sets, n, axes), generator=r).to(torch.int32)
    elif place == "near":
        p = torch.randint(-3, 4, (sets, n, axes), generator=r).to(torch.int32)
    else:
        p = 1000 * torch.randn(sets, n, axes, generator=r)
    return x, p


def _check(got, x, ref, place):
    """Cosine and sine are off by their angle's rounding (2^-27 half turns), the
    fraction's (2^-32 of a position) and two steps of their own, and each
    product and sum by half a step: under 8 of x's pair."""
    size = x.double().abs().amax(-1, keepdim=True)
    bound = 10 * R.U * size + R.half_step(x.dtype) * ref.abs()
    if place == "far":
        bound = bound + 2e-6 * size  # of the reference: 2^31 radians in 64 bits are known to 2^-22
    assert ((got.cpu().double() - ref).abs() <= bound + 2.0 ** -25).all()


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("place", ["near", "far", "centres"])
@pytest.mark.parametrize("shape,pairs", [((1, 1, 1, 2), (1,)), ((2, 3, 1, 8), (4,)), ((3, 1, 8, 64), (32,)),
                                         ((2, 33, 5, 64), (8, 12, 12)), ((1, 7, 3, 42), (11, 10)),
                                         ((2, 5, 4, 80), (16, 8, 8)), ((2, 5, 4, 77), (16, 8, 8)),
                                         ((1, 9, 33, 128), (0, 64)), ((1, 2, 2, 256), (128,))])
@pytest.mark.parametrize("halves", [True, False])
def test_both_directions(shape, pairs, kind, place, halves):
    x, p = _inputs(*shape, len(pairs), kind, place, seed=sum(shape))
    lut = g.rotary_lut(*pairs).cuda()
    for turn, sign in ((g.rotary, 1.0), (g.rotary_grad, -1.0)):
        got = turn(x.cuda(), p.cuda(), lut, halves=halves)
        assert got.dtype is x.dtype and got.shape == x.shape
        _check(got, x, R.rotary(x, p, pairs, halves, sign=sign), place)
        assert torch.equal(got[..., 2 * sum(pairs):].cpu(), x[..., 2 * sum(pairs):])


def test_far_positions_are_exact():
    """Positions whole turns of the slowest pair apart turn alike, and a turn
    there and back gives the vectors again."""
    lut = torch.tensor([[1 << 44, 1 << 50, -(1 << 62)], [0, 0, 0]], dtype=torch.int64, device="cuda")
    x = torch.randn(1, 2, 3, 6, device="cuda")
    p = torch.tensor([[[5], [5 + (1 << 20)]]], dtype=torch.int32, device="cuda")
    y = g.rotary(x[:, :1].expand(1, 2, 3, 6), p, lut)
    assert torch.equal(y[:, 0], y[:, 1])
    back = g.rotary_grad(g.rotary(x, p, lut), p, lut)
    assert (back - x).abs().max() <= 16 * R.U * x.abs().max()


def test_quarter_turns():
    lut = torch.tensor([[1 << 62], [0]], dtype=torch.int64, device="cuda")
    x = torch.tensor([3.0, 4.0], device="cuda").expand(1, 4, 1, 2)
    p = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4, 1)
    assert g.rotary(x, p, lut)[0, :, 0].tolist() == [[3, 4], [-4, 3], [-3, -4], [4, -3]]
    assert g.rotary(x, p.float() * 2, lut)[0, :, 0].tolist() == [[3, 4], [-3, -4], [3, 4], [-3, -4]]


def test_strides_sets_and_layouts():
    r = torch.Generator().manual_seed(1)
    packed = torch.randn(3, 10, 12, 32, generator=r).cuda()
    lut = g.rotary_lut(10, 6).cuda()
    p = torch.randint(0, 50, (3, 10, 2), generator=r).to(torch.int32).cuda()
    for x in (packed[:, :, :8], packed[:, :, 1:4], packed[:, :, :, ::2].repeat(1, 1, 1, 2), packed[:, 3:4].expand(3, 10, 12, 32),
              packed.permute(0, 1, 2, 3)[:, :, ::3], packed.transpose(2, 3)[..., :12].repeat(1, 1, 1, 3)[..., :32]):
        for halves in (True, False):
            y = g.rotary(x, p, lut, halves=halves)
            assert y.shape == x.shape and torch.equal(y, g.rotary(x.contiguous(), p, lut, halves=halves))
    heads_first = torch.randn(3, 5, 10, 32, generator=r).cuda().transpose(1, 2)  # lies as [batch, heads, tokens, dim]
    y = g.rotary(heads_first, p, lut)
    assert y.stride() == heads_first.stride() and torch.equal(y, g.rotary(heads_first.contiguous(), p, lut))
    one = g.rotary(packed, p[:1], lut)
    assert torch.equal(one, g.rotary(packed, p[:1].expand(3, 10, 2), lut))
    odd = torch.randn(3 * 10 * 12 * 32 + 1, generator=r).cuda()[1:].view(3, 10, 12, 32)
    assert torch.equal(g.rotary(odd, p, lut), g.rotary(odd.clone(), p, lut))


def test_unknown_positions_and_axes():
    lut = g.rotary_lut(4, 4)
    x = torch.randn(1, 5, 2, 20, device="cuda")
    p = torch.tensor([[float("nan"), 1.0], [float("inf"), 1.0], [-float("inf"), 1.0], [2.0 ** 31, 1.0], [7.5, 1.0]],
                     device="cuda")[None]
    y = g.rotary(x, p, lut.cuda())
    first = torch.cat([y[..., :4], y[..., 8:12]], -1)
    assert torch.isnan(first[:, :4]).all() and torch.isfinite(first[:, 4]).all()
    assert torch.isfinite(y[..., 4:8]).all() and torch.equal(y[..., 16:], x[..., 16:])
    lut[1, 0], lut[1, 5] = 2, -1  # axes that the positions do not have
    y = g.rotary(x, torch.ones(1, 5, 2, dtype=torch.int32, device="cuda"), lut.cuda())
    assert torch.equal(y[..., 0], x[..., 0]) and torch.equal(y[..., 8 + 5], x[..., 8 + 5])
    assert not torch.equal(y[..., 1], x[..., 1])


def test_empty():
    lut = g.rotary_lut(4).cuda()
    for shape in ((0, 5, 2, 8), (2, 0, 2, 8), (2, 5, 0, 8)):
        p = torch.zeros(shape[0], shape[1], 1, dtype=torch.int32, device="cuda")
        assert g.rotary(torch.empty(shape, device="cuda"), p, lut).shape == shape


def test_in_place_and_graph():
    x = torch.randn(2, 6, 3, 48, device="cuda", dtype=torch.bfloat16)
    p = torch.randint(0, 99, (2, 6, 1), dtype=torch.int32, device="cuda")
    lut = g.rotary_lut(24).cuda()
    y = g.rotary(x, p, lut)
    z = x.clone()
    s = z.stride()
    st = g.nms_rotary_run(z.data_ptr(), *s[:3], g.NMS_TYPE_BF16, 2, 6, 3, 48, p.data_ptr(), g.NMS_POSITION_I32, 2, 1,
                          lut.data_ptr(), 24, 1, 0, z.data_ptr(), *s[:3], torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == g.NMS_OK and torch.equal(z, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = g.rotary(x, p, lut)
    p.add_(1)
    graph.replay()
    assert torch.equal(got, g.rotary(x, p, lut)) and not torch.equal(got, y)
