"""Counter-based dropout (nms_dropout_run): the mask bit for bit against
Philox in Python integers, values after one rounding, residuals, lengths
around the generator's block, misaligned starts, element indices past 2^32."""
import pytest

import greedy_iou_nms_gb300 as g
import head_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.build()
    g.load()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [1, 7, 8, 9, 255, 4096, 5003])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999, 1.0])
def test_values_and_mask(t, n, p):
    r = torch.Generator().manual_seed(n)
    x, res = (torch.randn(n, generator=r).to(t) for _ in range(2))
    seed, offset = (1 << 64) - 3, (1 << 33) + n
    ref = R.drop(x.double(), p, seed, offset)
    got = g.dropout(x.cuda(), p, seed, offset)
    # One product in binary32 by a factor rounded to binary32, then the type's rounding.
    R.close(got, ref, 2 * R.EPS * ref.abs())
    if p:
        assert torch.equal(got.cpu() != 0, R.kept(n, p, seed, offset) & (x != 0))
    R.close(g.dropout(x.cuda(), p, seed, offset, residual=res.cuda()), ref + res.double(),
            3 * R.EPS * (ref.abs() + res.double().abs()))
    assert torch.equal(g.dropout_grad(x.cuda(), p, seed, offset), got)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shift", [1, 3, 4])
def test_misaligned_starts_and_strides(t, shift):
    base = torch.randn(3000, device="cuda").to(t)
    x = base[shift:shift + 2500]
    want = g.dropout(x.clone(), 0.3, 5, 6)
    assert torch.equal(g.dropout(x, 0.3, 5, 6), want)
    assert torch.equal(g.dropout(x.clone(), 0.3, 5, 6, residual=x), g.dropout(x, 0.3, 5, 6, residual=x.clone()))
    m = torch.randn(30, 50, device="cuda").to(t)
    assert torch.equal(g.dropout(m.T, 0.3, 5, 6), g.dropout(m.T.contiguous(), 0.3, 5, 6))


def test_a_dropped_element_is_zero_whatever_it_was():
    x = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0] * 64, device="cuda")
    keep = R.kept(256, 0.5, 9, 0).cuda()
    y = g.dropout(x, 0.5, 9)
    assert (y[~keep] == 0).all()
    assert torch.equal(y[keep].isnan(), x[keep].isnan()) and torch.equal(y[keep].isinf(), x[keep].isinf())


def test_share_kept_and_independence_of_offsets():
    n, p = 1 << 20, 0.3
    x = torch.ones(n, device="cuda")
    a, b = (g.dropout(x, p, 1, o) != 0 for o in (0, 1))
    c = g.dropout(x, p, 2, 0) != 0
    five = 5 * (n * p * (1 - p)) ** 0.5  # five standard deviations of the count
    for m in (a, b, c):
        assert abs(int(m.sum()) - n * (1 - p)) <= five
    both = (1 - p) ** 2
    for m in (b, c):
        assert abs(int((a & m).sum()) - n * both) <= 5 * (n * both * (1 - both)) ** 0.5


def test_indices_past_32_bits():
    """2^32 + 64 elements: element indices that 32 bits do not hold."""
    n = (1 << 32) + 64
    if torch.cuda.mem_get_info()[0] < 3 * 2 * n:
        pytest.skip("not enough device memory")
    x = torch.ones(n, dtype=torch.float16, device="cuda")
    y = g.dropout(x, 0.5, 3, 4)
    for start in (0, (1 << 32) - 64, 1 << 32):
        assert torch.equal((y[start:start + 64] != 0).cpu(), R.kept(64, 0.5, 3, 4, start=start))


def test_in_place_and_empty():
    x = torch.randn(1000, device="cuda")
    want = g.dropout(x, 0.2, 8)
    st = g.nms_dropout_run(x.data_ptr(), 0, g.NMS_TYPE_F32, 1000, 0.2, 8, 0, x.data_ptr(),
                           torch.cuda.current_stream().cuda_stream)
    assert st == g.NMS_OK and torch.equal(x, want)
    assert g.dropout(torch.empty(0, 4, device="cuda"), 0.5, 1).shape == (0, 4)


def test_refusals():
    x = torch.randn(16, device="cuda")
    for bad in (dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(seed=-1), dict(seed=1 << 64),
                dict(residual=x[:8]), dict(residual=x.half()), dict(residual=x.cpu())):
        with pytest.raises(ValueError):
            g.dropout(x, **{"p": 0.5, "seed": 0, **bad})
    for t in (x.cpu(), x.double(), x.int()):
        with pytest.raises(ValueError):
            g.dropout(t, 0.5, 0)
