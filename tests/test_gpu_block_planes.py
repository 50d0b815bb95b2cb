"""Binary32 products on the tensor cores keep all 24 bits of both operands: six
products of three bfloat16 parts each, none of which these tests would miss."""
import math

import pytest

import block_reference as R
import greedy_iou_nms_gb300 as g

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# Large enough for the tensor cores in all three products.
ROWS, INNER, OUTER = 300, 520, 520


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.build()
    g.load()


def _places(r, rows, columns):
    """A matrix with one signed power of two in each row, no two of them in one column."""
    m = torch.zeros(rows, columns)
    n = min(rows, columns)
    at = torch.randperm(columns, generator=r)[:n]
    m[torch.arange(n), at] = (1 - 2.0 * torch.randint(0, 2, (n,), generator=r)) * 2.0 ** torch.randint(-3, 4, (n,), generator=r)
    return m


def _odd(r, shape):
    """Odd whole numbers of 16 bits: two parts, none of them 0."""
    v = 32769.0 + 2.0 * torch.randint(0, 16384, shape, generator=r)
    return v * (1 - 2.0 * torch.randint(0, 2, shape, generator=r))


def _products(x, w, dy):
    """(x w^T, dz w, dz^T x) with dz = dy, its parts made by the pass over rows and by the one over slopes."""
    x, w, dy = x.cuda(), w.cuda(), dy.cuda()
    one = torch.ones_like(dy)
    yield g.linear_act(x, w).cpu(), *(v.cpu() for v in g.linear_act_grad(dy, x, w, need=(True, True, False))[:2])
    yield (None, *(v.cpu() for v in g.linear_act_grad(dy, x, w, one, act="relu")[:2]))


def _exact(x, w, dy):
    return x.double() @ w.double().T, dy.double() @ w.double(), dy.double().T @ x.double()


def _same(got, ref):
    assert got is None or torch.equal(got.double(), ref)


def test_numbers_of_24_bits_times_powers_of_two():
    """Exact, whichever operand has the 24 bits."""
    for seed in range(3):
        r = torch.Generator().manual_seed(seed)
        full = [torch.randn(s, generator=r) for s in ((ROWS, INNER), (OUTER, INNER), (ROWS, OUTER))]
        # The forward's first operand, its second; dz; the weight and x in the gradients.
        w = _places(r, OUTER, INNER)
        ref = _exact(full[0], w, full[2])
        for y, dx, _ in _products(full[0], w, full[2]):
            _same(y, ref[0])
            _same(dx, ref[1])
        x = _places(r, ROWS, INNER)
        ref = _exact(x, full[1], full[2])
        for y, _, dw in _products(x, full[1], full[2]):
            _same(y, ref[0])
            _same(dw, ref[2])
        dy = _places(r, ROWS, OUTER)
        ref = _exact(full[0], full[1], dy)
        for _, dx, dw in _products(full[0], full[1], dy):
            _same(dx, ref[1])
            _same(dw, ref[2])


def test_products_of_16_bit_numbers():
    """One product a result, of 32 bits: cut to 24 once and rounded once, where its second parts' product is 2^-18 of it."""
    r = torch.Generator().manual_seed(4)
    x, w, dy = (_odd(r, s) for s in ((ROWS, INNER), (OUTER, INNER), (ROWS, OUTER)))
    one_x, one_dy = ((_places(r, *v.shape) != 0) * v for v in (x, dy))
    for a, b, c, which in ((one_x, w, dy, (0, 2)), (x, w, one_dy, (1, 2))):
        ref = _exact(a, b, c)
        for got in _products(a, b, c):
            for i in which:
                if got[i] is not None:
                    assert ((got[i].double() - ref[i]).abs() <= 2.0 ** -22 * ref[i].abs()).all()
    assert float((ref[1] != 0).double().mean()) > 0.9


@pytest.mark.parametrize("rows,inner,outer", [(300, 256, 1024), (600, 520, 520), (130, 20000, 136), (20000, 136, 264),
                                              (400, 2600, 200), (1517, 333, 251)])
def test_errors_of_sums_do_not_grow_with_their_length(rows, inner, outer):
    """In the mean square, against S = sqrt(sum (a b)^2) of each result and in units of 2^-24 S.  Sums of 64, N of them, one
    after another, each rounded: sqrt(N / 6).  Within 64: 64 products and four sums, cut by 2^-25 and 2^-23 of the sum so
    far, half of that on average: 20, as the parts of 64 add up to S.  One of the three last pairs of parts left out would
    make 41 and more; stretches and clusters make chains shorter."""
    r = torch.Generator().manual_seed(rows)
    x, w, dy = (torch.randn(s, generator=r) for s in ((rows, inner), (outer, inner), (rows, outer)))
    y, dx, dw = next(_products(x, w, dy))
    for got, a, b in ((y, x, w.T), (dx, dy, w), (dw, dy.T, x)):
        a, b = a.double(), b.double()
        size = (a ** 2 @ b ** 2).sqrt()
        off = float((((got.double() - a @ b) / size) ** 2).mean().sqrt()) * 2.0 ** 24
        assert off <= 21 + math.sqrt(a.shape[1] / 64 / 6), off
    assert R.U == 2.0 ** -24
