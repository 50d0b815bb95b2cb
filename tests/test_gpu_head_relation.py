"""Relation weights (nms_relation_softmax_run), their gradient and the bucket
map against 64 bits.

Tolerances, fixed beforehand.  A weight's exponent is off by a few 2^-24 of
the logits' size and the row's sum by its chain of additions (K / 32 and the
joins), so a weight is right to (64 + K / 32) * 2^-24 * (1 + largest logit)
of itself, then rounded once.  da is right to (64 + K / 32) * 2^-24 of its
terms' size, and a table entry to 512 * 2^-24 of the sum of its terms' sizes
beside that."""
import math

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


def _inputs(seed, B, H, Q, K, t, nb, sets, masked=0.1):
    r = torch.Generator().manual_seed(seed)
    scores, dprobs = (torch.randn(B, H, Q, K, generator=r).to(t) for _ in range(2))
    scores = (scores.float() * 3).to(t)
    table = torch.randn(nb, H, generator=r)
    m = torch.randint(0, nb, (sets, Q, K), generator=r).to(torch.int16)
    m[torch.rand(sets, Q, K, generator=r) < masked] = -1
    return scores, dprobs, table, m


def _check(scores, dprobs, table, m, scale=0.7, key_mask=None):
    K = scores.shape[-1]
    t = scores.dtype
    km = None if key_mask is None else key_mask.cuda()
    got = g.relation_softmax(scores.cuda(), table.cuda(), m.cuda(), scale=scale, key_mask=km)
    ref, a = R.softmax(scores.double(), table.double(), m, scale, key_mask)
    big = float(a[torch.isfinite(a)].abs().max()) if torch.isfinite(a).any() else 0.0
    chain = (64 + K / 32) * R.EPS
    assert got.dtype == t and got.shape == scores.shape
    R.close(got, ref, chain * (1 + big) * ref)
    ok = R.valid_pairs(m, table.shape[0], key_mask).expand_as(ref)
    assert (got.cpu()[~ok] == 0).all()
    ds, dt = g.relation_softmax_grad(dprobs.cuda(), got, m.cuda(), table.shape[0], scale=scale, key_mask=km)
    (rs, rt), (ss, st) = R.softmax_grad(dprobs.double(), got.cpu().double(), m, table.shape[0], scale, key_mask)
    R.close(ds, rs, chain * ss)
    assert (ds.cpu()[~ok] == 0).all()
    assert dt.dtype == torch.float32
    R.close(dt, rt, (512 * R.EPS + chain) * st)
    again = g.relation_softmax_grad(dprobs.cuda(), got, m.cuda(), table.shape[0], scale=scale, key_mask=km)
    assert torch.equal(ds, again[0]) and torch.equal(dt, again[1])
    return got


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("B,H,Q,K,nb,per_image", [
    (2, 3, 5, 7, 4, True), (2, 2, 49, 49, 169, False), (3, 8, 64, 64, 225, False), (1, 1, 1, 1, 1, False),
    (2, 4, 1, 1000, 32, True), (2, 1, 33, 300, 225, True), (1, 2, 3, 2049, 32, False), (40, 2, 16, 16, 49, False),
    (1, 1, 2, 8192, 32, True), (3, 5, 17, 129, 9, True)])
def test_shapes(t, B, H, Q, K, nb, per_image):
    _check(*_inputs(K + Q, B, H, Q, K, t, nb, B if per_image else 1))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("K", [1, 2, 3, 15, 31, 32, 33, 63, 65, 127, 255, 256, 257, 511, 513, 1023, 1025, 4097, 20000])
def test_row_lengths(t, K):
    """Rows that start at every alignment and end inside every vector and tile."""
    _check(*_inputs(K, 2, 3, 3, K, t, 12, 2))


@pytest.mark.parametrize("nb", [1, 2, 225, 512, 961, 1024])
@pytest.mark.parametrize("per_image", [True, False])
def test_bucket_counts(nb, per_image):
    _check(*_inputs(nb, 3, 2, 40, 100, torch.float32, nb, 3 if per_image else 1))


@pytest.mark.parametrize("t", TYPES)
def test_key_masks_and_empty_rows(t):
    scores, dprobs, table, m = _inputs(3, 4, 2, 10, 70, t, 9, 4)
    mask = torch.rand(4, 70, generator=torch.Generator().manual_seed(1)) < 0.6
    mask[1] = False   # an image without keys
    mask[2] = True
    m[3, 4] = -1      # a query without pairs
    mask[0, 1:] = False  # a single key
    got = _check(scores, dprobs, table, m, key_mask=mask)
    assert (got[1] == 0).all() and (got[3, :, 4] == 0).all()
    # One map for all images, the mask alone differing; and bytes other than 0 and 1.
    _check(scores, dprobs, table, m[:1].contiguous(), key_mask=(mask * 7).to(torch.uint8))


def test_buckets_outside_the_table_mask():
    scores, dprobs, table, m = _inputs(4, 2, 2, 6, 50, torch.float32, 8, 2, masked=0.0)
    m[0, :, ::3] = 8
    m[1, :, ::5] = 32767
    m[1, 2] = -32768
    _check(scores, dprobs, table, m)


@pytest.mark.parametrize("t", TYPES)
def test_masked_places_are_not_looked_at(t):
    scores, dprobs, table, m = _inputs(5, 2, 2, 8, 40, t, 6, 2)
    mask = torch.ones(2, 40, dtype=torch.bool)
    mask[:, 30:] = False
    off = ~R.valid_pairs(m, 6, mask).expand_as(scores)
    clean = g.relation_softmax(scores.cuda(), table.cuda(), m.cuda(), key_mask=mask.cuda())
    want = g.relation_softmax_grad(dprobs.cuda(), clean, m.cuda(), 6, key_mask=mask.cuda())
    for junk in (float("nan"), float("inf"), -float("inf"), torch.finfo(t).max):
        s, d, p = scores.clone(), dprobs.clone(), clean.cpu().clone()
        s[off] = d[off] = p[off] = junk
        assert torch.equal(g.relation_softmax(s.cuda(), table.cuda(), m.cuda(), key_mask=mask.cuda()), clean)
        got = g.relation_softmax_grad(d.cuda(), p.cuda(), m.cuda(), 6, key_mask=mask.cuda())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("K", [20, 700, 9000])
def test_scores_of_the_types_lowest_value_and_infinities(t, K):
    scores, _, table, m = _inputs(6, 1, 1, 6, K, t, 4, 1, masked=0.0)
    table *= 0
    low = torch.finfo(t).min
    scores[0, 0, 0, 5:] = low            # a mask written into the scores
    scores[0, 0, 1] = low                # ... over the whole row: even weights
    scores[0, 0, 2, 7:] = -math.inf
    scores[0, 0, 3] = -math.inf          # nothing left: zero
    scores[0, 0, 4, 3] = math.inf        # inf - inf
    scores[0, 0, 5, K - 1] = math.nan
    got = g.relation_softmax(scores.cuda(), table.cuda(), m.cuda(), scale=1.0).cpu()
    assert (got[0, 0, 0, 5:] == 0).all() and (got[0, 0, 2, 7:] == 0).all() and (got[0, 0, 3] == 0).all()
    R.close(got[0, 0, 1], torch.full((K,), 1 / K, dtype=torch.float64), (64 + K / 32) * R.EPS)
    assert got[0, 0, 4].isnan().all() and got[0, 0, 5].isnan().all()
    ref, _ = R.softmax(scores[:, :, ::2, :].double()[:, :, :1], table.double(), m[:, :1], 1.0)
    R.close(got[0, 0, 0], ref[0, 0, 0], (64 + K / 32) * R.EPS * 16)


def test_strides_and_misaligned_starts():
    for t in TYPES:
        scores, dprobs, table, m = (v.cuda() for v in _inputs(7, 2, 3, 9, 33, t, 5, 2))
        want = g.relation_softmax(scores, table, m)
        grad = g.relation_softmax_grad(dprobs, want, m, 5)
        turned = scores.transpose(1, 2).contiguous().transpose(1, 2)
        assert torch.equal(g.relation_softmax(turned, table, m), want)
        for shift in (1, 3):
            def moved(v):
                base = torch.empty(v.numel() + shift, dtype=v.dtype, device="cuda")
                base[shift:].copy_(v.reshape(-1))
                return base[shift:].view(v.shape)
            assert torch.equal(g.relation_softmax(moved(scores), moved(table), moved(m)), want)
            got = g.relation_softmax_grad(moved(dprobs), moved(want), moved(m), 5)
            assert torch.equal(got[0], grad[0]) and torch.equal(got[1], grad[1])


def test_gradient_against_differences():
    """<dscores, v> + <dtable, w> against central differences of the 64-bit
    forward (an error of h^2, 1e-8, and the gradient's own roundings)."""
    scores, dprobs, table, m = _inputs(8, 2, 2, 12, 40, torch.float32, 7, 2)
    r = torch.Generator().manual_seed(2)
    vs, vt = (torch.randn(v.shape, generator=r, dtype=torch.float64) for v in (scores, table))

    def loss(h):
        return float((R.softmax(scores.double() + h * vs, table.double() + h * vt, m, 0.4)[0] * dprobs.double()).sum())

    h = 1e-5
    probs = g.relation_softmax(scores.cuda(), table.cuda(), m.cuda(), scale=0.4)
    ds, dt = g.relation_softmax_grad(dprobs.cuda(), probs, m.cuda(), 7, scale=0.4)
    terms = [ds.cpu().double() * vs, dt.cpu().double() * vt]
    size = sum(float(t.abs().sum()) for t in terms)
    assert abs(sum(float(t.sum()) for t in terms) - (loss(h) - loss(-h)) / (2 * h)) <= 1e-5 * size


def test_nothing_to_do():
    table = torch.randn(4, 2, device="cuda")
    for B, Q, K in ((0, 3, 5), (2, 0, 5), (2, 3, 0)):
        s = torch.empty(B, 2, Q, K, device="cuda")
        m = torch.zeros(1, Q, K, dtype=torch.int16, device="cuda")
        assert g.relation_softmax(s, table, m).shape == s.shape
        ds, dt = g.relation_softmax_grad(s, s, m, 4)
        assert ds.shape == s.shape and (dt == 0).all() and dt.shape == (4, 2)


# -------------------------------------------------------------------- the map

@pytest.mark.parametrize("qs,ks", [(1, 1), (3, 3), (1, 3), (3, 1)])
@pytest.mark.parametrize("axes", [1, 2, 3])
def test_buckets(qs, ks, axes):
    r = torch.Generator().manual_seed(axes)
    q = torch.randint(-40, 40, (qs, 13, axes), generator=r).to(torch.int32)
    k = torch.randint(-40, 40, (ks, 37, axes), generator=r).to(torch.int32)
    lut = torch.randint(-1, 9, (axes, 2 * 20 + 1), generator=r).to(torch.int32)
    assert torch.equal(g.relation_buckets(q.cuda(), k.cuda(), lut.cuda()).cpu(), R.buckets(q, k, lut))


def test_buckets_of_extreme_positions_and_sums():
    big = 2 ** 31 - 1
    q = torch.tensor([[[0], [big], [-big - 1]]], dtype=torch.int32)
    lut = torch.tensor([[7, 8, 9]], dtype=torch.int32)
    assert torch.equal(g.relation_buckets(q.cuda(), q.cuda(), lut.cuda()).cpu(), R.buckets(q, q, lut))
    lut2 = torch.tensor([[30000], [2767]], dtype=torch.int32)
    z = torch.zeros(1, 2, 2, dtype=torch.int32)
    assert (g.relation_buckets(z.cuda(), z.cuda(), lut2.cuda()) == 32767).all()
    assert (g.relation_buckets(z.cuda(), z.cuda(), (lut2 + 1).cuda()) == -1).all()


def test_tables_of_positions():
    """Windows and logarithmic distances through the library's own tables."""
    side = 5
    at = torch.arange(side * side)
    cell = torch.stack([at // side, at % side], -1).to(torch.int32)[None]
    lut = g.relation_lut_cells(side - 1, side - 1)
    m = g.relation_buckets(cell.cuda(), cell.cuda(), lut.cuda()).cpu()
    assert len(set(m.flatten().tolist())) == (2 * side - 1) ** 2 and (m[0].diagonal() == m[0, 0, 0]).all()
    pos = torch.arange(50, dtype=torch.int32)[None, :, None]
    m = g.relation_buckets(pos.cuda(), pos.cuda(), g.relation_lut_log(8, 16, ahead="mask").cuda()).cpu()[0]
    assert torch.equal(m < 0, torch.ones(50, 50).triu(1).bool())
    assert m.max() == 7 and (m.diagonal() == 0).all()


def test_refusals():
    s = torch.randn(2, 3, 4, 5, device="cuda")
    table = torch.randn(6, 3, device="cuda")
    m = torch.zeros(2, 4, 5, dtype=torch.int16, device="cuda")
    for a in ((s[0], table, m), (s.double(), table, m), (s.cpu(), table, m), (s, table[:, :2], m), (s, table.cpu(), m),
              (s, table, m.int()), (s, table, m[:, :3]), (s, table, m.cpu()), (s, table, m.repeat(2, 1, 1))):
        with pytest.raises(ValueError):
            g.relation_softmax(*a)
    for mask in (torch.ones(2, 4, device="cuda"), torch.ones(2, 4, device="cuda").bool(), torch.ones(2, 5).bool()):
        with pytest.raises(ValueError):
            g.relation_softmax(s, table, m, key_mask=mask)
    with pytest.raises(g.NmsError) as e:
        g.relation_softmax(s, torch.randn(1025, 3, device="cuda"), m)
    assert e.value.code == g.NMS_ERR_CAPACITY
    with pytest.raises(ValueError):
        g.relation_softmax_grad(s[:1], s, m, 6)
    with pytest.raises(g.NmsError):
        g.relation_softmax_grad(s, s, m, 0)
    p = torch.zeros(2, 3, 2, dtype=torch.int32, device="cuda")
    lut = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    for a in ((p.long(), p, lut), (p, p.cpu(), lut), (p, p[..., :1], lut), (p, p, lut[:, :4]), (p, p, lut[:1]),
              (p.repeat(2, 1, 1), p.repeat(3, 1, 1)[:3], lut)):
        with pytest.raises(ValueError):
            g.relation_buckets(*a)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("B,H,Q,K", [(9, 8, 49, 49), (5, 8, 33, 25), (6, 16, 9, 9), (3, 8, 81, 81), (7, 8, 40, 121),
                                     (5, 3, 49, 49), (4, 8, 65, 63), (2, 8, 1, 7)])
def test_short_odd_rows_by_image(t, B, H, Q, K):
    """Odd rows of one map for all images: an image's rows are a multiple of
    16 bytes or not, the last block's rows end inside a vector, images in
    fours and a remainder."""
    _check(*_inputs(B + K, B, H, Q, K, t, 31, 1))


def test_as_many_images_as_rows_may_be():
    """2^31 - 1 images of one pair: past 2^16 chunks and to the end of 32-bit
    counts.  da is 1/4 everywhere; the table's entry is chains of at most
    2^15 images and 2^13 partial sums."""
    n = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 32e9:
        pytest.skip("memory")
    m = torch.zeros(1, 1, 1, dtype=torch.int16, device="cuda")
    x = torch.zeros(n, 1, 1, 1, dtype=torch.float16, device="cuda")
    probs = g.relation_softmax(x, torch.ones(1, 1, device="cuda"), m)
    assert probs.min() == 1 and probs.max() == 1
    ds, dt = g.relation_softmax_grad(x.fill_(1.0), probs.fill_(0.5), m, 1)
    assert ds.min() == 0.25 and ds.max() == 0.25
    assert abs(float(dt) - n / 4) <= (2 ** 15 + 2 ** 13 + 64) * R.EPS * n / 4


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("nb", [100, 138, 225, 414, 415, 416, 440, 474, 475, 476, 831, 951, 1024])
@pytest.mark.parametrize("K", [5, 64, 100, 300, 1000])
def test_bucket_counts_by_head(t, nb, K):
    """A map by image: the gradient's tables of every size that changes how
    many columns and warps share the memory."""
    _check(*_inputs(nb + K, 2, 3, 7, K, t, nb, 2))


@pytest.mark.parametrize("t,K", [(torch.bfloat16, 1000), (torch.float16, 300), (torch.float32, 1000),
                                 (torch.float32, 46), (torch.bfloat16, 999), (torch.bfloat16, 128), (torch.float16, 64)])
@pytest.mark.parametrize("nb", [138, 225, 414, 440, 553])
def test_table_sums_of_lanes_that_share_a_column(t, K, nb):
    """Two lanes to a column of sums: no addition is lost where one lane's
    bucket is the other's a step before or behind, equal to it, or masked.
    Every weight is 2^-10 and the gradients are whole numbers that add up to 0
    in a row, so da = dprobs / 2^10 and its sums are exact in any order."""
    r = torch.Generator().manual_seed(K + nb)
    B, H, Q = 5, 2, 24
    dp = torch.randint(-8, 9, (B, H, Q, K), generator=r).float()
    half = K // 2
    dp[..., half:2 * half] = -dp[..., :half]
    if K % 2:
        dp[..., -1] = 0
    j = torch.arange(K)
    lane, e = j // 8 % 32, j % 8
    apart = torch.where(lane < 16, e, e - 1) + j // 256 * 8       # an element behind
    other = torch.where(lane < 16, e, e + 1) + j // 256 * 8       # an element ahead
    masked = torch.where(e % 2 == 0, -1, e)                       # masked in both lanes, or in one
    masked[::3] = -1
    rows = torch.stack([apart % nb, other % nb, j % 2, j * 0, masked, j % 16, j // 16 % nb,
                        torch.randint(0, nb, (K,), generator=r)])
    m = rows[torch.arange(B * Q) % 8].view(B, Q, K).to(torch.int16)
    m = torch.where((m < 0) & (torch.arange(K) >= 2 * half), torch.zeros_like(m), m)
    # A masked pair's partner of the row's other half is masked too: the row still adds up to 0.
    gone = m < 0
    gone[..., :half] |= gone[..., half:2 * half].clone()
    gone[..., half:2 * half] |= gone[..., :half].clone()
    m[gone] = -1
    probs = torch.full((B, H, Q, K), 2.0 ** -10).to(t).cuda()
    want = torch.zeros(nb + 1, H, dtype=torch.float64)
    at = torch.where(m < 0, nb, m.long())
    for h in range(H):
        want[:, h].index_add_(0, at.reshape(-1), dp[:, h].double().reshape(-1) / 1024)
    for _ in range(5):
        got = g.relation_softmax_grad(dp.to(t).cuda(), probs, m.cuda(), nb)[1]
        assert torch.equal(got.cpu().double(), want[:nb])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("K,nb", [(320, 40), (321, 40), (400, 225), (513, 225), (601, 9), (1000, 1000), (1100, 225),
                                  (1100, 32), (4100, 32)])
@pytest.mark.parametrize("B", [2, 3, 4, 7, 8, 15, 16, 63, 64])
def test_one_map_for_few_and_many_images(t, K, nb, B):
    """Both sides of every number of images at which the gradient goes another way."""
    _check(*_inputs(K + B, B, 1, 3, K, t, nb, 1))
