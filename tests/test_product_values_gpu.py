"""Adapters with infinities and NaN that are in use: they reach the rows of
their own requests and no others, wherever the rows lie in a tile.

The rows of other requests are compared bit for bit with a call in which the
same adapter holds finite values: nothing of it enters their sums.  Rows of the
adapter itself are compared by kind (finite, NaN, infinity and its sign) with
the formula in 64 bits, whose infinities and NaN are those of any order of the
sum, and the finite ones by the operators' documented error."""
import numpy as np
import pytest

from tests.test_product_gpu import TYPES, check, mods, normal, ref_lora

pytestmark = pytest.mark.gpu

# runs of 16 rows and more that share tiles; a short one; requests without an adapter among them
LENGTHS = [40, 20, 100, 33, 16, 200, 3, 64, 31, 700, 18, 256, 47]
IDS = [0, 1, 2, -1, 1, 3, 1, -1, 2, 1, 0, 3, 2]


def build(dtype, k, n, rank, copies=1):
    torch, _ = mods()
    lens = LENGTHS * copies
    off = 5 + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    ids = IDS * copies
    g = torch.Generator(device="cuda")
    g.manual_seed(31 * k + n + rank)
    x, w = normal(g, (int(off[-1]) + 7, k), dtype), normal(g, (n, k), dtype, k ** -0.5)
    a, b = normal(g, (4, rank, k), dtype, k ** -0.5), normal(g, (4, n, rank), dtype, rank ** -0.5)
    adapter = torch.tensor(ids, dtype=torch.int32, device="cuda")
    return off, ids, x, w, a, b, torch.from_numpy(off).cuda(), adapter


def rows_with(off, ids, used):
    torch, _ = mods()
    hit = torch.zeros(int(off[-1]) + 7, dtype=torch.bool, device="cuda")
    for s, i in enumerate(ids):
        if i == used:
            hit[int(off[s]):int(off[s + 1])] = True
    return hit


def same_kinds(got, want, where):
    torch, _ = mods()
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), (where, "NaN")
    assert torch.equal(torch.isposinf(got), torch.isposinf(want)), (where, "+inf")
    assert torch.equal(torch.isneginf(got), torch.isneginf(want)), (where, "-inf")


# n: one CTA per tile, a pair of CTAs, tiles of 64 columns
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k,n,rank,copies", ((200, 264, 16, 1), (264, 1288, 32, 2), (72, 72, 8, 1), (1104, 300, 33, 1), (96, 520, 128, 1),
                                             (64, 264, 5, 1)))
def test_values_of_b_stay_in_their_requests(dtype, k, n, rank, copies):
    torch, sr = mods()
    off, ids, x, w, a, b, do, adapter = build(dtype, k, n, rank, copies)
    scale = torch.tensor([0.5, -2.0, 1.0, 3.0], device="cuda")
    finite = sr.seg_lora(x, w, a, b, do, adapter, scale)
    y, m = ref_lora(x, w, a, b, off, ids, scale)
    check(finite, y, m, k + rank, (dtype, n, "finite"))
    bad = b.clone()
    bad[1, 3, 0] = float("inf")
    bad[1, n // 2, rank - 1] = float("nan")
    bad[1, n - 1, rank // 2] = float("-inf")
    if rank > 1:
        bad[1, 3, 1] = float("inf")          # with the one before: infinities of either sign in a sum
    got = sr.seg_lora(x, w, a, bad, do, adapter, scale)
    hit = rows_with(off, ids, 1)
    assert torch.equal(got[~hit], finite[~hit])
    y, m = ref_lora(x, w, a, bad, off, ids, scale)
    same_kinds(got[hit], y[hit], (dtype, n, rank))
    clean = torch.isfinite(y)
    check(got[clean], y[clean], torch.nan_to_num(m, 0.0, 0.0, 0.0)[clean], k + rank, (dtype, n, "finite columns"))
    assert torch.equal(got.view(torch.int32 if dtype == "float32" else torch.int16),
                       sr.seg_lora(x, w, a, bad, do, adapter, scale).view(torch.int32 if dtype == "float32" else torch.int16))
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k,n,rank,copies", ((200, 264, 16, 1), (264, 1288, 32, 2), (72, 72, 8, 1), (96, 300, 40, 1)))
def test_inner_products_that_are_not_finite_stay_in_their_rows(dtype, k, n, rank, copies):
    """An infinity in an adapter's a, one in a row of x, and NaN in every adapter's b at once."""
    torch, sr = mods()
    off, ids, x, w, a, b, do, adapter = build(dtype, k, n, rank, copies)
    finite = sr.seg_lora(x, w, a, b, do, adapter)
    bad_a = a.clone()
    bad_a[2, rank - 1, 7] = float("inf")
    got = sr.seg_lora(x, w, bad_a, b, do, adapter)
    hit = rows_with(off, ids, 2)
    assert torch.equal(got[~hit], finite[~hit])
    if dtype == "float32":                   # infinities may become NaN there
        assert not bool(torch.isfinite(got[hit]).any())
    else:
        y, _ = ref_lora(x, w, bad_a, b, off, ids, None)
        same_kinds(got[hit], y[hit], (dtype, n, rank, "a"))
    bad_x = x.clone()
    row = int(off[9]) + 300
    bad_x[row, 1] = float("inf")
    got = sr.seg_lora(bad_x, w, a, b, do, adapter)
    others = torch.arange(x.shape[0], device="cuda") != row
    assert torch.equal(got[others], finite[others]) and not bool(torch.isfinite(got[row]).any())
    bad_b = b.clone()
    bad_b[:, 11, 0] = float("nan")
    got = sr.seg_lora(x, w, a, bad_b, do, adapter)
    none = ~sum(rows_with(off, ids, i) for i in range(4)).bool()
    assert torch.equal(got[none], finite[none])
    columns = torch.arange(n, device="cuda") != 11
    assert torch.equal(got[:, columns], finite[:, columns]) and bool(torch.isnan(got[~none, 11]).all())
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_values_of_b_stay_in_their_requests_in_split_tiles(dtype):
    """Few rows and a long sum: the parts of a tile are added by a cluster."""
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    off, ids, k, n, rank = np.array([0, 20, 44, 60]), [0, 1, 2], 2048, 136, 12
    x, w = normal(g, (62, k), dtype), normal(g, (n, k), dtype, k ** -0.5)
    a, b = normal(g, (3, rank, k), dtype, k ** -0.5), normal(g, (3, n, rank), dtype)
    do, adapter = torch.from_numpy(off).cuda(), torch.tensor(ids, dtype=torch.int32, device="cuda")
    finite = sr.seg_lora(x, w, a, b, do, adapter)
    b[1, 100, 3], b[1, 5, 0] = float("nan"), float("inf")
    got = sr.seg_lora(x, w, a, b, do, adapter)
    others = torch.ones(62, dtype=torch.bool, device="cuda")
    others[20:44] = False
    assert torch.equal(got[others], finite[others])
    y, _ = ref_lora(x, w, a, b, off, ids, None)
    same_kinds(got[~others], y[~others], dtype)
    assert sr.device_status() == 0
