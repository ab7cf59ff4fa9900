"""Sums of one sign over many steps: the tensor cores' additions cut what they
shift out, always towards zero, so a sum in one accumulator drifts with its
length.  What is held is 32,768 steps at most, each 16 of them off by less than
2 * 2^-23 of the sum: 2^-11 of it.  Beside that a 16-bit result has its own
rounding, half a unit: 2^-8 of its size for bfloat16 and 2^-11 for float16,
whose smallest step is 2^-24."""
import numpy as np
import pytest

from tests.test_product_gpu import mods

pytestmark = pytest.mark.gpu

HALF_UNIT = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
HALF_STEP = {"bfloat16": 0.0, "float16": 2.0 ** -25}
DRIFT = 2.0 ** -11


def positive(g, shape, dtype, most):
    torch, _ = mods()
    return (torch.rand(shape, generator=g, device="cuda") * most).to(getattr(torch, dtype))


def check(got, want, dtype, where):
    err = (got.double() - want).abs()
    bad = ~(err <= (HALF_UNIT[dtype] + DRIFT) * want + HALF_STEP[dtype])
    assert not bool(bad.any()), (where, int(bad.sum()), float((err / want).max()))


@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("k,n", ((64, 64), (40, 24), (96, 136), (300, 8)))
@pytest.mark.parametrize("segments", (3, 1300, 2600))
def test_gradient_of_a_long_segment_among_many(dtype, k, n, segments):
    """Short segments, empty ones and two long ones, each before and after the other kind."""
    torch, sr = mods()
    rng = np.random.default_rng(segments + k)
    lens = rng.integers(0, 4, size=segments)
    lens[segments // 3], lens[-1] = 300_000, 100_001
    off = 7 + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    g = torch.Generator(device="cuda")
    g.manual_seed(k)
    rows = int(off[-1]) + 3
    x, dy = positive(g, (rows, k), dtype, 0.25), positive(g, (rows, n), dtype, 0.25)
    do = torch.from_numpy(off).cuda()
    got = sr.seg_matmul_grad_w(x, dy, do)
    for s in [segments // 3, segments - 1] + [int(i) for i in rng.integers(0, segments, 20)]:
        at = slice(int(off[s]), int(off[s + 1]))
        want = x[at].double().t() @ dy[at].double()
        if lens[s] == 0:
            assert bool((got[s] == 0).all())
        else:
            check(got[s], want, dtype, (k, n, segments, s))
    assert torch.equal(got, sr.seg_matmul_grad_w(x, dy, do))
    # every segment, against the one sum in float32 that is kept rounded
    full = sr.seg_matmul_grad_w(x, dy, do, out_dtype=torch.float32)
    assert bool(((got.float() - full).abs() <= (HALF_UNIT[dtype] + DRIFT) * full + 2.0 ** -24).all())
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("rows,k,n", ((5, 131_080, 72), (300, 70_000, 40), (300, 262_144, 64), (100, 1_048_576, 64), (2000, 65_600, 264), (700, 40_001, 1288)))
@pytest.mark.parametrize("trans", (False, True))
def test_long_rows(dtype, rows, k, n, trans):
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(k + n)
    off = np.array([2, rows // 2, rows // 2, rows - 1])
    x = positive(g, (rows, k), dtype, 0.125)
    w = positive(g, (3, n, k) if trans else (3, k, n), dtype, 0.125)
    out = torch.full((rows, n + 8), 7.0, dtype=x.dtype, device="cuda")
    got = sr.seg_matmul(x, w, torch.from_numpy(off).cuda(), transpose_w=trans, out=out[:, :n])
    for s in (0, 2):
        want = torch.zeros(int(off[s + 1] - off[s]), n, dtype=torch.float64, device="cuda")
        for i in range(0, k, 16384):
            ws = w[s, :, i:i + 16384].double().t() if trans else w[s, i:i + 16384].double()
            want += x[int(off[s]):int(off[s + 1]), i:i + 16384].double() @ ws
        check(got[int(off[s]):int(off[s + 1])], want, dtype, (rows, k, n, s))
    assert bool((got[:2] == 0).all()) and bool((got[rows - 1:] == 0).all()) and bool((out[:, n:] == 7).all())
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("lens,k,n,rank", (([1, 1, 1], 131_080, 72, 8), ([40, 100, 33], 70_000, 136, 16), ([300, 200, 20], 65_600, 264, 40)))
def test_adapters_of_long_rows(dtype, lens, k, n, rank):
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(k + n)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    rows = int(off[-1])
    x, w = positive(g, (rows, k), dtype, 0.125), positive(g, (n, k), dtype, 0.0625)
    a, b = positive(g, (2, rank, k), dtype, 0.0625), positive(g, (2, n, rank), dtype, 1.0 / rank)
    ids, do = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda"), torch.from_numpy(off).cuda()

    def want_of(b):
        y, u = torch.zeros(rows, n, dtype=torch.float64, device="cuda"), torch.zeros(2, rows, rank, dtype=torch.float64, device="cuda")
        for i in range(0, k, 16384):
            part = x[:, i:i + 16384].double()
            y += part @ w[:, i:i + 16384].double().t()
            u += part @ a[:, :, i:i + 16384].double().transpose(1, 2)
        for s, l in enumerate(ids.tolist()):
            if l >= 0:
                at = slice(int(off[s]), int(off[s + 1]))
                y[at] += u[l, at] @ b[l].double().t()
        return y
    got = sr.seg_lora(x, w, a, b, do, ids)
    # (the inner products and the sum drift, both by less than DRIFT)
    err = (got.double() - want_of(b)).abs() / want_of(b)
    assert float(err.max()) <= HALF_UNIT[dtype] + 2 * DRIFT, float(err.max())
    bad = b.clone()
    bad[1, 3, 0], bad[0, 5, 1] = float("nan"), float("inf")
    again = sr.seg_lora(x, w, a, bad, do, ids)
    y = want_of(bad)
    fine = torch.isfinite(y)
    assert torch.equal(again[fine], got[fine]) and torch.equal(torch.isnan(again), torch.isnan(y)) and torch.equal(torch.isposinf(again), torch.isposinf(y))
    assert sr.device_status() == 0
