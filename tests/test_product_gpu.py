"""The products over segments' rows (seg_matmul, seg_matmul_grad_w, seg_lora)
against the formulas in 64 bits.

Tolerance, from the operators' documented error: an output of n terms is
within (n * 2^-24 + 2^-20) * sum(|terms|) of the exact sum before it is
rounded once to its type (2^-24 of its size for float32, 2^-11 for float16
and 2^-8 for bfloat16 are whole units of that rounding; half a unit is the
error, and a rounding that the earlier error tips over costs no more than
the other half).  float16 also has a smallest step of 2^-24."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

TYPES = ("bfloat16", "float16", "float32")
UNIT = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11, "float32": 2.0 ** -24}


def mods():
    import torch
    import segmented_reduction_csr_gb300 as sr
    return torch, sr


def lengths_of(kind, rng):
    if kind == "mixed":         # both sides of the tile sizes, empty ones, single rows
        return [0, 1, 15, 16, 17, 0, 0, 63, 64, 65, 127, 128, 129, 1, 255, 256, 257, 2, 300, 0]
    if kind == "one":
        return [1]
    if kind == "empty":
        return [0, 0, 0]
    if kind == "single rows":
        return [1] * 37
    if kind == "skewed":
        return [3, 1500, 0, 9, 40]
    return list(rng.integers(0, 9, size=2500))       # "many": more segments than rows in a tile


def case(kind, seed, before=0, after=0, odt=None):
    torch, _ = mods()
    rng = np.random.default_rng(seed)
    lens = lengths_of(kind, rng)
    off = before + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    rows = int(off[-1]) + after
    do = torch.from_numpy(off).cuda()
    if odt == "uint32":
        do = torch.from_numpy(off.astype(np.int32)).cuda().view(torch.uint32)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return off, rows, do, g


def normal(g, shape, dtype, scale=1.0):
    torch, _ = mods()
    t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0, scale, generator=g)
    return t.to(getattr(torch, dtype))


def check(got, want, absum, terms, where, unit=None):
    torch, _ = mods()
    name = str(got.dtype).replace("torch.", "")
    tol = (unit or UNIT[name]) * want.abs() + (terms * 2.0 ** -24 + 2.0 ** -20) * absum
    if name == "float16":
        tol = tol + 2.0 ** -24
    err = (got.double() - want).abs()
    bad = ~(err <= tol)          # NaN counts as bad
    assert not bool(bad.any()), (where, int(bad.sum()), float(err.max()), float((err / (tol + 1e-300)).max()))


def ref_forward(x, w, off, trans):
    torch, _ = mods()
    n = w.shape[1] if trans else w.shape[2]
    y = torch.zeros(x.shape[0], n, dtype=torch.float64, device="cuda")
    a = torch.zeros_like(y)
    for s in range(len(off) - 1):
        if off[s + 1] > off[s]:
            xs = x[off[s]:off[s + 1]].double()
            ws = w[s].double().t() if trans else w[s].double()
            y[off[s]:off[s + 1]] = xs @ ws
            a[off[s]:off[s + 1]] = xs.abs() @ ws.abs()
    return y, a


def ref_grad(x, dy, off):
    torch, _ = mods()
    w = torch.zeros(len(off) - 1, x.shape[1], dy.shape[1], dtype=torch.float64, device="cuda")
    a = torch.zeros_like(w)
    for s in range(len(off) - 1):
        xs, ds = x[off[s]:off[s + 1]].double(), dy[off[s]:off[s + 1]].double()
        w[s] = xs.t() @ ds
        a[s] = xs.abs().t() @ ds.abs()
    return w, a


SIZES = [(64, 64), (1, 1), (7, 5), (16, 128), (63, 129), (65, 127), (72, 136), (200, 300), (256, 8), (8, 256), (520, 264), (136, 1104)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("trans", (False, True))
@pytest.mark.parametrize("k,n", SIZES)
def test_forward_sizes(dtype, trans, k, n):
    torch, sr = mods()
    off, rows, do, g = case("mixed", 1000 * k + n)
    x = normal(g, (rows, k), dtype)
    w = normal(g, (len(off) - 1, n, k) if trans else (len(off) - 1, k, n), dtype)
    got = sr.seg_matmul(x, w, do, transpose_w=trans)
    y, a = ref_forward(x, w, off, trans)
    check(got, y, a, k, (dtype, trans, k, n))
    assert torch.equal(got, sr.seg_matmul(x, w, do, transpose_w=trans))     # repeats bit for bit
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("trans", (False, True))
@pytest.mark.parametrize("k,n", ((64, 64), (63, 5), (128, 40), (600, 64), (1100, 24)))
def test_many_rows_of_few_columns(dtype, trans, k, n):
    """Tiles of many rows whose lanes are half used or less; sums of one block and of several pieces."""
    torch, sr = mods()
    lens = [9001, 0, 1, 128, 8209, 130, 4000]
    off = 3 + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    g = torch.Generator(device="cuda")
    g.manual_seed(k + n)
    x = normal(g, (int(off[-1]) + 5, k), dtype)
    w = normal(g, (len(lens), n, k) if trans else (len(lens), k, n), dtype)
    out = torch.full((x.shape[0], n + 12), 7.0, dtype=x.dtype, device="cuda")
    got = sr.seg_matmul(x, w, torch.from_numpy(off).cuda(), transpose_w=trans, out=out[:, 4:4 + n])
    y, a = ref_forward(x, w, off, trans)
    check(got, y, a, k, (dtype, trans, k, n))
    assert bool((out[:, :4] == 7).all()) and bool((out[:, 4 + n:] == 7).all())      # nothing beside the columns
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k,n", SIZES)
def test_grad_sizes(dtype, k, n):
    torch, sr = mods()
    off, rows, do, g = case("mixed", 2000 * k + n)
    x, dy = normal(g, (rows, k), dtype), normal(g, (rows, n), dtype)
    w, a = ref_grad(x, dy, off)
    for out_dtype in {x.dtype, torch.float32}:
        got = sr.seg_matmul_grad_w(x, dy, do, out_dtype=out_dtype)
        check(got, w, a, 300, (dtype, k, n, out_dtype))
        assert torch.equal(got, sr.seg_matmul_grad_w(x, dy, do, out_dtype=out_dtype))
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ("one", "empty", "single rows", "skewed", "many"))
@pytest.mark.parametrize("odt", ("int64", "uint32"))
def test_segment_shapes(dtype, kind, odt):
    torch, sr = mods()
    off, rows, do, g = case(kind, 77, before=5, after=9, odt=odt)
    k, n = (24, 40) if kind == "many" else (136, 200)
    x, dy = normal(g, (rows, k), dtype), normal(g, (rows, n), dtype)
    # rows in no segment hold NaN: they must reach nothing
    x[:5] = float("nan")
    dy[:5] = float("inf")
    x[int(off[-1]):] = float("inf")
    dy[int(off[-1]):] = float("nan")
    w = normal(g, (len(off) - 1, k, n), dtype)
    for s in range(len(off) - 1):
        if off[s] == off[s + 1]:
            w[s] = float("nan")
    got = sr.seg_matmul(x, w, do)
    y, a = ref_forward(x, w, off, False)
    check(got, y, a, k, (dtype, kind))
    got = sr.seg_matmul_grad_w(x, dy, do)
    y, a = ref_grad(x, dy, off)
    check(got, y, a, int(max(np.diff(off))), (dtype, kind, "grad"))
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_values_that_are_not_finite_stay_in_their_row_and_segment(dtype):
    torch, sr = mods()
    off, rows, do, g = case("mixed", 5)
    k, n = 136, 72
    x, dy = normal(g, (rows, k), dtype), normal(g, (rows, n), dtype)
    w = normal(g, (len(off) - 1, k, n), dtype)
    bad = [int(off[9]) + 3, int(off[14])]      # one row of two segments
    for r in bad:
        x[r, 11] = float("inf")
        dy[r, 3] = float("nan")
    got = sr.seg_matmul(x, w, do)
    fine = torch.ones(rows, dtype=torch.bool, device="cuda")
    fine[bad] = False
    assert bool(torch.isfinite(got[fine]).all()) and not bool(torch.isfinite(got[bad]).any())
    got = sr.seg_matmul_grad_w(x, dy, do)
    hit = [int(np.searchsorted(off, r, side="right") - 1) for r in bad]
    for s in range(len(off) - 1):
        assert bool(torch.isfinite(got[s]).all()) == (s not in hit), s


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_alignment(dtype):
    torch, sr = mods()
    off, rows, do, g = case("mixed", 6)
    s = len(off) - 1
    k, n = 72, 40
    for xcols, xat, wcols, wat, ocols, oat in ((96, 8, 64, 16, 56, 8), (75, 1, 43, 2, 47, 5), (73, 0, 40, 0, 41, 1)):
        x = normal(g, (rows, xcols), dtype)[:, xat:xat + k]
        w = normal(g, (s, k + 3, wcols), dtype)[:, 1:1 + k, wat:wat + n]
        big = torch.full((rows + 2, ocols), 7.0, device="cuda").to(x.dtype)
        out = big[1:-1, oat:oat + n]
        sr.seg_matmul(x, w, do, out=out)
        y, a = ref_forward(x, w, off, False)
        check(out, y, a, k, (dtype, xcols))
        wt = normal(g, (s, n + 1, xcols), dtype)[:, :n, xat:xat + k]
        sr.seg_matmul(x, wt, do, transpose_w=True, out=out)
        y, a = ref_forward(x, wt, off, True)
        check(out, y, a, k, (dtype, xcols, "transposed"))
        keep = torch.ones_like(big, dtype=torch.bool)
        keep[1:-1, oat:oat + n] = False
        assert bool((big[keep] == 7.0).all())            # nothing outside the view is written
        dy = normal(g, (rows, wcols), dtype)[:, wat:wat + n]
        got = sr.seg_matmul_grad_w(x, dy, do)
        y, a = ref_grad(x, dy, off)
        check(got, y, a, 300, (dtype, xcols, "grad"))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,segments,k,n", ((2, 8, 2048, 264), (128, 64, 520, 256), (2000, 3, 1032, 384)))
def test_few_rows_and_long_sums(dtype, rows, segments, k, n):
    """Where the sum is long and the output small the work is split along the sum."""
    torch, sr = mods()
    rng = np.random.default_rng(rows)
    lens = rng.multinomial(rows, np.ones(segments) / segments)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    do = torch.from_numpy(off).cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x, w = normal(g, (rows, k), dtype), normal(g, (segments, k, n), dtype, k ** -0.5)
    y, a = ref_forward(x, w, off, False)
    for rep in range(3):
        check(sr.seg_matmul(x, w, do), y, a, k, (dtype, rows, rep))
    # a long sum of the weight gradient: few columns, many rows
    big = normal(g, (60000, 24), dtype)
    dy = normal(g, (60000, 16), dtype)
    boff = np.array([0, 10, 10, 51000, 60000])
    y, a = ref_grad(big, dy, boff)
    for rep in range(3):
        check(sr.seg_matmul_grad_w(big, dy, torch.from_numpy(boff).cuda(), out_dtype=torch.float32), y, a, 51000, (dtype, rep))
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("trans", (False, True))
@pytest.mark.parametrize("rows,k,n", ((1, 63, 65), (3, 1023, 130), (7, 513, 301), (2, 200, 5)))
def test_odd_rows_of_few_of_many_matrices(dtype, trans, rows, k, n):
    """Operands that tensor copies cannot take and most matrices in no use (those hold NaN)."""
    torch, sr = mods()
    segments = 16
    rng = np.random.default_rng(k)
    lens = np.zeros(segments, dtype=np.int64)
    lens[rng.choice(segments, size=min(rows, 3), replace=False)] = 1
    lens[np.flatnonzero(lens)[-1]] += rows - lens.sum()
    off = np.concatenate([[0], np.cumsum(lens)]) + 1
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    x = normal(g, (rows + 2, k), dtype)
    w = normal(g, (segments, n, k) if trans else (segments, k, n), dtype, k ** -0.5)
    w[torch.from_numpy(lens == 0).cuda()] = float("nan")
    got = sr.seg_matmul(x, w, torch.from_numpy(off).cuda(), transpose_w=trans)
    y, a = ref_forward(x, w, off, trans)
    check(got, y, a, k, (dtype, trans, rows, k, n))
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_positive_values(dtype):
    """Sums that only grow show a bias in how they are added."""
    torch, sr = mods()
    off, rows, do, g = case("skewed", 8)
    x, w = normal(g, (rows, 4096), dtype).abs(), normal(g, (len(off) - 1, 4096, 72), dtype).abs()
    y, a = ref_forward(x, w, off, False)
    check(sr.seg_matmul(x, w, do), y, a, 4096, dtype)
    dy = normal(g, (rows, 72), dtype).abs()
    y, a = ref_grad(x, dy, off)
    check(sr.seg_matmul_grad_w(x, dy, do), y, a, 1500, (dtype, "grad"))


def test_zero_sizes():
    torch, sr = mods()
    off = torch.tensor([0, 2, 2], device="cuda")
    x = torch.ones(2, 0, device="cuda")
    assert bool((sr.seg_matmul(x, torch.ones(2, 0, 3, device="cuda"), off) == 0).all())
    assert sr.seg_matmul(torch.ones(2, 4, device="cuda"), torch.ones(2, 4, 0, device="cuda"), off).shape == (2, 0)
    none = torch.zeros(3, dtype=torch.int64, device="cuda")
    e = torch.ones(0, 4, device="cuda")
    assert sr.seg_matmul(e, torch.ones(2, 4, 3, device="cuda"), none).shape == (0, 3)
    assert bool((sr.seg_matmul_grad_w(e, torch.ones(0, 3, device="cuda"), none) == 0).all())
    y = sr.seg_matmul(torch.ones(3, 4, device="cuda"), torch.ones(0, 4, 5, device="cuda"), none[:1])
    assert y.shape == (3, 5) and bool((y == 0).all())        # no segments: every row is in none
    assert sr.seg_matmul_grad_w(torch.ones(3, 4, device="cuda"), torch.ones(3, 5, device="cuda"), none[:1]).shape == (0, 4, 5)


def test_malformed_offsets_touch_nothing_else():
    """Offsets past the rows or decreasing: unspecified results, but nothing outside the output is written."""
    torch, sr = mods()
    x = torch.ones(300, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(4, 64, 128, device="cuda", dtype=torch.bfloat16)
    for off in ([0, 200, 100, 900, 50], [-7, 400, 10, 20, 1 << 40], [300, 300, 0, 0, 0]):
        big = torch.full((302, 128), 7.0, device="cuda", dtype=torch.bfloat16)
        sr.seg_matmul(x, w, torch.tensor(off, device="cuda"), out=big[1:-1])
        grad = torch.full((6, 64, 128), 7.0, device="cuda")
        sr.seg_matmul_grad_w(x, big[1:-1], torch.tensor(off, device="cuda"), out=grad[1:-1])
        torch.cuda.synchronize()
        assert bool((big[0] == 7).all() and (big[-1] == 7).all() and (grad[0] == 7).all() and (grad[-1] == 7).all())
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_segment_matmul_gradients(dtype):
    """Against the formula, and (the function is linear in each argument) against differences."""
    torch, sr = mods()
    off, rows, do, g = case("mixed", 9)
    k, n = 40, 56
    x = normal(g, (rows, k), dtype).requires_grad_()
    w = normal(g, (len(off) - 1, k, n), dtype).requires_grad_()
    t = normal(g, (rows, n), dtype)
    y = sr.segment_matmul(x, w, do)
    dx, dw = torch.autograd.grad(y, (x, w), t)
    want, a = ref_forward(t, w.detach(), off, True)
    check(dx, want, a, n, (dtype, "dx"))
    want, a = ref_grad(x.detach(), t, off)
    check(dw, want, a, 300, (dtype, "dw"))
    if dtype == "float32":
        for arg, d in ((x, dx), (w, dw)):
            step = normal(g, arg.shape, dtype)
            lo, hi = ([v.detach() + sign * step if v is arg else v.detach() for v in (x, w)] for sign in (-0.5, 0.5))
            diff = ((sr.segment_matmul(*hi, do).double() - sr.segment_matmul(*lo, do).double()) * t.double()).sum()
            want = (d.double() * step.double()).sum()
            # each output is off by 1e-5 of its terms at most, and the two sums hold rows * n of them
            scale = (sr.seg_matmul(x.detach().abs(), w.detach().abs(), do).double() * t.double().abs()).sum()
            assert abs(float(diff - want)) <= 4e-5 * float(scale)
    # a sum's gradient comes with strides of 0; only what is asked for is computed
    dx, = torch.autograd.grad(sr.segment_matmul(x, w.detach(), do).sum(), (x,))
    want, a = ref_forward(torch.ones(rows, n, device="cuda", dtype=x.dtype), w.detach(), off, True)
    check(dx, want, a, n, (dtype, "sum"))


def ref_lora(x, w, a, b, off, ids, scale):
    y = x.double() @ w.double().t()
    m = x.double().abs() @ w.double().abs().t()
    for s in range(len(off) - 1):
        i = ids[s]
        if 0 <= i < a.shape[0] and off[s + 1] > off[s]:
            at = slice(int(off[s]), int(off[s + 1]))
            f = 1.0 if scale is None else float(scale[i])
            y[at] += f * (x[at].double() @ a[i].double().t()) @ b[i].double().t()
            m[at] += abs(f) * (x[at].double().abs() @ a[i].double().abs().t()) @ b[i].double().abs().t()
    return y, m


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ("one", "single rows", "mixed", "empty", "skewed"))
@pytest.mark.parametrize("k,n,rank", ((64, 128, 16), (200, 72, 8), (520, 300, 12), (63, 65, 1), (256, 264, 33), (128, 136, 64), (96, 40, 128)))
def test_lora(dtype, kind, k, n, rank):
    torch, sr = mods()
    off, rows, do, g = case(kind, 11 * k + rank, before=3, after=2)
    adapters = 5
    x, w = normal(g, (rows, k), dtype), normal(g, (n, k), dtype, k ** -0.5)
    a, b = normal(g, (adapters, rank, k), dtype, k ** -0.5), normal(g, (adapters, n, rank), dtype, rank ** -0.5)
    rng = np.random.default_rng(k + rank)
    ids = rng.integers(-1, adapters + 1, size=len(off) - 1)       # -1 and 5: no adapter
    ids[0] = 2
    used = set(ids.tolist())
    for i in range(adapters):
        if i not in used:                # an adapter that nobody uses may hold anything
            a[i] = float("nan")
            b[i] = float("inf")
    scale = torch.from_numpy(rng.uniform(-2, 2, adapters).astype(np.float32)).cuda()
    adapter = torch.from_numpy(ids.astype(np.int32)).cuda()
    for sc in (scale, None):
        got = sr.seg_lora(x, w, a, b, do, adapter, sc)
        y, m = ref_lora(x, w, a, b, off, ids, sc)
        check(got, y, m, k + rank, (dtype, kind, k, n, rank))
        assert torch.equal(got, sr.seg_lora(x, w, a, b, do, adapter, sc))
    assert sr.device_status() == 0


def test_lora_strides_and_no_adapters():
    torch, sr = mods()
    off, rows, do, g = case("mixed", 12)
    k, n, rank = 72, 88, 16
    x = normal(g, (rows, 96), "bfloat16")[:, 9:9 + k]
    w = normal(g, (n, 80), "bfloat16")[:, :k]
    a, b = normal(g, (2, rank, k), "bfloat16"), normal(g, (2, n, rank), "bfloat16")
    ids = np.arange(len(off) - 1) % 3 - 1
    adapter = torch.from_numpy(ids.astype(np.int32)).cuda()
    big = torch.full((rows, n + 6), 7.0, device="cuda", dtype=torch.bfloat16)
    sr.seg_lora(x, w, a, b, do, adapter, out=big[:, 3:3 + n])
    y, m = ref_lora(x, w, a, b, off, ids, None)
    check(big[:, 3:3 + n], y, m, k + rank, "strides")
    assert bool((big[:, :3] == 7).all() and (big[:, 3 + n:] == 7).all())
    got = sr.seg_lora(x, w, a[:0], b[:0], do, adapter)
    y, m = ref_lora(x, w, a[:0], b[:0], off, ids, None)
    check(got, y, m, k, "no adapters")


def test_products_on_other_streams():
    """Each (device, stream) has its own scratch: unordered calls on four streams do not disturb one another."""
    torch, sr = mods()
    off, rows, do, g = case("skewed", 13)
    x, w = normal(g, (rows, 1024), "bfloat16"), normal(g, (len(off) - 1, 1024, 136), "bfloat16", 1 / 32)
    dy = normal(g, (rows, 136), "bfloat16")
    small = x[:3].contiguous()
    so = torch.tensor([0, 1, 2, 3, 3, 3], device="cuda")
    a, b = normal(g, (2, 16, 1024), "bfloat16", 1 / 32), normal(g, (2, 136, 16), "bfloat16")
    adapter = torch.tensor([0, 1, -1, 0, 1], dtype=torch.int32, device="cuda")
    shared = w[0].t().contiguous()
    calls = [lambda: sr.seg_matmul(x, w, do), lambda: sr.seg_matmul(small, w, so),
             lambda: sr.seg_matmul_grad_w(x, dy, do), lambda: sr.seg_lora(x, shared, a, b, do, adapter)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for rep in range(3):
        for st, c in zip(streams, calls):
            with torch.cuda.stream(st):
                got.append(c())
    torch.cuda.synchronize()
    for i, v in enumerate(got):
        assert torch.equal(v, want[i % 4])
    assert sr.device_status() == 0


def test_offsets_past_32_bits_of_elements():
    """Rows whose element offsets pass 2^31: the last segment's rows against the formula."""
    torch, sr = mods()
    rows, k, n = 2_100_000, 1032, 24
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x[-700:] = normal(g, (700, k), "bfloat16")
    w = normal(g, (3, k, n), "bfloat16", 1 / 32)
    off = np.array([0, 5, rows - 600, rows])
    got = sr.seg_matmul(x, w, torch.from_numpy(off).cuda())
    y, a = ref_forward(x[-700:], w, np.array([0, 0, 100, 700]), False)
    check(got[-700:], y, a, k, "large rows")
    assert bool((got[:-700] == 0).all())
    dy = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    dy[-650:] = normal(g, (650, n), "bfloat16")
    got = sr.seg_matmul_grad_w(x, dy, torch.from_numpy(off).cuda())
    y, a = ref_grad(x[-650:], dy[-650:], np.array([0, 0, 50, 650]))
    check(got, y, a, 650, "large rows, grad")


def test_refusals():
    torch, sr = mods()
    x = torch.ones(4, 8, device="cuda")
    w = torch.ones(2, 8, 16, device="cuda")
    off = torch.tensor([0, 2, 4], device="cuda")
    ok = dict(x=x, w=w, offsets=off)
    for change, error in ((dict(x=x.double()), TypeError), (dict(x=x.int()), TypeError), (dict(w=w.half()), TypeError),
                          (dict(x=x.cpu()), ValueError), (dict(w=w.cpu()), ValueError), (dict(offsets=off.cpu()), ValueError),
                          (dict(offsets=off.int()), TypeError), (dict(x=x[0]), ValueError), (dict(w=w[0]), ValueError),
                          (dict(w=w[:, :7]), ValueError), (dict(w=w[:1]), ValueError), (dict(x=x.t()), ValueError),
                          (dict(x=torch.ones(8, 4, device="cuda").t()), ValueError),
                          (dict(w=torch.ones(2, 16, 8, device="cuda").transpose(1, 2)), ValueError),
                          (dict(x=x[:1].expand(4, 8)), ValueError),
                          (dict(out=torch.ones(4, 15, device="cuda")), ValueError),
                          (dict(out=torch.ones(4, 16, device="cuda").half()), TypeError),
                          (dict(out=torch.ones(16, 4, device="cuda").t()), ValueError),
                          (dict(w=w[:1].expand(2, 8, 16)), sr.SegReduceError)):
        with pytest.raises(error):
            sr.seg_matmul(**{**ok, **change})
    dy = torch.ones(4, 16, device="cuda")
    for args, kw in (((x, dy[:3], off), {}), ((x, dy.half(), off), {}), ((x, dy, off), dict(out_dtype=torch.float16)),
                     ((x, dy, off), dict(out=torch.ones(2, 16, 8, device="cuda").transpose(1, 2)))):
        with pytest.raises((ValueError, TypeError)):
            sr.seg_matmul_grad_w(*args, **kw)
    shared, a, b = torch.ones(16, 8, device="cuda"), torch.ones(3, 4, 8, device="cuda"), torch.ones(3, 16, 4, device="cuda")
    ids = torch.zeros(2, dtype=torch.int32, device="cuda")
    sr.seg_lora(x, shared, a, b, off, ids)
    for args in ((x, shared, a, b[:2], off, ids), (x, shared, a, b, off, ids.long()), (x, shared, a, b, off, ids[:1]),
                 (x, shared[:, :7], a, b, off, ids), (x, shared, a.half(), b, off, ids),
                 (x, shared, a, b, off, ids, torch.ones(3, device="cuda").double()),
                 (x, shared, a, b, off, ids, torch.ones(2, device="cuda")),
                 (x, shared, a, torch.ones(3, 4, 16, device="cuda").transpose(1, 2), off, ids)):
        with pytest.raises((ValueError, TypeError)):
            sr.seg_lora(*args)
    with pytest.raises(sr.SegReduceError):      # a rank above the limit
        sr.seg_lora(x, shared, torch.ones(1, 129, 8, device="cuda"), torch.ones(1, 16, 129, device="cuda"), off, ids)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rank", (8, 12, 40, 128))
def test_lora_runs_of_rows(dtype, rank):
    """Tiles of one adapter, of a few runs (an adapter twice among them) and of many, in one call and across its tiles."""
    torch, sr = mods()
    lens = [500, 20, 20, 300, 1, 1, 1, 2, 1, 1, 130, 0, 64] + [1] * 60 + [700]
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64) + 2
    rows = int(off[-1]) + 5
    do = torch.from_numpy(off).cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(rank)
    k, n, adapters = 1104, 264, 4
    x, w = normal(g, (rows, k), dtype), normal(g, (n, k), dtype, k ** -0.5)
    a, b = normal(g, (adapters, rank, k), dtype, k ** -0.5), normal(g, (adapters, n, rank), dtype, rank ** -0.5)
    ids = np.arange(len(lens)) % (adapters + 1) - 1
    ids[:4] = [1, 3, 1, -1]
    adapter = torch.from_numpy(ids.astype(np.int32)).cuda()
    scale = torch.tensor([0.5, -3.0, 1.0, 40.0], device="cuda")
    got = sr.seg_lora(x, w, a, b, do, adapter, scale)
    y, m = ref_lora(x, w, a, b, off, ids, scale)
    check(got, y, m, k + rank, (dtype, rank))
    for rep in range(3):
        assert torch.equal(got, sr.seg_lora(x, w, a, b, do, adapter, scale))
    assert sr.device_status() == 0


def test_lora_many_requests():
    """More requests than a CTA keeps offsets of, one row or none each."""
    torch, sr = mods()
    off, rows, do, g = case("many", 14)
    k, n, rank, adapters = 72, 136, 16, 7
    x, w = normal(g, (rows, k), "bfloat16"), normal(g, (n, k), "bfloat16", k ** -0.5)
    a, b = normal(g, (adapters, rank, k), "bfloat16", k ** -0.5), normal(g, (adapters, n, rank), "bfloat16")
    ids = np.random.default_rng(1).integers(-1, adapters, size=len(off) - 1)
    adapter = torch.from_numpy(ids.astype(np.int32)).cuda()
    got = sr.seg_lora(x, w, a, b, do, adapter)
    y, m = ref_lora(x, w, a, b, off, ids, None)
    check(got, y, m, k + rank, "many")
    bad = do.clone()
    bad[3], bad[5], bad[700] = 1 << 40, -9, 0        # malformed: unspecified, but nothing else is written
    big = torch.full((rows + 2, n), 7.0, device="cuda", dtype=torch.bfloat16)
    sr.seg_lora(x, w, a, b, bad, adapter, out=big[1:-1])
    torch.cuda.synchronize()
    assert bool((big[0] == 7).all() and (big[-1] == 7).all()) and sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_large_tiles(dtype):
    """Several tiles of rows, lanes and blocks of every kind, and a segment in hundreds of parts."""
    torch, sr = mods()
    rng = np.random.default_rng(5)
    lens = rng.multinomial(9000, [0.5, 0.3, 0.1, 0.05, 0.05])
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    do = torch.from_numpy(off).cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    k, n = 584, 1288
    x, w, dy = normal(g, (9000, k), dtype), normal(g, (5, k, n), dtype, k ** -0.5), normal(g, (9000, n), dtype)
    y, a = ref_forward(x, w, off, False)
    check(sr.seg_matmul(x, w, do), y, a, k, dtype)
    y, a = ref_forward(dy, w, off, True)
    check(sr.seg_matmul(dy, w, do, transpose_w=True), y, a, n, (dtype, "dx"))
    y, a = ref_grad(x, dy, off)
    check(sr.seg_matmul_grad_w(x, dy, do, out_dtype=torch.float32), y, a, int(max(lens)), (dtype, "dw"))
    long_x, long_dy = normal(g, (400000, 40), dtype), normal(g, (400000, 72), dtype)
    loff = np.array([0, 3, 399000, 400000])
    y, a = ref_grad(long_x, long_dy, loff)
    got = sr.seg_matmul_grad_w(long_x, long_dy, torch.from_numpy(loff).cuda(), out_dtype=torch.float32)
    check(got, y, a, 398997, (dtype, "long"))
    assert sr.device_status() == 0


def test_products_in_a_graph():
    """Captured and replayed, the calls give what they give outside."""
    torch, sr = mods()
    off, rows, do, g = case("skewed", 15)
    x, w = normal(g, (rows, 512), "bfloat16"), normal(g, (len(off) - 1, 512, 136), "bfloat16", 0.05)
    dy = normal(g, (rows, 136), "bfloat16")
    shared = normal(g, (136, 512), "bfloat16", 0.05)
    a, b = normal(g, (3, 16, 512), "bfloat16", 0.05), normal(g, (3, 136, 16), "bfloat16")
    adapter = torch.tensor([0, 1, 2, -1, 0], dtype=torch.int32, device="cuda")
    one = torch.arange(6, device="cuda")
    calls = [lambda: sr.seg_matmul(x, w, do), lambda: sr.seg_matmul_grad_w(x, dy, do), lambda: sr.seg_lora(x, shared, a, b, do, adapter),
             lambda: sr.seg_lora(x[:5], shared, a, b, one, adapter)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()        # whose scratch is first needed while it captures
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = [c() for c in calls]
        for rep in range(3):
            for v in got:
                v.zero_()
            graph.replay()
            stream.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(want, got)), rep
            for c, u in zip(calls, want):       # calls of the stream between the replays
                assert torch.equal(c(), u)
            if rep == 0:                        # and one that needs far more scratch
                big, many = normal(g, (200000, 128), "bfloat16"), normal(g, (200000, 136), "bfloat16")
                sr.seg_matmul_grad_w(big, many, torch.tensor([0, 200000], device="cuda"))
    assert sr.device_status() == 0


def test_example_layer():
    torch, sr = mods()
    from examples import expert_layer as ex
    losses = ex.train(tokens=513, width=128, hidden=136, experts=7, steps=4)
    assert losses[-1] < losses[0] and all(np.isfinite(losses))
    assert losses == ex.train(tokens=513, width=128, hidden=136, experts=7, steps=4)     # every sum has a fixed order
    prompts, tokens, offsets = ex.serve()
    same = prompts[offsets[1:] - 1].double()
    # the same sums in another order, then rounded to bfloat16
    assert bool(((same - tokens.double()).abs() <= 2.0 ** -8 * same.abs() + 1e-3).all())
