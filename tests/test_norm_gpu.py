"""Layer norm over the rows of segments (seg_layer_norm, seg_layer_norm_grad,
segment_layer_norm) against the formulas in 64 bits.

Tolerances, with u = 2^-24 and F columns.  A thread adds at most F / 256 or 64
values in a row, then a tree of 10 levels: sums are within c = (F / 256 + 80) u
of their terms' sizes.  So the mean is within dm = c mean|x|, the variance
within 2 c of itself and dm^2, rstd within c + 4 u + dm^2 rstd^2, and
y = z w + b within |w| (rstd dm + |z| (c + 8 u + dm^2 rstd^2)) + 2 u (|w z| +
|b|) before its rounding.  Gradients are compared at the mean and rstd that the
forward pass gave: z is within 3 u of itself, the row's two sums within c + 8 u
of their terms' sizes, and the sums over n rows within (n / 300 + 200) u (a block
has at most n / 300 + 32 of a segment's rows, a thread at most those).  A
rounding adds half a step."""
import numpy as np
import pytest

from tests.test_gated_gpu import close
from tests.test_product_gpu import TYPES, case, lengths_of, mods, normal

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def segments_of(off, rows):
    """Segment of each row (-1: none); off None: one of all rows."""
    torch, _ = mods()
    if off is None:
        return torch.zeros(rows, dtype=torch.int64, device="cuda")
    at = np.arange(rows)
    s = np.searchsorted(off, at, side="right") - 1
    s[(s < 0) | (s >= len(off) - 1)] = -1
    return torch.from_numpy(s).cuda()


def rows_of(t, seg, f, fill):
    """The weights of each row in 64 bits; t None: `fill`."""
    torch, _ = mods()
    if t is None:
        return torch.full((len(seg), f), fill, dtype=torch.float64, device="cuda")
    t = t.double().reshape(-1, f)
    if t.shape[0] == 0:
        return torch.zeros(len(seg), f, dtype=torch.float64, device="cuda")
    return t[seg.clamp(min=0)]


def check_forward(got, x, weight, bias, off, eps, where):
    torch, _ = mods()
    y, mean, rstd = got
    f = x.shape[1]
    seg = segments_of(off, x.shape[0])
    none = seg < 0
    xs = torch.where(none[:, None], torch.zeros_like(x), x).double()
    c = (f / 256 + 80) * U
    m = xs.mean(1, keepdim=True)
    v = (xs - m).square().mean(1, keepdim=True)
    r = 1 / torch.sqrt(v + eps)
    dm = c * xs.abs().mean(1, keepdim=True)
    rel = c + 8 * U + dm.square() * r.square()
    z, w, b = (xs - m) * r, rows_of(weight, seg, f, 1.0), rows_of(bias, seg, f, 0.0)
    want = torch.where(none[:, None], torch.zeros_like(xs), z * w + b)
    close(y, want, w.abs() * (r * dm + z.abs() * rel) + 2 * U * ((w * z).abs() + b.abs()), where)
    if mean is not None:
        zero = torch.zeros_like(m[:, 0])
        close(mean, torch.where(none, zero, m[:, 0]), dm[:, 0], (where, "mean"))
        close(rstd, torch.where(none, zero, r[:, 0]), (r * rel)[:, 0], (where, "rstd"))


def check_grad(got, x, dy, mean, rstd, weight, off, where):
    torch, _ = mods()
    dx, dweight, dbias = got
    rows, f = x.shape
    seg = segments_of(off, rows)
    none = (seg < 0)[:, None]
    zero = torch.zeros(rows, f, dtype=torch.float64, device="cuda")
    xs, ds = torch.where(none, zero, x.double()), torch.where(none, zero, dy.double())
    m, r = mean.double()[:, None], rstd.double()[:, None]
    w = rows_of(weight, seg, f, 1.0)
    z, g = (xs - m) * r, ds * w
    c = (f / 256 + 88) * U
    m1, m2 = g.mean(1, keepdim=True), (g * z).mean(1, keepdim=True)
    if dx is not None:
        want = torch.where(none, zero, r * (g - m1 - z * m2))
        tol = r * (4 * U * (g.abs() + m1.abs() + (z * m2).abs()) + c * (g.abs().mean(1, keepdim=True) + z.abs() * (g * z).abs().mean(1, keepdim=True)))
        close(dx, want, tol, (where, "dx"))
    s = 1 if off is None else len(off) - 1
    part = (rows / 300 + 200) * U

    def total(t):
        return torch.zeros(s, f, dtype=torch.float64, device="cuda").index_add_(0, seg.clamp(min=0), torch.where(none, zero, t))
    if s == 0:
        return
    if dweight is not None:
        close(dweight.reshape(s, f), total(ds * z), part * total((ds * z).abs()), (where, "dweight"))
    if dbias is not None:
        close(dbias.reshape(s, f), total(ds), part * total(ds.abs()), (where, "dbias"))


def weights(g, s, f, wdtype):
    torch, _ = mods()
    shape = (f,) if s is None else (s, f)
    return normal(g, shape, wdtype, 0.5), normal(g, shape, wdtype)


WIDTHS = (1, 2, 7, 8, 16, 63, 64, 65, 128, 200, 256, 333, 512, 1000, 1024, 2048, 2050, 4096, 4100, 5000, 8192, 12288, 16384, 16392, 20000)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("f", WIDTHS)
def test_widths(dtype, f):
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(f)
    rows = 37 if f > 4096 else 301
    x = normal(g, (rows, f), dtype) + 0.5
    dy = normal(g, (rows, f), dtype)
    for wdtype in {dtype, "float32"}:
        w, b = weights(g, None, f, wdtype)
        got = sr.seg_layer_norm(x, w, b, with_stats=True)
        check_forward(got, x, w, b, None, 1e-5, (dtype, f, wdtype))
        assert torch.equal(got[0], sr.seg_layer_norm(x, w, b))
        grads = sr.seg_layer_norm_grad(x, dy, *got[1:], w)
        check_grad(grads, x, dy, *got[1:], w, None, (dtype, f, wdtype))
        assert all(torch.equal(p, q) for p, q in zip(grads, sr.seg_layer_norm_grad(x, dy, *got[1:], w)))      # bit for bit


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ("mixed", "one", "empty", "single rows", "skewed", "many"))
@pytest.mark.parametrize("f", (24, 136, 1100, 2048))
def test_segment_shapes(dtype, kind, f):
    torch, sr = mods()
    if kind == "many" and f > 136:
        f = 72
    off, rows, do, g = case(kind, 7 + f, before=5, after=9, odt="uint32" if f == 136 else None)
    x, dy = normal(g, (rows, f), dtype), normal(g, (rows, f), dtype)
    x[:5], dy[:5], x[int(off[-1]):], dy[int(off[-1]):] = float("nan"), float("inf"), float("inf"), float("nan")
    w, b = weights(g, len(off) - 1, f, "float32" if f == 24 else dtype)
    got = sr.seg_layer_norm(x, w, b, do, with_stats=True)
    check_forward(got, x, w, b, off, 1e-5, (dtype, kind, f))
    check_grad(sr.seg_layer_norm_grad(x, dy, *got[1:], w, do), x, dy, *got[1:], w, off, (dtype, kind, f))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("f", (4104, 6001, 9000, 12288, 20000))
def test_wide_rows_of_segments(dtype, f):
    """Rows of a block's threads, from shared memory, read again, and in tiles of columns."""
    torch, sr = mods()
    lens = [3, 0, 1, 150, 0, 97, 1, 0]
    off = 2 + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    g = torch.Generator(device="cuda")
    g.manual_seed(f)
    x, dy = normal(g, (int(off[-1]) + 3, f), dtype), normal(g, (int(off[-1]) + 3, f), dtype)
    x[:2], dy[-3:] = float("nan"), float("inf")
    w, b = weights(g, len(lens), f, "float32" if f == 9000 else dtype)
    do = torch.from_numpy(off).cuda()
    got = sr.seg_layer_norm(x, w, b, do, with_stats=True)
    check_forward(got, x, w, b, off, 1e-5, (dtype, f))
    check_grad(sr.seg_layer_norm_grad(x, dy, *got[1:], w, do), x, dy, *got[1:], w, off, (dtype, f))


def test_what_follows_the_gradients_in_a_stream_sees_them():
    """Segments that lie in one block's rows each leave the adding kernel nothing to wait for but the backward pass."""
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x, dy = normal(g, (60000, 256), "bfloat16"), normal(g, (60000, 256), "bfloat16")
    off = torch.arange(0, 60001, 2, device="cuda")
    w = normal(g, (30000, 256), "bfloat16")
    _, mean, rstd = sr.seg_layer_norm(x, w, None, off, with_stats=True)
    want = [t.clone() for t in sr.seg_layer_norm_grad(x, dy, mean, rstd, w, off)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [t.clone() for t in sr.seg_layer_norm_grad(x, dy, mean, rstd, w, off)]
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("f", (16, 64, 72))
def test_many_rows(dtype, f):
    """Chunks that begin, end and lie inside of segments; more segments than chunks and fewer."""
    torch, sr = mods()
    for lens in ([30011, 1, 0, 9000, 70000], [100000], list(lengths_of("many", np.random.default_rng(3))) * 3, [40] * 2000 + [5000] + [0] * 50 + [3] * 999):
        off = np.concatenate([[2], 2 + np.cumsum(lens)]).astype(np.int64)
        g = torch.Generator(device="cuda")
        g.manual_seed(f)
        x, dy = normal(g, (int(off[-1]) + 3, f), dtype), normal(g, (int(off[-1]) + 3, f), dtype)
        w, b = weights(g, len(lens), f, dtype)
        do = torch.from_numpy(off).cuda()
        got = sr.seg_layer_norm(x, w, b, do, with_stats=True)
        check_forward(got, x, w, b, off, 1e-5, (dtype, f, len(lens)))
        check_grad(sr.seg_layer_norm_grad(x, dy, *got[1:], w, do), x, dy, *got[1:], w, off, (dtype, f, len(lens)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("f", (1, 5, 33, 50, 65, 130, 333, 700, 1501, 3001, 5001, 9001, 16001, 16385))
@pytest.mark.parametrize("many", (False, True))
def test_rows_that_begin_anywhere(dtype, f, many):
    """x, dy and out each with a beginning and a stride of its own, NaN all around; one to some rows a block."""
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(f)
    lens = [0, 4, 1, 60, 0, 0, 33, 1] if not many else [700, 0, 1, 2, 150, 3 if f > 4000 else 4000, 11]
    off = 3 + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    rows = int(off[-1]) + 2
    do = torch.from_numpy(off).cuda()

    def within(first, stride, fill):
        flat = torch.full((first + rows * stride + 9,), fill, dtype=getattr(torch, dtype), device="cuda")
        return flat, flat.as_strided((rows, f), (stride, 1), first)
    x, dy = within(1, f + 2, float("nan"))[1], within(3, f + 1, float("nan"))[1]
    x[3:-2], dy[3:-2] = normal(g, (rows - 5, f), dtype) + 0.5, normal(g, (rows - 5, f), dtype)
    flat, out = within(5, f + 3, 7.0)
    w, b = weights(g, len(lens), f, "float32" if f % 3 else dtype)
    got = sr.seg_layer_norm(x, w, b, do, with_stats=True, out=out)
    check_forward(got, x, w, b, off, 1e-5, (dtype, f))
    edges = flat.clone()
    edges.as_strided((rows, f), (f + 3, 1), 5).fill_(7.0)
    assert bool((edges == 7).all())
    grads = sr.seg_layer_norm_grad(x, dy, *got[1:], w, do)
    check_grad(grads, x, dy, *got[1:], w, off, (dtype, f))
    assert all(torch.equal(p, q) for p, q in zip(grads, sr.seg_layer_norm_grad(x, dy, *got[1:], w, do)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("f", (64, 65, 1000, 2001, 9001, 12288, 20000, 20001))
def test_in_place(dtype, f):
    """A row is read before it is written, whatever its neighbours' threads do meanwhile."""
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(f)
    x = normal(g, (1200 if f > 4000 else 9000, f), dtype)
    w, b = weights(g, None, f, dtype)
    want = sr.seg_layer_norm(x, w, b)
    assert sr.seg_layer_norm(x, w, b, out=x) is x and torch.equal(x, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("f", (7, 48, 1000))
@pytest.mark.parametrize("rows,segments", ((30, 58), (1, 1000), (5, 3000), (64, 2), (200, 150), (3, 1)))
def test_few_rows_in_many_segments(dtype, f, rows, segments):
    torch, sr = mods()
    rng = np.random.default_rng(rows)
    off = np.concatenate([[0], np.sort(rng.integers(0, rows + 1, segments - 1)), [rows]]).astype(np.int64)
    g = torch.Generator(device="cuda")
    g.manual_seed(f)
    x, dy = normal(g, (rows, f), dtype), normal(g, (rows, f), dtype)
    w, b = weights(g, segments, f, dtype)
    do = torch.from_numpy(off).cuda()
    got = sr.seg_layer_norm(x, w, b, do, with_stats=True)
    check_forward(got, x, w, b, off, 1e-5, (dtype, f))
    check_grad(sr.seg_layer_norm_grad(x, dy, *got[1:], w, do), x, dy, *got[1:], w, off, (dtype, f))


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_alignment_and_what_is_left_out(dtype):
    torch, sr = mods()
    off, rows, do, g = case("mixed", 6)
    f = 72
    for cols, at in ((96, 8), (75, 1), (73, 0)):
        x, dy = normal(g, (rows, cols), dtype)[:, at:at + f], normal(g, (rows, cols), dtype)[:, at:at + f]
        w, b = weights(g, len(off) - 1, f, "float32")
        big = torch.full((rows, cols), 7.0, dtype=x.dtype, device="cuda")
        out = big[:, at:at + f]
        for ww, bb in ((w, b), (w, None), (None, b), (None, None)):
            got = sr.seg_layer_norm(x, ww, bb, do, eps=0.1, with_stats=True, out=out)
            check_forward(got, x, ww, bb, off, 0.1, (dtype, at))
            assert bool((big[:, :at] == 7).all()) and bool((big[:, at + f:] == 7).all())
            grads = sr.seg_layer_norm_grad(x, dy, *got[1:], ww, do)
            check_grad(grads, x, dy, *got[1:], ww, off, (dtype, at))
            for keep in range(3):
                some = sr.seg_layer_norm_grad(x, dy, *got[1:], ww, do, with_dx=keep == 0, with_weight=keep == 1, with_bias=keep == 2)
                assert [t is not None for t in some] == [i == keep for i in range(3)] and torch.equal(some[keep], grads[keep])


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_that_are_constant_far_from_zero_or_not_finite(dtype):
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = normal(g, (9, 512), dtype)
    x[1] = 3.0                       # no variance: z is 0
    x[2] = x[2] * 2.0 ** -8 + 100    # a mean of many deviations
    x[3, 7], x[4, 8], x[5, 9] = float("inf"), float("nan"), float("-inf")
    x[6] = torch.finfo(x.dtype).max if dtype == "float16" else 1e15
    w, b = weights(g, None, 512, dtype)
    y, mean, rstd = sr.seg_layer_norm(x, w, b, with_stats=True)
    fine = [0, 1, 2, 6, 7, 8]
    check_forward((y[fine], mean[fine], rstd[fine]), x[fine], w, b, None, 1e-5, dtype)
    assert torch.equal(y[1], b) and not bool(torch.isfinite(y[3:6]).any())
    # eps 0: a row without variance is not a number, the others are
    y = sr.seg_layer_norm(x[:3], w, b, eps=0.0)
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isfinite(y[0]).all())


def test_empty_sizes():
    torch, sr = mods()
    do = torch.tensor([0, 2, 3], device="cuda")
    for rows, f in ((0, 8), (3, 0), (0, 0)):
        x, w = torch.ones(rows, f, device="cuda"), torch.ones(2, f, device="cuda")
        y, mean, rstd = sr.seg_layer_norm(x, w, w, do, with_stats=True)
        assert y.shape == x.shape
        dx, dw, db = sr.seg_layer_norm_grad(x, x, mean, rstd, w, do)
        assert dx.shape == x.shape and dw.shape == w.shape and not bool(dw.any()) and not bool(db.any())
    x = torch.ones(5, 8, device="cuda")
    none, w = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.ones(0, 8, device="cuda")
    y, mean, rstd = sr.seg_layer_norm(x, w, w, none, with_stats=True)
    dx, dw, db = sr.seg_layer_norm_grad(x, x, mean, rstd, w, none)
    assert not bool(y.any()) and not bool(mean.any()) and not bool(dx.any()) and dw.shape == (0, 8)


def test_offsets_that_decrease_or_pass_the_rows_do_no_harm():
    torch, sr = mods()
    x, w = torch.ones(1000, 64, device="cuda"), torch.ones(5, 64, device="cuda")
    for bad in ([0, 900, 20, 1000, 5, 100], [700, 600, 500, 400, 30, 20], [-5, 10, 1 << 40, 3, 7, 1 << 50]):
        do = torch.tensor(bad, device="cuda")
        _, mean, rstd = sr.seg_layer_norm(x, w, w, do, with_stats=True)
        sr.seg_layer_norm_grad(x, x, mean, rstd, w, do)
    torch.cuda.synchronize()
    y = sr.seg_layer_norm(x, w, w, torch.tensor([0, 200, 400, 600, 800, 1000], device="cuda"))
    assert bool((y == 1).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_differentiable(dtype):
    torch, sr = mods()
    off, rows, do, g = case("mixed", 8)
    x, dy = normal(g, (rows, 72), dtype).requires_grad_(), normal(g, (rows, 72), dtype)
    w, b = (t.requires_grad_() for t in weights(g, len(off) - 1, 72, "float32"))
    y = sr.segment_layer_norm(x, w, b, do)
    grads = torch.autograd.grad(y, (x, w, b), dy)
    _, mean, rstd = sr.seg_layer_norm(x.detach(), w.detach(), b.detach(), do, with_stats=True)
    check_grad(grads, x.detach(), dy, mean, rstd, w.detach(), off, dtype)
    # the bias alone, float32 beside any x, and the gradient of a sum (strides of 0)
    only, = torch.autograd.grad(sr.segment_layer_norm(x.detach(), None, b, do).sum(), (b,))
    assert only.dtype == torch.float32 and torch.equal(only, torch.from_numpy(np.diff(off)).cuda().float()[:, None].expand_as(b))
    # without offsets or weights
    dx, = torch.autograd.grad(sr.segment_layer_norm(x), (x,), dy)
    _, mean, rstd = sr.seg_layer_norm(x.detach(), with_stats=True)
    check_grad((dx, None, None), x.detach(), dy, mean, rstd, None, None, dtype)


def test_gradient_against_differences():
    """<grad, d> against (f(p + h d) - f(p - h d)) / 2 h, float32: the values are
    exact to 2^-20 of their sizes, over 2 h = 2^-6; the third derivative (rows of
    24 unit normals, moved by h of as much) costs 64 h^2 at most."""
    torch, sr = mods()
    off, rows, do, g = case("mixed", 8)
    f = 24
    x, dy = normal(g, (rows, f), "float32"), normal(g, (rows, f), "float32")
    w, b = weights(g, len(off) - 1, f, "float32")
    _, mean, rstd = sr.seg_layer_norm(x, w, b, do, with_stats=True)
    grads = sr.seg_layer_norm_grad(x, dy, mean, rstd, w, do)
    h = 2.0 ** -7
    for which in range(3):
        d = normal(g, (x, w, b)[which].shape, "float32")

        def value(t):
            p = [q + t * d if i == which else q for i, q in enumerate((x, w, b))]
            return sr.seg_layer_norm(*p, do).double() * dy.double()
        up, down = value(h), value(-h)
        got, want = (grads[which].double() * d.double()).sum(), (up - down).sum() / (2 * h)
        tol = (2.0 ** -14 + 64 * h * h) * float(up.abs().sum())
        assert abs(float(got - want)) <= tol, (which, float(got), float(want), tol)


def test_another_stream_and_graphs_at_the_same_time():
    torch, sr = mods()
    sets = []
    for seed, f, kind in ((1, 264, "skewed"), (2, 63, "mixed"), (3, 20000, "one")):
        off, rows, do, g = case(kind, seed)
        x, dy = normal(g, (rows, f), "bfloat16"), normal(g, (rows, f), "bfloat16")
        w, b = weights(g, len(off) - 1, f, "bfloat16")

        def step(stream=None, x=x, dy=dy, w=w, b=b, do=do):
            y, mean, rstd = sr.seg_layer_norm(x, w, b, do, with_stats=True, stream=stream)
            return (y, mean, rstd) + sr.seg_layer_norm_grad(x, dy, mean, rstd, w, do, stream=stream)
        sets.append(step)
    want = [step() for step in sets]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for _ in range(10):
        got = [step(stream) for step in sets]
        stream.synchronize()
        assert all(torch.equal(a, b) for p, q in zip(got, want) for a, b in zip(p, q))
    graphs = []
    for step in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        graphs.append((graph, got))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        for (graph, got), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for v in got:
                    v.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for (_, got), expect in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(got, expect))
