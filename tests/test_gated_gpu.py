"""The gated feed-forward block (seg_gated, seg_gated_grad, segment_gated)
against the formulas in 64 bits.

Tolerances.  The products g and u of K terms are within e = (K * 2^-24 + 2^-20) *
sum(|x w|) of the exact ones, as seg_matmul's are.  The activations have slopes
of at most 1.13 and are computed to 2^-15 of their size where that is a normal
number (exp of q, 88 at most: 2 + 1.2 q units of 2^-23, and 2 q for the rounding
of q), so before its rounding out is within 1.13 e_g (|u| + e_u) + |act(g)| e_u
+ 2^-15 |out| of the exact one.  A rounding
adds half a step, 2^-8, 2^-11 or 2^-24 of the value (float16: 2^-25 at least)."""
import numpy as np
import pytest

from tests.test_product_gpu import TYPES, UNIT, case, mods, normal

pytestmark = pytest.mark.gpu

ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")


def act64(kind, g):
    """The activation and its derivative, from their definitions."""
    torch, _ = mods()
    if kind == "relu":
        return g.clamp(min=0), (g > 0).to(g.dtype)
    if kind == "gelu":
        p = 0.5 * torch.special.erfc(-g / 2 ** 0.5)
        return g * p, p + g * torch.exp(-g * g / 2) / (2 * np.pi) ** 0.5
    if kind == "gelu_tanh":
        q = (8 / np.pi) ** 0.5 * (g + 0.044715 * g ** 3)
        s = torch.sigmoid(q)
        return g * s, s + g * s * (1 - s) * (8 / np.pi) ** 0.5 * (1 + 0.134145 * g ** 2)
    s = torch.sigmoid(g)
    return (s, s * (1 - s)) if kind == "sigmoid" else (g * s, s + g * s * (1 - s))


def products(x, w, off, trans):
    """pre and the sum of its terms' sizes, [R, 2 N] in 64 bits."""
    torch, _ = mods()
    both = w.shape[1] if trans else w.shape[2]
    y = torch.zeros(x.shape[0], both, dtype=torch.float64, device="cuda")
    a = torch.zeros_like(y)
    for s in range(len(off) - 1):
        if off[s + 1] > off[s]:
            xs = x[off[s]:off[s + 1]].double()
            ws = w[s].double().t() if trans else w[s].double()
            y[off[s]:off[s + 1]] = xs @ ws
            a[off[s]:off[s + 1]] = xs.abs() @ ws.abs()
    return y, a


def close(got, want, tol, where):
    torch, _ = mods()
    name = str(got.dtype).replace("torch.", "")
    tol = tol + UNIT[name] * (want.abs() + tol) + (2.0 ** -25 if name == "float16" else 2.0 ** -125)
    err = (got.double() - want).abs()
    bad = ~(err <= tol)          # NaN counts as bad
    assert not bool(bad.any()), (where, int(bad.sum()), float(err.max()), float((err / (tol + 1e-300)).max()))


def check_forward(out, pre, x, w, off, trans, act, where):
    k, n = x.shape[1], out.shape[1]
    y, a = products(x, w, off, trans)
    e = (k * 2.0 ** -24 + 2.0 ** -20) * a
    g, u = y[:, :n], y[:, n:]
    f, _ = act64(act, g)
    close(out, f * u, 1.13 * e[:, :n] * (u.abs() + e[:, n:]) + f.abs() * e[:, n:] + 2.0 ** -15 * (f * u).abs(), where)
    if pre is not None:
        close(pre, y, e, (where, "pre"))


def check_grad(dx, dw, x, w, pre, dy, off, trans, act, where):
    """Against the formula at the pre that the forward pass gave."""
    torch, _ = mods()
    n, k = dy.shape[1], x.shape[1]
    g, u, d = pre[:, :n].double(), pre[:, n:].double(), dy.double()
    f, slope = act64(act, g)
    dpre = torch.cat([d * u * slope, d * f], dim=1)
    name = str(x.dtype).replace("torch.", "")
    # computed to 2^-15 of the slope's largest size and of f, then rounded (float16: to 2^-25 at least)
    e = torch.cat([2.0 ** -15 * (d * u).abs(), 2.0 ** -15 * (d * f).abs()], dim=1) + UNIT[name] * dpre.abs()
    if name == "float16":
        e = e + 2.0 ** -24
    if dx is not None:
        want, tol = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for s in range(len(off) - 1):
            at = slice(int(off[s]), int(off[s + 1]))
            ws = w[s].double() if trans else w[s].double().t()
            want[at] = dpre[at] @ ws
            tol[at] = (e[at] + (2 * n * 2.0 ** -24 + 2.0 ** -20) * (dpre[at].abs() + e[at])) @ ws.abs()
        close(dx, want, tol, (where, "dx"))
    if dw is not None:
        want, tol = torch.zeros(w.shape, dtype=torch.float64, device="cuda"), torch.zeros(w.shape, dtype=torch.float64, device="cuda")
        for s in range(len(off) - 1):
            at = slice(int(off[s]), int(off[s + 1]))
            xs, rows = x[at].double(), int(off[s + 1] - off[s])
            if rows == 0:
                continue
            part, bound = xs.t() @ dpre[at], xs.abs().t() @ (e[at] + (rows * 2.0 ** -24 + 2.0 ** -20) * (dpre[at].abs() + e[at]))
            want[s], tol[s] = (part.t(), bound.t()) if trans else (part, bound)
        close(dw, want, tol, (where, "dw"))


def inputs(kind, seed, k, n, dtype, trans, **more):
    off, rows, do, g = case(kind, seed, **more)
    x = normal(g, (rows, k), dtype)
    w = normal(g, (len(off) - 1, 2 * n, k) if trans else (len(off) - 1, k, 2 * n), dtype, k ** -0.5)
    return off, do, g, x, w


SIZES = [(64, 64), (1, 1), (7, 5), (16, 128), (63, 33), (65, 127), (72, 136), (200, 300), (256, 8), (8, 256), (520, 264), (136, 600)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("trans", (False, True))
@pytest.mark.parametrize("k,n", SIZES)
def test_sizes(dtype, trans, k, n):
    torch, sr = mods()
    off, do, g, x, w = inputs("mixed", 1000 * k + n, k, n, dtype, trans)
    act = ACTS[(k + n) % 5]
    out = sr.seg_gated(x, w, do, act, transpose_w=trans)
    again, pre = sr.seg_gated(x, w, do, act, transpose_w=trans, with_pre=True)
    check_forward(out, pre, x, w, off, trans, act, (dtype, trans, k, n, act))
    assert torch.equal(out, again)
    dy = normal(g, out.shape, dtype)
    dx, dw = sr.seg_gated_grad(x, w, pre, dy, do, act, transpose_w=trans)
    check_grad(dx, dw, x, w, pre, dy, off, trans, act, (dtype, trans, k, n, act))
    if dtype != "float32":
        # products kept in 16 bits
        assert pre.dtype == torch.float32
        same, half = sr.seg_gated(x, w, do, act, transpose_w=trans, pre=torch.empty(pre.shape, dtype=x.dtype, device="cuda"))
        assert torch.equal(same, out) and torch.equal(half, pre.to(x.dtype))
        dx, dw = sr.seg_gated_grad(x, w, half, dy, do, act, transpose_w=trans)
        check_grad(dx, dw, x, w, half, dy, off, trans, act, (dtype, trans, k, n, act, "half"))
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
def test_activations(dtype, act):
    torch, sr = mods()
    off, do, g, x, w = inputs("skewed", 5, 136, 200, dtype, False)
    w = (w.float() * 6).to(w.dtype)         # far into both tails
    out, pre = sr.seg_gated(x, w, do, act, with_pre=True)
    check_forward(out, pre, x, w, off, False, act, (dtype, act))
    dy = normal(g, out.shape, dtype)
    dx, dw = sr.seg_gated_grad(x, w, pre, dy, do, act)
    check_grad(dx, dw, x, w, pre, dy, off, False, act, (dtype, act))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
def test_far_tails_and_border_values(dtype, act):
    """Products of any size: the largest of the type, infinities and NaN among them."""
    torch, sr = mods()
    top = torch.finfo(getattr(torch, dtype)).max
    g = torch.tensor([0.0, -0.0, 1e-6, -1e-6, 88.0, -88.0, 300.0, -300.0, 6e4, -6e4, top, -top, float("inf"), float("nan")], dtype=torch.float64, device="cuda")
    pre = torch.stack([g, torch.ones_like(g)], dim=1).to(getattr(torch, dtype))
    one = torch.ones(len(g), 1, dtype=pre.dtype, device="cuda")
    # the products by a matrix of the identity's two halves: pre = x @ w
    w = torch.tensor([[[1.0, 0.0], [0.0, 1.0]]], dtype=pre.dtype, device="cuda")
    do = torch.tensor([0, len(g)], device="cuda")
    if dtype != "float32":      # (float32 products make NaN of infinities)
        out = sr.seg_gated(pre[:12], w, do.clamp(max=12), act)
        f, _ = act64(act, pre[:12, 0].double())
        close(out[:, 0], f, 2.0 ** -15 * f.abs(), act)
    dx, _ = sr.seg_gated_grad(pre, w, pre, one, do, act, want_dw=False)
    slope = act64(act, pre[:12, 0].double())[1]
    if dtype != "float32":
        close(dx[:12, 0], torch.nan_to_num(slope, nan=0.0) if act == "gelu_tanh" else slope, torch.full_like(slope, 2.0 ** -15), act)
    assert not bool(torch.isfinite(dx[13]).all()) or act == "relu"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ("one", "empty", "single rows", "skewed", "many"))
@pytest.mark.parametrize("odt", ("int64", "uint32"))
def test_segment_shapes(dtype, kind, odt):
    torch, sr = mods()
    k, n = (24, 40) if kind == "many" else (136, 200)
    off, do, g, x, w = inputs(kind, 77, k, n, dtype, True, before=5, after=9, odt=odt)
    # rows in no segment hold NaN: they must reach nothing
    dy = normal(g, (x.shape[0], n), dtype)
    x[:5], dy[:5] = float("nan"), float("inf")
    x[int(off[-1]):], dy[int(off[-1]):] = float("inf"), float("nan")
    for s in range(len(off) - 1):
        if off[s] == off[s + 1]:
            w[s] = float("nan")
    out, pre = sr.seg_gated(x, w, do, transpose_w=True, with_pre=True)
    check_forward(out, pre, x, w, off, True, "silu", (dtype, kind))
    dx, dw = sr.seg_gated_grad(x, w, pre, dy, do, transpose_w=True)
    check_grad(dx, dw, x, w, pre, dy, off, True, "silu", (dtype, kind))
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("trans", (False, True))
@pytest.mark.parametrize("lens,k,n", (([1, 1], 2048, 1024), ([3, 0, 2, 1] * 16, 1024, 520), ([4100], 264, 512), ([900, 0, 3300, 77], 1000, 192), ([2500, 2600], 600, 40)))
def test_few_rows_long_sums_and_large_tiles(dtype, trans, lens, k, n):
    """Sums that are split, float32 sums of several pieces, tiles of a pair of CTAs."""
    torch, sr = mods()
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    g = torch.Generator(device="cuda")
    g.manual_seed(k + n)
    x = normal(g, (int(off[-1]), k), dtype)
    w = normal(g, (len(lens), 2 * n, k) if trans else (len(lens), k, 2 * n), dtype, k ** -0.5)
    do = torch.from_numpy(off).cuda()
    out, pre = sr.seg_gated(x, w, do, "gelu", transpose_w=trans, with_pre=True)
    check_forward(out, pre, x, w, off, trans, "gelu", (dtype, trans, k, n))
    assert torch.equal(out, sr.seg_gated(x, w, do, "gelu", transpose_w=trans))
    assert sr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("trans", (False, True))
def test_odd_matrices_most_of_which_are_in_no_use(dtype, trans):
    """Not copied to aligned rows: the products first, then the activation."""
    torch, sr = mods()
    k, n = 63, 33
    lens = [0] * 70 + [3] + [0] * 50 + [1]
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = normal(g, (4, k), dtype)
    w = normal(g, (len(lens), 2 * n, k) if trans else (len(lens), k, 2 * n), dtype, k ** -0.5)
    do = torch.from_numpy(off).cuda()
    out = sr.seg_gated(x, w, do, "sigmoid", transpose_w=trans)
    check_forward(out, None, x, w, off, trans, "sigmoid", (dtype, trans))
    for ptype in {x.dtype, torch.float32}:
        same, pre = sr.seg_gated(x, w, do, "sigmoid", transpose_w=trans, pre=torch.empty(4, 2 * n, dtype=ptype, device="cuda"))
        assert torch.equal(out, same)
        check_forward(out, pre, x, w, off, trans, "sigmoid", (dtype, trans, ptype))


@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
def test_sums_longer_than_an_accumulator_takes(dtype):
    torch, sr = mods()
    off = np.array([0, 4090])
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    k, n = 32776, 512
    x, w = normal(g, (4100, k), dtype), normal(g, (1, 2 * n, k), dtype, k ** -0.5)
    do = torch.from_numpy(off).cuda()
    out, pre = sr.seg_gated(x, w, do, transpose_w=True, with_pre=True)
    check_forward(out, pre, x, w, off, True, "silu", dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("trans", (False, True))
def test_strides_and_alignment(dtype, trans):
    torch, sr = mods()
    k, n = 72, 40
    for xcols, xat, wcols, wat, ocols, oat in ((96, 8, 104, 16, 104, 8), (75, 1, 83, 2, 87, 5), (73, 0, 80, 0, 81, 1), (72, 0, 81, 1, 80, 0)):
        off, rows, do, g = case("mixed", 6)
        s = len(off) - 1
        x = normal(g, (rows, xcols), dtype)[:, xat:xat + k]
        w = normal(g, (s, 2 * n, wcols) if trans else (s, k, wcols + 0), dtype, k ** -0.5)
        w = w[:, :, :k] if trans else w[:, :, wat:wat + 2 * n] if wcols >= wat + 2 * n else w[:, :, :2 * n]
        ptype = torch.float32 if xat == 0 else x.dtype
        big, pres = torch.full((rows, ocols), 7.0, dtype=x.dtype, device="cuda"), torch.full((rows, 2 * n + 9), 7.0, dtype=ptype, device="cuda")
        out, pre = big[:, oat:oat + n], pres[:, 3:3 + 2 * n]
        sr.seg_gated(x, w, do, transpose_w=trans, out=out, pre=pre)
        check_forward(out, pre, x, w, off, trans, "silu", (dtype, xat))
        assert bool((big[:, :oat] == 7).all()) and bool((big[:, oat + n:] == 7).all())
        assert bool((pres[:, :3] == 7).all()) and bool((pres[:, 3 + 2 * n:] == 7).all())
        dy = normal(g, (rows, n + 3), dtype)[:, 1:1 + n]
        dx, dw = sr.seg_gated_grad(x, w, pre, dy, do, transpose_w=trans, dw_dtype=torch.float32)
        check_grad(dx, dw, x, w, pre, dy, off, trans, "silu", (dtype, xat))


def test_empty_sizes():
    torch, sr = mods()
    do = torch.tensor([0, 2, 3], device="cuda")
    for rows, k, n in ((0, 8, 4), (3, 0, 4), (3, 8, 0)):
        x, w = torch.ones(rows, k, device="cuda"), torch.ones(2, k, 2 * n, device="cuda")
        out, pre = sr.seg_gated(x, w, do, with_pre=True)
        assert out.shape == (rows, n) and pre.shape == (rows, 2 * n) and not bool(out.any()) and not bool(pre.any())
        dx, dw = sr.seg_gated_grad(x, w, pre, torch.ones(rows, n, device="cuda"), do)
        assert dx.shape == x.shape and dw.shape == w.shape and not bool(dx.any()) and not bool(dw.any())
    # no segments at all: every row is in none
    x = torch.ones(5, 8, device="cuda")
    out = sr.seg_gated(x, torch.ones(0, 8, 6, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert out.shape == (5, 3) and not bool(out.any())


def test_offsets_that_decrease_or_pass_the_rows_do_no_harm():
    torch, sr = mods()
    x, w = torch.ones(100, 64, device="cuda", dtype=torch.bfloat16), torch.ones(5, 64, 128, device="cuda", dtype=torch.bfloat16)
    for bad in ([0, 90, 20, 1000, 5, 100], [70, 60, 50, 40, 30, 20], [-5, 10, 1 << 40, 3, 7, 1 << 50]):
        sr.seg_gated(x, w, torch.tensor(bad, device="cuda"))
    assert sr.device_status() == 0
    out = sr.seg_gated(x, w, torch.tensor([0, 20, 40, 60, 80, 100], device="cuda"))
    assert bool((out == 64 * 64).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("trans", (False, True))
def test_differentiable(dtype, trans):
    torch, sr = mods()
    off, do, g, x, w = inputs("mixed", 9, 72, 40, dtype, trans)
    x.requires_grad_()
    w.requires_grad_()
    y = sr.segment_gated(x, w, do, "gelu", trans)
    dy = normal(g, y.shape, dtype)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    pre = sr.seg_gated(x.detach(), w.detach(), do, "gelu", trans, with_pre=True)[1]
    check_grad(dx, dw, x.detach(), w.detach(), pre, dy, off, trans, "gelu", (dtype, trans))
    # one gradient alone, and that of a sum (strides of 0)
    only, = torch.autograd.grad(sr.segment_gated(x.detach(), w, do, "gelu", trans).sum(), (w,))
    want, = torch.autograd.grad(sr.segment_gated(x, w, do, "gelu", trans), (w,), torch.ones_like(y))
    assert torch.equal(only, want)


def test_gradient_against_differences():
    """<grad, d> against (f(p + h d) - f(p - h d)) / 2 h, float32.  The values are
    of size 1 and the difference of them exact to 2^-20 of the absolute sum, so
    to 2^-20 / 2^-6 of it over 2 h; the third derivative costs h^2 = 2^-14 of it."""
    torch, sr = mods()
    off, do, g, x, w = inputs("mixed", 19, 24, 40, "float32", False)
    dy = normal(g, (x.shape[0], 40), "float32")
    pre = sr.seg_gated(x, w, do, "gelu_tanh", with_pre=True)[1]
    dx, dw = sr.seg_gated_grad(x, w, pre, dy, do, "gelu_tanh")
    h = 2.0 ** -7
    for which in range(2):
        d = normal(g, (x, w)[which].shape, "float32")
        def f(t):
            a, b = (x + t * d, w) if which == 0 else (x, w + t * d)
            return sr.seg_gated(a, b, do, "gelu_tanh").double() * dy.double()
        up, down = f(h), f(-h)
        got = ((dx, dw)[which].double() * d.double()).sum()
        want = (up - down).sum() / (2 * h)
        # a direction moves a product by the sum of 24 terms: up to 5 times its size
        tol = (2.0 ** -14 + 125 * 2.0 ** -14) * float(up.abs().sum())
        assert abs(float(got - want)) <= tol, (which, float(got), float(want), tol)


def test_results_on_another_stream():
    torch, sr = mods()
    off, do, g, x, w = inputs("skewed", 21, 264, 200, "bfloat16", False)
    want, wpre = sr.seg_gated(x, w, do, with_pre=True)
    dy = normal(g, want.shape, "bfloat16")
    wdx, wdw = sr.seg_gated_grad(x, w, wpre, dy, do)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for _ in range(20):
        out, pre = sr.seg_gated(x, w, do, with_pre=True, stream=stream)
        dx, dw = sr.seg_gated_grad(x, w, pre, dy, do, stream=stream)
        stream.synchronize()
        assert torch.equal(out, want) and torch.equal(dx, wdx) and torch.equal(dw, wdw)


def test_graphs_of_one_capture_stream_at_the_same_time():
    torch, sr = mods()
    sets = []
    for seed, k, n in ((1, 264, 200), (2, 63, 65), (3, 1032, 96)):
        off, do, g, x, w = inputs("skewed", seed, k, n, "bfloat16", False)
        dy = normal(g, (x.shape[0], n), "bfloat16")
        def step(x=x, w=w, do=do, dy=dy):
            out, pre = sr.seg_gated(x, w, do, with_pre=True)
            return (out, pre) + sr.seg_gated_grad(x, w, pre, dy, do)
        sets.append(step)
    want = [step() for step in sets]
    torch.cuda.synchronize()
    graphs = []
    for step in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        graphs.append((graph, got))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        for (graph, got), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                for v in got:
                    v.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for (_, got), expect in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(got, expect))
    assert sr.device_status() == 0
