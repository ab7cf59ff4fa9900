"""The sums of segments without rows, where they are nearly all that a norm's
backward pass has to store: zeros there, and the other segments' sums as they are
without the empty segments.

Tolerance: at most 40 rows are added up, by blocks that may be others, so either sum
is within 40 * 2^-24 of its terms' sizes of the exact one, then rounded by half a step."""
import numpy as np
import pytest

from tests.test_product_gpu import TYPES, UNIT, mods, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,segments,f", ((1, 200, 16384), (10, 100000, 64), (20, 2000, 33), (3, 5000, 1), (1, 400, 1001), (7, 33, 20000), (40, 65, 4100), (0, 300, 40)))
@pytest.mark.parametrize("odt", ("int64", "uint32"))
def test_few_rows_beside_many_sums(dtype, rows, segments, f, odt):
    torch, sr = mods()
    rng = np.random.default_rng(rows + segments)
    g = torch.Generator(device="cuda")
    g.manual_seed(f)
    lens = np.bincount(rng.integers(0, segments, rows), minlength=segments)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    used = np.flatnonzero(lens)
    x, dy = normal(g, (rows, f), dtype), normal(g, (rows, f), dtype)
    w = normal(g, (segments, f), "float32" if f % 2 else dtype)

    def offsets(o):
        return torch.from_numpy(o).cuda() if odt == "int64" else torch.from_numpy(o.astype(np.int32)).cuda().view(torch.uint32)
    do, few = offsets(off), offsets(np.concatenate([[0], np.cumsum(lens[used])]).astype(np.int64))
    _, mean, rstd = sr.seg_layer_norm(x, w, None, do, with_stats=True)
    at = torch.from_numpy(used).cuda()
    if rows:
        want_dx, want_dw, want_db = sr.seg_layer_norm_grad(x, dy, mean, rstd, w[at], few)
    for with_weight, with_bias in ((True, True), (True, False), (False, True)):
        # what is there before is not zeros
        torch.full((2, segments, f), float("nan"), dtype=w.dtype, device="cuda")
        dx, dw, db = sr.seg_layer_norm_grad(x, dy, mean, rstd, w, do, with_weight=with_weight, with_bias=with_bias)
        assert (dw is not None) == with_weight and (db is not None) == with_bias
        if rows:
            assert torch.equal(dx, want_dx)
        for got, name in ((dw, "dw"), (db, "db")):
            if got is None:
                continue
            want = torch.zeros(segments, f, dtype=w.dtype, device="cuda")
            if rows:
                want[at] = want_dw if name == "dw" else want_db
            size = torch.zeros(segments, f, dtype=torch.float64, device="cuda")
            if rows:
                z = (x.double() - mean.double()[:, None]) * rstd.double()[:, None] if name == "dw" else torch.ones_like(x, dtype=torch.float64)
                size.index_add_(0, torch.from_numpy(np.repeat(np.arange(segments), lens)).cuda(), (dy.double() * z).abs())
            tol = 2 * 40 * 2.0 ** -24 * size
            # (float16's smallest step is 2^-24)
            tol = tol + 2 * UNIT[str(w.dtype).replace("torch.", "")] * (want.double().abs() + tol) + 2.0 ** -24
            close = (got.double() - want.double()).abs() <= tol
            assert bool(close.all()) and not bool(got[torch.from_numpy(lens == 0).cuda()].any()), name


def test_clearing_in_a_graph_and_on_another_stream():
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, dy, w = normal(g, (3, 1000), "bfloat16"), normal(g, (3, 1000), "bfloat16"), normal(g, (700, 1000), "float32")
    off = torch.zeros(701, dtype=torch.int64, device="cuda")
    off[300:] = 1
    off[500:] = 3
    _, mean, rstd = sr.seg_layer_norm(x, w, None, off, with_stats=True)
    want = sr.seg_layer_norm_grad(x, dy, mean, rstd, w, off)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = sr.seg_layer_norm_grad(x, dy, mean, rstd, w, off, stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sr.seg_layer_norm_grad(x, dy, mean, rstd, w, off)
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert float(want[1].abs().sum(1).count_nonzero()) == 2
