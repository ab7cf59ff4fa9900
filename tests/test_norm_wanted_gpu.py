"""Gradients of the norm that are asked for one at a time are those of all
together, for every way that rows are worked on: also where the rows' two sums,
which dx alone needs, come from a kernel of their own (more than 16,384 columns)."""
import numpy as np
import pytest

from tests.test_product_gpu import TYPES, mods, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("f", (40, 333, 2048, 9000, 9001, 16392, 20000, 33001))
def test_one_gradient_at_a_time(dtype, f):
    torch, sr = mods()
    lens = [3, 0, 70, 0, 0, 1, 300 if f < 5000 else 60, 0]
    off = 2 + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    g = torch.Generator(device="cuda")
    g.manual_seed(f)
    x, dy = normal(g, (int(off[-1]) + 3, f), dtype), normal(g, (int(off[-1]) + 3, f), dtype)
    x[:2], dy[-3:] = float("nan"), float("inf")
    w = normal(g, (len(lens), f), "float32")
    do = torch.from_numpy(off).cuda()
    _, mean, rstd = sr.seg_layer_norm(x, w, None, do, with_stats=True)
    want = sr.seg_layer_norm_grad(x, dy, mean, rstd, w, do)
    assert all(bool(torch.isfinite(t).all()) for t in want)
    for keep in ((0,), (1,), (2,), (0, 1), (1, 2)):
        got = sr.seg_layer_norm_grad(x, dy, mean, rstd, w, do, with_dx=0 in keep, with_weight=1 in keep, with_bias=2 in keep)
        assert [t is not None for t in got] == [i in keep for i in range(3)]
        assert all(torch.equal(got[i], want[i]) for i in keep), keep
