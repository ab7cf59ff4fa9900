"""Gradients of hundreds and thousands of segments of very uneven length, of which some are split into parts."""
import numpy as np
import pytest

from tests.test_product_gpu import TYPES, check, mods, normal, ref_grad

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("segments,rows,k,n", ((350, 60000, 64, 64), (1000, 200000, 64, 64), (1100, 90000, 33, 130), (1215, 120000, 64, 20)))
def test_gradients_of_uneven_segments(dtype, segments, rows, k, n):
    torch, sr = mods()
    rng = np.random.default_rng(segments)
    share = 1.0 / np.arange(1, segments + 1) ** 1.3
    share[rng.random(segments) < 0.1] = 0
    lens = rng.permutation(rng.multinomial(rows, share / share.sum()))
    off = 11 + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    g = torch.Generator(device="cuda")
    g.manual_seed(k)
    x, dy = normal(g, (rows + 20, k), dtype), normal(g, (rows + 20, n), dtype)
    do = torch.from_numpy(off).cuda()
    want, a = ref_grad(x, dy, off)
    for out_dtype in {x.dtype, torch.float32}:
        got = sr.seg_matmul_grad_w(x, dy, do, out_dtype=out_dtype)
        check(got, want, a, int(lens.max()), (dtype, segments, out_dtype))
        assert torch.equal(got, sr.seg_matmul_grad_w(x, dy, do, out_dtype=out_dtype))
    assert sr.device_status() == 0


def test_malformed_offsets_of_many_segments_touch_nothing_else():
    """Decreasing offsets and ones past the rows: unspecified results, but nothing outside the output is written."""
    torch, sr = mods()
    rng = np.random.default_rng(1)
    x = torch.ones(70000, 24, device="cuda", dtype=torch.bfloat16)
    dy = torch.ones(70000, 40, device="cuda", dtype=torch.bfloat16)
    for segments in (900, 1500):
        off = rng.integers(-1000, 90000, segments + 1)
        off[7], off[300] = 1 << 40, -5
        for out_dtype in (torch.bfloat16, torch.float32):
            big = torch.full((segments + 2, 24, 40), 7.0, device="cuda", dtype=out_dtype)
            sr.seg_matmul_grad_w(x, dy, torch.from_numpy(off).cuda(), out=big[1:-1])
            torch.cuda.synchronize()
            assert bool((big[0] == 7).all() and (big[-1] == 7).all())
    assert sr.device_status() == 0
