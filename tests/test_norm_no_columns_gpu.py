"""Rows without columns: the statistics are zeros, not what the memory held."""
import pytest

from tests.test_product_gpu import mods

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("segments", (False, True))
@pytest.mark.parametrize("another", (False, True))
def test_statistics_of_rows_without_columns(segments, another):
    torch, sr = mods()
    rows = 5000
    stream = torch.cuda.Stream() if another else None
    x = torch.empty(rows, 0, device="cuda")
    off = torch.tensor([0, 3000, rows], device="cuda") if segments else None
    with torch.cuda.stream(stream):
        # memory that the results may be given
        for t in [torch.full((rows,), float("nan"), device="cuda") for _ in range(4)]:
            del t
    torch.cuda.synchronize()
    y, mean, rstd = sr.seg_layer_norm(x, offsets=off, with_stats=True, stream=stream)
    torch.cuda.synchronize()
    assert y.shape == (rows, 0) and torch.equal(mean, torch.zeros(rows, device="cuda")) and torch.equal(rstd, mean)
