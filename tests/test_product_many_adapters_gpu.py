"""Adapters, most of them in no use, whose rows tensor copies cannot take: every row of long requests gets its part."""
import numpy as np
import pytest

from tests.test_product_gpu import TYPES, check, mods, normal, ref_lora

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,requests,adapters,k,rank", ((20000, 10, 50000, 33, 8), (20000, 300, 40001, 33, 4)))
def test_every_row_gets_its_adapter(dtype, rows, requests, adapters, k, rank):
    torch, sr = mods()
    rng = np.random.default_rng(rows + requests)
    lens = rng.multinomial(rows, np.ones(requests) / requests)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    n = 24
    x, w = normal(g, (rows, k), dtype), normal(g, (n, k), dtype, k ** -0.5)
    a, b = normal(g, (adapters, rank, k), dtype, k ** -0.5), normal(g, (adapters, n, rank), dtype)
    ids = rng.integers(0, adapters, requests)
    adapter, do = torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(off).cuda()
    # what scratch holds from a call before is not what this call needs
    sr.seg_lora(-x, w, a, b, do, torch.roll(adapter, 1))
    got = sr.seg_lora(x, w, a, b, do, adapter)
    y, m = ref_lora(x, w, a, b, off, ids, None)
    check(got, y, m, k + rank, (dtype, requests))
    assert sr.device_status() == 0
