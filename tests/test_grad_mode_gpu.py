"""Serving a model of parameters: with gradients off the gated block allocates its
result alone, not the [R, 2 N] float32 products, and the results are those of training."""
import pytest

from tests.test_product_gpu import mods, normal

pytestmark = pytest.mark.gpu


def test_no_products_with_gradients_off():
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows, k, n = 4096, 256, 1024
    x, w = normal(g, (rows, k), "bfloat16"), torch.nn.Parameter(normal(g, (4, k, 2 * n), "bfloat16", k ** -0.5))
    b = torch.nn.Parameter(normal(g, (4, k), "float32"))
    off = torch.tensor([0, 1000, 1000, 3000, rows], device="cuda")

    def run():
        return sr.segment_layer_norm(x, None, b, off), sr.segment_gated(x, w, off)

    def peak():
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        y = run()
        torch.cuda.synchronize()
        return torch.cuda.max_memory_allocated() - before, y
    products, results = rows * 2 * n * 4, rows * (n + k) * 2
    kept, want = peak()
    assert kept >= products + results
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            kept, got = peak()
        assert results <= kept < results + products // 8
        assert all(torch.equal(p, q) for p, q in zip(got, want)) and not any(p.requires_grad for p in got)
