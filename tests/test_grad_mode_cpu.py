"""What the differentiable calls keep for a backward pass: the products of the
gated block and the norm's statistics where a gradient is recorded, nothing where
gradients are off, also with parameters.  The operators themselves are stood in
for by functions of the host that say how they were called."""
import pytest

import segmented_reduction_csr_gb300 as sr


@pytest.fixture
def calls(monkeypatch):
    torch = pytest.importorskip("torch")
    seen = []

    def gated(x, w, offsets, activation="silu", transpose_w=False, with_pre=False):
        seen.append(with_pre)
        out = torch.ones(x.shape[0], w.shape[2] // 2)
        return (out, torch.ones(x.shape[0], w.shape[2])) if with_pre else out

    def norm(x, weight=None, bias=None, offsets=None, eps=1e-5, with_stats=False):
        seen.append(with_stats)
        return (torch.ones_like(x), torch.ones(x.shape[0]), torch.ones(x.shape[0])) if with_stats else torch.ones_like(x)
    monkeypatch.setattr(sr, "seg_gated", gated)
    monkeypatch.setattr(sr, "seg_layer_norm", norm)
    return seen


def both(torch, grad):
    """Each call with a parameter among its arguments, and with none."""
    x, off = torch.ones(4, 8), torch.tensor([0, 2, 4])
    w, b = torch.ones(2, 8, 6), torch.ones(2, 8)
    if grad:
        w, b = torch.nn.Parameter(w), torch.nn.Parameter(b)
    return sr.segment_gated(x, w, off), sr.segment_layer_norm(x, None, b, off)


def test_with_gradients_they_are_kept(calls):
    torch = pytest.importorskip("torch")
    assert all(y.requires_grad for y in both(torch, True)) and calls == [True, True]


def test_without_they_are_not(calls):
    torch = pytest.importorskip("torch")
    with torch.no_grad():
        assert not any(y.requires_grad for y in both(torch, True))
    with torch.inference_mode():
        both(torch, True)
    assert not any(y.requires_grad for y in both(torch, False))
    assert calls == [False] * 6


def test_gradients_that_are_on_within_no_grad(calls):
    torch = pytest.importorskip("torch")
    with torch.no_grad():
        with torch.enable_grad():
            assert all(y.requires_grad for y in both(torch, True))
    assert calls == [True, True]
