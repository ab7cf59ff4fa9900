"""The products' host checks: every bad argument is refused before any CUDA call."""
import pytest

import segmented_reduction_csr_gb300 as sr
from segmented_reduction_csr_gb300 import build as srbuild


@pytest.fixture(scope="module")
def lib():
    srbuild.build()
    return sr.load_library()


def test_matmul_host_checks(lib):
    def call(x=64, dtype=4, R=10, K=8, ldx=8, w=64, N=16, ldw=16, stride=128, trans=0, off=64, odt=1, S=3, out=64, ldo=16):
        return lib.seg_matmul(x, dtype, R, K, ldx, w, N, ldw, stride, trans, off, odt, S, out, ldo, None)
    assert call(R=0) == 0 and call(N=0, ldw=0, ldo=0, stride=0) == 0      # nothing to do
    for bad in (dict(dtype=0), dict(dtype=1), dict(dtype=5), dict(odt=2), dict(R=-1), dict(K=-1), dict(N=-1), dict(S=-1),
                dict(ldx=7), dict(ldw=15), dict(ldo=15), dict(trans=2), dict(stride=127), dict(stride=-1),
                dict(trans=1, ldw=7), dict(x=None), dict(w=None), dict(off=None), dict(out=None), dict(x=65), dict(w=65),
                dict(out=65), dict(off=68), dict(dtype=2, x=66), dict(dtype=2, w=66), dict(dtype=2, out=66)):
        assert call(**bad) == 1, bad
    for bad in (dict(R=1 << 31), dict(S=1 << 31), dict(K=(1 << 20) + 1, ldx=1 << 21), dict(N=(1 << 20) + 1, ldw=1 << 21, ldo=1 << 21)):
        assert call(**bad) == 2, bad


def test_grad_host_checks(lib):
    def call(x=64, dtype=3, R=10, K=8, ldx=8, dy=64, N=16, ldy=16, off=64, odt=0, S=3, out=64, odtype=3):
        return lib.seg_matmul_grad_w(x, dtype, R, K, ldx, dy, N, ldy, off, odt, S, out, odtype, None)
    assert call(S=0) == 0 and call(K=0, ldx=0) == 0 and call(N=0, ldy=0) == 0
    for bad in (dict(dtype=0), dict(odtype=4), dict(odtype=0), dict(ldy=15), dict(ldx=7), dict(dy=None), dict(x=None),
                dict(out=None), dict(off=None), dict(dy=65), dict(out=65), dict(odtype=2, out=66), dict(off=66), dict(odt=7)):
        assert call(**bad) == 1, bad
    assert call(R=1 << 31) == 2


def test_lora_host_checks(lib):
    def call(x=64, dtype=4, R=10, K=8, ldx=8, w=64, N=16, ldw=8, a=64, b=64, L=4, rank=16, off=64, odt=1, S=3, adapter=64,
             scale=64, out=64, ldo=16):
        return lib.seg_lora(x, dtype, R, K, ldx, w, N, ldw, a, b, L, rank, off, odt, S, adapter, scale, out, ldo, None)
    assert call(R=0) == 0 and call(N=0, ldo=0) == 0
    for bad in (dict(dtype=1), dict(rank=0), dict(L=-1), dict(ldw=7), dict(ldo=15), dict(a=None), dict(b=None), dict(w=None),
                dict(adapter=None), dict(out=None), dict(adapter=66), dict(scale=66), dict(a=65), dict(b=65)):
        assert call(**bad) == 1, bad
    for bad in (dict(rank=129), dict(L=1 << 31)):
        assert call(**bad) == 2, bad


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x, w, off = torch.ones(4, 8), torch.ones(2, 8, 16), torch.tensor([0, 2, 4])
    with pytest.raises(ValueError, match="CUDA"):
        sr.seg_matmul(x, w, off)
    with pytest.raises(ValueError, match="CUDA"):
        sr.seg_matmul_grad_w(x, torch.ones(4, 16), off)
    with pytest.raises(ValueError, match="CUDA"):
        sr.seg_lora(x, w[0].t(), w, w, off, off)
