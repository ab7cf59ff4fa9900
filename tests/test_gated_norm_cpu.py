"""The host checks of the gated block and of the norm: every bad argument is
refused before any CUDA call."""
import pytest

import segmented_reduction_csr_gb300 as sr
from segmented_reduction_csr_gb300 import build as srbuild


@pytest.fixture(scope="module")
def lib():
    srbuild.build()
    return sr.load_library()


def test_gated_host_checks(lib):
    def call(x=64, dtype=4, R=10, K=8, ldx=8, w=64, N=16, ldw=32, stride=256, trans=0, off=64, odt=1, S=3, act=0, out=64, ldo=16, pre=64, pt=None, ldp=32):
        return lib.seg_gated(x, dtype, R, K, ldx, w, N, ldw, stride, trans, off, odt, S, act, out, ldo, pre, dtype if pt is None else pt, ldp, None)
    assert call(R=0) == 0 and call(N=0, ldw=0, ldo=0, stride=0, ldp=0) == 0      # nothing to do
    assert call(R=0, pre=None, ldp=0) == 0
    for bad in (dict(dtype=0), dict(dtype=5), dict(odt=2), dict(R=-1), dict(K=-1), dict(N=-1), dict(S=-1), dict(act=-1), dict(act=5),
                dict(ldx=7), dict(ldw=31), dict(ldo=15), dict(ldp=31), dict(trans=2), dict(stride=255), dict(stride=-1),
                dict(trans=1, ldw=7), dict(trans=1, ldw=8, stride=255), dict(x=None), dict(w=None), dict(off=None), dict(out=None),
                dict(x=65), dict(w=65), dict(out=65), dict(pre=65), dict(pt=3), dict(pt=2, pre=66), dict(dtype=2, pt=4), dict(off=68), dict(dtype=2, x=66), dict(dtype=2, out=66), dict(dtype=2, pre=66)):
        assert call(**bad) == 1, bad
    for bad in (dict(R=1 << 31), dict(S=1 << 31), dict(K=(1 << 20) + 1, ldx=1 << 21, stride=1 << 40), dict(N=(1 << 19) + 1, ldw=1 << 21, stride=1 << 40, ldo=1 << 21, ldp=1 << 21)):
        assert call(**bad) == 2, bad


def test_gated_grad_host_checks(lib):
    def call(pre=64, pt=2, R=10, N=16, ldp=32, dy=64, dtype=3, ldy=16, act=1, dpre=64, ldd=32):
        return lib.seg_gated_grad(pre, pt, R, N, ldp, dy, dtype, ldy, act, dpre, ldd, None)
    assert call(R=0) == 0 and call(N=0, ldp=0, ldy=0, ldd=0) == 0
    for bad in (dict(dtype=1), dict(R=-1), dict(N=-1), dict(ldp=31), dict(ldy=15), dict(ldd=31), dict(act=9), dict(pre=None), dict(dy=None),
                dict(dpre=None), dict(pre=66), dict(pt=4), dict(dtype=2, pt=3), dict(dy=65), dict(dpre=65), dict(dtype=2, dy=66)):
        assert call(**bad) == 1, bad
    assert call(R=1 << 31) == 2 and call(N=(1 << 19) + 1, ldp=1 << 21, ldy=1 << 21, ldd=1 << 21) == 2


def test_layer_norm_host_checks(lib):
    def call(x=64, dtype=4, R=10, F=8, ldx=8, w=64, b=64, wt=2, off=64, odt=1, S=3, eps=1e-5, out=64, ldo=8, mean=64, rstd=64):
        return lib.seg_layer_norm(x, dtype, R, F, ldx, w, b, wt, off, odt, S, eps, out, ldo, mean, rstd, None)
    assert call(R=0) == 0 and call(F=0, ldx=0, ldo=0) == 0 and call(R=0, off=None, S=1) == 0 and call(R=0, w=None, b=None) == 0
    for bad in (dict(dtype=0), dict(dtype=5), dict(wt=3), dict(wt=0), dict(R=-1), dict(F=-1), dict(S=-1), dict(off=None), dict(off=None, S=0),
                dict(ldx=7), dict(ldo=7), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(out=None),
                dict(x=65), dict(out=65), dict(w=66), dict(b=66), dict(mean=66), dict(rstd=66), dict(off=68), dict(odt=3)):
        assert call(**bad) == 1, bad
    for bad in (dict(R=1 << 31), dict(S=1 << 31), dict(F=(1 << 20) + 1, ldx=1 << 21, ldo=1 << 21)):
        assert call(**bad) == 2, bad


def test_layer_norm_grad_host_checks(lib):
    def call(x=64, dtype=4, R=10, F=8, ldx=8, dy=64, ldy=8, mean=64, rstd=64, w=64, wt=2, off=64, odt=1, S=3, dx=64, lddx=8, dw=64, db=64):
        return lib.seg_layer_norm_grad(x, dtype, R, F, ldx, dy, ldy, mean, rstd, w, wt, off, odt, S, dx, lddx, dw, db, None)
    assert call(F=0, ldx=0, ldy=0, lddx=0) == 0 and call(dx=None, dw=None, db=None) == 0
    for bad in (dict(dtype=1), dict(wt=3), dict(ldx=7), dict(ldy=7), dict(lddx=7), dict(x=None), dict(dy=None), dict(mean=None), dict(rstd=None),
                dict(off=None), dict(dy=65), dict(dx=65), dict(dw=66), dict(db=66), dict(w=66), dict(mean=66), dict(rstd=66), dict(off=66)):
        assert call(**bad) == 1, bad
    assert call(R=1 << 31) == 2


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    x, w, off = torch.ones(4, 8), torch.ones(2, 8, 16), torch.tensor([0, 2, 4])
    with pytest.raises(ValueError, match="CUDA"):
        sr.seg_gated(x, w, off)
    with pytest.raises(ValueError, match="CUDA"):
        sr.seg_gated_grad(x, w, x, x, off)
    with pytest.raises(ValueError, match="CUDA"):
        sr.seg_layer_norm(x)
    with pytest.raises(ValueError, match="CUDA"):
        sr.seg_layer_norm(x, offsets=off)
    with pytest.raises(ValueError, match="CUDA"):
        sr.seg_layer_norm_grad(x, x, x[0], x[0])


def test_binding_refuses_arguments_that_do_not_fit():
    """On tensors without data that say that they are on a GPU."""
    torch = pytest.importorskip("torch")

    class Like:
        """The shape, type and strides of a tensor, on cuda:0."""
        def __init__(self, *shape, dtype=torch.float32, step=None):
            self.t = torch.empty(shape, dtype=dtype, device="meta")
            self.shape, self.dtype, self.is_cuda, self.device = self.t.shape, dtype, True, torch.device("cuda:0")
            self.step = step

        def dim(self):
            return len(self.shape)

        def numel(self):
            return self.t.numel()

        def is_contiguous(self):
            return self.step is None

        def stride(self, i=None):
            s = list(self.t.stride())
            if self.step is not None:
                s[-1] = self.step
            return s if i is None else s[i]

        def data_ptr(self):
            raise AssertionError("the call was not refused")

    x, w, off = Like(4, 8), Like(2, 8, 16), Like(3, dtype=torch.int64)
    gated = [
        (ValueError, dict(w=Like(2, 8, 15))), (ValueError, dict(w=Like(8, 16))), (ValueError, dict(w=Like(2, 9, 16))), (ValueError, dict(w=Like(3, 8, 16))),
        (TypeError, dict(w=Like(2, 8, 16, dtype=torch.float16))), (ValueError, dict(x=Like(4, 8, 2))), (ValueError, dict(x=Like(4, 8, step=2))),
        (ValueError, dict(activation="swish")), (ValueError, dict(out=Like(4, 7))), (TypeError, dict(out=Like(4, 8, dtype=torch.float16))),
        (ValueError, dict(pre=Like(4, 8))), (TypeError, dict(pre=Like(4, 16, dtype=torch.bfloat16))), (ValueError, dict(offsets=Like(3, 1, dtype=torch.int64))), (TypeError, dict(x=Like(4, 8, dtype=torch.float64))),
    ]
    for error, bad in gated:
        with pytest.raises(error):
            sr.seg_gated(**{**dict(x=x, w=w, offsets=off, out=Like(4, 8), pre=Like(4, 16)), **bad})
    grad = [(ValueError, dict(pre=Like(4, 8))), (ValueError, dict(dy=Like(4, 16))), (TypeError, dict(dy=Like(4, 8, dtype=torch.bfloat16))),
            (TypeError, dict(dw_dtype=torch.float16)), (ValueError, dict(dy=Like(4, 8, step=0)))]
    for error, bad in grad:
        with pytest.raises(error):
            sr.seg_gated_grad(**{**dict(x=x, w=w, pre=Like(4, 16), dy=Like(4, 8), offsets=off), **bad})
    norm = [(ValueError, dict(weight=Like(8))), (ValueError, dict(bias=Like(3, 8))), (TypeError, dict(bias=Like(2, 8, dtype=torch.float16))),
            (TypeError, dict(weight=Like(2, 8, dtype=torch.float16))), (ValueError, dict(eps=-1.0)), (ValueError, dict(eps=float("nan"))),
            (ValueError, dict(out=Like(4, 9))), (ValueError, dict(offsets=None)), (ValueError, dict(weight=Like(2, 8, step=2))),
            (ValueError, dict(x=Like(8)))]
    for error, bad in norm:
        with pytest.raises(error):
            sr.seg_layer_norm(**{**dict(x=x, weight=Like(2, 8), bias=Like(2, 8), offsets=off, out=Like(4, 8)), **bad})
    back = [(ValueError, dict(dy=Like(4, 7))), (ValueError, dict(mean=Like(5))), (TypeError, dict(rstd=Like(4, dtype=torch.float16))),
            (TypeError, dict(weight=None, weight_dtype=torch.float16)), (ValueError, dict(weight=Like(8)))]
    for error, bad in back:
        with pytest.raises(error):
            sr.seg_layer_norm_grad(**{**dict(x=x, dy=Like(4, 8), mean=Like(4), rstd=Like(4), weight=Like(2, 8), offsets=off), **bad})
