"""Layer norm of rows far from zero: where a row's mean is more than half its
deviation, it is corrected by the mean of what is left, so that neither the first
mean's rounding nor that of 1 / F is enlarged by rstd (up to 316 with eps 1e-5).

Tolerances, with u = 2^-24, F columns and c = (F / 256 + 80) u for a sum (as in
the tests of the norm).  The first mean is within dm = c mean|x|.  What is left of
a value, d = x - mean, is within u of itself; its mean, the correction, is within
c mean|d| <= c (mean|x - m| + dm).  So z = (d - correction) rstd is within
rstd (c + 4 u) (mean|x - m| + |x - m| + 2 dm) of the exact one beside rstd's own
error.  The squares' sum exceeds F var by F dm^2 at most, which is taken away
again: the variance is within 2 c (var + 2 dm^2), rstd within c + 8 u + 4 c dm^2
rstd^2 of itself.  Where |m| rstd is at most 1/2 (0.51 here, for the roundings of
the comparison) the mean may be left as it is: dm more for it, rstd dm for z, dm^2
rstd^2 for rstd.  A rounding adds half a step."""
import pytest

from tests.test_gated_gpu import close
from tests.test_product_gpu import TYPES, mods, normal

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# aligned and not, a few threads to a block's for a row, rows from shared memory, rows that are read again
WIDTHS = (3, 24, 41, 100, 333, 1000, 1001, 3001, 5000, 9000, 9001, 12296, 16392, 16385, 20000, 40000)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("f", WIDTHS)
def test_constant_rows_give_the_bias(dtype, f):
    """No variance: z is 0 whatever the value, and with eps 0 it is no number."""
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(f)
    values = [3.0, 100.0, 1000.0, 1.0 / 3, 1234.567, -7.7e-3, 0.0, 6e4]
    x = torch.tensor(values, device="cuda")[:, None].expand(-1, f).to(getattr(torch, dtype)).contiguous()
    b = normal(g, (f,), "float32")
    y, mean, rstd = sr.seg_layer_norm(x, None, b, with_stats=True)
    assert torch.equal(y, b.to(x.dtype).expand_as(x))
    assert torch.equal(mean, x[:, 0].float())
    close(rstd, torch.full_like(rstd, 1e-5 ** -0.5).double(), 8 * U * 317, (dtype, f))
    assert bool(torch.isnan(sr.seg_layer_norm(x, None, b, eps=0.0)).all())


def check(y, mean, rstd, x, w, b, eps, where):
    torch, _ = mods()
    f = x.shape[1]
    c = (f / 256 + 80) * U
    xs = x.double()
    m = xs.mean(1, keepdim=True)
    left = xs - m
    v = left.square().mean(1, keepdim=True)
    r = 1 / torch.sqrt(v + eps)
    dm, size = c * xs.abs().mean(1, keepdim=True), left.abs().mean(1, keepdim=True)
    near = (m.abs() * r <= 0.51).double() * dm          # of a mean that is not corrected
    rel = c + 8 * U + 4 * c * dm.square() * r.square() + near.square() * r.square()
    z, ww, bb = left * r, w.double(), b.double()
    tol = r * (c + 4 * U) * (size + left.abs() + 2 * dm) + r * near + z.abs() * rel
    close(y, z * ww + bb, ww.abs() * tol + 2 * U * ((ww * z).abs() + bb.abs()), where)
    close(mean, m[:, 0], ((c + 4 * U) * (size + 2 * dm) + near + 2 * U * m.abs())[:, 0], (where, "mean"))
    close(rstd, r[:, 0], (r * rel)[:, 0], (where, "rstd"))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("f", WIDTHS)
def test_rows_far_from_zero_with_a_small_spread(dtype, f):
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(f)
    at = torch.tensor([0.0, 3.0, 100.0, 1000.0, -1234.567, 3e4, 0.1, -50.0, 700.0], device="cuda")[:, None]
    spread = torch.tensor([1.0, 0.1, 0.01, 0.25, 1e-3, 2.0, 1e-4, 1e-2, 0.0], device="cuda")[:, None]
    x = (at + spread * normal(g, (9, f), "float32")).to(getattr(torch, dtype))
    x[8, f // 2] += 4          # one value alone is another
    w, b = normal(g, (f,), "float32"), normal(g, (f,), "float32")
    check(*sr.seg_layer_norm(x, w, b, with_stats=True), x, w, b, 1e-5, (dtype, f))


@pytest.mark.parametrize("f", (41, 1000, 9001, 16392, 16385))
def test_values_whose_squares_pass_float32s_range(f):
    """Constant rows of any size still give the bias, others of that size rows of it too (rstd is 0)."""
    torch, sr = mods()
    x = torch.full((3, f), 1e33, device="cuda")
    x[1] = -3.3e29
    x[2, 0] = 2e33
    b = torch.ones(f, device="cuda")
    assert torch.equal(sr.seg_layer_norm(x, None, b), torch.ones_like(x))


@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_at_rows_far_from_zero(dtype):
    """The mean that is kept for the backward pass is the corrected one: constant rows have z = 0 there too."""
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for f in (41, 1000):
        x = torch.full((7, f), 1000.0, device="cuda").to(getattr(torch, dtype))
        dy = normal(g, (7, f), dtype)
        _, mean, rstd = sr.seg_layer_norm(x, with_stats=True)
        dx, dw, _ = sr.seg_layer_norm_grad(x, dy, mean, rstd)
        assert not bool(dw.any())
        d = dy.double()
        want = (d - d.mean(1, keepdim=True)) * 1e-5 ** -0.5
        close(dx, want, 317 * 100 * U * (d.abs() + d.abs().mean(1, keepdim=True)), (dtype, f))
