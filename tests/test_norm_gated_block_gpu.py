"""A block as it is used: rows normalised with their expert's own weights, the
gated feed-forward block, and the projection back, forward and backward in one
autograd graph, eager and captured.

The stages' own errors are tested where they are; here the whole is compared
with the same formulas in 64 bits.  Each of the three stages rounds to 16 bits
(2^-8 or 2^-11 of each value; backward as many times again), and the sums behind
a rounding average its errors: outputs and gradients are within 12 roundings of
their tensor's root mean square size, which 5 standard deviations of 6 of them
in a row are."""
import numpy as np
import pytest

from tests.test_gated_gpu import act64
from tests.test_product_gpu import case, mods, normal

pytestmark = pytest.mark.gpu


def block64(x, weight, bias, w, v, off, act):
    """The block's result in 64 bits, with its graph."""
    torch, _ = mods()
    parts = [torch.zeros(int(off[0]), v.shape[2], dtype=torch.float64, device="cuda")]
    for s in range(len(off) - 1):
        xs = x[int(off[s]):int(off[s + 1])]
        c = xs - xs.mean(1, keepdim=True)
        z = c / torch.sqrt(c.square().mean(1, keepdim=True) + 1e-5)
        pre = (z * weight[s] + bias[s]) @ w[s]
        n = pre.shape[1] // 2
        parts.append((act64(act, pre[:, :n])[0] * pre[:, n:]) @ v[s])
    parts.append(torch.zeros(x.shape[0] - int(off[-1]), v.shape[2], dtype=torch.float64, device="cuda"))
    return torch.cat(parts)


def inputs(kind, seed, dtype, k=136, n=88):
    torch, _ = mods()
    off, rows, do, g = case(kind, seed, before=3, after=4)
    s = len(off) - 1
    leaves = [normal(g, (rows, k), dtype), 1 + 0.1 * normal(g, (s, k), "float32"), 0.1 * normal(g, (s, k), "float32"),
              normal(g, (s, k, 2 * n), dtype, k ** -0.5), normal(g, (s, n, k), dtype, n ** -0.5)]
    return off, do, leaves, normal(g, (rows, k), dtype)


def block(leaves, do, act="silu"):
    _, sr = mods()
    x, weight, bias, w, v = leaves
    return sr.segment_matmul(sr.segment_gated(sr.segment_layer_norm(x, weight, bias, do), w, do, act), v, do)


@pytest.mark.parametrize("dtype,unit", (("bfloat16", 2.0 ** -8), ("float16", 2.0 ** -11), ("float32", 2.0 ** -18)))
@pytest.mark.parametrize("kind", ("mixed", "skewed", "single rows"))
def test_block_forward_and_backward(dtype, unit, kind):
    torch, sr = mods()
    off, do, leaves, dy = inputs(kind, 11, dtype)
    for t in leaves:
        t.requires_grad_()
    y = block(leaves, do)
    grads = torch.autograd.grad(y, leaves, dy)
    exact = [t.detach().double().requires_grad_() for t in leaves]
    want = block64(*exact, off, "silu")
    wgrads = torch.autograd.grad(want, exact, dy.double())
    for name, a, b in zip(("y", "x", "weight", "bias", "w", "v"), (y, *grads), (want, *wgrads)):
        assert a.shape == b.shape
        scale = float(b.detach().square().mean().sqrt())
        err = (a.detach().double() - b.detach()).abs()
        # large values have larger roundings of their own
        assert bool((err <= 12 * unit * (scale + b.detach().abs())).all()), (name, float((err / (scale + b.detach().abs())).max()) / unit)
    assert sr.device_status() == 0


def test_block_in_a_graph():
    """Forward and backward captured together, replayed on new values in the same places."""
    torch, sr = mods()
    off, do, leaves, dy = inputs("mixed", 12, "bfloat16")
    new = inputs("mixed", 13, "bfloat16")[2]
    x, weight, bias, w, v = leaves

    def step():
        y0, mean, rstd = sr.seg_layer_norm(x, weight, bias, do, with_stats=True)
        h, pre = sr.seg_gated(y0, w, do, with_pre=True)
        y = sr.seg_matmul(h, v, do)
        dh, dv = sr.seg_matmul(dy, v, do, transpose_w=True), sr.seg_matmul_grad_w(h, dy, do)
        dy0, dw = sr.seg_gated_grad(y0, w, pre, dh, do)
        return (y, dv, dw) + sr.seg_layer_norm_grad(x, dy0, mean, rstd, weight, do)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for old, value in zip(leaves, new):
        old.copy_(value)
    graph.replay()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sr.device_status() == 0


def test_two_threads_at_once():
    """Calls from two threads on streams of their own, each with its own scratch."""
    import threading
    torch, sr = mods()
    sets = [inputs(kind, seed, "bfloat16") for kind, seed in (("mixed", 21), ("skewed", 22))]
    want = [block(leaves, do) for _, do, leaves, _ in sets]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        _, do, leaves, _ = sets[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                if not torch.equal(block(leaves, do), want[i]):
                    bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_example_with_gated_experts():
    torch, sr = mods()
    from examples import expert_layer as ex
    losses = ex.train(tokens=257, width=128, hidden=72, experts=5, steps=3, gated=True)
    assert all(np.isfinite(losses)) and losses == ex.train(tokens=257, width=128, hidden=72, experts=5, steps=3, gated=True)
    # its gradients against differences: the loss along a direction of the norm's and the gate's weights
    torch.manual_seed(3)
    layer = ex.ExpertLayer(64, 40, 3, gated=True, dtype=torch.float32)
    x = torch.randn(50, 64, device="cuda")
    leaves = [layer.norm_weight, layer.norm_bias, layer.up]

    def value():
        return layer(x).double().square().sum()
    grads = torch.autograd.grad(value(), leaves)
    h = 2.0 ** -8
    for t, g in zip(leaves, grads):
        d = torch.randn_like(t)
        with torch.no_grad():
            t.add_(d, alpha=h)
            up = value()
            t.add_(d, alpha=-2 * h)
            down = value()
            t.add_(d, alpha=h)
        got, num = float((g.double() * d.double()).sum()), float((up - down) / (2 * h))
        # float32 values (2^-18 of the sum, over 2 h = 2^-7) and third derivatives
        assert abs(got - num) <= (2.0 ** -11 + 64 * h * h) * float(up.abs() + down.abs()), (got, num)
