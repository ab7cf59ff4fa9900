"""Products in graphs: every graph has scratch of its own, so graphs that were
captured from one stream may run at the same time on others, beside calls on
the stream of the capture, and give the scratch back when they go."""
import gc

import numpy as np
import pytest

from tests.test_product_gpu import mods, normal

pytestmark = pytest.mark.gpu


def make_calls(seed, rows, k=1024, n=1288, rank=16):
    """Calls that keep intermediate values in scratch: inner products, packed operands, partial sums."""
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    off = torch.tensor([0, rows // 3, rows - 5, rows], device="cuda")
    x, w = normal(g, (rows, k), "bfloat16"), normal(g, (n, k), "bfloat16", k ** -0.5)
    a, b = normal(g, (3, rank, k), "bfloat16", k ** -0.5), normal(g, (3, n, rank), "bfloat16")
    ids = torch.tensor([0, 2, 1], dtype=torch.int32, device="cuda")
    odd, dy = normal(g, (rows, 63), "bfloat16"), normal(g, (rows, 65), "bfloat16")
    wo = normal(g, (3, 63, 65), "bfloat16")
    return [lambda: sr.seg_lora(x, w, a, b, off, ids), lambda: sr.seg_matmul(odd, wo, off), lambda: sr.seg_matmul_grad_w(odd, dy, off)]


def capture(calls, times=1):
    torch, _ = mods()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):       # torch's own capture stream, the same one every time
        for _ in range(times):
            got = [c() for c in calls]
    return graph, got


def test_graphs_of_one_capture_stream_at_the_same_time():
    torch, sr = mods()
    sets = [make_calls(seed, rows) for seed, rows in ((1, 4000), (2, 3000), (3, 700))]
    want = [[c() for c in calls] for calls in sets]
    torch.cuda.synchronize()
    graphs = [capture(calls, times=3) for calls in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for rep in range(10):
        for (graph, got), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                for v in got:
                    v.zero_()
                for _ in range(3):
                    graph.replay()
        # and calls on the stream of the captures meanwhile
        with torch.cuda.stream(torch.cuda.graph.default_capture_stream):
            between = [c() for c in sets[rep % 3]]
        torch.cuda.synchronize()
        for (_, got), expect in zip(graphs, want):
            assert all(torch.equal(u, v) for u, v in zip(got, expect)), rep
        assert all(torch.equal(u, v) for u, v in zip(between, want[rep % 3]))
    assert sr.device_status() == 0


def test_two_streams_of_one_capture():
    """Branches of a graph run at the same time."""
    torch, sr = mods()
    sets = [make_calls(seed, rows) for seed, rows in ((4, 3000), (5, 2500))]
    want = [[c() for c in calls] for calls in sets]
    torch.cuda.synchronize()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            other = [c() for c in sets[1]]
        own = [c() for c in sets[0]]
        main.wait_stream(side)
    for rep in range(5):
        for v in own + other:
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(own + other, want[0] + want[1])), rep
    assert sr.device_status() == 0


def test_scratch_of_graphs_that_are_gone_is_used_again():
    torch, sr = mods()
    calls = make_calls(6, 60000, k=264, n=136, rank=128)      # 30 MB of inner products
    want = [c() for c in calls]
    free = []
    for rep in range(6):
        graph, got = capture(calls)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want))
        del graph, got
        gc.collect()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        free.append(torch.cuda.mem_get_info()[0])
    # (other processes may hold memory of the same GPU: the most that is free stands for this one)
    assert max(free[3:]) >= free[0] - (16 << 20), np.array(free) / 2 ** 20
