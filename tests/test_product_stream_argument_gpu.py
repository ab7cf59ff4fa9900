"""Products with ``stream=``: the memory they read and write is not anyone
else's meanwhile.  Shown by the addresses that the allocator gives out; nothing
here writes memory that another stream may be using."""
import pytest

from tests.test_product_gpu import mods, normal

pytestmark = pytest.mark.gpu


def calls():
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows, k, n = 4096, 520, 1032
    off = torch.tensor([0, 1000, 4096], device="cuda")
    x, w, dy = normal(g, (rows, k), "bfloat16"), normal(g, (2, k, n), "bfloat16", 0.05), normal(g, (rows, n), "bfloat16")
    shared = normal(g, (n, k), "bfloat16", 0.05)
    a, b, ids = normal(g, (2, 8, k), "bfloat16", 0.05), normal(g, (2, n, 8), "bfloat16"), torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    return {"matmul": (lambda x=x, **kw: sr.seg_matmul(x, w, off, **kw), x),
            "grad": (lambda x=x, **kw: sr.seg_matmul_grad_w(x, dy, off, **kw), x),
            "lora": (lambda x=x, **kw: sr.seg_lora(x, shared, a, b, off, ids, **kw), x)}


@pytest.mark.parametrize("name", ("matmul", "grad", "lora"))
def test_a_result_is_memory_of_the_stream_that_writes_it(name):
    torch, sr = mods()
    call, _ = calls()[name]
    stream = torch.cuda.Stream()
    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # a block of the current stream that has just been let go, of a result's size
    block = torch.empty_like(want)
    at = block.data_ptr()
    del block
    got = call(stream=stream)
    torch.cuda.synchronize()
    assert got.data_ptr() != at and torch.equal(got, want)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    assert call(stream=stream, out=out) is out
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("name", ("matmul", "grad", "lora"))
def test_an_input_that_goes_keeps_its_memory_until_the_stream_is_through(name):
    torch, sr = mods()
    call, x = calls()[name]
    stream = torch.cuda.Stream()
    want = call()
    call(stream=stream)      # scratch and kernels are there
    mine = x.clone()
    torch.cuda.synchronize()
    at = mine.data_ptr()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)       # some 50 ms before the call's turn
    got = call(mine, stream=stream)
    size = mine.shape
    del mine
    others = [torch.empty(size, dtype=x.dtype, device="cuda") for _ in range(4)]
    assert at not in [o.data_ptr() for o in others]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
