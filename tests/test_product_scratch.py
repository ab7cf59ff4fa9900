"""How the products' scratch grows: the old buffer goes, and a call is refused only where what it needs is not there."""
import subprocess

import pytest

from segmented_reduction_csr_gb300 import build as srbuild

SOURCE = r"""
#include <cstdio>
#include <map>
#include "seg_scratch.cuh"
using namespace segred;

static size_t room = 0, held = 0, calls = 0;
static std::map<void*, size_t> live;

static bool grow(Scratch& sc, size_t bytes) {
    return grow_scratch(
        sc, bytes,
        [](void** p, size_t n) {
            ++calls;
            if (held + n > room) return false;
            *p = reinterpret_cast<void*>(calls);
            live[*p] = n, held += n;
            return true;
        },
        [](void* p) { held -= live.at(p), live.erase(p); });
}

#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }

int main() {
    const size_t M = size_t(1) << 20, G = size_t(1) << 30;
    room = 24 * G;
    Scratch sc;
    CHECK(grow(sc, 1) && sc.bytes == M && held == M);                       // the least
    CHECK(grow(sc, M) && calls == 1);                                       // it fits
    CHECK(grow(sc, M + 1) && sc.bytes == 2 * M && held == 2 * M);           // twice, and the old one is gone
    CHECK(grow(sc, 20 * G) && held == sc.bytes && sc.bytes == 20 * G);
    CHECK(grow(sc, 21 * G) && held == sc.bytes && sc.bytes == 21 * G + 256 * M);     // not twice a large one
    CHECK(grow(sc, 24 * G - M) && sc.bytes == 24 * G - M && held == sc.bytes);       // and what is needed where there is no more
    CHECK(!grow(sc, 25 * G) && sc.ptr == nullptr && sc.bytes == 0 && held == 0);     // refused: nothing is held
    CHECK(grow(sc, 3 * M) && sc.bytes == 3 * M);                            // and the next call starts anew
    size_t before = calls;
    for (size_t n = 3 * M; n < 4 * G; n += M / 2) CHECK(grow(sc, n) && sc.bytes >= n && live.size() == 1);
    CHECK(calls - before < 40);                                             // a little more each time does not allocate each time
    std::printf("ok\n");
    return 0;
}
"""


def test_growth(tmp_path):
    src, exe = tmp_path / "scratch.cpp", tmp_path / "scratch"
    src.write_text(SOURCE)
    subprocess.run([srbuild._nvcc(), "-std=c++17", "-I", srbuild.CSRC, "-o", str(exe), str(src)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.gpu
def test_growth_does_not_keep_the_old_buffer_or_double_a_large_one():
    torch = pytest.importorskip("torch")
    import segmented_reduction_csr_gb300 as sr
    rank, rows = 128, (2_000_000, 2_400_000)        # 1.02 and 1.23 GB of inner products
    x = torch.ones(rows[1], 8, dtype=torch.bfloat16, device="cuda")
    w, out = torch.ones(8, 8, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    a, b = torch.ones(1, rank, 8, dtype=torch.bfloat16, device="cuda"), torch.ones(1, 8, rank, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(1, dtype=torch.int32, device="cuda")
    offs = [torch.tensor([0, r], device="cuda") for r in rows]
    stream = torch.cuda.Stream()        # its scratch is first needed here
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for r, off in zip(rows, offs):
        sr.seg_lora(x[:r], w, a, b, off, ids, out=out[:r], stream=stream)
        torch.cuda.synchronize()
        assert bool((out[:r] == 8 + 8 * rank).all())
    assert free - torch.cuda.mem_get_info()[0] < 1_900_000_000
