"""Which kernel computes the adapters' inner products: dot products by rows where
that was measured faster, tiles where they were, and the same results on both
sides of the rule."""
import os
import subprocess

import numpy as np
import pytest

from segmented_reduction_csr_gb300 import build as srbuild

# (requests, rows of each, rank): measured faster by rows, and by tiles
ROWS = [(1, 1, 16), (1, 4, 64), (16, 4, 64), (96, 1, 16), (96, 4, 16), (256, 4, 8), (1024, 2, 16), (4096, 1, 16), (4096, 2, 16), (4096, 1, 8), (96, 1, 64)]
TILES = [(96, 4, 64), (256, 2, 64), (1024, 1, 64), (1024, 4, 64), (4096, 1, 64), (4096, 4, 64), (4096, 4, 16), (4096, 4, 8), (1024, 4, 16), (16, 20, 8), (1, 300, 16)]

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include "seg_product.cuh"
int main(int argc, char** argv) {
    segred::ProductParams p{};
    p.S = std::atoll(argv[1]), p.R = p.S * std::atoll(argv[2]), p.N = std::atoll(argv[3]), p.K = 4096;
    std::printf("%d\n", segred::lora_by_rows(p) ? 1 : 0);
}
"""


def test_rule(tmp_path):
    lib = srbuild.build()
    src, exe = tmp_path / "rule.cpp", tmp_path / "rule"
    src.write_text(SOURCE)
    subprocess.run([srbuild._nvcc(), "-std=c++17", "-I", srbuild.CSRC, "-o", str(exe), str(src), lib, "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib)],
                   check=True, capture_output=True, text=True)
    for cases, by_rows in ((ROWS, "1"), (TILES, "0")):
        for c in cases:
            assert subprocess.run([str(exe), *map(str, c)], capture_output=True, text=True, check=True).stdout.strip() == by_rows, c


@pytest.mark.gpu
@pytest.mark.parametrize("requests,rows,rank", ((64, 4, 64), (65, 4, 64), (128, 3, 44), (1300, 2, 16), (1300, 2, 17), (1300, 3, 16), (4096, 4, 64), (4097, 1, 8)))
def test_both_sides(requests, rows, rank):
    from tests.test_product_gpu import check, mods, normal, ref_lora
    torch, sr = mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(requests + rank)
    k, n, adapters = 96, 136, 9
    off = 1 + rows * np.arange(requests + 1)
    x, w = normal(g, (int(off[-1]) + 2, k), "bfloat16"), normal(g, (n, k), "bfloat16", k ** -0.5)
    a, b = normal(g, (adapters, rank, k), "bfloat16", k ** -0.5), normal(g, (adapters, n, rank), "bfloat16", rank ** -0.5)
    ids = np.random.default_rng(rank).integers(-1, adapters, requests)
    got = sr.seg_lora(x, w, a, b, torch.from_numpy(off).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda())
    y, m = ref_lora(x, w, a, b, off, ids, None)
    check(got, y, m, k + rank, (requests, rows, rank))
    assert sr.device_status() == 0
