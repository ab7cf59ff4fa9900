"""The products' planner and launcher agree on the tile: a plan counts as many
tiles of rows as the kernel that is launched for it can need.

Evaluated on the host for many shapes, by a small program linked with the
library: the plan of each shape, the columns of the tile that is launched for
it, and the most tiles that rows in so many segments can take."""
import os
import subprocess

import pytest

from segmented_reduction_csr_gb300 import build as srbuild

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include "seg_product.cuh"
using namespace segred;

// The most tiles of `size` rows that `rows` rows in at most `segments` segments can take.
static int64_t most_tiles(int64_t rows, int64_t segments, int64_t size) {
    const int64_t used = segments < rows ? segments : rows;
    // a row in all but one of them, and of those as many as can be a row above whole tiles
    return used == 0 ? 0 : used + (rows - used) / size;
}

int main() {
    std::mt19937_64 rng(1);
    auto log = [&](double top) { return static_cast<int64_t>(std::exp2(std::uniform_real_distribution<double>(0, top)(rng))); };
    int64_t tried = 0, loaders = 0, bad = 0;
    for (int i = 0; i < 400000; ++i) {
        ProductParams p{};
        const int types[3] = {PT_F32, PT_F16, PT_BF16};
        p.type = p.out_type = types[rng() % 3];
        const int size = p.type == PT_F32 ? 4 : 2;
        p.R = log(17), p.K = log(12), p.N = rng() % 2 ? 1 + rng() % 128 : log(12), p.S = log(14);
        p.trans = rng() % 2;
        p.sms = rng() % 2 ? 152 : 1 + rng() % 200;
        p.ldx = p.K + (rng() % 2 ? rng() % 9 : 0);
        p.ldw = (p.trans ? p.K : p.N) + (rng() % 2 ? rng() % 9 : 0);
        p.stride_w = (p.trans ? p.N : p.K) * p.ldw + (rng() % 2 ? rng() % 9 : 0);
        p.ldo = p.N;
        p.x = reinterpret_cast<void*>(uintptr_t(1 << 20) + (rng() % 2 ? rng() % 8 * size : 0));
        p.w = reinterpret_cast<void*>(uintptr_t(1 << 20) + (rng() % 2 ? rng() % 8 * size : 0));
        p.out = reinterpret_cast<void*>(uintptr_t(1 << 20));
        int mode = PRODUCT_FORWARD;
        const int kind = rng() % 3;
        if (kind == 1) {                 // the adapters' inner products
            p.index = reinterpret_cast<const int32_t*>(uintptr_t(1 << 20));
            p.L = log(18);
            p.N = 1 + rng() % 128;
            p.trans = 1, p.ldw = p.K, p.stride_w = p.N * p.K, p.ldo = p.N, p.out_type = PT_F32;
        } else if (kind == 2) {
            mode = PRODUCT_ADAPTERS;
            p.trans = 1, p.ldw = p.K, p.rank = 1 + rng() % 128, p.L = log(18);
        }
        const ProductPlan d = plan_product(mode, p);
        if (d.empty || d.too_many) continue;
        ++tried;
        loaders += !d.tensor;
        const int64_t size_n = TILE_COLUMNS;
        const int64_t need = most_tiles(p.R, mode == PRODUCT_ADAPTERS ? 1 : p.S, size_n);
        if (d.row_tiles < need && ++bad <= 5)
            std::printf("mode %d type %d R %lld S %lld K %lld N %lld L %lld sms %d: tensor %d narrow %d, row_tiles %lld of %lld\n", mode, p.type,
                        (long long)p.R, (long long)p.S, (long long)p.K, (long long)p.N, (long long)p.L, p.sms, d.tensor, d.narrow,
                        (long long)d.row_tiles, (long long)need);
    }
    std::printf("tried %lld loaders %lld bad %lld\n", (long long)tried, (long long)loaders, (long long)bad);
    return bad != 0 || tried < 300000 || loaders < 1000;
}
"""


def run(tmp_path, tile):
    lib = srbuild.build()
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(SOURCE.replace("TILE_COLUMNS", tile).replace("#include <random>", "#include <cmath>\n#include <random>"))
    subprocess.run([srbuild._nvcc(), "-std=c++17", "-O1", "-I", srbuild.CSRC, "-o", str(exe), str(src), lib,
                    "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib)], check=True, capture_output=True, text=True)
    return subprocess.run([str(exe)], capture_output=True, text=True)


def test_plans_count_the_tiles_that_are_launched(tmp_path):
    r = run(tmp_path, "product_tile_columns(p, d)")
    assert r.returncode == 0, r.stdout
