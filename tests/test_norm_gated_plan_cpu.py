"""The planners of the norm and of the gated block, evaluated on the host for many
shapes: a norm's plan has threads and registers for every column, blocks for
every row and shared memory that an SM has; a gated block's counts as many tiles
of rows as the kernel that is launched for it can need, and leaves no operand
that a tensor copy cannot take."""
import os
import subprocess

from segmented_reduction_csr_gb300 import build as srbuild

SOURCE = r"""
#include <cmath>
#include <cstdio>
#include <random>
#include "seg_norm.cuh"
#include "seg_product.cuh"
using namespace segred;

int main() {
    std::mt19937_64 rng(1);
    auto log = [&](double top) { return static_cast<int64_t>(std::exp2(std::uniform_real_distribution<double>(0, top)(rng))); };
    auto at = [&](int size) { return reinterpret_cast<void*>(uintptr_t(1 << 20) + (rng() % 2 ? rng() % 8 * size : 0)); };
    const int types[3] = {PT_F32, PT_F16, PT_BF16};
    long bad = 0, wide = 0, odd = 0, tiled = 0, fused = 0, unfused = 0, tried = 0;
    auto wrong = [&](const char* what, long long a, long long b, long long c) {
        if (++bad <= 8) std::printf("%s %lld %lld %lld\n", what, a, b, c);
    };
    for (int i = 0; i < 300000; ++i) {
        const bool grad = rng() % 2;
        NormParams p{};
        p.type = types[rng() % 3];
        const int size = p.type == PT_F32 ? 4 : 2, v = 16 / size;
        p.weight_type = rng() % 2 ? p.type : PT_F32;
        p.R = log(31) > (1ll << 31) - 4096 ? 1 : log(30.9), p.F = rng() % 3 ? log(15) : log(20), p.S = log(20);
        if (rng() % 4 && p.F > v) p.F = p.F / v * v;
        p.ldx = p.F + (rng() % 2 ? 0 : rng() % 17), p.ldy = p.F, p.ldo = p.F;
        p.x = at(size), p.dy = at(size), p.out = rng() % 4 ? at(size) : nullptr;
        p.weight = at(size), p.bias = nullptr;
        p.sms = rng() % 2 ? 152 : 1 + rng() % 200;
        if (!grad && !p.out) p.out = at(size);
        const NormPlan d = plan_norm(grad, p);
        ++tried;
        const int64_t held = int64_t(d.group) * d.per * v * d.tiles;
        if (d.per > 0 && held < p.F) wrong("columns", p.F, held, d.group);
        if (d.per > 0 && d.per * v > 32) wrong("registers", p.F, d.per, d.group);
        if (d.threads % d.group != 0 || d.threads > 1024) wrong("threads", d.threads, d.group, p.F);
        const bool by_row = d.per == 0 && !(d.aligned && d.group == 512);       // a block strides over the rows
        if (by_row ? d.chunks < 1 : d.chunk * d.chunks < p.R) wrong("rows", p.R, d.chunk, d.chunks);
        if (!by_row && d.chunk * (d.chunks - 1) >= p.R) wrong("a block without rows", p.R, d.chunk, d.chunks);
        if (d.chunks > INT32_MAX || d.tiles > 65535) wrong("grid", d.chunks, d.tiles, p.F);
        if (grad && d.partial_bytes < d.chunks * 4 * p.F * 4) wrong("partials", d.partial_bytes, d.chunks, p.F);
        if (d.tiles > 1 && d.sums_bytes < p.R * 8) wrong("sums", d.sums_bytes, p.R, p.F);
        if (d.per == 0 && grad) wrong("no shape", p.F, d.group, 0);
        if (d.per == 0 && d.aligned && d.group == 512 && 3 * p.F * size > 216 * 1024) wrong("ring", p.F, size, 0);
        wide += d.per == 0, odd += !d.aligned, tiled += d.tiles > 1;
    }
    for (int i = 0; i < 300000; ++i) {
        ProductParams p{};
        p.type = p.out_type = types[rng() % 3];
        const int size = p.type == PT_F32 ? 4 : 2, v = 16 / size;
        const int64_t n = rng() % 2 ? 1 + rng() % 128 : log(12);
        p.R = log(17), p.K = log(16.5), p.N = 2 * n, p.S = log(14);
        p.trans = rng() % 2;
        p.sms = rng() % 2 ? 152 : 1 + rng() % 200;
        p.ldx = p.K + (rng() % 2 ? rng() % 9 : 0);
        p.ldw = (p.trans ? p.K : p.N) + (rng() % 2 ? rng() % 9 : 0);
        p.stride_w = (p.trans ? p.N : p.K) * p.ldw + (rng() % 2 ? rng() % 9 : 0);
        p.ldo = n;
        p.x = at(size), p.w = at(size), p.out = at(16);
        const ProductPlan d = plan_product(PRODUCT_GATED, p);
        if (d.empty || d.too_many) continue;
        ++tried;
        const int64_t columns = product_tile_columns(p, d), used = p.S < p.R ? p.S : p.R, need = used + (p.R - used) / columns;
        if (d.row_tiles < need) wrong("tiles", d.row_tiles, need, columns);
        if (int64_t(d.mtiles) * 64 * (d.pair ? 2 : 1) < n) wrong("lanes", d.mtiles, d.pair, n);
        if (d.fused && !d.tensor) wrong("fused without copies", p.K, n, p.S);
        auto whole = [&](int64_t e) { return e % v == 0; };
        const bool fits = reinterpret_cast<uintptr_t>(p.w) % 16 == 0 && whole(p.ldw) && (p.S == 1 || whole(p.stride_w)) && (p.trans || whole(n));
        if (d.fused && !fits && !d.pack_w) wrong("an operand as it is", p.ldw, n, p.trans);
        const int64_t rows = (p.trans ? p.N : p.K) * p.S, cols = p.trans ? p.K : n, halves = p.trans ? 1 : 2;
        if (d.pack_w && d.pack_w_bytes < rows * halves * ((cols * size + 15) / 16 * 16)) wrong("packed", d.pack_w_bytes, rows, cols);
        if (d.fused && p.type != PT_F32 && d.parts == 1 && p.K > 32768) wrong("a sum too long", p.K, 0, 0);
        if (d.fused && p.type == PT_F32 && d.parts == 1 && p.K > 512) wrong("a float32 sum in pieces", p.K, 0, 0);
        fused += d.fused, unfused += !d.fused;
    }
    std::printf("tried %ld bad %ld wide %ld odd %ld tiled %ld fused %ld unfused %ld\n", tried, bad, wide, odd, tiled, fused, unfused);
    return bad != 0 || tried < 400000 || wide < 1000 || odd < 1000 || tiled < 1000 || fused < 1000 || unfused < 1000;
}
"""


def test_plans_have_room_for_every_row_and_column(tmp_path):
    lib = srbuild.build()
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(SOURCE)
    subprocess.run([srbuild._nvcc(), "-std=c++17", "-O1", "-I", srbuild.CSRC, "-o", str(exe), str(src), lib,
                    "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
