"""The norm's planner on the host: no block of the backward pass has more than 64 KB
of sums to clear, however many segments without rows there are beside few rows;
where it would, a kernel of its own has the blocks for it."""
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
    std::mt19937_64 rng(2);
    auto log = [&](double top) { return static_cast<int64_t>(std::exp2(std::uniform_real_distribution<double>(0, top)(rng))); };
    long bad = 0, own = 0, shared = 0;
    auto wrong = [&](const char* what, const NormParams& p, const NormPlan& d) {
        if (++bad <= 8) std::printf("%s R %lld S %lld F %lld chunks %lld clear %d\n", what, (long long)p.R, (long long)p.S, (long long)p.F, (long long)d.chunks, d.clear_blocks);
    };
    const int types[3] = {PT_F32, PT_F16, PT_BF16};
    auto at = [](int i) { return reinterpret_cast<void*>(uintptr_t(i) << 20); };
    for (int i = 0; i < 200000; ++i) {
        NormParams p{};
        p.type = types[rng() % 3];
        p.weight_type = rng() % 2 ? p.type : PT_F32;
        p.R = log(20), p.F = log(rng() % 4 ? 14 : 20), p.S = log(21);
        p.ldx = p.ldy = p.ldo = p.F;
        p.x = at(1), p.dy = at(2), p.out = rng() % 3 ? at(3) : nullptr;
        p.dweight = rng() % 3 ? at(4) : nullptr, p.dbias = rng() % 3 ? at(5) : nullptr;
        const bool by_segment = rng() % 8;
        p.offsets = by_segment ? at(6) : nullptr;
        if (!by_segment) p.S = 1;
        p.sms = 152;
        const NormPlan d = plan_norm(true, p);
        const double bytes = double(p.S) * p.F * (p.weight_type == PT_F32 ? 4 : 2) * ((p.dweight ? 1 : 0) + (p.dbias ? 1 : 0));
        if (!by_segment && d.clear_blocks) wrong("nothing to clear", p, d);
        if (by_segment && d.clear_blocks == 0 && bytes > 65536.0 * d.chunks * d.tiles) wrong("few blocks clear", p, d);
        // 32 segments x 512 columns a warp, or all the blocks that an SM has room for
        const int64_t tiles = (p.S + 31) / 32 * ((p.F + 511) / 512);
        if (d.clear_blocks && d.clear_blocks < 152 * 8 && int64_t(d.clear_blocks) * 8 < tiles) wrong("tiles", p, d);
        if (d.clear_blocks < 0 || plan_norm(false, p).clear_blocks) wrong("blocks", p, d);
        own += d.clear_blocks > 0, shared += by_segment && d.clear_blocks == 0;
    }
    std::printf("bad %ld own %ld shared %ld\n", bad, own, shared);
    return bad != 0 || own < 10000 || shared < 10000;
}
"""


def test_no_block_clears_much(tmp_path):
    lib = srbuild.build()
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(SOURCE)
    subprocess.run([srbuild._nvcc(), "-std=c++17", "-O1", "-I", srbuild.CSRC, "-o", str(exe), str(src), lib,
                    "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
