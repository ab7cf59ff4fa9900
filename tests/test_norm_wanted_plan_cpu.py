"""The norm's backward pass asks for no scratch that the gradients in question do not
use: the rows' two sums are for dx, the parts of the column sums for the weight's
and the bias's gradients."""
import os
import subprocess

from segmented_reduction_csr_gb300 import build as srbuild

SOURCE = r"""
#include <cstdio>
#include "seg_norm.cuh"
#include "seg_product.cuh"
using namespace segred;

int main() {
    long bad = 0, some = 0;
    for (int64_t f : {64, 1000, 9001, 16384, 20000, 1000000})
        for (int64_t rows : {1, 513, 100000})
            for (int type : {PT_F32, PT_BF16})
                for (int want = 0; want < 8; ++want) {
                    NormParams p{};
                    auto at = [](int i) { return reinterpret_cast<void*>(uintptr_t(i) << 20); };
                    p.type = p.weight_type = type;
                    p.R = rows, p.F = p.ldx = p.ldy = p.ldo = f, p.S = 1, p.sms = 152;
                    p.x = at(1), p.dy = at(2);
                    if (want & 1) p.out = at(3);
                    if (want & 2) p.dweight = at(4);
                    if (want & 4) p.dbias = at(5);
                    const NormPlan d = plan_norm(true, p);
                    const int64_t sums = want & 1 && d.tiles > 1 ? rows * 8 : 0, parts = want & 6 ? d.chunks * 4 * f * 4 : 0;
                    auto fits = [](int64_t given, int64_t need) { return need ? given >= need && given < need + 256 : given == 0; };
                    if (!fits(d.sums_for(p), sums) || !fits(d.parts_for(p), parts)) ++bad, std::printf("%lld x %lld, %d\n", (long long)rows, (long long)f, want);
                    some += sums > 0;
                }
    return bad != 0 || some == 0;
}
"""


def test_scratch_is_what_is_wanted(tmp_path):
    lib = srbuild.build()
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(SOURCE)
    subprocess.run([srbuild._nvcc(), "-std=c++17", "-O1", "-I", srbuild.CSRC, "-o", str(exe), str(src), lib,
                    "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
