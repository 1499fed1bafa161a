"""The GPU tests of the layer with 16-bit activations reach the many-row kernel at the lengths it exists for,
and its workspace regions do not overlap."""
import os
import shutil
import subprocess

import pytest

from tests import test_gpu_a16_long_sums
from tests.plan_rules import ROOT, ask
from tests.test_a16_plan import rules  # noqa: F401  (the fixture)

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")

LAYOUT = r"""
#include <cstdio>
#include "twq_moe.h"
int main() {
    for (int64_t b : {65, 100, 1000, 4001, 100003})
        for (int64_t m : {128, 1152, 8192})
            for (int64_t n : {4112, 33040, 131072})
                for (int64_t r : {0, 16, 128, 256}) {
                    const twq::A16Plan p = twq::plan_a16(b, m, n, r);
                    if (!p.many) continue;
                    const size_t at[] = {p.t, p.x16, p.xe, p.mul, p.mask, p.small, p.unit, p.t16, p.twide, p.te, p.total};
                    const size_t bytes[] = {(size_t)p.tks * b * r * 4, (size_t)b * m * 2, (size_t)b * 4, (size_t)(m / 128 * n) * 4,
                                            (size_t)(m / 128 * n) * 4, (size_t)n * 4, (size_t)n * 4, (size_t)b * r * 4,
                                            (size_t)b * r * 4, (size_t)b * 4};
                    for (int i = 0; i < 10; ++i)
                        if (at[i] % 256 != 0 || at[i] + bytes[i] > at[i + 1]) return std::printf("region %d\n", i), 1;
                    std::printf("ok\n");
                }
    return 0;
}
"""


def test_workspace_regions(tmp_path):
    src, exe, csrc = tmp_path / "layout.cpp", str(tmp_path / "layout"), os.path.join(ROOT, "w4a4_rank_gemm_amd", "csrc")
    src.write_text(LAYOUT)
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + csrc,
                    os.path.join(csrc, "plan.cpp"), str(src), "-o", exe], check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.count("ok") > 20, r.stdout[-200:]


def test_long_sums_reach_the_many_row_kernel(rules):  # noqa: F811
    cases = test_gpu_a16_long_sums.LONG + [test_gpu_a16_long_sums.LONGEST]
    plans = ask(rules, [("a16", *c) for c in cases])
    assert all(p[0] for p in plans) and all(c[1] >= 4096 for c in cases)
    assert {p[1] for p, c in zip(plans, cases) if c[1] >= 8192 and p[4] >= 8} == {64, 128}
    assert max(p[4] for p in plans) == 16 and max(c[1] for c in cases) == 131072
    narrow = ask(rules, [("a16", *c) for c in test_gpu_a16_long_sums.NARROW])
    assert {p[2] for p in narrow if not p[0]} == {1, 2} and not any(p[0] for p in narrow)
