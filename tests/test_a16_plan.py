"""The shapes of the GPU tests of the 16-bit-activation and routed layers reach every variant that the
launch rules choose from, and the rules choose no other anywhere."""
import os
import shutil
import subprocess

import pytest

from tests import test_gpu_a16, test_gpu_moe
from tests.moe_reference import few
from tests.plan_rules import ROOT, ask

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")

ROWS = (1, 2, 3, 4, 5, 9, 16, 17, 32, 33, 64, 65, 100, 128, 129, 256, 1000, 2048, 5000, 1 << 20)


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    exe = os.path.join(str(tmp_path_factory.mktemp("plan")), "a16_plan_driver")
    csrc = os.path.join(ROOT, "w4a4_rank_gemm_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + csrc,
                    os.path.join(csrc, "plan.cpp"), os.path.join(ROOT, "tests", "a16_plan_driver.cpp"), "-o", exe],
                   check=True, capture_output=True, text=True)
    return exe


def _a16(rules, cases):
    """(rows of a CTA, panels of a wave, waves that share K, one or more K slices, low-rank part: none, T of a
    launch before, T of the CTA's own) of each."""
    got = ask(rules, [("a16", *c) for c in cases])
    for (b, m, n, r), (many, rows, fn, kw, tks, ks) in zip(cases, got):
        assert many == (not few(b, n)) and (b <= rows or rows >= 64) and 1 <= ks <= m // 128 and tks <= 64 and (tks == 0 or r > 0)
        assert many or m // 128 >= kw or rows > 16
    return {(rows, fn, kw, ks > 1, 0 if r == 0 else 1 if tks else 2) for (_, _, _, r), (many, rows, fn, kw, tks, ks) in zip(cases, got)}


def test_layer_variants(rules):
    reached = _a16(rules, test_gpu_a16.CASES)
    grid = [(b, m, n, r) for b in ROWS for m in (128, 256, 512, 1152, 4096, 5120, 8192, 14336, 131072)
            for n in (16, 272, 1024, 4096, 6144, 8192, 14336, 16400, 22016, 28672, 65536, 1 << 20) for r in (0, 16, 64)]
    chosen = _a16(rules, grid)
    assert {v[:4] for v in chosen} == {v[:4] for v in reached}
    assert {v[:2] for v in reached} == {(4, 1), (16, 1), (16, 2), (32, 1), (64, 1), (64, 2), (64, 0), (128, 0)}
    for low in (0, 1):
        assert {v[:2] for v in reached if v[4] == low} == {v[:2] for v in reached}
    assert {v[:2] for v in reached if v[4] == 2} == {v[:2] for v in chosen if v[4] == 2} == {(4, 1), (16, 1), (16, 2)}


def test_router_variants(rules):
    reached = {tuple(p) for p in ask(rules, [("route", b, m, e) for b, m, e, _ in test_gpu_moe.ROUTES])}
    grid = [("route", b, m, e) for b in ROWS if b <= 256 for m in (128, 512, 1024, 2048, 4096, 7168, 131072) for e in (1, 8, 64, 128, 256, 512)]
    assert {tuple(p) for p in ask(rules, grid)} == reached
    assert {s for t, s in reached if t} >= {1, 4, 8}


def test_routed_layer_variants(rules):
    reached = {tuple(p) for p in ask(rules, [("moe", b, m, f, e, k) for b, m, f, e, k, _ in test_gpu_moe.LAYERS])}
    grid = [("moe", b, m, f, e, k) for b in ROWS if b <= 256 for m in (128, 1024, 2048, 4096, 16384) for f in (128, 768, 1408, 14336)
            for e in (1, 8, 60, 128, 512) for k in (1, 2, 8, 16)]
    chosen = {tuple(p) for p in ask(rules, grid)}
    # few tokens: waves that share K; more: gate and up by waves or shared, rows of a down tile, K slices or none
    assert {p[2] for p in chosen if p[0]} == {p[2] for p in reached if p[0]}
    assert {p[2] for p in chosen if not p[0] and not p[1]} == {p[2] for p in reached if not p[0] and not p[1]}
    assert {(p[1], p[3], p[4] > 1) for p in chosen if not p[0]} == {(p[1], p[3], p[4] > 1) for p in reached if not p[0]}
