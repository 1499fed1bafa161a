"""The shapes of the GPU tests reach every kernel variant that the launch rules choose from, so
that a changed rule cannot leave one without a test."""
import shutil

import pytest

from tests import plan_rules, test_gpu_adapters_many, test_gpu_dx_kernels

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    return plan_rules.build(tmp_path_factory.mktemp("plan"))


def test_input_gradient_variants(rules):
    cases = test_gpu_dx_kernels.CASES
    got = plan_rules.ask(rules, [("dx", *c) for c in cases])
    variants = {(bt, kg, ks > 1, r > 0) for (bt, kg, ks, *_), (_, _, _, r) in zip(got, cases)}
    tiles = [(32, 1, False), (32, 1, True), (64, 1, False), (64, 1, True), (128, 1, False), (128, 2, False), (128, 2, True)]
    assert variants == {(*t, lowrank) for t in tiles for lowrank in (False, True)}
    for (b, m, n, r), (bt, kg, ks, stages, trows, tks) in zip(cases, got):
        assert n % 64 and b % bt or (b, n) == (2000, 1088)  # ends inside a stage and inside a tile
        assert kg * ks == 1 or stages % (kg * ks)           # slices and groups of unequal lengths
    # the row maxima's launch: each row tile with each rank tile (128-row tiles alone take 128 ranks at once)
    low = {(trows, min(16 * (1 if r <= 16 else 2 if r <= 32 else 4 if r <= 64 or trows < 128 else 8), 128))
           for (*_, trows, _), (_, _, _, r) in zip(got, cases) if r}
    assert low == {(t, k) for t in (16, 64, 128) for k in (16, 32, 64, 128) if k < 128 or t == 128}
    # nothing else is chosen anywhere
    grid = [(b, m, n, r) for b in (1, 16, 60, 65, 128, 200, 500, 1000, 2048, 2049, 4096, 8192, 40000)
            for m in (128, 512, 1152, 4096, 8192, 28672) for n in (16, 512, 1040, 4096, 14336, 65536) for r in (0, 64)]
    assert {(bt, kg, ks > 1) for bt, kg, ks, *_ in plan_rules.ask(rules, [("dx", *c) for c in grid])} == set(tiles)


def test_adapter_variants(rules):
    shapes = test_gpu_adapters_many.SHAPES
    got = plan_rules.ask(rules, [("rows", b) for b, *_ in shapes])
    # rows of a tile with the ranks' matrix blocks, in the first product (powers of two up to 64, or 128
    # with the largest tiles) and in the second (up to 256)
    first = {(t, next(k for k in (16, 32, 64, 128) if r <= k or k == (128 if t == 128 else 64)))
             for (t, _), (_, _, _, r, *_) in zip(got, shapes)}
    assert first == {(t, k) for t in (16, 64, 128) for k in (16, 32, 64, 128) if k < 128 or t == 128}
    second = {(t, next(k for k in (32, 64, 128, 256) if r <= k)) for (t, _), (_, _, _, r, *_) in zip(got, shapes)}
    assert second == {(t, k) for t in (16, 64, 128) for k in (32, 64, 128, 256)}
    # an adapter of several weight-gradient pieces, at each length of a piece
    assert {c for (_, c), (b, _, _, _, count, kind) in zip(got, shapes) if kind in ("one", "runs") and b > count * c} == \
        {512, 1024, 2048}
