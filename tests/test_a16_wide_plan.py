"""The layer of the graph, stream and thread tests takes the many-row kernel, with tiles of both heights."""
import shutil

import pytest

from tests.plan_rules import ask
from tests.test_a16_plan import rules  # noqa: F401  (the fixture)
from tests.test_gpu_a16_wide_use import M, N, R, TOKENS

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")


def test_layers_in_use_reach_the_many_row_kernel(rules):  # noqa: F811
    plans = ask(rules, [("a16", b, M, N, R) for b in TOKENS])
    assert all(p[0] and p[4] >= 1 for p in plans) and {p[1] for p in plans} == {64, 128}
