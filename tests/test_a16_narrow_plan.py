"""Panels of a wave in the layer with 16-bit activations: a second panel a wave is taken only where it makes
fewer CTAs, and no more than there are compute units. Without that, waves of narrow layers own no second
panel and multiply for nothing."""
import shutil

import pytest

from tests.moe_reference import few
from tests.plan_rules import ask
from tests.test_a16_plan import rules  # noqa: F401  (the fixture)

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")


def _ctas(b, n, fn):
    return -(-n // (128 * fn)) * -(-b // 64)


def test_second_panels_of_narrow_layers(rules):  # noqa: F811
    shapes = [(b, m, n, 0) for b in (65, 200, 700, 3000, 6000, 8000, 10000, 12000, 16448, 17000, 20000, 32768) for m in (512, 4096)
              for n in (16, 32, 112, 128, 144, 192, 256, 272, 384, 400, 512, 528, 640, 1024, 4096, 14336) if few(b, n)]
    plans = ask(rules, [("a16", *s) for s in shapes])
    two = 0
    for (b, _, n, _), (many, rows, fn, _, _, _) in zip(shapes, plans):
        assert not many and rows == 64
        if fn == 2:
            assert _ctas(b, n, 2) <= 256 < _ctas(b, n, 1), (b, n)
        two += fn == 2
    assert 0 < two < len(shapes)
