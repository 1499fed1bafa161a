"""bf16 rows and scales far from 1 in opposite directions: Y is an ordinary number whatever is formed on the way,
with few rows and with many (both tile heights)."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import moe_reference as ref
from tests.adapter_reference import check
from tests.test_gpu_adapters import _gen, _say
from tests.test_gpu_a16 import _layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("s,x", [(100, -100), (112, -100), (118, -112), (-100, 100), (-118, 104)])
@pytest.mark.parametrize("b,m,n", [(3, 640, 400), (40, 640, 400), (100, 640, 33040), (300, 1152, 16400), (3000, 640, 4112)])
def test_large_scales_and_small_rows(b, m, n, s, x):
    """Scales about 2^s and rows about 2^x; beside small rows the low-rank pair, whose T is about 2^x too."""
    _say(f"linear_a16 scales 2^{s}, rows 2^{x} b={b} m={m} n={n}")
    g = _gen(b + n + s)
    qw, sw, l1t, l2t = _layer(m, n, 16 if x < 0 else 0, g)
    sw = sw * 2.0 ** s
    v = (torch.randn(b, m, generator=g, device="cuda") * 2.0 ** x).bfloat16()
    value, bound = ref.linear_a16(v, qw, sw, l1t, l2t)
    assert float(value.abs().max()) < 2.0 ** 30 and bool(bound.isfinite().all())
    check(twq.linear_a16(v, qw, sw, l1t, l2t), (value, bound), "y")
    assert float((twq.linear_a16(v, qw, sw, l1t, l2t).double() - value).norm() / value.norm()) <= 2.0 ** -8
