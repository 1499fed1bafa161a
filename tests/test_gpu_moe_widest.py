"""The experts of a routed layer at the ends of its sizes: 131072 input and 131072 inner channels, 4096 pairs of
token and choice beside them (inner rows of 2 GB), 512 experts."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import moe_reference as ref
from tests.adapter_reference import check
from tests.test_gpu_adapters import TYPES, _gen, _say
from tests.test_gpu_moe import _choice, _experts

pytestmark = pytest.mark.gpu

# b, m, f, experts, k, choices
LAYERS = [
    (1, 131072, 128, 3, 2, "spread"), (4, 131072, 128, 2, 16, "twice"), (40, 131072, 128, 3, 2, "none"), (256, 131072, 128, 2, 2, "one"),
    (1, 128, 131072, 2, 2, "spread"), (4, 128, 131072, 2, 16, "twice"), (30, 128, 131072, 3, 2, "spread"),
    (256, 128, 131072, 2, 16, "twice"), (256, 128, 128, 512, 16, "spread"), (4, 128, 128, 512, 16, "spread"), (256, 128, 128, 512, 1, "spread"),
]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,f,e,k,kind", LAYERS)
def test_experts(b, m, f, e, k, kind, dt):
    """Against the definition, the first and the last rows and two between (with 16 choices not those)."""
    _say(f"moe_experts b={b} m={m} f={f} experts={e} k={k} {kind} {dt}")
    g = _gen(b + m + f + e + k)
    gate_up, down = _experts(m, f, e, b + e)
    ids, w = _choice(b, e, k, kind, g)
    x = torch.randn(b, m, generator=g, device="cuda").to(dt)
    out = torch.full((b, m), float("nan"), dtype=dt, device="cuda")
    twq.moe_experts(x, ids, w, gate_up, down, out=out)
    rows = sorted({0, b - 1} if k == 16 else {0, 1 % b, b // 2, b - 1})
    check(out[rows], ref.experts(x[rows], ids[rows], w[rows], gate_up, down), "y")
    assert bool(out.isfinite().all())
    assert torch.equal(twq.moe_experts(x, ids, w, gate_up, down), out)
