"""The low-rank pair of linear_a16 when a row's T = X L1 spans many powers of two: each of its elements is
taken to 16 significant bits, with few rows and with many (both tile heights)."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import moe_reference as ref
from tests.adapter_reference import F64, U, check, rounded
from tests.test_gpu_adapters import TYPES, _gen, _say
from tests.test_gpu_a16 import _layer

pytestmark = pytest.mark.gpu

SHAPES = [(3, 640, 400, 32), (40, 640, 400, 48), (100, 640, 33040, 16), (300, 1152, 16400, 48), (3000, 640, 4112, 256)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n,r", SHAPES)
def test_small_elements_beside_large_ones(b, m, n, r, dt):
    """One element of T is 2^30 and more times the others and its rank has no weight in L2; every third
    row has no such element. The weight is zero and each channel has one rank, so that Y is one
    product: X in {-1, 0, 1} and integers times 2^-24 or 2^14 in L1 make T's sums exact (integers below 2^18),
    16 bits of T are off by 2^-17 of it, and the sums of at most four products of parts by a few half steps."""
    _say(f"linear_a16 T over many powers of two b={b} m={m} n={n} r={r} {dt}")
    g = _gen(b + n)
    qw, sw, _, _ = _layer(m, n, 0, g)
    sw.zero_()
    wide = r // 2
    l1t = torch.randint(-200, 201, (r, m), generator=g, device="cuda") * 2.0 ** -24
    l1t[wide] = 0
    l1t[wide, :128] = torch.randint(1, 4, (128,), generator=g, device="cuda") * 2.0 ** 14
    l2t = torch.zeros(n, r, device="cuda")
    rank = torch.arange(n, device="cuda") % (r - 1)
    rank += rank >= wide
    l2t[torch.arange(n, device="cuda"), rank] = (0.5 + torch.rand(n, generator=g, device="cuda")) * 2.0 ** 10
    l1t, l2t = l1t.half(), l2t.half()
    x = torch.randint(-1, 2, (b, m), generator=g, device="cuda")
    x[:, :128] = x[:, :1] * 2 + 1  # -1, 1 or 3: nothing cancels
    x[1::3, :128] = 0
    x = x.to(dt)
    t = x.to(F64) @ l1t.to(F64).T
    rest = torch.cat([t[:, :wide], t[:, wide + 1:]], 1).abs()
    assert float((t[0::3, wide].abs() / rest[0::3].amax(1)).min()) > 2 ** 30 and not bool(t[1::3, wide].any())
    assert float(rest.max()) < 2.0 ** -6
    value = t @ l2t.to(F64).T
    check(twq.linear_a16(x, qw, sw, l1t, l2t), (value, rounded(value, (2.0 ** -17 + 16 * U) * value.abs(), dt)), "y")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,n", [(100, 33040), (3000, 4112)])
def test_beside_the_weight(b, n, dt):
    """The same rows with a weight, against the definition with its usual bounds."""
    _say(f"linear_a16 T over many powers of two beside a weight b={b} n={n} {dt}")
    g = _gen(b)
    m, r = 512, 32
    qw, sw, l1t, l2t = _layer(m, n, r, g)
    l1t[3] = (l1t[3].float() * 2.0 ** 12).half()
    l1t[8:] = (l1t[8:].float() * 2.0 ** -12).half()
    l2t[:, 3] = (l2t[:, 3].float() * 2.0 ** -12).half()
    x = torch.randn(b, m, generator=g, device="cuda").to(dt)
    check(twq.linear_a16(x, qw, sw, l1t, l2t), ref.linear_a16(x, qw, sw, l1t, l2t), "y")
