"""Scales far apart in a channel: a row counts in every group it is non-zero in, whatever the scales of the
groups where it is zero, with few rows and with many (both tile heights)."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import moe_reference as ref
from tests.adapter_reference import F64, U, check, rounded
from tests.test_gpu_adapters import TYPES, _gen, _say
from tests.test_gpu_a16 import _layer

pytestmark = pytest.mark.gpu

# few rows; tiles of 64 rows (two ragged ones), of 128
SHAPES = [(3, 640, 400), (40, 640, 400), (100, 640, 33040), (300, 1152, 16400), (3000, 640, 4112)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n", SHAPES)
def test_small_scales_beside_large_ones(b, m, n, dt):
    """Two channels in three have a group whose scale is 2^100 times the others'; rows are zero there, so that
    the others make all of Y. Sums of m products and one multiplication by a scale (or its ratio) a group in
    binary32: (m + 3 m / 128 + 40) half steps of sum |x w|, as for any other scales; the groups with
    the large scales add products that are zero."""
    _say(f"linear_a16 scales 2^100 apart b={b} m={m} n={n} {dt}")
    g = _gen(b + n)
    qw, sw, _, _ = _layer(m, n, 0, g)
    groups = m // 128
    big = torch.randint(0, groups, (1,), generator=g, device="cuda").item()
    sw[big, 1::3] *= 2.0 ** 100
    sw[big, 2::3] *= -2.0 ** 95
    sw[(big + 1) % groups, 2::3] = 0
    x = torch.randint(-64, 65, (b, m), generator=g, device="cuda").to(dt)  # exact in both types
    x[:, big * 128:(big + 1) * 128] = 0
    one = (big + 2) % groups  # every fourth row lives in one group alone
    x[::4, :one * 128] = 0
    x[::4, (one + 1) * 128:] = 0
    w, x64 = ref.dense(qw, sw), x.to(F64)
    w[:, big * 128:(big + 1) * 128] = 0  # times zero
    value, err = x64 @ w.T, (m + 3 * groups + 40) * U * (x64.abs() @ w.abs().T)
    check(twq.linear_a16(x, qw, sw), (value, rounded(value, err, dt)), "y")


@pytest.mark.parametrize("b,n", [(100, 33040), (3000, 4112)])
def test_small_scales_count_among_large_ones(b, n):
    """bf16 rows without zeros and scales from 2^-120 to 2^20 in a channel; rows of 2^-30 to 2^30."""
    _say(f"linear_a16 scales from 2^-120 on b={b} n={n}")
    g = _gen(b)
    m = 1152
    qw, sw, l1t, l2t = _layer(m, n, 16, g)
    sw *= torch.exp2(torch.randint(-112, 28, (m // 128, n), generator=g, device="cuda").float())
    x = torch.randn(b, m, generator=g, device="cuda") * torch.exp2(torch.randint(-30, 31, (b, 1), generator=g, device="cuda").float())
    x = x.bfloat16()
    check(twq.linear_a16(x, qw, sw, l1t, l2t), ref.linear_a16(x, qw, sw, l1t, l2t), "y")
    # each row in one group alone, in all of them over the rows
    lone = torch.zeros_like(x)
    for i in range(m // 128):
        lone[i::m // 128, i * 128:(i + 1) * 128] = x[i::m // 128, i * 128:(i + 1) * 128]
    w, x64 = ref.dense(qw, sw), lone.to(F64)
    err = (128 + 3 * (m // 128) + 40) * U * (x64.abs() @ w.abs().T)
    # elements below 2^-28 of their row's largest are off by 2^-39 of it: those of this group
    for i in range(m // 128):
        k = slice(i * 128, (i + 1) * 128)
        err[i::m // 128] += 2.0 ** -39 * x64[i::m // 128].abs().amax(1, keepdim=True) * w[:, k].abs().sum(1)
    value = x64 @ w.T
    check(twq.linear_a16(lone, qw, sw), (value, rounded(value, err, torch.bfloat16)), "rows of one group")


@pytest.mark.parametrize("b,n", [(40, 400), (100, 33040), (3000, 4112)])
def test_groups_of_zeros_under_a_least_scale(b, n):
    """Pruned groups whose scale is the smallest normal number instead of zero: Y is that of zero scales, bit for
    bit, and one such group with codes beside them counts in rows that live there."""
    _say(f"linear_a16 pruned groups under a least scale b={b} n={n}")
    g = _gen(b + 7)
    m = 1152
    codes = torch.clamp(torch.round(torch.randn(n, m, generator=g, device="cuda") * 2.2), -7, 7)
    sw = 0.002 + 0.008 * torch.rand(m // 128, n, generator=g, device="cuda")
    least = torch.finfo(torch.float32).tiny
    for i in (1, 2, 5, 8):
        codes[:, i * 128:(i + 1) * 128] = 0
        sw[i] = least
    qw = ref.pack(codes)
    x = torch.randn(b, m, generator=g, device="cuda").bfloat16()
    zero = torch.where(sw == least, torch.zeros_like(sw), sw)
    assert torch.equal(twq.linear_a16(x, qw, sw), twq.linear_a16(x, qw, zero))
    codes[5::16, 128:256] = 1
    qw = ref.pack(codes)
    x[0] = 0
    x[0, 128:256] = 2.0 ** 20
    y = twq.linear_a16(x, qw, sw)
    assert torch.equal(y[1:], twq.linear_a16(x, qw, zero)[1:])
    want = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    want[5::16] = 2.0 ** 27 * least  # 128 times 2^20
    assert torch.equal(y[0], want)
