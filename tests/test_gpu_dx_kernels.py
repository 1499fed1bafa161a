"""Every kernel variant that the frozen layer's input gradient chooses from, on an MI355X:
against the binary64 definition, and bit for bit on inputs whose sums are exact in binary32.
tests/test_plan_coverage.py asserts that the shapes here reach every variant."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import adapter_reference as ref
from tests.test_gpu_adapters import TYPES, _gen, _packed, _say

pytestmark = pytest.mark.gpu

# b, m, n, ranks: ragged token tiles, channels that end inside a stage, input columns that end
# inside a tile, slices and wave groups with unequal numbers of stages
SHAPES = [
    (30, 512, 400, (0, 16, 48)),              # 32 token rows
    (20, 640, 8208, (0, 32, 128)),            # the same, slices of the channels
    (2000, 4096, 1088, (0, 48, 128)),         # 64 token rows
    (120, 4096, 16400, (0, 48, 128)),         # the same, slices
    (4200, 4224, 1040, (0, 16, 32, 48, 128, 256)),  # 128 token rows
    (2000, 4096, 2064, (0, 48, 128)),         # two wave groups
    (500, 2048, 16400, (0, 16, 32, 48, 256)),  # the same, slices
]
CASES = [(b, m, n, r) for b, m, n, ranks in SHAPES for r in ranks]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n,r", CASES)
def test_linear_dx(b, m, n, r, dt):
    """Elementwise within the bound, which grows with n where the value grows with its root; so in
    the 2-norm too. There the errors of dY s_W and of the last rounding are independent and at
    most 2^-11 (fp16; bf16 2^-11 and 2^-8) times the element, uniform within that: sqrt(1/3 + 1/3)
    of 2^-11 together (bf16: sqrt(1/3) of 2^-8), below 2^-11 (2^-8)."""
    _say(f"linear_dx b={b} m={m} n={n} r={r} {dt}")
    g = _gen(b + m + n + r)
    qw, sw, codes = _packed(n, m, g)
    l1t = (torch.randn(r, m, generator=g, device="cuda") * 0.01).half() if r else None
    l2t = (torch.randn(n, r, generator=g, device="cuda") * 0.01).half() if r else None
    dy = torch.randn(b, n, generator=g, device="cuda") * torch.exp2(torch.randint(-8, 3, (b, 1), generator=g, device="cuda"))
    dy[3::7] = 0
    dy = dy.to(dt)
    out = torch.full((b, m), float("nan"), dtype=dt, device="cuda")
    twq.linear_dx(dy, qw, sw, l1t, l2t, out=out)
    value, bound = ref.linear_dx(dy, codes, sw, l1t, l2t)
    ref.check(out, (value, bound), "dx")
    norm = float((out.double() - value).norm() / value.norm())
    assert norm <= (2.0 ** -11 if dt == torch.float16 else 2.0 ** -8), norm


def _pack(codes):
    """int8 codes [n][m] in the library's panels."""
    n, m = codes.shape
    u = codes.view(torch.uint8) & 15
    rows = u[:, 0::2] | (u[:, 1::2] << 4)
    return rows.view(n // 16, 16, m // 128, 64).transpose(1, 2).contiguous().view(n, m // 2)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n,r", CASES)
def test_exact_sums(b, m, n, r, dt):
    """dY: integers up to 15 times a power of two a row; s_W: powers of two; L1 and L2: -1, 0, 1.
    dY s_W is exact in fp16, T in two parts, and all sums are integers below 2^24 of one unit, so
    that dX is the definition's value rounded once. One channel or slice lost or counted twice
    shows in nearly every element."""
    _say(f"exact sums b={b} m={m} n={n} r={r} {dt}")
    g = _gen(b + m + n + r + 1)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda")

    codes = ints(-7, 7, n, m).to(torch.int8)
    sw = torch.exp2(ints(-3, 0, n).float())
    d = ints(-15, 15, b, n)
    d[2::9] = 0
    power = torch.exp2(ints(-9, -6, b, 1).float())
    dy = (d * power).to(dt)
    l1t = ints(-1, 1, r, m).half() if r else None
    l2t = ints(-1, 1, n, r).half() if r else None
    units = d.double() * sw.double()
    want, most = units @ codes.double(), units.abs() @ codes.double().abs()
    if r:
        t = d.double() @ l2t.double()
        want += t @ l1t.double()
        most += t.abs() @ l1t.double().abs()
        assert float((d.double().abs() @ l2t.double().abs()).max()) < 2 ** 22
    assert float(most.max()) * 8 < 2 ** 24
    want = (want * power.double()).float().to(dt)
    assert bool(want.isfinite().all())
    assert torch.equal(twq.linear_dx(dy, _pack(codes), sw, l1t, l2t), want)
