"""The packed layer with 16-bit activations on an MI355X: every variant of its kernels against the
binary64 definition, bit for bit where sums are exact, and the inputs where it could go wrong."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import moe_reference as ref
from tests.adapter_reference import check
from tests.test_gpu_adapters import TYPES, _gen, _say

pytestmark = pytest.mark.gpu

# b, m, n, ranks: each row tile, panels a wave, waves a panel and K slices of the few-row kernels, and
# each tile and slicing of the many-row kernel; ragged rows, panels that do not fill a CTA
SHAPES = [
    (1, 128, 16, (0, 16)),
    (1, 256, 48, (0, 48)),
    (2, 640, 400, (0, 16, 256)),
    (3, 512, 96, (32, 64)),
    (4, 2048, 272, (16,)),
    (7, 256, 96, (80, 128)),
    (16, 128, 8224, (112,)),
    (4, 4096, 4096, (0, 32)),
    (3, 1024, 28688, (0, 128)),
    (1, 512, 57360, (16,)),
    (5, 384, 80, (0, 48)),
    (6, 128, 48, (0, 16)),
    (10, 512, 32, (0, 16)),
    (6, 128, 8208, (0, 16)),
    (11, 1152, 8208, (0, 32)),
    (16, 4096, 4112, (0, 16, 128)),
    (9, 1152, 14352, (0, 64)),
    (13, 512, 28704, (0, 16)),
    (17, 256, 48, (0, 256)),
    (32, 4096, 4096, (0, 32)),
    (25, 896, 28704, (0, 48)),
    (29, 2176, 6160, (0, 48)),
    (21, 128, 6160, (0, 16)),
    (50, 512, 24592, (0, 16)),
    (37, 2176, 24592, (0, 16)),
    (40, 128, 16400, (0, 16)),
    (45, 2176, 528, (0, 32)),
    (33, 384, 112, (0, 16)),
    (61, 8192, 1040, (0, 64)),
    (64, 2048, 14352, (0, 128)),
    (65, 128, 16, (0, 16)),
    (70, 4224, 272, (0, 48)),
    (200, 1024, 1040, (0, 256)),
    (130, 384, 4112, (0, 48)),
    (450, 256, 4096, (0, 64)),
    (700, 1152, 4112, (0, 16)),
    (600, 256, 272, (128,)),
    (1000, 8320, 400, (0, 16)),
    (5000, 128, 16, (0, 16)),
    (33000, 256, 32, (0, 16)),
    (300, 256, 16400, (0, 32)),
    (100, 1152, 65536, (0, 16)),
    (2100, 1152, 4112, (0, 16, 128)),
    (3000, 1152, 4112, (0, 16, 256)),
    (4200, 384, 4368, (0, 64)),
]
CASES = [(b, m, n, r) for b, m, n, ranks in SHAPES for r in ranks]


def _layer(m, n, r, g, low=0.05):
    codes = torch.clamp(torch.round(torch.randn(n, m, generator=g, device="cuda") * 2.2), -7, 7)
    sw = 0.002 + 0.008 * torch.rand(m // 128, n, generator=g, device="cuda")
    l1t = (torch.randn(r, m, generator=g, device="cuda") * low).half() if r else None
    l2t = (torch.randn(n, r, generator=g, device="cuda") * low).half() if r else None
    return ref.pack(codes), sw, l1t, l2t


def _x(b, m, dt, g):
    x = torch.randn(b, m, generator=g, device="cuda") * torch.exp2(torch.randint(-8, 3, (b, 1), generator=g, device="cuda"))
    x[:, ::97] *= 30
    return x.to(dt)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n,r", CASES)
def test_against_the_definition(b, m, n, r, dt):
    """Elementwise within the bound, and in the 2-norm within half the last rounding's largest step
    (its errors are spread within that: at most 1 / sqrt(3) of it)."""
    _say(f"linear_a16 b={b} m={m} n={n} r={r} {dt}")
    g = _gen(b + m + n + r)
    qw, sw, l1t, l2t = _layer(m, n, r, g)
    x = _x(b, m, dt, g)
    out = torch.full((b, n), float("nan"), dtype=dt, device="cuda")
    twq.linear_a16(x, qw, sw, l1t, l2t, out=out)
    value, bound = ref.linear_a16(x, qw, sw, l1t, l2t)
    check(out, (value, bound), "y")
    norm = float((out.double() - value).norm() / value.norm())
    assert norm <= (2.0 ** -11 if dt == torch.float16 else 2.0 ** -8), norm
    assert torch.equal(twq.linear_a16(x, qw, sw, l1t, l2t), out)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n", sorted({c[:3] for c in CASES}))
def test_exact_sums(b, m, n, dt):
    """X in {-1, 0, 1}, scales powers of two within 2^4: every partial sum is an integer below 2^24
    times the least scale, so Y is the definition rounded once, bit for bit. T = X L1 of a pair with
    entries in {-1, 0, 1} is at most m <= 2^13 (2^16 holds in two parts of 8 bits)."""
    _say(f"linear_a16 exact b={b} m={m} n={n} {dt}")
    g = _gen(b * 3 + m + n)
    r = 32
    codes = torch.randint(-7, 8, (n, m), generator=g, device="cuda")
    qw = ref.pack(codes)
    sw = torch.exp2(torch.randint(-4, 1, (m // 128, n), generator=g, device="cuda").float())
    x = torch.randint(-1, 2, (b, m), generator=g, device="cuda").to(dt)
    l1t = torch.randint(-1, 2, (r, m), generator=g, device="cuda").half()
    l2t = torch.randint(-1, 2, (n, r), generator=g, device="cuda").half()
    w = ref.dense(qw, sw)
    assert float((x.double().abs() @ w.abs().T).max()) * 16 + r * m < 2 ** 24
    want = (x.double() @ w.T).to(dt)
    assert torch.equal(twq.linear_a16(x, qw, sw), want)
    t = x.double() @ l1t.double().T
    assert torch.equal(twq.linear_a16(x, qw, sw, l1t, l2t), (x.double() @ w.T + t @ l2t.double().T).to(dt))


def test_packed_weights_of_the_library():
    """The weight pack_weight_grouped makes is the one linear_a16 reads: Y is near X W^T, by the
    quantizer's half step."""
    g = _gen(3)
    m, n, b = 512, 272, 40
    w = torch.randn(n, m, generator=g, device="cuda") * 0.02
    qw, sw = twq.pack_weight_grouped(w)
    x = torch.randn(b, m, generator=g, device="cuda").half()
    check(twq.linear_a16(x, qw, sw), ref.linear_a16(x, qw, sw, None, None), "y")
    step = (ref.dense(qw, sw) - w.double()).abs()
    assert bool((step <= sw.double().T.repeat_interleave(128, dim=1) * 0.5 * (1 + 1e-6)).all())


@pytest.mark.parametrize("b", [1, 7, 40, 90, 300, 11000])
@pytest.mark.parametrize("dt", TYPES)
def test_non_finite_rows_stay_alone(b, dt):
    g = _gen(b)
    qw, sw, l1t, l2t = _layer(384, 272, 16, g)
    x = _x(b, 384, dt, g)
    want = twq.linear_a16(x, qw, sw, l1t, l2t)
    x2 = x.clone()
    rows = sorted({0, b // 2, b - 1})[:2] if b > 1 else [0]
    for i, v in zip(rows, (float("nan"), float("inf"))):
        x2[i, 5 + 200 * i % 384] = v
    out = twq.linear_a16(x2, qw, sw, l1t, l2t)
    keep = torch.ones(b, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.equal(out[keep], want[keep]) and not bool(out[~keep].isfinite().any())


@pytest.mark.parametrize("b", [1, 16, 64, 65, 200, 11000])
@pytest.mark.parametrize("dt", TYPES)
def test_scales_of_any_size(b, dt):
    """Groups of scale zero (whatever their codes), channels of zeros, scales 2^80 apart within a
    channel and past the 2^90 that the many-row kernel tells apart, tiny and negative ones."""
    g = _gen(b)
    m, n = 1024, 288
    qw, sw, _, _ = _layer(m, n, 0, g)
    sw[::3, ::2] = 0
    sw[:, 7] = 0
    sw[1, 5::16] *= 2.0 ** -80
    sw[2, 6::16] *= 2.0 ** -100
    sw[:, 8] *= 2.0 ** -120
    sw[:, 9] *= 2.0 ** 60
    sw[3, 10::16] *= -1
    sw[0, 11::16] = 0
    sw[7, 12::16] = 0
    x = torch.randn(b, m, generator=g, device="cuda")
    if dt == torch.float16:
        sw[:, 9] = 0
    x[b // 2, 128:] = 0  # only the first group's scale matters there
    x = x.to(dt)
    check(twq.linear_a16(x, qw, sw), ref.linear_a16(x, qw, sw, None, None), "y")


@pytest.mark.parametrize("b", [3, 16, 64, 130, 16500])
def test_bf16_ranges(b):
    """bf16 rows from 2^-90 to 2^100, rows of zeros, and elements 2^-20 of their row's largest, whose
    codes are the only ones."""
    g = _gen(b)
    m, n, r = 512, 144, 16
    qw, sw, l1t, l2t = _layer(m, n, r, g)
    x = torch.randn(b, m, generator=g, device="cuda")
    x *= torch.exp2(torch.linspace(-90, 100, b, device="cuda").round())[:, None]
    x[1] = 0
    x = x.bfloat16()
    check(twq.linear_a16(x, qw, sw, l1t, l2t), ref.linear_a16(x, qw, sw, l1t, l2t), "y")
    codes = torch.zeros(n, m, device="cuda")
    codes[:, 128:] = torch.randint(-7, 8, (n, m - 128), generator=g, device="cuda")
    qw = ref.pack(codes)
    x = torch.randn(b, m, generator=g, device="cuda")
    x[:, :128] *= 2.0 ** 20
    x = x.bfloat16()
    value, bound = ref.linear_a16(x, qw, sw, None, None)
    out = twq.linear_a16(x, qw, sw)
    check(out, (value, bound), "beside outliers")
    assert float((out.double() - value).norm() / value.norm()) <= 2.0 ** -8


def test_fp16_subnormals():
    """fp16 rows below the normal range count."""
    g = _gen(8)
    for b in (2, 20, 100, 33000):
        qw, sw, _, _ = _layer(256, 48, 0, g)
        x = (torch.randn(b, 256, generator=g, device="cuda") * 2.0 ** -20).half()
        sw = sw * 2.0 ** 14
        check(twq.linear_a16(x, qw, sw), ref.linear_a16(x, qw, sw, None, None), f"b={b}")


def test_largest_sizes():
    """m = 131072, n = 2^22, 2^20 token rows; the last rows and columns are checked."""
    g = _gen(9)
    _say("linear_a16 m=131072")
    for b in (2, 20, 70):
        qw, sw, l1t, l2t = _layer(131072, 32, 16, g, low=0.002)
        x = torch.randn(b, 131072, generator=g, device="cuda").bfloat16()
        check(twq.linear_a16(x, qw, sw, l1t, l2t), ref.linear_a16(x, qw, sw, l1t, l2t), f"m=131072 b={b}")
    n = 1 << 22
    qw, sw, _, _ = _layer(128, n, 0, g)
    for b in (1, 20, 600):  # 600: 2.5e9 outputs
        _say(f"linear_a16 n=2^22 b={b}")
        x = torch.randn(b, 128, generator=g, device="cuda").half()
        y = twq.linear_a16(x, qw, sw)
        for c in (slice(0, 64), slice(n - 64, n)):
            part = qw.view(n // 16, -1)[c.start // 16:c.stop // 16].reshape(64, -1)
            check(y[-3:, c], ref.linear_a16(x[-3:], part, sw[:, c], None, None, tokens=b, channels=n), f"n=2^22 {c}")
        del y
    b = 1 << 20
    _say("linear_a16 b=2^20")
    qw, sw, l1t, l2t = _layer(256, 2064, 16, g)  # 2.2e9 outputs
    x = torch.randn(b, 256, generator=g, device="cuda").half()
    y = twq.linear_a16(x, qw, sw, l1t, l2t)
    for rows in (slice(0, 130), slice(b - 130, b)):
        check(y[rows], ref.linear_a16(x[rows], qw, sw, l1t, l2t, tokens=b), f"rows {rows}")


def test_refusals():
    g = _gen(1)
    qw, sw, l1t, l2t = _layer(256, 48, 16, g)
    x = torch.zeros(40, 256, device="cuda").half()
    bad = [lambda: twq.linear_a16(x.float(), qw, sw), lambda: twq.linear_a16(x[:, :128].contiguous(), qw, sw),
           lambda: twq.linear_a16(x.T.contiguous().T, qw, sw), lambda: twq.linear_a16(x, qw, sw[:1]),
           lambda: twq.linear_a16(x, qw, sw.T.contiguous()), lambda: twq.linear_a16(x, qw, sw, l1t),
           lambda: twq.linear_a16(x, qw, sw, None, l2t), lambda: twq.linear_a16(x, qw, sw, l1t, l2t[:32]),
           lambda: twq.linear_a16(x, qw, sw, l1t.bfloat16(), l2t.bfloat16()), lambda: twq.linear_a16(x, qw, sw[0]),
           lambda: twq.linear_a16(x, qw, sw, out=torch.zeros(40, 48, device="cuda")),
           lambda: twq.linear_a16(x, qw, sw, out=torch.zeros(80, 48, device="cuda").half()[::2]),
           lambda: twq.linear_a16(x, qw, sw, out=x.view(-1)[:40 * 48].view(40, 48)),
           lambda: twq.linear_a16(x.cpu(), qw, sw), lambda: twq.linear_a16(x, qw.cpu(), sw), lambda: twq.linear_a16(x, qw.int(), sw)]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(twq.TwqError):  # ranks of 16
        twq.linear_a16(x, qw, sw, l1t[:8].contiguous(), l2t[:, :8].contiguous())
    with pytest.raises(twq.TwqError):  # not 16-byte aligned
        twq.linear_a16(torch.zeros(40 * 256 + 4, device="cuda").half()[4:].view(40, 256), qw, sw)
    assert twq.linear_a16(x[:0], qw, sw, l1t, l2t).shape == (0, 48)
    assert twq.linear_a16(x, qw[:0], sw[:, :0].contiguous()).shape == (40, 0)
