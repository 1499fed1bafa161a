"""The many-row kernel of the layer with 16-bit activations at the lengths that it exists for: tens to a
thousand groups, T joined from 8 to 16 K slices, ragged rows and channels, both tile heights; and
narrow layers of very many rows."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import moe_reference as ref
from tests.adapter_reference import U, check
from tests.test_gpu_adapters import TYPES, _gen, _say
from tests.test_gpu_a16 import _layer, _x

pytestmark = pytest.mark.gpu

# b, m, n, ranks: tiles of 64 rows, then of 128
SHAPES = [
    (100, 8320, 33040, (0, 64)),
    (520, 4224, 8208, (0, 128)),
    (300, 14336, 16400, (256,)),
    (3000, 8320, 4112, (0, 64)),
    (2100, 8192, 6160, (16,)),
    (2048, 4096, 14336, (32,)),
]
LONG = [(b, m, n, r) for b, m, n, ranks in SHAPES for r in ranks]
LONGEST = (70, 131072, 32784, 16)
# few-row kernel: more rows than 256 CTAs of one block hold, in CTAs whose waves own few panels
NARROW = [(17000, 256, 128, 16), (10000, 384, 272, 0), (20000, 640, 16, 0), (12000, 256, 192, 32)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n,r", LONG + NARROW)
def test_against_the_definition(b, m, n, r, dt):
    """Elementwise within the bound, in the 2-norm within half the last rounding's largest step, and along the
    definition's own direction, where a drift of the sums would add up: there the last rounding is noise of
    at most h |y| / sqrt(3) an element (6 deviations are allowed), and a product passes through m / 16 sums
    and three roundings a group."""
    _say(f"linear_a16 b={b} m={m} n={n} r={r} {dt}")
    g = _gen(b + m + n + r)
    qw, sw, l1t, l2t = _layer(m, n, r, g)
    x = _x(b, m, dt, g)
    out = torch.full((b, n), float("nan"), dtype=dt, device="cuda")
    twq.linear_a16(x, qw, sw, l1t, l2t, out=out)
    value, bound = ref.linear_a16(x, qw, sw, l1t, l2t)
    check(out, (value, bound), "y")
    half = 2.0 ** -11 if dt == torch.float16 else 2.0 ** -8
    assert float((out.double() - value).norm() / value.norm()) <= half
    along = float(((out.double() - value) * value).sum() / value.square().sum())
    noise = half * float((value.double() ** 4).sum().sqrt() / value.square().sum()) / 3 ** 0.5
    assert abs(along) <= 6 * noise + (m / 16 + 3 * m / 128 + 40) * U, (along, noise)
    assert torch.equal(twq.linear_a16(x, qw, sw, l1t, l2t), out)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n", sorted({c[:3] for c in LONG + NARROW}))
def test_exact_sums(b, m, n, dt):
    """Integers below 2^24 in every sum: the definition rounded once, bit for bit (T is at most m < 2^14)."""
    _say(f"linear_a16 exact b={b} m={m} n={n} {dt}")
    g = _gen(b * 3 + m + n)
    r = 32
    qw = ref.pack(torch.randint(-7, 8, (n, m), generator=g, device="cuda"))
    sw = torch.exp2(torch.randint(-4, 1, (m // 128, n), generator=g, device="cuda").float())
    x = torch.randint(-1, 2, (b, m), generator=g, device="cuda").to(dt)
    l1t = torch.randint(-1, 2, (r, m), generator=g, device="cuda").half()
    l2t = torch.randint(-1, 2, (n, r), generator=g, device="cuda").half()
    w = ref.dense(qw, sw)
    assert float(w.abs().sum(1).max()) * 16 + r * m < 2 ** 24
    y = x.double() @ w.T
    assert torch.equal(twq.linear_a16(x, qw, sw), y.to(dt))
    y += (x.double() @ l1t.double().T) @ l2t.double().T
    assert torch.equal(twq.linear_a16(x, qw, sw, l1t, l2t), y.to(dt))


def test_longest_rows():
    """131072 input channels, 2 GB of codes; the first, some middle and the last output channels are checked."""
    b, m, n, r = LONGEST
    _say(f"linear_a16 b={b} m={m} n={n} r={r}")
    g = _gen(9)
    qw = torch.randint(0, 256, (n, m // 2), dtype=torch.uint8, generator=g, device="cuda")
    for part in qw.split(4096):  # codes are -7 .. 7
        part ^= ((part & 15) == 8).to(torch.uint8) * 8
        part ^= ((part >> 4) == 8).to(torch.uint8) * 128
    sw = 0.002 + 0.008 * torch.rand(m // 128, n, generator=g, device="cuda")
    l1t = (torch.randn(r, m, generator=g, device="cuda") * 0.002).half()
    l2t = (torch.randn(n, r, generator=g, device="cuda") * 0.05).half()
    x = torch.randn(b, m, generator=g, device="cuda").bfloat16()
    y = twq.linear_a16(x, qw, sw, l1t, l2t)
    for c in (slice(0, 64), slice(n // 32 * 16, n // 32 * 16 + 64), slice(n - 64, n)):
        part = qw.view(n // 16, -1)[c.start // 16:c.stop // 16].reshape(64, m // 2)
        check(y[:, c], ref.linear_a16(x, part, sw[:, c], l1t, l2t[c], tokens=b, channels=n), f"channels {c}")
