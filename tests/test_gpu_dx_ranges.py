"""The frozen layer's input gradient at the ends of bfloat16's range, on an MI355X: rows whose
products with the channel scales are below binary32's normal numbers, and rows whose only
nonzero elements meet channels of scale zero."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import adapter_reference as ref
from tests.test_gpu_adapters import _gen, _packed, _say

pytestmark = pytest.mark.gpu


def _pair(n, m, r, g):
    return ((torch.randn(r, m, generator=g, device="cuda") * 0.1).half(),
            (torch.randn(n, r, generator=g, device="cuda") * 0.1).half())


@pytest.mark.parametrize("r", [0, 48])
@pytest.mark.parametrize("exponent", [-96, -108, -118, -124])
def test_tiny_rows_keep_their_bits(exponent, r):
    """Beside the usual bound: the product dY s_W, when below 2^-126, is off by half a step of the
    subnormals, 2^-150. The scaling of a row ends at 2^126, so G and T may be off by half a step
    of fp16's subnormals times 2^-126, 2^-151. Sums of T, in binary32, may add 2^-150 a channel
    where they are subnormal."""
    b, m, n = 33, 256, 1024
    _say(f"tiny rows 2^{exponent} r={r}")
    g = _gen(40)
    qw, sw, codes = _packed(n, m, g)
    l1t, l2t = _pair(n, m, r, g) if r else (None, None)
    dy = torch.randn(b, n, generator=g, device="cuda") * 2.0 ** exponent
    dy[::4] = 0
    dy[1] *= 2.0 ** 60  # an ordinary row among them
    dy = dy.to(torch.bfloat16)
    got = twq.linear_dx(dy, qw, sw, l1t, l2t)
    value, bound = ref.linear_dx(dy, codes, sw, l1t, l2t)
    bound += 3 * 2.0 ** -151 * codes.double().abs().sum(0)
    if r:
        bound += (n * 2.0 ** -150 + 2.0 ** -151) * l1t.double().abs().sum(0)
    ref.check(got, (value, bound * (1 + 2.0 ** -8)), "dx")
    # what the row's own scaling keeps: the relative 2-norm of each row is that of G's 11 bits and
    # the output's 8 while the values are normal
    live = value.abs().amax(1) > 0
    norm = (got.double() - value)[live].norm(dim=1) / value[live].norm(dim=1)
    assert float(norm.max()) <= 2.0 ** -7


def test_channels_of_scale_zero():
    """The low-rank part of a row without a quantized one keeps its own scaling, however small."""
    b, m, n, r = 20, 256, 512, 32
    g = _gen(41)
    qw, sw, codes = _packed(n, m, g)
    sw[::2] = 0
    l1t, l2t = _pair(n, m, r, g)
    dy = torch.randn(b, n, generator=g, device="cuda") * 2.0 ** -90
    dy[:, 1::2] = 0
    dy[3] = torch.randn(n, generator=g, device="cuda")
    dy[4] = 0
    dy = dy.to(torch.bfloat16)
    got = twq.linear_dx(dy, qw, sw, l1t, l2t)
    ref.check(got, ref.linear_dx(dy, codes, sw, l1t, l2t), "dx")
    assert not bool(got[4].any())
