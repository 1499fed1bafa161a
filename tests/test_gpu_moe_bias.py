"""The router with a bias where scores vanish or saturate: the choice and the weights are the definition's, and
weights are zero where the chosen scores are all zero."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import moe_reference as ref
from tests.test_gpu_adapters import TYPES, _gen, _say
from tests.test_gpu_moe import _router

pytestmark = pytest.mark.gpu

# both kernels of the logits
SHAPES = [(3, 70, 8), (40, 300, 16), (256, 64, 4), (130, 512, 8)]


def _same(got, want, score):
    """ids equal; weights rounded once to binary32, after scores in binary64 that keep 2^-44 of themselves (an
    exponent of at most 745 is off by 2^-43 of 1), and next to nothing where a score is subnormal."""
    (ids, w), (wids, ww) = got, want
    assert torch.equal(ids.long(), wids), score
    live = ww.isfinite().all(1)  # elsewhere the formula divides 0 by 0
    assert bool(((w.double() - ww).abs() <= 2.0 ** -22 * ww.abs() + 1e-37)[live].all())
    assert not bool(w[~live].any())
    return int((~live).sum())


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("b,e,k", SHAPES)
def test_far_logits_with_a_bias(b, e, k, score, dt):
    """Logits of several hundred: most softmax scores are 0 or tiny, sigmoid scores 0 or 1, so that the bias
    (binary32 values, all different) decides among them."""
    _say(f"moe_route with a bias, far logits b={b} experts={e} k={k} {score} {dt}")
    x, wr, bias = _router(b, 256, e, dt, 5)
    assert len(set(bias.tolist())) == e
    x = x * 100
    for kw in (dict(), dict(norm=False), dict(scale=2.5)):
        _same(twq.moe_route(x, wr, k, bias=bias, score=score, **kw), ref.route(x, wr, k, bias=bias, score=score, **kw), score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("b,e,k", SHAPES)
def test_vanished_scores_have_zero_weights(b, e, k, score):
    """The bias asks for experts whose logits are 2000 below the others' (softmax) or below zero (sigmoid):
    their scores are 0 in binary64 too. Every other row is an ordinary one."""
    _say(f"moe_route vanished scores b={b} experts={e} k={k} {score}")
    g = _gen(b + e)
    wr = (torch.randn(e, 256, generator=g, device="cuda") / 16).bfloat16()
    wr[:, 0] = torch.where(torch.arange(e, device="cuda") % 2 == 0, 0.0, -1.0) if score == "softmax" else -1.0
    x = torch.randn(b, 256, generator=g, device="cuda").bfloat16()
    x[:, 0] = 0
    x[::2, 0] = 2048
    bias = torch.rand(e, generator=g, device="cuda")
    bias[1::2] += 4  # the odd experts, whatever their scores
    assert len(set(bias.tolist())) == e
    zero = _same(twq.moe_route(x, wr, k, bias=bias, score=score), ref.route(x, wr, k, bias=bias, score=score), score)
    assert zero == (b + 1) // 2
    ids, w = twq.moe_route(x, wr, k, bias=bias, score=score, norm=False)
    assert bool((ids % 2 == 1).all()) and not bool(w[::2].any()) and bool((w[1::2] > 0).all())
