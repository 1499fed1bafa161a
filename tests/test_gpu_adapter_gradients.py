"""Gradients against differences along their own direction, on an MI355X: there the difference is a
sum of squares, far above what roundings can move it by, so that a lost, halved or flipped
gradient cannot pass. Steps are eight times as long as the operand."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import adapter_reference as ref
from tests.test_gpu_adapters import TYPES, _case, _gen, _packed, _say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b", [70, 500, 2200])
def test_adapter_gradients(b, dt):
    """out (from zero) is linear in A, in B and in x: <dY, out(A + D) - out(A)> = <dA, D>, and so on.
    Each side's error is summed from its elementwise bounds; dB's takes the H of the forward
    pass, off by its own bound."""
    m, n, r, count = 256, 272, 32, 3
    idx, x, at, bt, _, scale = _case(b, m, n, r, count, "random", dt, seed=12)
    scale += 1.0
    dy = torch.randn(b, n, generator=_gen(78), device="cuda").to(dt)
    plan = twq.adapter_plan(idx, count)
    out, h = twq.adapters(x, at, bt, plan, None, scale, keep_h=True)
    grads = twq.adapters_grad(dy, x, h, at, bt, plan, scale)
    bounds = [w[1] for w in ref.adapters_grad(dy, x.double(), h, at, bt, idx, scale, None)]
    (_, base), (_, eh) = ref.adapters(x, at, bt, idx, None, scale)
    for name, t0, grad, bound, args in (("A", at, grads[0], bounds[0], lambda t: (x, t, bt)),
                                        ("B", bt, grads[1], bounds[1], lambda t: (x, at, t)),
                                        ("x", x, grads[2], bounds[2], lambda t: (t, at, bt))):
        t1 = (t0.double() + 8 * t0.double().norm() / grad.double().norm() * grad.double()).to(dt)
        step = t1.double() - t0.double()
        moved = twq.adapters(*args(t1), plan, None, scale)
        err = (dy.double().abs() * (ref.adapters(*args(t1), idx, None, scale)[0][1] + base)).sum() + (bound * step.abs()).sum()
        if name == "B":
            for a in range(count):
                err += float(scale[a]) * (dy[idx == a].double().abs() * (eh[idx == a] @ step[a].abs().T)).sum()
        left, right = float((dy.double() * (moved.double() - out.double())).sum()), float((grad.double() * step).sum())
        _say(f"differences {name} b={b} {dt}: {left} {right} bound {float(err)}")
        assert right > 10 * float(err) and abs(left - right) <= float(err)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b", [50, 4200])
def test_input_gradient(b, dt):
    """<dY, V W> = <dX, V> with V = dX, for the layer's dense weight W in binary64."""
    m, n, r = 4224, 1040, 32
    g = _gen(22)
    qw, sw, codes = _packed(n, m, g)
    l1t = (torch.randn(r, m, generator=g, device="cuda") * 0.01).half()
    l2t = (torch.randn(n, r, generator=g, device="cuda") * 0.01).half()
    dy = torch.randn(b, n, generator=g, device="cuda").to(dt)
    dx = twq.linear_dx(dy, qw, sw, l1t, l2t)
    v = dx.double()
    w = codes.double() * sw.double()[:, None] + l2t.double() @ l1t.double()
    left, right = float((dy.double() * (v @ w.T)).sum()), float((v * v).sum())
    err = float((ref.linear_dx(dy, codes, sw, l1t, l2t)[1] * v.abs()).sum())
    _say(f"adjoint b={b} {dt}: {left} {right} bound {err}")
    assert right > 10 * err and abs(left - right) <= err * (1 + 1e-9)
