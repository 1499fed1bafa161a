"""What the binding of the adapter and input-gradient operators says to operands that are no
matrices or no tensors, on an MI355X."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests.test_gpu_adapters import _case

pytestmark = pytest.mark.gpu


def test_wrong_kinds_are_named():
    idx, x, at, bt, y, scale = _case(40, 256, 272, 16, 3, "random", torch.float16)
    plan = twq.adapter_plan(idx, 3)
    _, h = twq.adapters(x, at, bt, plan, y, keep_h=True)
    qw, sw = twq.pack_weight(torch.randn(272, 256, device="cuda"))
    scalar = torch.zeros((), dtype=torch.float16, device="cuda")
    for error, name, call in (
            (TypeError, "at", lambda: twq.adapters(x, None, bt, plan, y)),
            (TypeError, "bt", lambda: twq.adapters(x, at, None, plan, y)),
            (ValueError, "at", lambda: twq.adapters(x, at[0], bt, plan, y)),
            (ValueError, "bt", lambda: twq.adapters_grad(y, x, h, at, bt[0], plan)),
            (TypeError, "bt", lambda: twq.adapters_grad(y, x, h, at, 3, plan)),
            (ValueError, "x", lambda: twq.adapters(scalar, at, bt, plan, y)),
            (ValueError, "x", lambda: twq.adapters(x.view(-1), at, bt, plan, y)),
            (ValueError, "dy", lambda: twq.adapters_grad(scalar, x, h, at, bt, plan)),
            (ValueError, "dy", lambda: twq.linear_dx(scalar, qw, sw)),
            (TypeError, "l1t", lambda: twq.linear_dx(y, qw, sw, None, torch.zeros(272, 16, device="cuda").half())),
            (TypeError, "x", lambda: twq.adapters_grad(y, None, h, at, bt, plan)),
            (TypeError, "h", lambda: twq.adapters_grad(y, x, None, at, bt, plan)),
            (ValueError, "x", lambda: twq.checkpoint_act(scalar))):
        with pytest.raises(error, match=rf"^{name} must"):
            call()
