"""The adapter operators at 2^24 token rows, the limit, on an MI355X."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import adapter_reference as ref
from tests.test_gpu_adapters import _gen, _say

pytestmark = pytest.mark.gpu


def test_most_token_rows():
    """Most rows without an adapter; those of adapter 0 lie at the start, of 1 in runs and of 2 at the
    end. Rows that the plan misplaced, or launches cut off by a grid's limit, show."""
    b, m, n, r, count = 1 << 24, 128, 16, 16, 3
    _say(f"adapters b={b} m={m} n={n} r={r}")
    g = _gen(25)
    idx = torch.full((b,), -1, dtype=torch.int32, device="cuda")
    idx[:100] = 0
    idx[1 << 23:(1 << 23) + 40000] = 1
    idx[(1 << 23) + 500:(1 << 23) + 40000:3] = -5
    idx[-300:] = 2
    on = (idx >= 0).nonzero()[:, 0]
    x = torch.randn(b, m, generator=g, device="cuda", dtype=torch.float16)
    y = torch.randn(b, n, generator=g, device="cuda", dtype=torch.float16)
    at = (torch.randn(count, r, m, generator=g, device="cuda") / m ** 0.5).half()
    bt = (torch.randn(count, n, r, generator=g, device="cuda") * 0.3).half()
    scale = torch.rand(count, generator=g, device="cuda") + 0.5
    plan = twq.adapter_plan(idx, count)
    out, h = twq.adapters(x, at, bt, plan, y, scale, keep_h=True)
    want, wh = ref.adapters(x[on], at, bt, idx[on], y[on], scale)
    ref.check(h[on], wh, "h")
    ref.check(out[on], want, "out")
    off = idx < 0
    assert torch.equal(out[off], y[off]) and not bool(h[off].any())
    del out
    dy = torch.randn(b, n, generator=g, device="cuda", dtype=torch.float16) * 2.0 ** -6
    dat, dbt, dx = twq.adapters_grad(dy, x, h, at, bt, plan, scale, dx=x)
    wants = ref.adapters_grad(dy[on], x[on].double(), h[on], at, bt, idx[on], scale, x[on])
    for name, o, w in zip(("dat", "dbt", "dx"), (dat, dbt, dx[on]), wants):
        ref.check(o, w, name)
    assert torch.equal(dx[off], x[off])


def test_every_adapter_and_many_rows():
    """4096 adapters, the limit, over 200000 rows: each row's own adapter is found."""
    b, m, n, r, count = 200000, 128, 16, 16, 4096
    _say(f"adapters b={b} m={m} n={n} r={r} count={count}")
    g = _gen(26)
    idx = torch.randint(-1, count, (b,), generator=g, device="cuda").to(torch.int32)
    at = torch.zeros(count, r, m, dtype=torch.float16, device="cuda")
    at[:, 0] = 1 / 64  # H[0] = sum x / 64
    number = torch.arange(count, device="cuda")
    bt = torch.zeros(count, n, r, dtype=torch.float16, device="cuda")
    bt[:, 0, 0], bt[:, 1, 0] = (number % 64).half(), (number // 64).half()
    x = torch.full((b, m), 0.5, dtype=torch.float16, device="cuda")  # H[0] = 1
    out = twq.adapters(x, at, bt, twq.adapter_plan(idx, count), None)
    want = torch.zeros(b, n, dtype=torch.float16, device="cuda")
    want[:, 0], want[:, 1] = (idx % 64).half(), (idx // 64).half()
    want[idx < 0] = 0
    assert torch.equal(out, want)


WIDE = 1 << 22  # the largest n


def _columns(g):
    """Some columns of WIDE, the last among them."""
    cols = torch.randint(0, WIDE, (1000,), generator=g, device="cuda")
    cols[:24] = torch.arange(WIDE - 24, WIDE, device="cuda")
    return cols.unique()


@pytest.mark.parametrize("b", [40, 300])
def test_widest_adapters(b):
    m, r, count = 128, 16, 2
    _say(f"adapters b={b} m={m} n={WIDE} r={r}")
    g = _gen(27)
    idx = torch.randint(-1, count, (b,), generator=g, device="cuda").to(torch.int32)
    x = torch.randn(b, m, generator=g, device="cuda").half()
    at = (torch.randn(count, r, m, generator=g, device="cuda") / m ** 0.5).half()
    bt = torch.randn(count, WIDE, r, generator=g, device="cuda", dtype=torch.float16)
    y = torch.randn(b, WIDE, generator=g, device="cuda", dtype=torch.float16)
    cols = _columns(g)
    plan = twq.adapter_plan(idx, count)
    out, h = twq.adapters(x, at, bt, plan, y, keep_h=True)
    ref.check(out[:, cols], ref.adapters(x, at, bt[:, cols], idx, y[:, cols], None)[0], "out")
    del out, y
    dy = torch.zeros(b, WIDE, dtype=torch.float16, device="cuda")
    dy[:, cols] = torch.randn(b, len(cols), generator=g, device="cuda").half() * 2.0 ** -6
    dat, dbt, dx = twq.adapters_grad(dy, x, h, at, bt, plan)
    wants = ref.adapters_grad(dy[:, cols], x.double(), h, at, bt[:, cols], idx, None, None)
    for name, o, w in zip(("dat", "dbt", "dx"), (dat, dbt[:, cols], dx), wants):
        ref.check(o, w, name)
    assert int(dbt.count_nonzero()) == int(dbt[:, cols].count_nonzero())


@pytest.mark.parametrize("b,r", [(20, 16), (200, 0), (200, 32)])
def test_widest_input_gradient(b, r):
    m = 128
    _say(f"linear_dx b={b} m={m} n={WIDE} r={r}")
    g = _gen(28)
    qw, sw = twq.pack_weight(torch.randn(WIDE, m, generator=g, device="cuda"))
    rows = qw.view(WIDE // 16, 1, 16, 64).reshape(WIDE, m // 2)
    l1t = torch.randn(r, m, generator=g, device="cuda").half() if r else None
    l2t = torch.randn(WIDE, r, generator=g, device="cuda", dtype=torch.float16) if r else None
    cols = _columns(g)
    dy = torch.zeros(b, WIDE, dtype=torch.float16, device="cuda")
    dy[:, cols] = torch.randn(b, len(cols), generator=g, device="cuda").half() * 2.0 ** -6
    codes = torch.stack((rows[cols] & 15, rows[cols] >> 4), dim=2).view(len(cols), m).to(torch.int16)
    codes = torch.where(codes > 7, codes - 16, codes)
    got = twq.linear_dx(dy, qw, sw, l1t, l2t)
    ref.check(got, ref.linear_dx(dy[:, cols], codes, sw[cols], l1t, l2t[cols] if r else None), "dx")
