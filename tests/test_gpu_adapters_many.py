"""The adapter kernels for every row tile and rank, on an MI355X: against the binary64
definitions, and bit for bit on inputs whose sums are exact in binary32.
tests/test_plan_coverage.py asserts that the shapes here reach every variant."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import adapter_reference as ref
from tests.test_gpu_adapters import TYPES, _case, _gen, _index, _say

pytestmark = pytest.mark.gpu

# b, m, n, r, adapters, order of the rows: 16-, 64- and 128-row tiles with every rank class;
# adapters of several weight-gradient pieces (512, 1024 and 2048 rows) with a remainder; the
# last row count of one tile size and the first of the next
SHAPES = [
    (13, 512, 272, 16, 4, "random"), (60, 256, 144, 128, 3, "runs"), (100, 256, 272, 32, 2, "one"),
    (256, 384, 400, 64, 5, "random"), (200, 128, 144, 160, 3, "strays"), (257, 256, 528, 16, 3, "random"),
    (400, 256, 272, 96, 3, "runs"), (700, 384, 272, 64, 4, "strays"),
    (1300, 256, 528, 256, 2, "one"), (2047, 128, 144, 32, 3, "runs"),
    (2048, 256, 144, 128, 2, "runs"), (2049, 128, 272, 16, 3, "random"), (2200, 384, 272, 64, 2, "random"),
    (2300, 256, 144, 112, 3, "runs"), (2600, 128, 80, 32, 1, "one"), (4100, 256, 272, 256, 2, "runs"),
    (8300, 256, 144, 64, 1, "one"), (8192, 128, 528, 16, 3, "runs"), (9000, 128, 144, 128, 2, "random"),
    (8200, 128, 80, 240, 3, "runs"), (8250, 128, 272, 32, 2, "strays"),
]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n,r,count,kind", SHAPES)
def test_forward_and_gradients(b, m, n, r, count, kind, dt):
    _say(f"b={b} m={m} n={n} r={r} count={count} {kind} {dt}")
    idx, x, at, bt, y, scale = _case(b, m, n, r, count, kind, dt, seed=3)
    g = _gen(b + r)
    plan = twq.adapter_plan(idx, count)
    out, h = twq.adapters(x, at, bt, plan, y, scale, keep_h=True)
    want_out, want_h = ref.adapters(x, at, bt, idx, y, scale)
    ref.check(h, want_h, "h")
    ref.check(out, want_out, "out")
    dy = (torch.randn(b, n, generator=g, device="cuda") * 2.0 ** -9).to(dt)
    dy[::5] = 0
    dx = (torch.randn(b, m, generator=g, device="cuda") * 2.0 ** -9).to(dt)
    qc, sc = twq.checkpoint_act(x)
    x8 = qc.double() * sc.double().T.repeat_interleave(128, dim=1)
    for saved, x64 in ((x, x.double()), ((qc, sc), x8)):
        got = twq.adapters_grad(dy, saved, h, at, bt, plan, scale, dx=dx)
        for name, o, w in zip(("dat", "dbt", "dx"), got, ref.adapters_grad(dy, x64, h, at, bt, idx, scale, dx)):
            ref.check(o, w, name)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n,r,count,kind", SHAPES)
def test_exact_sums(b, m, n, r, count, kind, dt):
    """Small integers times powers of two, so that H and G fit the two 16-bit parts (bf16: 16 bits
    together) and every sum is an integer below 2^24 of one unit: the outputs are the
    definitions' values rounded once. A row lost, counted twice or given to another adapter
    shows."""
    _say(f"exact sums b={b} m={m} n={n} r={r} count={count} {kind} {dt}")
    g = _gen(b + m + n + r)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda")

    idx = _index(b, count, kind, g)
    scale = torch.exp2(ints(-1, 1, count).float())
    x, y, at, bt = ints(-4, 4, b, m), ints(-100, 100, b, n), ints(-1, 1, count, r, m), ints(-1, 1, count, n, r)
    at[torch.rand(at.shape, generator=g, device="cuda") < 0.5] = 0
    bt[torch.rand(bt.shape, generator=g, device="cuda") < 0.5] = 0
    dy, dx = ints(-3, 3, b, n), ints(-50, 50, b, m)
    dy[1::6] = 0
    small = 2.0 ** -9  # of dY and dx: gradients inside fp16's range
    qc, sc = ints(-15, 15, b, m).to(torch.int8), torch.exp2(ints(-1, 0, m // 128, b).float())
    x8 = qc.double() * sc.double().T.repeat_interleave(128, dim=1)

    h = torch.zeros(b, r, dtype=torch.float64, device="cuda")
    out, dxo = y.double(), dx.double()
    dat = [torch.zeros(count, r, m, dtype=torch.float64, device="cuda") for _ in range(2)]
    dbt = torch.zeros(count, n, r, dtype=torch.float64, device="cuda")
    units = []  # the largest sums of magnitudes, in units of the smallest step
    for a in range(count):
        on = idx == a
        c = float(scale[a])
        h[on] = x[on].double() @ at[a].double().T
        d, ha = dy[on].double(), h[on]
        gg = d @ bt[a].double()
        if len(ha):  # below 2^16
            units += [2 * c * ha.abs().max() * 2 ** 8, 2 * c * gg.abs().max() * 2 ** 8]
        out[on] += c * (ha @ bt[a].double().T)
        dxo[on] += c * (gg @ at[a].double())
        dbt[a] = c * (d.T @ ha)
        sums = [(ha.abs() @ bt[a].double().abs().T) * 2, (gg.abs() @ at[a].double().abs()) * 2, (d.abs().T @ ha.abs()) * 2]
        for k, xx in enumerate((x.double(), x8)):
            dat[k][a] = c * (gg.T @ xx[on])
            sums.append((gg.abs().T @ xx[on].abs()) * (2, 4)[k])
        units += [c * v.max() for v in sums if v.numel()]
    assert max(float(u) for u in units) < 2 ** 24

    def once(v):
        v = v.float().to(dt)
        assert bool(v.isfinite().all())
        return v

    xt, att, btt = x.to(dt), at.to(dt), bt.to(dt)
    plan = twq.adapter_plan(idx, count)
    got, hh = twq.adapters(xt, att, btt, plan, y.to(dt), scale, keep_h=True)
    assert torch.equal(hh.double(), h) and torch.equal(got, once(out))
    for k, saved in enumerate((xt, (qc, sc))):
        ga, gb, gx = twq.adapters_grad((dy * small).to(dt), saved, hh, att, btt, plan, scale, dx=(dx * small).to(dt))
        assert torch.equal(gx, once(dxo * small)), f"dx, {k}"
        assert torch.equal(gb, once(dbt * small)), f"dbt, {k}"
        assert torch.equal(ga, once(dat[k] * small)), f"dat, {k}"
