"""Low-rank adapters of many requests beside the shared layer, their gradients, 8-bit
activation checkpoints and the frozen layer's input gradient, on an MI355X, against the
binary64 definitions and bounds of tests/adapter_reference.py."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import adapter_reference as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]


def _say(msg):
    print(msg, flush=True)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _index(b, count, kind, g):
    dev = "cuda"
    if kind == "one":
        return torch.full((b,), count - 1, dtype=torch.int32, device=dev)
    if kind == "none":
        return torch.full((b,), -1, dtype=torch.int32, device=dev)
    if kind == "runs":
        cuts = torch.randint(0, b + 1, (2 * count,), generator=g, device=dev).sort().values
        own = torch.randint(0, count, (2 * count + 1,), generator=g, device=dev)
        return own[torch.bucketize(torch.arange(b, device=dev), cuts, right=True)].to(torch.int32)
    idx = torch.randint(-1, count, (b,), generator=g, device=dev).to(torch.int32)
    if kind == "strays":  # values that name no adapter
        idx[::3] = torch.tensor([-7, count, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=dev).repeat(b)[:len(idx[::3])]
    return idx


def _case(b, m, n, r, count, kind, dt, seed=0):
    g = _gen(seed + b + m + n + r)
    idx = _index(b, count, kind, g)
    x = torch.randn(b, m, generator=g, device="cuda")
    x[:, ::37] *= 20.0
    at = (torch.randn(count, r, m, generator=g, device="cuda") / m ** 0.5).to(dt)
    bt = (torch.randn(count, n, r, generator=g, device="cuda") * 0.05).to(dt)
    y = torch.randn(b, n, generator=g, device="cuda").to(dt)
    scale = torch.rand(count, generator=g, device="cuda") * 2 - 0.5
    return idx, x.to(dt), at, bt, y, scale


# tokens 1 to long, tiles that end inside, K tails (n a multiple of 16 only), every rank tiling
SHAPES = [(1, 128, 16, 16, 1, "one"), (1, 512, 528, 16, 4, "random"), (3, 256, 80, 48, 2, "random"),
          (17, 1024, 272, 32, 5, "random"), (40, 384, 1040, 64, 40, "random"), (64, 128, 64, 96, 1, "one"),
          (65, 640, 144, 128, 3, "runs"), (130, 256, 512, 256, 2, "strays"), (300, 2048, 336, 16, 7, "runs"),
          (9, 256, 64, 16, 3, "none"), (33, 256, 48, 16, 4096, "random"), (1500, 256, 160, 32, 6, "random"),
          (2200, 128, 96, 16, 2, "runs")]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n,r,count,kind", SHAPES)
def test_adapters(b, m, n, r, count, kind, dt):
    _say(f"adapters b={b} m={m} n={n} r={r} count={count} {kind} {dt}")
    idx, x, at, bt, y, scale = _case(b, m, n, r, count, kind, dt)
    plan = twq.adapter_plan(idx, count)
    out, h = twq.adapters(x, at, bt, plan, y, scale, keep_h=True)
    torch.cuda.synchronize()
    want_out, want_h = ref.adapters(x, at, bt, idx, y, scale)
    ref.check(h, want_h, "h")
    ref.check(out, want_out, "out")
    # in place, without h, without a scale, without y
    y2 = y.clone()
    assert twq.adapters(x, at, bt, plan, y2, scale, out=y2) is y2
    assert torch.equal(y2, out)
    ref.check(twq.adapters(x, at, bt, plan, None), ref.adapters(x, at, bt, idx, None, None)[0], "out without y")


@pytest.mark.parametrize("saved", ["full", "int8"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n,r,count,kind", SHAPES)
def test_adapters_grad(b, m, n, r, count, kind, dt, saved):
    _say(f"adapters_grad b={b} m={m} n={n} r={r} count={count} {kind} {dt} {saved}")
    idx, x, at, bt, y, scale = _case(b, m, n, r, count, kind, dt, seed=5)
    g = _gen(b)
    dy = (torch.randn(b, n, generator=g, device="cuda") * 2.0 ** -9).to(dt)
    dy[::5] = 0
    dx = (torch.randn(b, m, generator=g, device="cuda") * 2.0 ** -9).to(dt)
    plan = twq.adapter_plan(idx, count)
    _, h = twq.adapters(x, at, bt, plan, y, scale, keep_h=True)
    if saved == "int8":
        act = twq.checkpoint_act(x)
        x64 = act[0].double() * act[1].double().T.repeat_interleave(128, dim=1)
    else:
        act, x64 = x, x.double()
    got = twq.adapters_grad(dy, act, h, at, bt, plan, scale, dx=dx)
    torch.cuda.synchronize()
    want = ref.adapters_grad(dy, x64, h, at, bt, idx, scale, dx)
    for name, o, w in zip(("dat", "dbt", "dx"), got, want):
        ref.check(o, w, name)
    dx2 = dx.clone()
    again = twq.adapters_grad(dy, act, h, at, bt, plan, scale, dx=dx2, out=dx2)
    assert again[2] is dx2
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    ref.check(twq.adapters_grad(dy, act, h, at, bt, plan)[2],
              ref.adapters_grad(dy, x64, h, at, bt, idx, None, None)[2], "dx from zero")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m", [(1, 128), (3, 384), (16, 512), (17, 1152), (300, 2048)])
def test_checkpoint(b, m, dt):
    _say(f"checkpoint b={b} m={m} {dt}")
    g = _gen(b + m)
    x = torch.randn(b, m, generator=g, device="cuda") * torch.exp2(torch.randint(-12, 12, (b, 1), generator=g, device="cuda"))
    x[:, 5] *= 100
    x[0, :128] = 0  # an empty group
    x = x.to(dt)
    if b > 2:  # half-way codes: max 127 gives s = 1
        x[2, :128] = 0
        x[2, :8] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 63.5, -126.5], device="cuda").to(dt)
        x[1, :4] = torch.tensor([6e-8, -6e-8, 0.0, 0.0], device="cuda").to(dt)
        x[1, 4:128] = 0
    qc, sc = twq.checkpoint_act(x)
    back = twq.restore_act(qc, sc, dt)
    other = twq.restore_act(qc, sc, TYPES[1 - TYPES.index(dt)])
    q64, s64 = ref.checkpoint(x)
    assert ref.same(sc, s64)
    assert torch.equal(qc, q64)
    value = (q64.float() * s64.T.repeat_interleave(128, dim=1))
    assert ref.same(back, value.to(dt)) and ref.same(other, value.to(other.dtype))


def test_checkpoint_tiny_and_non_finite():
    """bf16 reaches scales below binary32's normal range; a group with a NaN or infinity
    restores as NaN and leaves its neighbours alone."""
    g = _gen(3)
    x = torch.randn(4, 512, generator=g, device="cuda")
    x[0, :128] *= 2.0 ** -124
    x[1, 128:256] *= 2.0 ** -131
    x = x.to(torch.bfloat16)
    qc, sc = twq.checkpoint_act(x)
    q64, s64 = ref.checkpoint(x)
    assert torch.equal(sc, s64) and torch.equal(qc, q64)
    for dt in TYPES:
        z = torch.randn(3, 384, generator=g, device="cuda").to(dt)
        clean, _ = twq.checkpoint_act(z)
        z[1, 130] = float("nan")
        z[2, 5] = float("-inf")
        qc, sc = twq.checkpoint_act(z)
        back = twq.restore_act(qc, sc, dt)
        bad = torch.zeros(3, 3, dtype=torch.bool, device="cuda")
        bad[1, 1] = bad[2, 0] = True
        assert torch.equal(sc.T.isnan(), bad)
        assert torch.equal(back.isnan(), bad.repeat_interleave(128, dim=1))
        assert torch.equal(qc[~bad.repeat_interleave(128, dim=1)], clean[~bad.repeat_interleave(128, dim=1)])


def _packed(n, m, g):
    w = torch.randn(n, m, generator=g, device="cuda") * 0.02
    qw, sw = twq.pack_weight(w)
    codes = torch.round(w.double() / sw.double()[:, None]).clamp(-7, 7)
    # the layer's own codes, from the packed panels
    rows = qw.view(n // 16, m // 128, 16, 64).transpose(1, 2).reshape(n, m // 2).to(torch.int16)
    c = torch.stack((rows & 15, rows >> 4), dim=2).view(n, m)
    c = torch.where(c > 7, c - 16, c)
    assert float((c - codes).abs().max()) <= 1  # the same rounding up to ties
    return qw, sw, c


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,n,r", [(1, 128, 16, 0), (1, 512, 528, 16), (16, 512, 512, 16), (33, 384, 80, 48),
                                     (64, 256, 2064, 0), (65, 1152, 1040, 32), (129, 2048, 336, 128), (31, 4096, 4096, 32),
                                     (300, 640, 1616, 256), (1000, 256, 192, 16), (5, 128, 8192, 64)])
def test_linear_dx(b, m, n, r, dt):
    _say(f"linear_dx b={b} m={m} n={n} r={r} {dt}")
    g = _gen(b + m + n)
    qw, sw, codes = _packed(n, m, g)
    l1t = (torch.randn(r, m, generator=g, device="cuda") * 0.1).half() if r else None
    l2t = (torch.randn(n, r, generator=g, device="cuda") * 0.1).half() if r else None
    dy = torch.randn(b, n, generator=g, device="cuda") * torch.exp2(torch.randint(-10, 4, (b, 1), generator=g, device="cuda"))
    dy[::4] = 0
    dy = dy.to(dt)
    out = torch.full((b, m), float("nan"), dtype=dt, device="cuda")
    assert twq.linear_dx(dy, qw, sw, l1t, l2t, out=out) is out
    ref.check(out, ref.linear_dx(dy, codes, sw, l1t, l2t), "dx")


def test_linear_dx_small_gradients():
    """Rows whose products with the scales lie below fp16's range keep their bits."""
    g = _gen(11)
    qw, sw, codes = _packed(256, 256, g)
    dy = (torch.randn(40, 256, generator=g, device="cuda") * 2.0 ** -60).to(torch.bfloat16)
    ref.check(twq.linear_dx(dy, qw, sw), ref.linear_dx(dy, codes, sw, None, None), "dx")
