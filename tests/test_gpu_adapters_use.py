"""The adapter operators as they are used together, on an MI355X: a training step over the
frozen layer, gradients against differences, graph replays, streams, what the binding refuses,
rows that must not be touched, and arrays whose offsets pass 32 bits."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import adapter_reference as ref
from tests.test_gpu_adapters import TYPES, _case, _gen, _index, _packed, _say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,m,n,r,ra,count", [(5, 256, 272, 16, 16, 3), (300, 512, 528, 32, 48, 4)])
def test_training_step(b, m, n, r, ra, count):
    """Two adapted layers over frozen weights, activations kept in 8 bits: every gradient against
    the binary64 formulas on the values the step itself saw."""
    _say(f"training step b={b} m={m} n={n} r={r} adapters {count} of rank {ra}")
    g = _gen(b)

    def layer(fan_in, fan_out):
        w = torch.randn(fan_out, fan_in, generator=g, device="cuda") * 0.05
        l1t = (torch.randn(r, fan_in, generator=g, device="cuda") * 0.1).half()
        l2t = (torch.randn(fan_out, r, generator=g, device="cuda") * 0.1).half()
        at = (torch.randn(count, ra, fan_in, generator=g, device="cuda") / fan_in ** 0.5).half()
        bt = (torch.randn(count, fan_out, ra, generator=g, device="cuda") * 0.05).half()
        return twq.DualLinear(w, l1t, l2t), at, bt

    up, at1, bt1 = layer(m, n * 8)
    down, at2, bt2 = layer(n * 8, m)
    scale = torch.rand(count, generator=g, device="cuda") + 0.5
    index = _index(b, count, "random", g)
    plan = twq.adapter_plan(index, count)
    x = torch.randn(b, m, generator=g, device="cuda").half()

    y1, h1 = up.adapted(x, at1, bt1, plan, scale, keep_h=True)
    c1 = twq.checkpoint_act(x)
    y2, h2 = down.adapted(y1, at2, bt2, plan, scale, keep_h=True)
    c2 = twq.checkpoint_act(y1)
    dy2 = (torch.randn(b, m, generator=g, device="cuda") * 2.0 ** -6).half()
    base2 = down.grad_input(dy2)
    da2, db2, dy1 = twq.adapters_grad(dy2, c2, h2, at2, bt2, plan, scale, dx=base2, out=base2.clone())
    base1 = up.grad_input(dy1)
    da1, db1, dx = twq.adapters_grad(dy1, c1, h1, at1, bt1, plan, scale, dx=base1)
    torch.cuda.synchronize()

    # forward: the frozen layer's output plus the adapters'
    ref.check(y1, ref.adapters(x, at1, bt1, index, up(x), scale)[0], "y1")
    ref.check(y2, ref.adapters(y1, at2, bt2, index, down(y1), scale)[0], "y2")
    # backward
    for name, (lay, dy, c, h, at, bt, base, got) in {
            "down": (down, dy2, c2, h2, at2, bt2, base2, (da2, db2, dy1)),
            "up": (up, dy1, c1, h1, at1, bt1, base1, (da1, db1, dx))}.items():
        rows = lay.qw.view(lay.n // 16, lay.m // 128, 16, 64).transpose(1, 2).reshape(lay.n, lay.m // 2).to(torch.int16)
        codes = torch.stack((rows & 15, rows >> 4), dim=2).view(lay.n, lay.m)
        codes = torch.where(codes > 7, codes - 16, codes)
        ref.check(base, ref.linear_dx(dy, codes, lay.sw, lay.l1t, lay.l2t), f"{name}: frozen dx")
        x64 = c[0].double() * c[1].double().T.repeat_interleave(128, dim=1)
        for part, o, w in zip(("dat", "dbt", "dx"), got, ref.adapters_grad(dy, x64, h, at, bt, index, scale, base)):
            ref.check(o, w, f"{name}: {part}")


@pytest.mark.parametrize("dt", TYPES)
def test_gradients_against_differences(dt):
    """out is linear in A, in B and in x, so a difference over a full step is the derivative:
    <dY, out(A + D) - out(A)> = <dA, D>, and so on. Each side's error is summed from its
    elementwise bounds."""
    b, m, n, r, count = 70, 256, 272, 32, 3
    idx, x, at, bt, y, scale = _case(b, m, n, r, count, "random", dt, seed=9)
    g = _gen(77)
    dy = torch.randn(b, n, generator=g, device="cuda").to(dt)
    plan = twq.adapter_plan(idx, count)
    out, h = twq.adapters(x, at, bt, plan, y, scale, keep_h=True)
    dat, dbt, dx = twq.adapters_grad(dy, x, h, at, bt, plan, scale)
    wants = ref.adapters_grad(dy, x.double(), h, at, bt, idx, scale, None)
    # dB is taken with the H that the forward pass returned
    (_, _), (h64, eh) = ref.adapters(x, at, bt, idx, y, scale)
    base = ref.adapters(x, at, bt, idx, y, scale)[0][1]

    def shifted(t, amount):
        return (t.float() + amount * torch.randn(t.shape, generator=g, device="cuda")).to(dt)

    for name, grad, bound, args in (
            ("A", dat, wants[0][1], lambda t: (x, t, bt)), ("B", dbt, wants[1][1], lambda t: (x, at, t)),
            ("x", dx, wants[2][1], lambda t: (t, at, bt))):
        t0 = {"A": at, "B": bt, "x": x}[name]
        t1 = shifted(t0, {"A": 0.1, "B": 0.1, "x": 2.0}[name])
        step = t1.double() - t0.double()
        moved = twq.adapters(*args(t1), plan, y, scale)
        bound1 = ref.adapters(*args(t1), idx, y, scale)[0][1]
        left = float((dy.double() * (moved.double() - out.double())).sum())
        right = float((grad.double() * step).sum())
        err = float((dy.double().abs() * (bound1 + base)).sum() + (bound * step.abs()).sum())
        if name == "B":
            c = torch.zeros(b, 1, device="cuda", dtype=torch.float64)
            on = (idx >= 0) & (idx < count)
            c[on, 0] = scale.double()[idx[on].long()].abs()
            err += float((dy.double().abs().sum(1) * (c[:, 0] * eh.amax(1))).sum() * float(step.abs().sum(2).max()))
        _say(f"differences {name} {dt}: {left} {right} bound {err}")
        assert abs(left - right) <= err and abs(right) > 0


def test_dx_is_the_adjoint():
    """<dX, V> = <dY, V W> for the layer's dense weight W in binary64."""
    g = _gen(21)
    m, n, r, b = 384, 336, 32, 50
    qw, sw, codes = _packed(n, m, g)
    l1t = (torch.randn(r, m, generator=g, device="cuda") * 0.1).half()
    l2t = (torch.randn(n, r, generator=g, device="cuda") * 0.1).half()
    dy = torch.randn(b, n, generator=g, device="cuda").half()
    v = torch.randn(b, m, generator=g, device="cuda").double()
    w = codes.double() * sw.double()[:, None] + l2t.double() @ l1t.double()
    dx = twq.linear_dx(dy, qw, sw, l1t, l2t)
    err = (ref.linear_dx(dy, codes, sw, l1t, l2t)[1] * v.abs()).sum()
    assert abs(float((dx.double() * v).sum() - (dy.double() * (v @ w.T)).sum())) <= float(err) * (1 + 1e-9)


def _everything(idx, x, at, bt, y, scale, dy, qw, sw, outs=None):
    """One call of each operator; returns every output."""
    plan = twq.adapter_plan(idx, at.shape[0])
    out, h = twq.adapters(x, at, bt, plan, y, scale, keep_h=True)
    qc, sc = twq.checkpoint_act(x)
    dx = twq.linear_dx(dy, qw, sw)
    dat, dbt, dx2 = twq.adapters_grad(dy, (qc, sc), h, at, bt, plan, scale, dx=dx)
    return [out, h, qc, sc, twq.restore_act(qc, sc, x.dtype), dx, dat, dbt, dx2]


def _inputs(b, dt, seed):
    m, n, r, count = 512, 528, 32, 5
    idx, x, at, bt, y, scale = _case(b, m, n, r, count, "random", dt, seed=seed)
    g = _gen(seed)
    qw, sw, _ = _packed(n, m, g)
    dy = torch.randn(b, n, generator=g, device="cuda").to(dt)
    return [idx, x, at, bt, y, scale, dy, qw, sw]


@pytest.mark.parametrize("b", [7, 400])
def test_graph_replays_follow_their_inputs(b):
    """Two graphs captured one after the other and replayed in turn, their inputs (the adapter
    index among them) replaced between replays, with eager calls in between."""
    _say(f"graphs b={b}")
    dev = torch.device("cuda:0")
    sets = [[_inputs(b, torch.float16, s) for s in range(k, k + 3)] for k in (0, 10)]
    live = [[t.clone() for t in s[0]] for s in sets]
    side = torch.cuda.Stream(dev)
    graphs, outs = [], []
    for inp in live:
        _everything(*inp)
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream(dev))
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            outs.append(_everything(*inp))
        graphs.append(gr)
    torch.cuda.synchronize()
    for rep in range(3):
        want = []
        for k in range(2):
            for dst, src in zip(live[k], sets[k][rep]):
                dst.copy_(src)
            want.append([o.clone() for o in _everything(*sets[k][rep])])
        torch.cuda.synchronize()
        for k in range(2):
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            for i, (o, w) in enumerate(zip(outs[k], want[k])):
                assert torch.equal(o, w), f"replay {rep}, graph {k}, output {i}"


def test_streams_do_not_share_scratch():
    """The same operators on two streams at once give what they give alone."""
    ins = [_inputs(400, torch.bfloat16, 3), _inputs(150, torch.bfloat16, 4)]
    want = [[o.clone() for o in _everything(*i)] for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[], []]
    for _ in range(4):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] = _everything(*ins[k])
    torch.cuda.synchronize()
    for k in range(2):
        for i, (o, w) in enumerate(zip(got[k], want[k])):
            assert torch.equal(o, w), f"stream {k}, output {i}"


def test_repeats_are_bitwise_equal():
    ins = _inputs(900, torch.float16, 8)
    first = _everything(*ins)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, _everything(*ins)))


@pytest.mark.parametrize("b", [40, 400])
@pytest.mark.parametrize("dt", TYPES)
def test_rows_without_an_adapter_are_not_read(b, dt):
    """NaN in such rows of x, dy and h changes nothing else, and their outputs are y and dx
    bit for bit; unused adapters may hold anything."""
    idx, x, at, bt, y, scale = _case(b, 384, 400, 32, 6, "random", dt, seed=2)
    idx[::4] = -1
    idx[idx == 3] = 2  # adapter 3 has no rows
    g = _gen(b)
    dy = torch.randn(b, 400, generator=g, device="cuda").to(dt)
    dx = torch.randn(b, 384, generator=g, device="cuda").to(dt)
    plan = twq.adapter_plan(idx, 6)
    want, h = twq.adapters(x, at, bt, plan, y, scale, keep_h=True)
    grads = twq.adapters_grad(dy, x, h, at, bt, plan, scale, dx=dx)
    off = idx < 0
    nan = float("nan")
    x2, dy2, h2, at2, bt2, s2 = x.clone(), dy.clone(), h.clone(), at.clone(), bt.clone(), scale.clone()
    x2[off], dy2[off], h2[off] = nan, nan, nan
    at2[3], bt2[3], s2[3] = nan, float("inf"), nan
    out, hh = twq.adapters(x2, at2, bt2, plan, y, s2, keep_h=True)
    assert torch.equal(out, want) and torch.equal(hh, h) and torch.equal(out[off], y[off])
    assert not bool(hh[off].any())
    again = twq.adapters_grad(dy2, x2, h2, at2, bt2, plan, s2, dx=dx)
    for p, q in zip(grads, again):
        assert torch.equal(p, q)
    assert torch.equal(again[2][off], dx[off]) and not bool(again[0][3].any()) and not bool(again[1][3].any())


@pytest.mark.parametrize("dt", TYPES)
def test_non_finite_rows_stay_alone(dt):
    """A NaN or infinity in one row of x or dY makes that row non-finite and no other."""
    idx, x, at, bt, y, scale = _case(90, 256, 272, 16, 3, "one", dt, seed=6)
    plan = twq.adapter_plan(idx, 3)
    want = twq.adapters(x, at, bt, plan, y, scale)
    x2 = x.clone()
    x2[17, 5], x2[60, 200] = float("nan"), float("inf")
    out = twq.adapters(x2, at, bt, plan, y, scale)
    keep = torch.ones(90, dtype=torch.bool, device="cuda")
    keep[17] = keep[60] = False
    assert torch.equal(out[keep], want[keep]) and not bool(out[~keep].isfinite().any())
    g = _gen(1)
    qw, sw, _ = _packed(272, 256, g)
    l1t = (torch.randn(16, 256, generator=g, device="cuda") * 0.1).half()
    l2t = (torch.randn(272, 16, generator=g, device="cuda") * 0.1).half()
    dy = torch.randn(90, 272, generator=g, device="cuda").to(dt)
    want = twq.linear_dx(dy, qw, sw, l1t, l2t)
    dy[17, 5], dy[60, 200] = float("nan"), float("inf")
    out = twq.linear_dx(dy, qw, sw, l1t, l2t)
    assert torch.equal(out[keep], want[keep]) and not bool(out[~keep].isfinite().any())


def test_large_values_in_fp16():
    """H beyond fp16's range, and far below it, reaches the output through its row's power of two."""
    b, m, n, r = 20, 256, 64, 16
    g = _gen(4)
    x = (torch.randn(b, m, generator=g, device="cuda") * torch.exp2(torch.arange(b, device="cuda") - 12.0)[:, None]).half()
    at = (torch.randn(1, r, m, generator=g, device="cuda") * 100).half()
    bt = (torch.randn(1, n, r, generator=g, device="cuda") * 2.0 ** -14).half()
    idx = torch.zeros(b, dtype=torch.int32, device="cuda")
    scale = torch.full((1,), 2.0 ** -4, device="cuda")
    plan = twq.adapter_plan(idx, 1)
    out, h = twq.adapters(x, at, bt, plan, None, scale, keep_h=True)
    assert float(h.abs().max()) > 65504
    want, wh = ref.adapters(x, at, bt, idx, None, scale)
    ref.check(h, wh, "h")
    ref.check(out, want, "out")


def test_empty_batches():
    at, bt = torch.randn(2, 16, 256, device="cuda").half(), torch.randn(2, 32, 16, device="cuda").half()
    x, dy = torch.empty(0, 256, device="cuda").half(), torch.empty(0, 32, device="cuda").half()
    plan = twq.adapter_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 2)
    out, h = twq.adapters(x, at, bt, plan, None, keep_h=True)
    assert out.shape == (0, 32) and h.shape == (0, 16)
    dat, dbt, dx = twq.adapters_grad(dy, x, h, at, bt, plan)
    assert not bool(dat.any()) and not bool(dbt.any()) and dx.shape == (0, 256)
    qc, sc = twq.checkpoint_act(x)
    assert twq.restore_act(qc, sc).shape == (0, 256)
    # no adapters at all: the output is y
    y = torch.randn(5, 32, device="cuda").half()
    plan = twq.adapter_plan(torch.zeros(5, dtype=torch.int32, device="cuda"), 0)
    assert torch.equal(twq.adapters(torch.zeros(5, 256, device="cuda").half(), at[:0], bt[:0], plan, y), y)


def test_refusals():
    idx, x, at, bt, y, scale = _case(40, 256, 272, 16, 3, "random", torch.float16)
    plan = twq.adapter_plan(idx, 3)
    _, h = twq.adapters(x, at, bt, plan, y, keep_h=True)
    dy, bad = torch.zeros_like(y), [
        lambda: twq.adapters(x[:39], at, bt, plan, y[:39]),                       # a plan of another batch
        lambda: twq.adapters(x, at[:2], bt[:2], plan, y),                         # another number of adapters
        lambda: twq.adapters(x, at, bt, plan, y, scale[:2]),
        lambda: twq.adapters(x.T.contiguous().T, at, bt, plan, y),                # strides
        lambda: twq.adapters(x, at, bt, plan, y, out=y[:39]),
        lambda: twq.adapters(x, at, bt, plan, y, out=torch.empty(80, 272, device="cuda").half()[::2]),
        lambda: twq.adapters(x, at, bt, plan, None, out=x.view(-1)[:40 * 128].view(40, 128)),
        lambda: twq.adapters_grad(dy, x[:, :128].contiguous(), h, at, bt, plan),
        lambda: twq.adapters_grad(dy, (x, h), h, at, bt, plan),
        lambda: twq.adapters_grad(dy, x, h, at, bt, plan, out=x),                 # over the activations
        lambda: twq.linear_dx(dy, torch.zeros(272, 128, dtype=torch.uint8, device="cuda"), scale),
        lambda: twq.restore_act(torch.zeros(4, 256, dtype=torch.int8, device="cuda"), torch.zeros(4, 2, device="cuda")),
        lambda: twq.adapter_plan(idx, 5000),
        lambda: twq.adapters(x, at.bfloat16(), bt, plan, y),
        lambda: twq.adapters(x.float(), at.float(), bt.float(), plan, None),
        lambda: twq.adapters(x, at, bt, "plan", y),
        lambda: twq.restore_act(torch.zeros(4, 256, dtype=torch.int8, device="cuda"), torch.zeros(2, 4, device="cuda"),
                                torch.float32),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            call()
            pytest.fail(f"call {i} was not refused")
    # overlap that starts elsewhere than at y
    both = torch.zeros(41, 272, device="cuda").half()
    with pytest.raises(ValueError):
        twq.adapters(x, at, bt, plan, both[:40], out=both[1:])
    # ranks, rows of 128: the library's own checks
    with pytest.raises(twq.TwqError):
        twq.adapters(x, at[:, :8].contiguous(), bt[:, :, :8].contiguous(), plan, y)
    with pytest.raises(twq.TwqError):
        twq.checkpoint_act(torch.zeros(4, 192, device="cuda").half())
    with pytest.raises(twq.TwqError):  # not 16-byte aligned
        twq.adapters(x, at, bt, plan, y, torch.zeros(4, device="cuda")[1:])


def test_offsets_past_32_bits():
    """Adapters, outputs, activations and the scaled copy of dY beyond 2^31 elements; the last
    rows are checked."""
    g = _gen(31)
    # at holds 2.3e9 elements
    count, r, m, n, b = 1100, 16, 131072, 16, 6
    at = torch.zeros(count, r, m, dtype=torch.float16, device="cuda")
    for a in (0, 1023, 1099):
        at[a] = torch.randn(r, m, generator=g, device="cuda").half() * 0.01
    bt = torch.randn(count, n, r, generator=g, device="cuda").half()
    x = torch.randn(b, m, generator=g, device="cuda").half()
    idx = torch.tensor([1099, 0, -1, 1023, 1099, 1050], dtype=torch.int32, device="cuda")
    plan = twq.adapter_plan(idx, count)
    out, h = twq.adapters(x, at, bt, plan, None, keep_h=True)
    used = [0, 1023, 1050, 1099]
    small = torch.tensor([3, 0, -1, 1, 3, 2], dtype=torch.int32, device="cuda")
    want, wh = ref.adapters(x, at[used], bt[used], small, None, None)
    ref.check(h, wh, "h")
    ref.check(out, want, "out")
    dy = torch.randn(b, n, generator=g, device="cuda").half()
    dat, dbt, dx = twq.adapters_grad(dy, x, h, at, bt, plan)
    wants = ref.adapters_grad(dy, x.double(), h, at[used], bt[used], small, None, None)
    ref.check(dat[used], wants[0], "dat")
    ref.check(dx, wants[2], "dx")
    del at, dat, x, dx
    # out holds 2.6e9 elements
    b, m, n = 40000, 128, 65536
    idx = torch.full((b,), -1, dtype=torch.int32, device="cuda")
    idx[-3:] = 0
    x = torch.randn(b, m, generator=g, device="cuda").half()
    at, bt = torch.randn(1, 16, m, generator=g, device="cuda").half(), torch.randn(1, n, 16, generator=g, device="cuda").half()
    out = twq.adapters(x, at, bt, twq.adapter_plan(idx, 1), None)
    ref.check(out[-4:], ref.adapters(x[-4:], at, bt, idx[-4:], None, None)[0], "last rows")
    assert not bool(out[:-3].any())
    # and so does dY, with its copy in the workspace
    qw, sw, codes = _packed(n, m, g)
    out.zero_()
    out[-2:] = torch.randn(2, n, generator=g, device="cuda").half()
    dx = twq.linear_dx(out, qw, sw)
    ref.check(dx[-3:], ref.linear_dx(out[-3:], codes, sw, None, None), "last rows of dx")
    assert not bool(dx[:-2].any())
    del out
    x = torch.zeros(20000, 131072, dtype=torch.float16, device="cuda")
    x[-2:] = torch.randn(2, 131072, generator=g, device="cuda").half()
    qc, sc = twq.checkpoint_act(x)
    q, s = ref.checkpoint(x[-3:])
    assert torch.equal(qc[-3:], q) and torch.equal(sc[:, -3:], s)
    assert torch.equal(twq.restore_act(qc, sc)[-3:], (q.float() * s.T.repeat_interleave(128, dim=1)).half())


def test_most_token_rows():
    """2^24 token rows, the limit, without a low-rank pair: the rows' maxima are found by a launch
    of a CTA a row."""
    b, m, n = 1 << 24, 128, 16
    _say(f"linear_dx b={b} m={m} n={n} r=0")
    g = _gen(24)
    qw, sw, codes = _packed(n, m, g)
    dy = (torch.randn(b, n, generator=g, device="cuda") * 2.0 ** -5).half()
    dx = twq.linear_dx(dy, qw, sw)
    for rows in (slice(0, 3), slice(b // 2 - 2, b // 2 + 2), slice(b - 3, b)):
        ref.check(dx[rows], ref.linear_dx(dy[rows], codes, sw, None, None), f"rows {rows}")
