"""The router and the routed layer on an MI355X, against the binary64 definitions."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import moe_reference as ref
from tests.adapter_reference import check
from tests.test_gpu_adapters import TYPES, _gen, _say

pytestmark = pytest.mark.gpu

# b, m, experts, k: both logit kernels, every number of keys a lane
ROUTES = [(1, 128, 1, 1), (1, 2048, 64, 8), (3, 256, 5, 5), (5, 640, 65, 7), (17, 4096, 100, 16), (64, 1152, 256, 8),
          (130, 512, 129, 4), (256, 384, 512, 16), (100, 7168, 250, 10), (256, 256, 64, 2), (33, 131072, 512, 3), (150, 2048, 130, 6)]


def _router(b, m, e, dt, seed):
    g = _gen(seed)
    x = torch.randn(b, m, generator=g, device="cuda")
    x[:, ::67] *= 30
    wr = (torch.randn(e, m, generator=g, device="cuda") / m ** 0.5).to(dt)
    return x.to(dt), wr, torch.randn(e, generator=g, device="cuda") * 0.1


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("b,m,e,k", ROUTES)
def test_route(b, m, e, k, score, dt):
    """The choice is the definition's; weights are its, rounded once to binary32 (a few binary64
    roundings before that: 2^-23 in all)."""
    _say(f"moe_route b={b} m={m} experts={e} k={k} {score} {dt}")
    x, wr, bias = _router(b, m, e, dt, b + m + e)
    for kw in (dict(), dict(bias=bias), dict(norm=False), dict(bias=bias, norm=False, scale=2.5)):
        ids, w = twq.moe_route(x, wr, k, score=score, **kw)
        want, ww = ref.route(x, wr, k, score=score, **kw)
        assert torch.equal(ids.long(), want), kw
        assert bool(((w.double() - ww).abs() <= 2.0 ** -23 * ww.abs() + 1e-37).all()), kw


@pytest.mark.parametrize("b,e", [(4, 96), (200, 96), (200, 512)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_logits_go_to_the_lowest_index(b, e, score):
    """Expert rows repeated three times, and all rows the same."""
    g = _gen(b)
    x = torch.randn(b, 256, generator=g, device="cuda").half()
    third = (torch.randn(e // 3, 256, generator=g, device="cuda") / 16).half()
    wr = third.repeat(3, 1)
    wr = torch.cat([wr, wr[:e - wr.shape[0]]]).contiguous()
    ids, w = twq.moe_route(x, wr, 7, score=score)
    want, ww = ref.route(x, wr, 7, score=score)
    # binary64 sums of equal rows are equal in the kernels; the reference's may not be, so it is asked by row
    group = torch.arange(e, device="cuda") % (e // 3)
    assert torch.equal(group[ids.long()], group[want])
    same = group[ids.long()][:, 1:] == group[ids.long()][:, :-1]
    assert bool((ids[:, 1:] > ids[:, :-1])[same].all())
    assert bool(((w.double() - ww).abs() <= 2.0 ** -22 * ww).all())
    ids, w = twq.moe_route(x, third[:1].repeat(e, 1).contiguous(), 7, score=score)
    assert torch.equal(ids, torch.arange(7, dtype=torch.int32, device="cuda").expand(b, 7))
    assert torch.equal(twq.moe_route(torch.zeros_like(x), wr, 3, bias=torch.zeros(e, device="cuda"))[0],
                       torch.arange(3, dtype=torch.int32, device="cuda").expand(b, 3))


def test_close_logits():
    """Logits one part in 2^40 apart, which binary32 sums could not order: x = (1, 2^-20, ..) against
    rows (1, j 2^-20, 0, ..)."""
    e = 64
    for b in (2, 256):
        x = torch.zeros(b, 256, device="cuda", dtype=torch.bfloat16)
        x[:, 0], x[:, 1] = 1, 2.0 ** -20
        wr = torch.zeros(e, 256, device="cuda", dtype=torch.bfloat16)
        order = torch.randperm(e, generator=_gen(b), device="cuda")
        wr[:, 0] = 1
        wr[:, 1] = order.float() * 2.0 ** -20
        ids, _ = twq.moe_route(x, wr, 8)
        assert torch.equal(ids.long(), torch.argsort(order, descending=True)[:8].expand(b, 8))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("b,e,k", [(3, 70, 8), (256, 64, 4)])
def test_extreme_and_non_finite_logits(b, e, k, score):
    """Logits far apart (scores that vanish), and rows with infinities and NaN: ids always name k
    different experts, and other rows are untouched."""
    x, wr, bias = _router(b, 256, e, torch.bfloat16, 5)
    x = x * 100
    for kw in (dict(), dict(norm=False), dict(bias=bias)):
        ids, w = twq.moe_route(x, wr, k, score=score, **kw)
        want, ww = ref.route(x, wr, k, score=score, **kw)
        live = ww.isfinite().all(1)  # all chosen scores zero: 0 / 0 in the formula, zeros here
        assert torch.equal(ids[live].long(), want[live]) or kw.get("bias") is not None
        if kw.get("bias") is None:
            assert bool(((w.double() - ww).abs() <= 2.0 ** -22 * ww.abs() + 1e-37)[live].all())
        assert bool(w.isfinite().all())
        bad = x.clone()
        bad[0, 3], bad[b // 2, 9], bad[b - 1] = float("nan"), float("inf"), float("-inf")
        ids2, w2 = twq.moe_route(bad, wr, k, score=score, **kw)
        keep = torch.ones(b, dtype=torch.bool, device="cuda")
        keep[[0, b // 2, b - 1]] = False
        assert torch.equal(ids2[keep], ids[keep]) and torch.equal(w2[keep], w[keep])
        assert bool(((ids2 >= 0) & (ids2 < e)).all())
        assert all(len(set(r)) == k for r in ids2.tolist())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("b,e", [(3, 64), (200, 96)])
def test_nan_logits_give_nan_weights(b, e, score):
    """A row of NaN logits has NaN weights, whether they are divided by their sum or not."""
    x, wr, bias = _router(b, 256, e, torch.float16, 7)
    x[b // 2, 5] = float("nan")
    for kw in (dict(), dict(norm=False), dict(bias=bias), dict(bias=bias, norm=False)):
        w = twq.moe_route(x, wr, 4, score=score, **kw)[1]
        assert bool(w[b // 2].isnan().all()) and int(w.isnan().sum()) == 4, kw


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_masked_by_the_bias(score):
    """A bias of -inf, or of the type's lowest value, takes an expert out while others are left."""
    for b, e, k in ((2, 20, 8), (150, 130, 8)):
        x, wr, bias = _router(b, 256, e, torch.bfloat16, 8)
        for low in (float("-inf"), torch.finfo(torch.float32).min):
            bias[::2] = low
            ids, w = twq.moe_route(x, wr, k, bias=bias, score=score)
            want, ww = ref.route(x, wr, k, bias=bias, score=score)
            assert torch.equal(ids.long(), want) and bool((ids % 2 == 1).all())
            assert bool(((w.double() - ww).abs() <= 2.0 ** -23 * ww.abs() + 1e-37).all())


@pytest.mark.parametrize("b", [1, 4, 5, 40])
def test_weights_of_no_expert_are_not_used(b):
    """Choices outside the range carry NaN weights, as a masked router's may."""
    gate_up, down = _experts(256, 128, 6, 1)
    g = _gen(b)
    ids, w = _choice(b, 6, 4, "spread", g)
    ids[:, 1], ids[:, 3] = -1, 6
    x = torch.randn(b, 256, generator=g, device="cuda").half()
    w2 = w.clone()
    w[:, 1::2], w2[:, 1::2] = float("nan"), 0
    assert torch.equal(twq.moe_experts(x, ids, w, gate_up, down), twq.moe_experts(x, ids, w2, gate_up, down))


@pytest.mark.parametrize("k", [1, 3, 8])
def test_rows_of_a_larger_batch(k):
    """Slices of a batch's ids and weights start at no multiple of 16 bytes."""
    gate_up, down = _experts(256, 128, 9, 1)
    g = _gen(k)
    b = 21
    ids, w = _choice(b, 9, k, "spread", g)
    x = torch.randn(b, 256, generator=g, device="cuda").half()
    for lo, hi in ((3, 20), (5, 6)):
        args = [t[lo:hi] for t in (x, ids, w)]
        out = twq.moe_experts(*args, gate_up, down)
        check(out, ref.experts(*args, gate_up, down), "y")
        assert torch.equal(out, twq.moe_experts(*[t.clone() for t in args], gate_up, down))


def test_packing_refusals():
    for shape in ((2, 24, 128), (2, 32, 100)):
        with pytest.raises(ValueError):
            twq.pack_experts(torch.zeros(shape, device="cuda"))
    with pytest.raises(ValueError):
        twq.pack_experts(torch.zeros(2, 128, 32, device="cuda").transpose(1, 2))
    with pytest.raises(TypeError):
        twq.pack_experts(torch.zeros(2, 32, 128, device="cuda").half())


def _experts(m, f, e, seed):
    g = _gen(seed)

    def packed(n, kk, size):
        codes = torch.clamp(torch.round(torch.randn(e * n, kk, generator=g, device="cuda") * 2.2), -7, 7)
        s = (0.5 + torch.rand(kk // 128, e * n, generator=g, device="cuda")) * size
        return ref.pack(codes).view(e, n, kk // 2), s

    return packed(2 * f, m, 0.5 / m ** 0.5), packed(m, f, 0.3 / f ** 0.5)


def _choice(b, e, k, kind, g):
    if kind == "spread":
        ids = torch.stack([torch.randperm(e, generator=g, device="cuda")[:k] for _ in range(b)])
    elif kind == "one":  # every token asks the same experts
        ids = (torch.arange(k, device="cuda") % e).expand(b, k).clone()
    elif kind == "twice":  # experts named more than once by a token
        ids = torch.randint(0, max(1, e // 2), (b, k), generator=g, device="cuda")
    else:  # some choices and some tokens without an expert
        ids = torch.randint(-2, e + 2, (b, k), generator=g, device="cuda")
        ids[::3] = -1
        ids[1, 0] = 2 ** 31 - 1
    w = torch.rand(b, k, generator=g, device="cuda") - 0.2
    return ids.to(torch.int32).contiguous(), w


# b, m, f, experts, k, choices
LAYERS = [
    (1, 128, 128, 1, 1, "spread"), (1, 2048, 768, 16, 8, "spread"), (1, 512, 1408, 3, 3, "spread"), (2, 256, 128, 40, 4, "spread"),
    (4, 384, 256, 8, 3, "one"), (5, 256, 384, 12, 4, "twice"), (3, 640, 128, 7, 5, "none"), (13, 1024, 384, 60, 4, "spread"),
    (16, 256, 256, 4, 4, "one"), (17, 128, 128, 20, 3, "none"), (30, 512, 256, 5, 2, "spread"), (64, 256, 256, 16, 8, "spread"),
    (37, 256, 128, 2, 16, "twice"), (100, 128, 384, 512, 2, "spread"), (256, 256, 128, 8, 2, "spread"), (256, 128, 128, 3, 16, "none"),
    (200, 128, 256, 30, 4, "one"), (2, 1024, 128, 6, 2, "spread"), (3, 4096, 128, 9, 2, "twice"), (6, 2048, 128, 9, 3, "spread"),
    (7, 4096, 256, 6, 2, "none"), (40, 128, 1024, 8, 2, "spread"), (128, 128, 1024, 8, 2, "spread"), (96, 256, 4096, 8, 2, "spread"),
    (128, 128, 1024, 40, 2, "twice"), (130, 1024, 1152, 64, 4, "none"), (64, 2176, 2048, 16, 8, "one"),
]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,f,e,k,kind", LAYERS)
def test_experts(b, m, f, e, k, kind, dt):
    _say(f"moe_experts b={b} m={m} f={f} experts={e} k={k} {kind} {dt}")
    g = _gen(b + m + f + e + k)
    gate_up, down = _experts(m, f, e, b + e)
    ids, w = _choice(b, e, k, kind, g)
    x = torch.randn(b, m, generator=g, device="cuda").to(dt)
    out = torch.full((b, m), float("nan"), dtype=dt, device="cuda")
    twq.moe_experts(x, ids, w, gate_up, down, out=out)
    rows = list(range(b)) if b * k <= 150 else [0, 1, 2, b // 2, b - 2, b - 1]
    check(out[rows], ref.experts(x[rows], ids[rows], w[rows], gate_up, down), "y")
    none = ((ids < 0) | (ids >= e)).all(1)
    assert not bool(out[none].any())
    for _ in range(2):
        assert torch.equal(twq.moe_experts(x, ids, w, gate_up, down), out)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,m,f,e,k", [(1, 512, 256, 16, 4), (9, 256, 128, 6, 2), (20, 256, 384, 24, 3), (150, 128, 128, 70, 8)])
def test_whole_layer(b, m, f, e, k, dt):
    """moe is moe_route and moe_experts, bit for bit; RoutedLayer calls it on weights it packs."""
    _say(f"moe b={b} m={m} f={f} experts={e} k={k} {dt}")
    x, wr, bias = _router(b, m, e, dt, b)
    g = _gen(b + 1)
    up = torch.randn(e, 2 * f, m, generator=g, device="cuda") / m ** 0.5
    dn = torch.randn(e, m, f, generator=g, device="cuda") / f ** 0.5
    for kw in (dict(), dict(bias=bias, score="sigmoid", norm=False, scale=1.5)):
        layer = twq.RoutedLayer(wr, up, dn, k, **kw)
        ids, w = layer.route(x)
        want = twq.moe_experts(x, ids, w, layer.gate_up, layer.down)
        out = torch.full_like(x, float("nan"))
        assert layer(x, out=out) is out and torch.equal(out, want)
        assert torch.equal(twq.moe(x, wr, k, layer.gate_up, layer.down, **kw), want)
        rows = [0, b // 2, b - 1]
        check(out[rows], ref.experts(x[rows], ids[rows], w[rows], layer.gate_up, layer.down), "y")
        one = twq.pack_weight_grouped(up[e - 1])
        assert torch.equal(layer.gate_up[0][e - 1], one[0]) and torch.equal(layer.gate_up[1].view(-1, e, 2 * f)[:, e - 1], one[1])


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("b,k", [(1, 2), (6, 3), (16, 4), (40, 4), (200, 2)])
def test_rows_of_a_batch_do_not_touch_each_other(b, k, dt):
    """A token's output does not depend on the other tokens' values: NaN and infinities elsewhere
    change no bit of it."""
    e, m, f = 5, 256, 256
    gate_up, down = _experts(m, f, e, 1)
    g = _gen(b)
    ids, w = _choice(b, e, k, "spread", g)
    x = torch.randn(b, m, generator=g, device="cuda").to(dt)
    want = twq.moe_experts(x, ids, w, gate_up, down)
    x2, w2 = x.clone(), w.clone()
    x2[0, 7] = float("nan")
    x2[b // 2, 100] = float("inf")
    w2[b - 1, 0] = float("inf")
    out = twq.moe_experts(x2, ids, w2, gate_up, down)
    keep = torch.ones(b, dtype=torch.bool, device="cuda")
    keep[[0, b // 2, b - 1]] = False
    assert torch.equal(out[keep], want[keep]) and not bool(out[~keep].isfinite().all(1).any())


@pytest.mark.parametrize("dt", TYPES)
def test_large_and_small_inner_values(dt):
    """Inner rows past fp16's range reach a finite output; gates where silu vanishes or is the identity."""
    m, f, e, k, b = 256, 128, 3, 2, 6
    gate_up, down = _experts(m, f, e, 2)
    gate_up, down = (gate_up[0], gate_up[1] * 200), (down[0], down[1] * 2.0 ** -12)
    g = _gen(11)
    ids, w = _choice(b, e, k, "spread", g)
    x = torch.randn(b, m, generator=g, device="cuda").to(dt)
    gu = x.double() @ ref.dense(gate_up[0][0], gate_up[1][:, :2 * f]).T
    assert float((gu[:, :f] * gu[:, f:]).abs().max()) > 65504 and float(gu[:, :f].min()) < -90
    check(twq.moe_experts(x, ids, w, gate_up, down), ref.experts(x, ids, w, gate_up, down), "y")


def test_offsets_past_32_bits():
    """Codes of all experts beyond 2^32 bytes: the last expert is checked."""
    m, f, e = 8192, 14336, 80
    _say("moe_experts, 14 GB of codes")
    q1 = torch.zeros(e, 2 * f, m // 2, dtype=torch.uint8, device="cuda")
    q2 = torch.zeros(e, m, f // 2, dtype=torch.uint8, device="cuda")
    s1 = torch.zeros(m // 128, e * 2 * f, device="cuda")
    s2 = torch.zeros(f // 128, e * m, device="cuda")
    (a1, t1), (a2, t2) = _experts(m, f, 1, 3)
    q1[-1], q2[-1] = a1[0], a2[0]
    s1.view(-1, e, 2 * f)[:, -1], s2.view(-1, e, m)[:, -1] = t1, t2
    g = _gen(4)
    for b in (1, 20):
        x = torch.randn(b, m, generator=g, device="cuda").bfloat16()
        ids = torch.full((b, 1), e - 1, dtype=torch.int32, device="cuda")
        w = torch.ones(b, 1, device="cuda")
        out = twq.moe_experts(x, ids, w, (q1, s1), (q2, s2))
        rows = [0, b - 1]
        check(out[rows], ref.experts(x[rows], ids[rows] * 0, w[rows], (a1, t1), (a2, t2)), f"b={b}")


def test_refusals():
    m, f, e, k, b = 256, 128, 4, 2, 5
    gate_up, down = _experts(m, f, e, 1)
    (q1, s1), (q2, s2) = gate_up, down
    x, wr, bias = _router(b, m, e, torch.float16, 1)
    ids, w = twq.moe_route(x, wr, k)
    bad = [lambda: twq.moe_route(x, wr.bfloat16(), k), lambda: twq.moe_route(x, wr[:, :128].contiguous(), k),
           lambda: twq.moe_route(x, wr, k, bias=bias[:3]), lambda: twq.moe_route(x, wr, k, bias=bias.half()),
           lambda: twq.moe_route(x, wr, k, score="relu"), lambda: twq.moe_route(x.T.contiguous().T, wr, k),
           lambda: twq.moe_experts(x, ids.long(), w, gate_up, down), lambda: twq.moe_experts(x, ids, w.half(), gate_up, down),
           lambda: twq.moe_experts(x, ids[:, :1].contiguous(), w, gate_up, down), lambda: twq.moe_experts(x[:3], ids, w, gate_up, down),
           lambda: twq.moe_experts(x, ids, w, (q1, s1[:1]), down), lambda: twq.moe_experts(x, ids, w, (q1[:3], s1), down),
           lambda: twq.moe_experts(x, ids, w, gate_up, (q2[:3], s2)), lambda: twq.moe_experts(x, ids, w, down, gate_up),
           lambda: twq.moe_experts(x, ids, w, gate_up, down, out=x), lambda: twq.moe(x, wr, k, gate_up, down, out=x[:4]),
           lambda: twq.moe(x, wr[:3].contiguous(), k, gate_up, down), lambda: twq.moe(x, wr, k, (q1.cpu(), s1), down),
           lambda: twq.moe(x.float(), wr.float(), k, gate_up, down)]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: twq.moe_route(x, wr, 5), lambda: twq.moe_route(x, wr, 0), lambda: twq.moe(x, wr, 17, gate_up, down),
                 lambda: twq.moe(torch.zeros(257, m, device="cuda").half(), wr, k, gate_up, down)):
        with pytest.raises((twq.TwqError, ValueError, RuntimeError)):
            call()
    assert twq.moe(x[:0], wr, k, gate_up, down).shape == (0, m)
    ids, w = twq.moe_route(x[:0], wr, k)
    assert ids.shape == (0, k) and w.shape == (0, k) and twq.moe_experts(x[:0], ids, w, gate_up, down).shape == (0, m)
