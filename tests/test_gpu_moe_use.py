"""The 16-bit-activation and routed layers as they are used, on an MI355X: a block of a decoder with
adapters beside it, graph replays whose inputs change, streams, calls of several threads."""
import threading

import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import moe_reference as ref
from tests.adapter_reference import check
from tests.test_gpu_adapters import TYPES, _gen, _say

pytestmark = pytest.mark.gpu

M, N, R, F, E, K = 512, 528, 16, 256, 12, 3


class Block:
    """A projection with its low-rank pair and its requests' adapters, then a routed layer."""

    def __init__(self, dt, seed=1):
        g = _gen(seed)

        def randn(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        w = randn(M, M) / M ** 0.5
        self.qw, self.sw = twq.pack_weight_grouped(w)
        self.l1t, self.l2t = (randn(R, M) * 0.03).half(), (randn(M, R) * 0.03).half()
        self.at, self.bt = (randn(4, 32, M) * 0.03).to(dt), (randn(4, M, 32) * 0.03).to(dt)
        self.routed = twq.RoutedLayer((randn(E, M) / M ** 0.5).to(dt), randn(E, 2 * F, M) / M ** 0.5, randn(E, M, F) / F ** 0.5, K,
                                      bias=randn(E) * 0.1, score="sigmoid")

    def __call__(self, x, index):
        """Every value on the way."""
        y = twq.linear_a16(x, self.qw, self.sw, self.l1t, self.l2t)
        z = twq.adapters(x, self.at, self.bt, twq.adapter_plan(index, 4), y)
        ids, w = self.routed.route(z)
        return [y, z, ids, w, self.routed(z)]


def _inputs(b, dt, seed):
    g = _gen(seed)
    return [torch.randn(b, M, generator=g, device="cuda").to(dt),
            torch.randint(-1, 4, (b,), generator=g, device="cuda").to(torch.int32)]


@pytest.mark.parametrize("b", [1, 13, 70])
@pytest.mark.parametrize("dt", TYPES)
def test_block(b, dt):
    """Each step against its binary64 definition on the values the block itself saw."""
    from tests import adapter_reference
    _say(f"block b={b} {dt}")
    block = Block(dt)
    x, index = _inputs(b, dt, b)
    y, z, ids, w, out = block(x, index)
    check(y, ref.linear_a16(x, block.qw, block.sw, block.l1t, block.l2t), "projection")
    check(z, adapter_reference.adapters(x, block.at, block.bt, index, y, None)[0], "adapters")
    want, ww = ref.route(z, block.routed.wr, K, block.routed.bias, "sigmoid")
    assert torch.equal(ids.long(), want) and bool(((w.double() - ww).abs() <= 2.0 ** -23 * ww).all())
    check(out, ref.experts(z, ids, w, block.routed.gate_up, block.routed.down), "routed layer")


@pytest.mark.parametrize("b", [1, 6, 33, 100])
def test_graph_replays_follow_their_inputs(b):
    """Two graphs of the block, replayed in turn with other inputs each time (other experts among
    them), eager calls in between; both share nothing with each other or with those."""
    _say(f"graphs of the block, b={b}")
    block = Block(torch.float16)
    sets = [[_inputs(b, torch.float16, s + 10 * q) for s in range(3)] for q in range(2)]
    live = [[t.clone() for t in s[0]] for s in sets]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for inp in live:
        block(*inp)
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs.append(block(*inp))
        graphs.append(graph)
    torch.cuda.synchronize()
    for rep in range(3):
        want = []
        for q in range(2):
            for dst, src in zip(live[q], sets[q][rep]):
                dst.copy_(src)
            want.append([o.clone() for o in block(*sets[q][rep])])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for q in range(2):
            with torch.cuda.stream(streams[q]):
                graphs[q].replay()
        torch.cuda.synchronize()
        for q in range(2):
            for i, (o, w) in enumerate(zip(outs[q], want[q])):
                assert torch.equal(o, w), f"replay {rep}, graph {q}, output {i}"


def test_streams_and_threads_do_not_share_scratch():
    """The block on two streams at once, and from four host threads, gives what it gives alone."""
    block = Block(torch.bfloat16)
    sizes = [70, 9, 1, 150]
    ins = [_inputs(b, torch.bfloat16, b) for b in sizes]
    want = [[o.clone() for o in block(*i)] for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [None] * 4
    for _ in range(4):
        for q, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[q] = block(*ins[q])
    torch.cuda.synchronize()
    for q in range(4):
        assert all(torch.equal(o, w) for o, w in zip(got[q], want[q])), f"stream {q}"

    def work(q):
        with torch.cuda.stream(streams[q]):
            for _ in range(4):
                got[q] = block(*ins[q])
            streams[q].synchronize()

    threads = [threading.Thread(target=work, args=(q,)) for q in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for q in range(4):
        assert all(torch.equal(o, w) for o, w in zip(got[q], want[q])), f"thread {q}"


def test_same_weight_with_activations_of_each_width():
    """One packed weight serves linear_grouped (4-bit activations) and linear_a16: on activations
    that 4 bits hold exactly, both give the same product up to their roundings."""
    g = _gen(6)
    qw, sw = twq.pack_weight_grouped(torch.randn(N, M, generator=g, device="cuda") * 0.02)
    x = torch.randint(-7, 8, (40, M), generator=g, device="cuda").half()
    x[:, ::128] = 7  # each group's scale is then 1
    a, b = twq.linear_a16(x, qw, sw), twq.linear_grouped(x, qw, sw)
    value, bound = ref.linear_a16(x, qw, sw, None, None)
    check(a, (value, bound), "linear_a16")
    assert float((b.double() - value).abs().max()) <= 2e-3 * float(value.abs().max())
