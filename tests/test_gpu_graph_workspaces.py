"""Captured layers own their scratch memory, on an MI355X: replays neither write the workspaces of
eager calls nor, where two graphs run at once, each other's."""
import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests.test_gpu_adapters import _case, _gen, _say

pytestmark = pytest.mark.gpu

B, M, N, R = 300, 1024, 2064, 32


def _layers(seed):
    g = _gen(seed)
    x = torch.randn(B, M, generator=g, device="cuda").half()
    w = torch.randn(N, M, generator=g, device="cuda") * 0.02
    l1t = (torch.randn(R, M, generator=g, device="cuda") / M ** 0.5).half()
    l2t = (torch.randn(N, R, generator=g, device="cuda") * 0.05).half()
    qw, sw = twq.pack_weight(w)
    qg, sg = twq.pack_weight_grouped(w)
    lp = twq.pack_lowrank_int4(l1t, l2t)
    layer = twq.DualLinear(w, l1t, l2t)
    idx, _, at, bt, _, scale = _case(B, M, N, 16, 3, "random", torch.float16, seed=seed)
    plan = twq.adapter_plan(idx, 3)
    return {"linear": lambda: [twq.linear(x, qw, sw, l1t, l2t)],
            "linear_grouped": lambda: [twq.linear_grouped(x, qg, sg, l1t, l2t)],
            "linear_a8": lambda: [twq.linear_a8(x, qw, sw, l1t, l2t)],
            "linear_lr4": lambda: [twq.linear_lr4(x, qw, sw, lp)],
            "quantize_act": lambda: list(twq.quantize_act(x, l1t)),
            "adapted": lambda: list(layer.adapted(x, at, bt, plan, scale, keep_h=True))}


def _capture(fn, stream):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = fn()
    torch.cuda.synchronize()
    return graph, outs


@pytest.mark.parametrize("name", ["linear", "linear_grouped", "linear_a8", "linear_lr4", "quantize_act", "adapted"])
def test_replays_leave_eager_workspaces_alone(name):
    """Eager calls on the capture stream first, as a warm-up does, so that it has a workspace."""
    _say(f"workspaces {name}")
    fn = _layers(1)[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in fn()]
    torch.cuda.synchronize()
    graph, outs = _capture(fn, side)
    mine = list(twq._workspaces.values())
    for ws in mine:
        ws.fill_(0xA5)
    torch.cuda.synchronize()
    for rep in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), f"replay {rep}"
    assert all(bool((ws == 0xA5).all()) for ws in mine)


def test_two_graphs_at_once():
    """Captured on one stream, replayed on two, with eager calls on a third."""
    layers = [_layers(2), _layers(3)]
    side, streams = torch.cuda.Stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    want, captured = [], []
    for lay in layers:
        def everything(lay=lay):
            return [t for fn in lay.values() for t in fn()]
        want.append([t.clone() for t in everything()])
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        captured.append(_capture(everything, side))
    for rep in range(4):
        for (_, outs) in captured:
            for o in outs:
                o.zero_()
        torch.cuda.synchronize()
        for s, (graph, _) in zip(streams, captured):
            with torch.cuda.stream(s):
                graph.replay()
        eager = [t for fn in layers[0].values() for t in fn()]
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(eager, want[0])), f"eager, replay {rep}"
        for k, (_, outs) in enumerate(captured):
            assert all(torch.equal(o, w) for o, w in zip(outs, want[k])), f"graph {k}, replay {rep}"
