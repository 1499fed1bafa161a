"""The many-row kernel of the layer with 16-bit activations, whose call has the largest workspace and the most
launches, as it is used: graphs replayed beside each other with changing inputs, streams, threads."""
import threading

import pytest
import torch

import w4a4_rank_gemm_amd as twq
from tests import moe_reference as ref
from tests.adapter_reference import check
from tests.test_gpu_adapters import TYPES, _gen, _say

pytestmark = pytest.mark.gpu

M, N, R = 512, 33024, 16
TOKENS = (100, 700, 130)  # tiles of 64, 128, 64 rows


class Wide:
    """Up to a wide layer with its low-rank pair, down again, and up once more."""

    def __init__(self, dt, seed=1):
        g = _gen(seed)

        def randn(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.up = twq.pack_weight_grouped(randn(N, M) / M ** 0.5)
        self.down = twq.pack_weight_grouped(randn(M, N) / N ** 0.5)
        self.l1t, self.l2t = (randn(R, M) * 0.03).half(), (randn(N, R) * 0.03).half()

    def __call__(self, x):
        y = twq.linear_a16(x, *self.up, self.l1t, self.l2t)
        z = twq.linear_a16(y, *self.down)
        return [y, z, twq.linear_a16(z, *self.up, self.l1t, self.l2t)]


def _x(b, dt, seed):
    return torch.randn(b, M, generator=_gen(seed), device="cuda").to(dt)


@pytest.mark.parametrize("dt", TYPES)
def test_each_step(dt):
    wide = Wide(dt)
    for b in TOKENS:
        _say(f"wide block b={b} {dt}")
        assert not ref.few(b, N)
        x = _x(b, dt, b)
        y, z, w = wide(x)
        check(y, ref.linear_a16(x, *wide.up, wide.l1t, wide.l2t), "up")
        check(z, ref.linear_a16(y, *wide.down, None, None), "down")
        check(w, ref.linear_a16(z, *wide.up, wide.l1t, wide.l2t), "up again")


@pytest.mark.parametrize("b", TOKENS)
@pytest.mark.parametrize("dt", TYPES)
def test_graph_replays_follow_their_inputs(b, dt):
    """Two graphs replayed at once on two streams, with other inputs each time and eager calls in between."""
    _say(f"graphs of the wide block, b={b} {dt}")
    wide = Wide(dt)
    sets = [[_x(b, dt, s + 10 * q) for s in range(4)] for q in range(2)]
    live = [s[0].clone() for s in sets]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for x in live:
        wide(x)
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs.append(wide(x))
        graphs.append(graph)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(4):
        want = []
        for q in range(2):
            live[q].copy_(sets[q][rep])
            want.append([o.clone() for o in wide(sets[q][rep])])
        torch.cuda.synchronize()
        for q in range(2):
            with torch.cuda.stream(streams[q]):
                graphs[q].replay()
        eager = wide(sets[0][rep])  # beside both
        torch.cuda.synchronize()
        for q in range(2):
            assert all(torch.equal(o, w) for o, w in zip(outs[q], want[q])), f"replay {rep}, graph {q}"
        assert all(torch.equal(o, w) for o, w in zip(eager, want[0])), f"eager call beside replay {rep}"


@pytest.mark.parametrize("dt", TYPES)
def test_streams_and_threads_do_not_share_scratch(dt):
    wide = Wide(dt)
    sizes = list(TOKENS) + [9]
    ins = [_x(b, dt, b) for b in sizes]
    want = [[o.clone() for o in wide(x)] for x in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [None] * len(ins)
    for _ in range(4):
        for q, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[q] = wide(ins[q])
    torch.cuda.synchronize()
    for q in range(len(ins)):
        assert all(torch.equal(o, w) for o, w in zip(got[q], want[q])), f"stream {q}"

    def work(q):
        with torch.cuda.stream(streams[q]):
            for _ in range(4):
                got[q] = wide(ins[q])
            streams[q].synchronize()

    threads = [threading.Thread(target=work, args=(q,)) for q in range(len(ins))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for q in range(len(ins)):
        assert all(torch.equal(o, w) for o, w in zip(got[q], want[q])), f"thread {q}"
