"""paged_attention in CUDA graphs without a workspace of the caller's: every
capture has scratch of its own, ready whichever graph runs first, on
whichever stream."""
from __future__ import annotations

import pytest

from paged_util import PagedCase

pytestmark = pytest.mark.gpu

ROWS = [(5000, 1), (100, 40), (3000, 3)]   # units that several CTAs share


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from speculative_decoding_verification_25_gb300 import build as b
    b.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _case(D=128, seed=1):
    """A case and its result, computed with a workspace that the caller zeroed."""
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N
    c = PagedCase(ROWS, 8, 2, D, 16, "bf16", seed=seed)
    want = c.run(workspace=torch.zeros(N.spec_paged_attention_workspace_bytes(D), dtype=torch.uint8, device="cuda:0"))
    c.check(want)
    return c, want


def _same(got, want):
    import torch
    torch.cuda.synchronize()
    assert torch.equal(got.out.view(torch.int16), want.out.view(torch.int16)) and torch.equal(got.lse, want.lse)


def _capture(c, stream, pool=None, calls=1):
    import torch
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream, pool=pool):
        got = [c.run() for _ in range(calls)]
    return graph, got


def _dirty_pool(stream, D):
    """A memory pool for captures whose blocks hold 0xff bytes, and the graph that keeps it."""
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N
    pool, graph = torch.cuda.graph_pool_handle(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream, pool=pool):
        block = torch.empty(N.spec_paged_attention_workspace_bytes(D), dtype=torch.uint8, device="cuda:0")
        block.fill_(255)
        del block
    graph.replay()
    torch.cuda.synchronize()
    return pool, graph


@pytest.mark.parametrize("D", [64, 128])
def test_two_cold_graphs_the_second_first(D):
    import torch
    c, want = _case(D)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pool, keep = _dirty_pool(side, D)
    first, got_first = _capture(c, side, pool)
    second, got_second = _capture(c, side, pool)
    for graph, got in ((second, got_second), (first, got_first), (second, got_second)):
        got[0].out.fill_(float("nan"))
        got[0].lse.fill_(float("nan"))
        graph.replay()
        _same(got[0], want)


def test_calls_outside_a_graph_after_a_cold_capture():
    import torch
    c, want = _case()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pool, keep = _dirty_pool(side, 128)
    graph, got = _capture(c, side, pool)
    with torch.cuda.stream(side):
        _same(c.run(), want)
    _same(c.run(stream=side), want)
    graph.replay()
    _same(got[0], want)


def test_graphs_of_one_stream_replayed_on_two():
    """Captured on one stream, replayed at the same time on others, beside calls on that stream."""
    import torch
    cases = [_case(seed=s) for s in (1, 2, 3)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = [_capture(c, side, calls=2) for c, _ in cases[:2]]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(40):
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        got = cases[2][0].run(stream=side)
        _same(got, cases[2][1])
        for (_, results), (_, want) in zip(graphs, cases):
            for r in results:
                _same(r, want)


def test_a_capture_over_two_streams():
    """The streams of one capture run at the same time and share nothing."""
    import torch
    (c, want), (d, want_d) = _case(seed=4), _case(seed=5)
    side, fork = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph, got, got_d = torch.cuda.CUDAGraph(), [], []
    with torch.cuda.graph(graph, stream=side):
        for k in range(3):
            fork.wait_stream(side)
            got_d.append(d.run(stream=fork))
            got.append(c.run())
        side.wait_stream(fork)
    for _ in range(20):
        graph.replay()
    for r in got:
        _same(r, want)
    for r in got_d:
        _same(r, want_d)
