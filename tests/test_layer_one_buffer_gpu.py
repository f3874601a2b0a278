"""Calls of the layer for a few tokens on one buffer at the same time: each has its own workspace, and the
buffer's layout is left alone."""
import pytest
import torch

from test_fp4_gpu import gen, make_ids
from test_moe_layer_gpu import FORMATS, Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_streams_and_two_graphs(fmt):
    layer = Layer(1024, 512, 16, 4, fmt, seed=1)
    g = gen(1)
    calls = []
    for i, T in enumerate((3, 16)):
        calls.append((torch.randn((T, 1024), device="cuda", generator=g).bfloat16(),
                      torch.rand((T, 4), device="cuda", generator=g), make_ids(T, 16, 4, i)))
    want = [layer.run(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        got = [layer.run(*c, stream=s) for c, s in zip(calls, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer.run(*c)
            for _ in range(3):
                out = layer.run(*c)
        graphs.append(graph)
        outs.append(out)
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert layer.buf.device_error() == 0
    del graphs, graph
    layer.buf.close()
