"""Workspaces of the operators around the SSD: calls without one, inside and outside of captured graphs."""
import pytest
import torch

import mamba_ssd_prefill_gb300 as m
from test_layer_ops import scan_inputs

gpu = pytest.mark.gpu
F32 = torch.float32


def scan(t, **kw):
    return m.ssd_selective_scan(**t, state_dtype=F32, **kw)


def captured(fn, stream):
    """fn() captured on `stream`: (graph, its outputs)."""
    graph = torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        out = fn()
    torch.cuda.current_stream().wait_stream(stream)
    return graph, out


@gpu
def test_a_captured_prompt_keeps_its_scratch():
    """A scan in segments, captured without a workspace; then longer ones on the same stream, whose memory other tensors
    take; then the replay: it gives the same values and leaves the others alone."""
    t, longer = scan_inputs(1, 700, 64, 16, seed=1), scan_inputs(1, 9000, 96, 16, seed=2)
    want = scan(t, workspace=m.Workspace("cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        scan(t)  # the stream has a workspace of this size
        graph, out = captured(lambda: scan(t), side)
        scan(longer)
        side.synchronize()
        fillers = [torch.full((n,), 3.0, device="cuda") for n in (64, 4096, 1 << 16, 1 << 18, 1 << 20) for _ in range(24)]
        side.synchronize()
        for _ in range(2):
            out[0].zero_()
            graph.replay()
            side.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert all(bool((f == 3).all()) for f in fillers)


@gpu
def test_graphs_of_one_stream_replayed_on_two():
    ts = [scan_inputs(1, 3000, 64, 16, seed=3 + i) for i in range(2)]
    wants = [scan(t, workspace=m.Workspace("cuda")) for t in ts]
    side = torch.cuda.Stream()
    graphs = [captured(lambda: scan(t), side) for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    for _ in range(20):
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, out), want in zip(graphs, wants):
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@gpu
def test_a_first_call_inside_a_capture():
    """A stream's first calls are captured ones: eager calls on it before the first replay find a workspace in order."""
    t = scan_inputs(1, 900, 64, 16, seed=7)
    want = scan(t, workspace=m.Workspace("cuda"))
    side = torch.cuda.Stream()
    graph, out = captured(lambda: scan(t), side)
    with torch.cuda.stream(side):
        eager = scan(t)
        assert torch.equal(eager[0], want[0])
        graph.replay()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@gpu
def test_a_stream_s_workspace_grows_between_calls():
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for L in (300, 1500, 6000, 700):
        t = scan_inputs(1, L, 64, 16, seed=L)
        want = scan(t, workspace=m.Workspace("cuda"))
        side.wait_stream(torch.cuda.current_stream())
        got = scan(t, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
