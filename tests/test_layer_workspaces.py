"""Workspaces of the operators around the SSD: calls without one, inside and outside of captured graphs."""
import pytest
import torch

import layer_oracle as lo
import mamba_ssd_prefill_gb300 as m
from test_layer_ops import ok, scan_inputs

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


def call_of(kind, ws, L=700, larger=False):
    """A call of the SSD or of the selective scan; `larger`: one that needs more workspace."""
    if kind == "ssd":
        from mamba_ssd_prefill_gb300.inputs import WORKLOADS, make_inputs

        inp = make_inputs(WORKLOADS["m130-bf16"].with_(batch=6 if larger else 1, seqlen=L, nheads=4, seed=11),
                          device="cuda")
        return lambda: m.ssd_fwd(**inp, workspace=ws)
    t = scan_inputs(1, 20000 if larger else L, 64, 16, seed=11)
    return lambda: scan(t, workspace=ws)


@gpu
@pytest.mark.parametrize("kind", ["ssd", "scan"])
def test_a_workspace_keeps_what_a_graph_uses(kind):
    """A Workspace that grows after a capture: the graph's buffer stays its own."""
    ws = m.Workspace("cuda")
    small, large = call_of(kind, ws), call_of(kind, ws, larger=True)
    want = [o.clone() for o in call_of(kind, m.Workspace("cuda"))()]
    small()
    before = ws.buffers()[-1].numel()
    side = torch.cuda.Stream()
    graph, out = captured(small, side)
    at = ws.buffers()[-1].data_ptr()
    with torch.cuda.stream(side):
        large()
        assert ws.buffers()[-1].numel() > before and at in [b.data_ptr() for b in ws.buffers()[:-1]]
        fillers = [torch.full((before // 4,), 3.0, device="cuda") for _ in range(8)]
        for _ in range(2):
            graph.replay()
            assert all(torch.equal(o, w) for o, w in zip(out, want))
        assert all(bool((f == 3).all()) for f in fillers)
    m.check(ws, side)
    plain = m.Workspace("cuda")  # without a graph nothing is held
    for larger in (False, True):
        call_of(kind, plain, larger=larger)()
    assert len(plain.buffers()) == 1
    m.check(plain)


@gpu
@pytest.mark.parametrize("kind", ["ssd", "scan"])
def test_a_workspace_first_used_inside_a_capture(kind):
    ws = m.Workspace("cuda")
    call = call_of(kind, ws, 900)
    want = [o.clone() for o in call_of(kind, m.Workspace("cuda"), 900)()]
    side = torch.cuda.Stream()
    graph, out = captured(call, side)
    with torch.cuda.stream(side):
        m.check(ws, side)  # nothing has run, nothing is reported
        assert all(torch.equal(o, w) for o, w in zip(call(), want))
        for _ in range(3):
            graph.replay()
            assert all(torch.equal(o, w) for o, w in zip(out, want))
    m.check(ws, side)


@gpu
def test_a_process_whose_first_call_is_captured():
    """The header of calls without a workspace does not exist before the capture."""
    import os
    import subprocess
    import sys

    code = """if True:
        import torch, mamba_ssd_prefill_gb300 as m
        x = torch.randn(4, 256, device="cuda").bfloat16()
        t = dict(x=torch.ones(1, 900, 64, device="cuda"), dt_raw=torch.zeros(1, 900, 64, device="cuda"), dt_bias=None,
                 A=-torch.ones(64, 16, device="cuda"), B=torch.ones(1, 900, 1, 16, device="cuda"),
                 C=torch.ones(1, 900, 1, 16, device="cuda"))
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            n = m.ssd_group_norm(x)
            y, f = m.ssd_selective_scan(**t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, m.ssd_group_norm(x))
        y2, f2 = m.ssd_selective_scan(**t)
        assert torch.equal(y, y2) and torch.equal(f, f2)
        print("same")
    """
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


BAD = [0, 300, 200, 900]  # offsets that decrease


@gpu
def test_errors_of_calls_without_a_workspace_are_reported():
    """Malformed offsets, in a scan with a workspace of its stream, in one that needs only the header, in the
    convolution, in a stream's workspace that grew since, and in replays of a graph."""
    bad = torch.tensor(BAD, dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 200, 300, 900], dtype=torch.int32, device="cuda")
    t = scan_inputs(1, 900, 64, 16, lengths=[200, 100, 600], seed=3)
    tiny = scan_inputs(1, 9, 64, 16, lengths=[2, 3, 4], seed=3)
    tiny_bad = {**tiny, "cu_seqlens": torch.tensor([0, 3, 2, 9], dtype=torch.int32, device="cuda")}
    w = torch.ones(64, 4, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def reports():
        with pytest.raises(m.SsdError) as e:
            m.check()
        assert e.value.status == 1
        m.check()  # read once

    with torch.cuda.stream(side):
        m.check()
        scan({**t, "cu_seqlens": bad})
        reports()
        scan(tiny_bad)
        reports()
        m.ssd_conv(t["x"], w, cu_seqlens=bad)
        reports()
        scan({**t, "cu_seqlens": bad})
        scan(scan_inputs(1, 30000, 64, 16, seed=5))  # the workspace grows
        reports()
    offsets = good.clone()
    graph, _ = captured(lambda: scan({**t, "cu_seqlens": offsets}), side)
    with torch.cuda.stream(side):
        graph.replay()
        m.check()
        offsets.copy_(bad)
        graph.replay()
        offsets.copy_(good)
        graph.replay()
        reports()
    m.check(stream=side)
    m.check()


@gpu
def test_one_workspace_for_the_ssd_and_the_operators_around_it():
    """The scan's states do not land on the tags that ssd_fwd's calls leave behind, nor the other way round."""
    ws = m.Workspace("cuda")
    calls = [call_of(k, ws, L) for k, L in (("ssd", 700), ("scan", 3000), ("ssd", 300), ("scan", 900))]
    wants = [[o.clone() for o in call_of(k, m.Workspace("cuda"), L)()]
             for k, L in (("ssd", 700), ("scan", 3000), ("ssd", 300), ("scan", 900))]
    for _ in range(3):
        for call, want in zip(calls, wants):
            assert all(torch.equal(o, w) for o, w in zip(call(), want))
            m.check(ws)
    t = scan_inputs(1, 900, 64, 16, lengths=[200, 100, 600], seed=3)
    scan({**t, "cu_seqlens": torch.tensor(BAD, dtype=torch.int32, device="cuda")}, workspace=ws)
    calls[0]()
    with pytest.raises(m.SsdError) as e:
        m.check(ws)
    assert e.value.status == 1
    m.check(ws)


def sums_of_segments(ws, nseq, Dc, N, size):
    """The steps' sums [segments, Dc] in a scan's workspace: behind the header and the segments' states, before a copy of
    the initial states, each at a multiple of 256 bytes."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for items in range(1, 1 << 14):
        sums = up(256 + items * Dc * N * 4)
        if up(up(sums + items * Dc * 4) + nseq * Dc * N * 4) == size:
            return ws[sums:sums + items * Dc * 4].view(F32).reshape(items, Dc)
    raise AssertionError("no number of segments has this size")


@gpu
@pytest.mark.parametrize("N", [3, 4, 8, 16, 40])
def test_every_segment_of_packed_sequences_has_a_sum_or_a_mark(N):
    """Segments cut anywhere, also where one sequence ends and the next begins: each channel's sum of steps is written, or
    NaN where no sequence goes on. Channels that fill one tile of the kernel and part of another."""
    import ctypes
    import struct

    Dc, L = 150, 4096
    lengths = [1024, 64, 960, 0, 1, 1023, 512, 512]
    t = scan_inputs(1, L, Dc, N, lengths=lengths, seed=N)
    n = ctypes.c_size_t(0)
    problem = struct.pack("@5q4i", len(lengths), L, Dc, N, 1, 1, 0, 1, 1)
    assert m.lib().ssd_selective_scan_workspace_size(problem, ctypes.byref(n)) == 0 and n.value > 256
    ws = torch.full((n.value,), 0x5a, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    got = scan(t, workspace=ws)
    m.check(ws)
    sums = sums_of_segments(ws, len(lengths), Dc, N, n.value)
    assert len(sums) > 20
    assert not bool((sums.view(torch.int32) == 0x5a5a5a5a).any())
    marked = torch.isnan(sums)
    assert bool((marked == marked[:, :1]).all()) and bool((sums[~marked] > 0).all())
    yr, fr, ey, ef = lo.scan(**t)
    ok(got[0], yr, ey, t["x"].dtype)
    ok(got[1], fr, ef, F32)


@gpu
@pytest.mark.parametrize("kind", ["ssd", "scan"])
def test_memory_of_a_capture_outlives_its_workspace(kind):
    """What a Workspace takes inside a capture is the graph's: it stays when the Workspace goes."""
    want = [o.clone() for o in call_of(kind, m.Workspace("cuda"))()]
    ws = m.Workspace("cuda")
    call = call_of(kind, ws)
    inputs = call.__closure__  # the graph reads them
    side = torch.cuda.Stream()
    graph, out = captured(call, side)
    at, size = ws.buffers()[-1].data_ptr(), ws.buffers()[-1].numel()
    pools = [tuple(s["segment_pool_id"]) for s in torch.cuda.memory_snapshot()
             if s["address"] <= at < s["address"] + s["total_size"]]
    assert pools and pools[0] != (0, 0)
    ws.held, ws.buf, ws.layer = [], None, None
    torch.cuda.empty_cache()
    fillers = [torch.full((size // 4,), 3.0, device="cuda") for _ in range(8)]
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(o, w) for o, w in zip(out, want))
    assert inputs and all(bool((f == 3).all()) for f in fillers)
