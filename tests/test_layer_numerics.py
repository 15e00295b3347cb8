"""Accuracy of the operators around the SSD where their bounds are tightest: softplus far from its bend, the gate, and
scans joined from many segments."""
import pytest
import torch

import layer_oracle as lo
import mamba_ssd_prefill_gb300 as m
from test_layer_ops import ok, run_scan, scan_inputs

gpu = pytest.mark.gpu
F32 = torch.float32


def units(v):
    """The bound of the relative error of softplus(v) and of v sigmoid(v): the exponent's argument |v| log2(e), rounded
    once and with a rounded constant, is off by 1.3 |v| units of 2^-24 in e; 2^x by 4; the rest by 4. For v >= 0 the
    exponential is at most half of the result, and its error |v| e stays below 1."""
    return torch.where(v < 0, 1.3 * v.abs(), 0.0) + 8


@gpu
@pytest.mark.parametrize("L", [1, 2, 700])
def test_softplus_is_accurate_from_minus_80(L):
    """With x = B = 1 in the first token and x = 0 behind it, A = 0 and no initial state, the final state is the first
    step itself: of one token, of a prompt, of a prompt in segments."""
    Dc = 4096
    v = torch.cat([torch.linspace(-80, 0, Dc - 1024), torch.linspace(0, 40, 1024)])
    raw, x = torch.zeros(1, L, Dc), torch.zeros(1, L, Dc)
    raw[0, 0], x[0, 0] = v, 1
    ones = torch.ones(1, L, 1, 4, device="cuda")
    _, fin = m.ssd_selective_scan(x.cuda(), raw.cuda(), None, torch.zeros(Dc, 4, device="cuda"), ones, ones)
    d = v.double()
    want = d.clamp(min=0) + torch.log1p(torch.exp(-d.abs()))
    off = (fin[0].cpu().double() - want[:, None]).abs() / want[:, None] * 2.0 ** 24
    assert bool((off <= units(d)[:, None]).all()), float((off - units(d)[:, None]).max())


@gpu
def test_the_gate_is_accurate_from_minus_80():
    """(norm(x) weight + bias) act(z) with weight 0 and bias 1 is v sigmoid(v) of the gate alone."""
    z = torch.linspace(-80, 80, 8192)[None]
    x, one, none = torch.ones(1, 8192, device="cuda"), torch.ones(8192, device="cuda"), torch.zeros(8192, device="cuda")
    y = m.ssd_group_norm(x, none, one, z=z.cuda())
    d = z.double()
    want = lo.silu(d)
    off = (y.cpu().double() - want).abs() / want.abs().clamp(min=1e-300) * 2.0 ** 24
    assert bool((off <= units(d)).all()), float((off - units(d)).max())


@gpu
@pytest.mark.parametrize("L,Dc,N,kw", [
    (4000, 24, 16, {}), (3500, 40, 4, dict(io=F32)), (4100, 16, 100, {}), (4100, 16, 200, dict(state=torch.float16)),
    (4100, 200, 8, dict(lengths=[1500, 0, 1, 2599])), (4100, 33, 24, dict(lengths=[4100], init=False)),
    (4100, 48, 33, dict(lengths=[7] * 100 + [3400])),
], ids=lambda v: None)
def test_scans_joined_from_more_segments_than_a_round_holds(L, Dc, N, kw):
    """The join takes 128 segments a round: these have more."""
    import ctypes
    import struct

    lengths, state = kw.get("lengths"), kw.get("state", F32)
    n, small = ctypes.c_size_t(0), 2 if state is torch.float16 else 4
    problem = struct.pack("@5q4i", len(lengths) if lengths else 1, L, Dc, N, 1, 1,
                          2 if small == 2 else 0, int(bool(lengths)), 1)
    assert m.lib().ssd_selective_scan_workspace_size(problem, ctypes.byref(n)) == 0
    assert n.value > 128 * Dc * (N + 1) * 4
    t = scan_inputs(1, L, Dc, N, seed=L, **kw)
    y, fin = run_scan(t, state)
    yr, fr, ey, ef = lo.scan(**t)
    ok(y, yr, ey, t["x"].dtype, "y")
    ok(fin, fr, ef + lo.TINY[state], state, "final states")  # fp16 states may be subnormal
