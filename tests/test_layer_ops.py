"""The operators around the SSD (selective scan, convolution by itself, group norm, e4m3 projections): refusals on the
CPU, values on the GPU against 64-bit forms with derived bounds (layer_oracle.py)."""
import ctypes
import os
import struct

import pytest
import torch

import layer_oracle as lo
import mamba_ssd_prefill_gb300 as m

gpu = pytest.mark.gpu
F32, BF16, F16, E4M3 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(m.LIB_PATH):
        from mamba_ssd_prefill_gb300 import _build

        _build.build()


def gen(seed):
    return torch.Generator("cpu").manual_seed(seed)


def ok(got, want, err, dtype, what=""):
    good, excess = lo.within(got, want, err, dtype)
    assert good, f"{what}: {excess} outside the bound"


# ------------------------------------------------------------------------------------------------ selective scan

def scan_inputs(b, L, Dc, N, G=1, io=BF16, state=F32, seed=0, gate=True, init=True, D=True, bias=True, lengths=None,
                dt_mid=0.0, device="cuda"):
    g = gen(seed)
    r = lambda *s, scale=1.0: torch.randn(*s, generator=g) * scale  # noqa: E731
    nseq = len(lengths) if lengths is not None else b
    dt0 = torch.exp(torch.rand(Dc, generator=g) * 4.6 - 6.9 + dt_mid)
    t = dict(x=r(b, L, Dc).to(io), dt_raw=r(b, L, Dc).to(io),
             dt_bias=torch.log(torch.expm1(dt0)) if bias else None,
             A=-torch.arange(1, N + 1) * torch.exp(r(Dc, N, scale=0.1)), B=r(b, L, G, N).to(io),
             C=r(b, L, G, N).to(io), D=r(Dc) if D else None, z=r(b, L, Dc).to(io) if gate else None,
             init_states=r(nseq, Dc, N, scale=0.3).to(state) if init else None,
             cu_seqlens=None if lengths is None else
             torch.tensor([sum(lengths[:i]) for i in range(nseq + 1)], dtype=torch.int32))
    return {k: v if v is None else v.to(device) for k, v in t.items()}


def run_scan(t, state=F32, **kw):
    ws = m.Workspace("cuda")
    y, fin = m.ssd_selective_scan(**t, state_dtype=state, workspace=ws, **kw)
    m.check(ws)
    return y, fin


def check_scan(t, state=F32, **kw):
    y, fin = run_scan(t, state, **kw)
    yr, fr, ey, ef = lo.scan(**t)
    ok(y, yr, ey, t["x"].dtype, "y")
    ok(fin, fr, ef, state, "final states")
    return y, fin


SCAN = [
    # b, L, Dc, N, extra
    (1, 1, 1536, 16, {}),                                        # one token
    (5, 1, 130, 16, dict(state=F16)),                            # tokens of several sequences, odd channels
    (3, 1, 64, 1, dict(io=F32, gate=False)),                     # one state
    (2, 1, 96, 256, dict(G=2)),                                  # the most states
    (2, 2, 64, 16, {}),
    (2, 33, 96, 16, dict(io=F16)),                               # ends inside a tile
    (1, 64, 1, 16, {}),                                          # one channel
    (1, 257, 40, 7, dict(G=5, io=F32)),                          # odd states, groups of 8 channels
    (3, 100, 130, 24, dict(G=2, state=F16)),
    (1, 129, 66, 33, dict(io=F16, D=False, gate=False, init=False)),
    (1, 70, 36, 100, dict(io=F32, bias=False)),
    (1, 65, 24, 256, dict(G=3)),
    (1, 1500, 70, 16, {}),                                       # long: several segments where it is cut
    (2, 700, 8, 4, dict(io=F32)),
    (1, 300, 200, 16, dict(dt_mid=4.0)),                         # large steps: states forgotten at once
]


@gpu
@pytest.mark.parametrize("b,L,Dc,N,kw", SCAN, ids=[f"scan{i}" for i in range(len(SCAN))])
def test_scan_values(b, L, Dc, N, kw):
    state = kw.get("state", F32)
    check_scan(scan_inputs(b, L, Dc, N, **kw, seed=L + Dc), state)


PACKED = [
    ([33, 1, 0, 64, 31], 40, 16, dict(G=2)),
    ([0, 0, 5, 0], 64, 16, dict(io=F32)),
    ([1] * 9, 70, 8, dict(state=F16)),
    ([700, 3, 500, 0, 1, 300], 66, 24, dict(io=F16, gate=False)),
    ([1300], 34, 16, dict(init=False)),
    ([64, 64, 128, 32, 32], 32, 16, dict(io=F32)),               # boundaries on tile edges
]


@gpu
@pytest.mark.parametrize("lengths,Dc,N,kw", PACKED, ids=[f"packed{i}" for i in range(len(PACKED))])
def test_scan_packed(lengths, Dc, N, kw):
    state = kw.get("state", F32)
    check_scan(scan_inputs(1, sum(lengths), Dc, N, lengths=lengths, **kw, seed=len(lengths)), state)


@gpu
def test_scan_packed_equals_regular_batch():
    t = scan_inputs(4, 90, 64, 16, seed=5)
    y, fin = run_scan(t)
    p = {k: v.reshape(1, 360, *v.shape[2:]) if k in ("x", "dt_raw", "B", "C", "z") else v for k, v in t.items()}
    p["cu_seqlens"] = torch.tensor([0, 90, 180, 270, 360], dtype=torch.int32, device="cuda")
    yr, fr, ey, ef = lo.scan(**t)
    yp, fp = run_scan(p)
    ok(yp.reshape(y.shape), yr, ey, BF16)
    ok(fp, fr, ef, F32)


@gpu
@pytest.mark.parametrize("io", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_scan_slices_of_wider_rows(io, off):
    """x, z, B and C as column slices: strides of the rows, and starts that are not 16-byte aligned."""
    t = scan_inputs(2, 75, 72, 16, io=io, seed=9)
    y0, f0 = run_scan(t)
    wide = torch.full((2, 75, 2 * 72 + 32 + 41), float("nan"), dtype=io, device="cuda")
    s = dict(t)
    at = off
    for k, w in (("x", 72), ("z", 72), ("B", 16), ("C", 16)):
        wide[..., at:at + w] = t[k].reshape(2, 75, w)
        s[k] = wide[..., at:at + w] if w == 72 else wide[..., at:at + w].unflatten(-1, (1, w))
        at += w + (off > 0)
    out = torch.full((2, 75, 100), 7.0, dtype=io, device="cuda")
    y, f = run_scan(s, y=out[..., off:off + 72])
    assert torch.equal(y, y0) and torch.equal(f, f0)
    assert bool((out[..., :off] == 7).all()) and bool((out[..., off + 72:] == 7).all())


@gpu
def test_scan_expanded_inputs():
    """Rows at stride 0 (one B for all tokens, one x for all sequences)."""
    t = scan_inputs(3, 50, 64, 16, seed=3)
    t["B"] = t["B"][:, :1].expand(3, 50, 1, 16)
    t["x"] = t["x"][:1].expand(3, 50, 64)
    check_scan(t)


@gpu
@pytest.mark.parametrize("L", [1, 40, 900])
def test_scan_state_in_place(L):
    t = scan_inputs(2, L, 64, 16, seed=11)
    y0, f0 = run_scan(t)
    st = t["init_states"]
    y, f = run_scan(t, final_states=st)
    assert f is st and torch.equal(y, y0) and torch.equal(f, f0)


@gpu
@pytest.mark.parametrize("T1", [1, 64, 333, 399])
def test_scan_split_continues(T1):
    """[0, T1) then [T1, L) from its final states, and single tokens, agree with the 64-bit scan of the whole."""
    t = scan_inputs(2, 400, 48, 16, io=F32, seed=13)
    yr, fr, ey, ef = lo.scan(**t)
    cut = lambda a, b: {k: v[:, a:b] if k in ("x", "dt_raw", "B", "C", "z") else v for k, v in t.items()}  # noqa: E731
    y1, f1 = run_scan(cut(0, T1))
    second = cut(T1, 400)
    second["init_states"] = f1
    y2, f2 = run_scan(second)
    ok(torch.cat([y1, y2], 1), yr, ey, F32)
    ok(f2, fr, ef, F32)


@gpu
def test_scan_decode_loop_matches_prefill():
    t = scan_inputs(3, 24, 80, 16, seed=17)
    yr, fr, ey, ef = lo.scan(**t)
    st = t["init_states"].clone()
    ys = []
    for i in range(24):
        step = {k: v[:, i:i + 1] if k in ("x", "dt_raw", "B", "C", "z") else v for k, v in t.items()}
        step["init_states"] = st
        ys.append(run_scan(step, final_states=st)[0])
    ok(torch.cat(ys, 1), yr, ey, BF16)
    ok(st, fr, ef, F32)


@gpu
def test_scan_without_softplus_and_options():
    t = scan_inputs(1, 60, 64, 16, io=F32, seed=19)
    t["dt_raw"] = t["dt_raw"].abs() * 0.1
    t["dt_bias"] = None
    y, fin = run_scan(t, softplus=False)
    yr, fr, ey, ef = lo.scan(**t, softplus=False)
    ok(y, yr, ey, F32)
    ok(fin, fr, ef, F32)
    y2, none = m.ssd_selective_scan(**t, softplus=False, return_final_states=False)
    assert none is None and torch.equal(y, y2)


@gpu
def test_scan_extreme_steps():
    """dt_raw far below and above softplus's bend, A = 0 and a state decay that underflows."""
    t = scan_inputs(1, 40, 32, 16, io=F32, seed=23)
    t["dt_raw"][0, ::3] = -60.0
    t["dt_raw"][0, 1::3] = 45.0
    t["dt_bias"] = None
    t["A"][:, 0] = 0.0
    check_scan(t)


@gpu
def test_scan_nan_stays_in_its_channel_and_sequence():
    t = scan_inputs(2, 80, 64, 16, seed=29)
    y0, f0 = run_scan(t)
    t["x"][1, 40, 5] = float("nan")
    y, f = run_scan(t)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1, 40:, 5] = True
    assert bool(torch.isnan(y[bad]).all()) and torch.equal(y[~bad], y0[~bad])
    assert bool(torch.isnan(f[1, 5]).all()) and torch.equal(f[0], f0[0])


@gpu
def test_scan_empty():
    for kw in (dict(b=0, L=5), dict(b=2, L=0)):
        t = scan_inputs(kw["b"], kw["L"], 64, 16)
        y, fin = run_scan(t)
        assert y.shape == (kw["b"], kw["L"], 64) and torch.equal(fin, t["init_states"])
    t = scan_inputs(2, 0, 64, 16, init=False)
    assert not run_scan(t)[1].any()
    t = scan_inputs(1, 0, 64, 16, lengths=[0, 0])
    assert torch.equal(run_scan(t)[1], t["init_states"])


@gpu
@pytest.mark.parametrize("cu", [[0, 30, 20, 64], [0, 30, 50, 60], [5, 30, 50, 64], [0, 2000000000, 50, 64],
                                [0, -7, 50, 64]])
def test_scan_and_conv_bad_offsets_reported(cu):
    t = scan_inputs(1, 64, 64, 16, lengths=[30, 20, 14])
    want = run_scan(t)[0]
    good = t["cu_seqlens"]
    t["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ws = m.Workspace("cuda")
    m.ssd_selective_scan(**t, workspace=ws)
    with pytest.raises(m.SsdError) as e:
        m.check(ws)
    assert e.value.status == 1
    t["cu_seqlens"] = good
    y, _ = m.ssd_selective_scan(**t, workspace=ws)  # the workspace works again
    m.check(ws)
    assert torch.equal(y, want)
    w = torch.ones(64, 4, device="cuda")
    m.ssd_conv(t["x"], w, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), workspace=ws)
    with pytest.raises(m.SsdError) as e:
        m.check(ws)
    assert e.value.status == 1


@gpu
def test_scan_repeats_bit_for_bit():
    t = scan_inputs(1, 2000, 96, 16, seed=31)
    y, f = run_scan(t)
    for _ in range(3):
        y2, f2 = run_scan(t)
        assert torch.equal(y, y2) and torch.equal(f, f2)


@gpu
def test_scan_offsets_past_32_bits():
    """Rows so wide that the last tokens lie more than 2^32 bytes and 2^31 elements from the first."""
    L, wide, Dc = 600, 4_000_000, 32
    t = scan_inputs(1, L, Dc, 16, seed=37)
    buf = torch.empty(1, L, wide, dtype=BF16, device="cuda")
    for i, k in enumerate(("x", "dt_raw", "z")):
        buf[..., i * Dc:(i + 1) * Dc] = t[k]
        t[k] = buf[..., i * Dc:(i + 1) * Dc]
    y = buf[..., 3 * Dc:4 * Dc]
    check_scan(t, y=y)


# ---------------------------------------------------------------------------------------------------- convolution

def conv_inputs(b, L, Dc, k, io=BF16, seed=0, state=True, bias=True, lengths=None):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    nseq = len(lengths) if lengths is not None else b
    return (r(b, L, Dc).to(io).cuda(), (r(Dc, k) * k ** -0.5).cuda(), (r(Dc) * 0.1).cuda() if bias else None,
            r(nseq, Dc, k - 1).to(io).cuda() if state else None,
            None if lengths is None else torch.tensor([sum(lengths[:i]) for i in range(nseq + 1)],
                                                      dtype=torch.int32).cuda())


CONV = [
    (1, 1, 1536, 4, {}), (64, 1, 130, 4, {}), (2, 3, 64, 4, {}), (2, 2, 64, 8, {}), (1, 100, 5376, 4, {}),
    (3, 67, 33, 4, dict(io=F32)), (1, 31, 1, 3, dict(io=F16)), (2, 200, 72, 2, dict(io=F16)),
    (2, 40, 64, 1, dict(io=F32)), (1, 129, 40, 8, dict(state=False)), (2, 70, 48, 5, dict(bias=False)),
    (1, 50, 24, 6, {}), (1, 50, 24, 7, dict(io=F32)),
    (1, 76, 40, 4, dict(lengths=[33, 1, 0, 2, 40])), (1, 9, 64, 8, dict(lengths=[1] * 9)),
    (1, 300, 66, 4, dict(lengths=[0, 128, 0, 3, 169, 0], io=F16)), (1, 64, 8, 4, dict(lengths=[64], state=False)),
    (2, 140, 1030, 4, {}), (1, 90, 258, 2, dict(io=F16)), (2, 77, 5, 8, dict(io=F32)), (3, 1, 35, 4, dict(io=F32)),
    (1, 200, 131, 3, dict(lengths=[1, 150, 0, 49], io=F32)), (1, 200, 130, 5, dict(lengths=[64, 64, 72])),
]


@gpu
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("b,L,Dc,k,kw", CONV, ids=[f"conv{i}" for i in range(len(CONV))])
def test_conv_values(b, L, Dc, k, kw, act):
    x, w, bias, state, cu = conv_inputs(b, L, Dc, k, seed=L, **kw)
    out, cache = m.ssd_conv(x, w, bias, state, cu, act)
    ref, cref, err = lo.conv(x, w, bias, state, cu, act)
    ok(out, ref, err, x.dtype)
    assert torch.equal(cache.cpu().double(), cref)


@gpu
@pytest.mark.parametrize("L,lengths", [(1, None), (2, None), (50, None), (50, [1, 0, 49])])
def test_conv_state_in_place(L, lengths):
    x, w, bias, state, cu = conv_inputs(1 if lengths else 3, L, 72, 4, lengths=lengths, seed=2)
    out0, c0 = m.ssd_conv(x, w, bias, state, cu)
    out, c = m.ssd_conv(x, w, bias, state, cu, conv_state_out=state)
    assert c is state and torch.equal(out, out0) and torch.equal(c, c0)


@gpu
@pytest.mark.parametrize("off", [0, 1, 2, 8])
def test_conv_slices_and_strided_output(off):
    x, w, bias, state, _ = conv_inputs(2, 45, 72, 4, seed=4)
    out0, c0 = m.ssd_conv(x, w, bias, state)
    wide = torch.full((2, 45, 120), float("nan"), dtype=BF16, device="cuda")
    wide[..., off:off + 72] = x
    to = torch.full((2, 45, 99), 3.0, dtype=BF16, device="cuda")
    out, c = m.ssd_conv(wide[..., off:off + 72], w, bias, state, out=to[..., off:off + 72])
    assert torch.equal(out, out0) and torch.equal(c, c0)
    assert bool((to[..., :off] == 3).all()) and bool((to[..., off + 72:] == 3).all())


@gpu
def test_conv_prefill_then_tokens():
    x, w, bias, state, _ = conv_inputs(2, 30, 64, 4, seed=6)
    out0, c0 = m.ssd_conv(x, w, bias, state)
    out1, c = m.ssd_conv(x[:, :20], w, bias, state)
    outs = [out1]
    for i in range(20, 30):
        o, c = m.ssd_conv(x[:, i:i + 1], w, bias, c, conv_state_out=c)
        outs.append(o)
    assert torch.equal(c, c0)
    ref, _, err = lo.conv(x, w, bias, state)
    ok(torch.cat(outs, 1), ref, err, BF16)


@gpu
def test_conv_agrees_with_the_convolution_in_front_of_the_ssd():
    from mamba_ssd_prefill_gb300.inputs import WORKLOADS, make_conv_inputs

    w = WORKLOADS["m130-bf16"].with_(batch=2, seqlen=150, nheads=4)
    ci = make_conv_inputs(w, 4, device="cuda", seed=3)
    _, _, cache, rows = m.ssd_fwd_conv(**ci, nheads=4, headdim=64, ngroups=1, dstate=128)
    out, c = m.ssd_conv(ci["xbc"], ci["conv_weight"], ci["conv_bias"], ci["conv_state"])
    # its SiLU goes through the 2^-11 hyperbolic tangent
    assert torch.allclose(out.float(), rows.float(), atol=2e-2, rtol=2 ** -7) and torch.equal(c, cache)


@gpu
def test_conv_empty():
    x, w, bias, state, _ = conv_inputs(2, 0, 64, 4)
    out, c = m.ssd_conv(x, w, bias, state)
    assert out.shape == (2, 0, 64) and torch.equal(c, state)
    out, c = m.ssd_conv(x, w, bias)
    assert not c.any()


@gpu
def test_conv_offsets_past_32_bits():
    x, w, bias, state, _ = conv_inputs(1, 600, 64, 4, seed=8)
    buf = torch.empty(1, 600, 4_000_000, dtype=BF16, device="cuda")
    buf[..., :64] = x
    out, c = m.ssd_conv(buf[..., :64], w, bias, state, out=buf[..., 64:128])
    ref, cref, err = lo.conv(x, w, bias, state)
    ok(out, ref, err, BF16)
    assert torch.equal(c.cpu().double(), cref)


# ----------------------------------------------------------------------------------------------------- group norm

NORM = [
    # rows, channels, groups, io
    (1, 1536, 1, BF16), (7, 1536, 24, BF16), (33, 5120, 8, BF16), (5, 200, 8, F32), (3, 1, 1, F32), (4, 7, 7, F16),
    (9, 130, 2, F16), (2, 8192, 1, F32), (3, 20000, 1, BF16), (2, 1000, 1, F16), (300, 64, 1, BF16), (65, 96, 3, F32),
    (2, 33000, 2, BF16), (700, 1538, 1, BF16), (9, 300, 10, F16), (3, 8190, 1, BF16), (2, 9006, 1, F16), (5, 2, 1, BF16),
]
MODES = [dict(), dict(z=True), dict(z=True, gate_first=True), dict(center=True, activation="none"),
         dict(z=True, center=True), dict(z=True, gate_first=True, center=True), dict(plain=True)]


def norm_inputs(rows, Dc, io, mode, seed):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    kw = {k: v for k, v in mode.items() if k not in ("z", "plain")}
    x = (r(rows, Dc) + 0.5).to(io).cuda()
    if not mode.get("plain"):
        kw.update(weight=(1 + 0.1 * r(Dc)).cuda(), bias=(0.1 * r(Dc)).cuda())
    if mode.get("z"):
        kw["z"] = r(rows, Dc).to(io).cuda()
    return x, kw


@gpu
@pytest.mark.parametrize("mode", MODES, ids=[f"mode{i}" for i in range(len(MODES))])
@pytest.mark.parametrize("rows,Dc,G,io", NORM, ids=[f"norm{i}" for i in range(len(NORM))])
def test_norm_values(rows, Dc, G, io, mode):
    x, kw = norm_inputs(rows, Dc, io, mode, rows + Dc)
    y = m.ssd_group_norm(x, ngroups=G, **kw)
    ref, err = lo.group_norm(x, ngroups=G, **kw)
    ok(y, ref, err, io)


@gpu
@pytest.mark.parametrize("mode", MODES[:4], ids=[f"mode{i}" for i in range(4)])
@pytest.mark.parametrize("rows,Dc,G,io", [(5, 1536, 1, BF16), (33, 5120, 8, BF16), (4, 256, 2, F32), (3, 200, 1, F16),
                                          (2, 1, 1, F32), (6, 20000, 1, BF16), (9, 1001, 1, F32)])
def test_norm_to_e4m3(rows, Dc, G, io, mode):
    """The values that come back are the norm, rounded once to e4m3 under its block's scale."""
    x, kw = norm_inputs(rows, Dc, io, mode, Dc)
    q, scales = m.ssd_group_norm(x, ngroups=G, quantize=True, **kw)
    assert q.dtype is E4M3 and q.shape == x.shape and scales.shape == (rows, -(-Dc // 128))
    ref, err = lo.group_norm(x, ngroups=G, **kw)
    pad = lambda t: torch.nn.functional.pad(t, (0, -Dc % 128)).reshape(rows, -1, 128)  # noqa: E731
    want, most = pad(ref).abs().amax(-1) / 448, pad(err).amax(-1) / 448
    assert bool(((scales.cpu().double() - want).abs() <= most + 4 * lo.U * want).all())
    s = scales.cpu().double().repeat_interleave(128, 1)[:, :Dc]
    v = ref / s
    half = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 4)  # half the spacing of e4m3
    off = (q.float().cpu().double() - v).abs()
    # an e4m3 of a value next to a power of two may have the next spacing up
    assert bool((off <= half * 1.001 + err / s + v.abs() * 8 * lo.U + (v.abs() > 447) * 2).all())


@gpu
def test_norm_in_place_strided_and_leading_dimensions():
    x, kw = norm_inputs(24, 96, BF16, MODES[1], 3)
    y0 = m.ssd_group_norm(x, ngroups=3, **kw)
    assert torch.equal(m.ssd_group_norm(x.reshape(2, 3, 4, 96), ngroups=3, **{**kw, "z": kw["z"].reshape(2, 3, 4, 96)}),
                       y0.reshape(2, 3, 4, 96))
    for off in (0, 1, 8):
        wide = torch.full((24, 240), float("nan"), dtype=BF16, device="cuda")
        wide[:, off:off + 96], wide[:, off + 110:off + 206] = x, kw["z"]
        s = {**kw, "z": wide[:, off + 110:off + 206]}
        to = torch.full((24, 130), 5.0, dtype=BF16, device="cuda")
        y = m.ssd_group_norm(wide[:, off:off + 96], ngroups=3, y=to[:, off:off + 96], **s)
        assert torch.equal(y, y0)
        assert bool((to[:, :off] == 5).all()) and bool((to[:, off + 96:] == 5).all())
    xi = x.clone()
    assert m.ssd_group_norm(xi, ngroups=3, y=xi, **kw) is xi and torch.equal(xi, y0)


@gpu
def test_norm_of_constant_rows_and_nonfinite_ones():
    """A constant row has no variance; a NaN or an infinity stays in its row and group."""
    x = torch.full((3, 64), 2.5, device="cuda")
    y = m.ssd_group_norm(x, center=True, activation="none")
    assert not y.any()
    assert not m.ssd_group_norm(torch.zeros(3, 64, device="cuda"), activation="none").any()
    x, kw = norm_inputs(6, 256, F32, MODES[0], 1)
    y0 = m.ssd_group_norm(x, ngroups=2, **kw)
    x[2, 200] = float("nan")
    y = m.ssd_group_norm(x, ngroups=2, **kw)
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[2, 128:] = True
    assert bool(torch.isnan(y[bad]).all()) and torch.equal(y[~bad], y0[~bad])
    q, s = m.ssd_group_norm(x, ngroups=2, quantize=True, **kw)
    assert bool(torch.isnan(s[2, 1])) and int(torch.isnan(s).sum()) == 1


@gpu
def test_norm_empty():
    assert m.ssd_group_norm(torch.zeros(0, 64, device="cuda")).shape == (0, 64)


# -------------------------------------------------------------------------------------------------------- e4m3

@gpu
@pytest.mark.parametrize("io", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols,br", [(1, 128, 1), (5, 2560, 1), (3, 200, 1), (7, 1, 1), (300, 96, 1), (2, 77, 1),
                                          (128, 128, 128), (300, 200, 128), (1, 16, 128), (129, 640, 128)])
def test_quantize_bits(rows, cols, br, io):
    x = torch.randn(rows, cols, generator=gen(rows + cols)).to(io)
    x[rows // 2, :] = 0
    q, s = m.ssd_fp8_quantize(x.cuda(), br)
    qr, sr = lo.quantize(x, br)
    assert torch.equal(q.cpu().view(torch.uint8) & 0x7f, qr.view(torch.uint8) & 0x7f)
    assert torch.equal(q.cpu().float(), qr.float()) and torch.equal(s.cpu(), sr)


@gpu
def test_quantize_extremes():
    """Magnitudes whose 448 / m overflows, zeros, infinities and NaN."""
    x = torch.randn(6, 256, generator=gen(1))
    x[1] *= 1e-37
    x[2] = 0
    x[3, 5] = float("inf")
    x[4, 200] = float("nan")
    x[5] *= 1e37
    q, s = m.ssd_fp8_quantize(x.cuda())
    qr, sr = lo.quantize(x, 1)
    keep = torch.tensor([0, 1, 2, 5])
    assert torch.equal(q.cpu().float()[keep], qr.float()[keep]) and torch.equal(s.cpu()[keep], sr[keep])
    assert torch.isnan(s.cpu()).tolist() == [[False, False]] * 3 + [[True, False], [False, True], [False, False]]
    assert not torch.isnan(q.float().cpu()[3, 128:]).any()


@gpu
def test_quantize_strided_and_leading_dimensions():
    x = torch.randn(4, 6, 150, generator=gen(2)).to(BF16).cuda()
    q, s = m.ssd_fp8_quantize(x[..., 9:139])
    q2, s2 = m.ssd_fp8_quantize(x[..., 9:139].reshape(24, 130).contiguous())
    assert q.shape == (4, 6, 130) and s.shape == (4, 6, 2)
    assert torch.equal(q.reshape(24, 130).view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s.reshape(24, 2), s2)


MATMUL = [
    # m, n, k, out type, bias
    (1, 128, 128, BF16, False), (1, 10576, 2560, BF16, False), (16, 300, 256, F32, True), (17, 129, 144, F16, False),
    (33, 1000, 16, F32, False), (64, 640, 1280, BF16, True), (65, 257, 400, F16, True), (128, 256, 512, F32, False),
    (129, 513, 2560, BF16, False), (200, 1, 640, F32, True), (300, 2560, 5120, BF16, False), (777, 350, 272, F16, False),
    (1030, 768, 1536, F32, True), (2, 8, 8192, BF16, False), (500, 130, 112, BF16, True),
]


@gpu
@pytest.mark.parametrize("M,N,K,out,bias", MATMUL, ids=[f"mm{i}" for i in range(len(MATMUL))])
def test_matmul_values(M, N, K, out, bias):
    g = gen(M + N + K)
    a, sa = lo.quantize(torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g)), 1)
    b, sb = lo.quantize(torch.randn(N, K, generator=g) * K ** -0.5, 128)
    bv = torch.randn(N, generator=g) if bias else None
    y, err = lo.matmul(a, sa, b, sb, bv)
    ws = m.Workspace("cuda")
    got = m.ssd_fp8_matmul(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), None if bv is None else bv.cuda(),
                           out_dtype=out, workspace=ws)
    m.check(ws)
    ok(got, y, err, out)


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 130, 272), (20, 256, 1024), (130, 300, 2560), (600, 512, 384)])
def test_matmul_of_whole_numbers_is_exact(M, N, K):
    """Small whole numbers under scales that are powers of two: every sum is exact whatever its order."""
    g = gen(M)
    a = torch.randint(-2, 3, (M, K), generator=g).float().to(E4M3)
    b = torch.randint(-2, 3, (N, K), generator=g).float().to(E4M3)
    sa = torch.exp2(torch.randint(-3, 4, (M, -(-K // 128)), generator=g).float())
    sb = torch.exp2(torch.randint(-3, 4, (-(-N // 128), -(-K // 128)), generator=g).float())
    got = m.ssd_fp8_matmul(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=F32)
    assert torch.equal(got.cpu().double(), lo.values(a, sa, 1) @ lo.values(b, sb, 128).t())


@gpu
def test_matmul_strided_output_zero_k_and_empty():
    g = gen(5)
    a, sa = lo.quantize(torch.randn(40, 256, generator=g), 1)
    b, sb = lo.quantize(torch.randn(90, 256, generator=g), 128)
    args = (a.cuda(), sa.cuda(), b.cuda(), sb.cuda())
    want = m.ssd_fp8_matmul(*args)
    to = torch.full((40, 131), 4.0, dtype=BF16, device="cuda")
    out = m.ssd_fp8_matmul(*args, out=to[:, 3:93])
    assert torch.equal(out, want) and bool((to[:, :3] == 4).all()) and bool((to[:, 93:] == 4).all())
    lead = m.ssd_fp8_matmul(args[0].reshape(5, 8, 256), args[1].reshape(5, 8, 2), *args[2:])
    assert torch.equal(lead.reshape(40, 90), want)
    z = m.ssd_fp8_matmul(args[0][:, :0].contiguous(), args[1][:, :0].contiguous(), args[2][:, :0].contiguous(),
                         args[3][:, :0].contiguous(), torch.arange(90.0, device="cuda"))
    assert torch.equal(z.float(), torch.arange(90.0, device="cuda").to(BF16).float().expand(40, 90))
    assert m.ssd_fp8_matmul(args[0][:0], args[1][:0], *args[2:]).shape == (0, 90)


@gpu
def test_matmul_nan_scale_stays_in_its_row():
    g = gen(6)
    x = torch.randn(70, 384, generator=g)
    b, sb = (t.cuda() for t in lo.quantize(torch.randn(200, 384, generator=g), 128))
    q, s = m.ssd_fp8_quantize(x.cuda())
    want = m.ssd_fp8_matmul(q, s, b, sb)
    x[31, 7] = float("inf")
    q, s = m.ssd_fp8_quantize(x.cuda())
    got = m.ssd_fp8_matmul(q, s, b, sb)
    assert bool(torch.isnan(got[31]).all())
    keep = torch.arange(70, device="cuda") != 31
    assert torch.equal(got[keep], want[keep])


@gpu
@pytest.mark.parametrize("M", [3, 150])
def test_matmul_repeats_bit_for_bit(M):
    g = gen(7)
    a, sa = (t.cuda() for t in lo.quantize(torch.randn(M, 5120, generator=g), 1))
    b, sb = (t.cuda() for t in lo.quantize(torch.randn(640, 5120, generator=g), 128))
    first = m.ssd_fp8_matmul(a, sa, b, sb, out_dtype=F32)
    for _ in range(3):
        assert torch.equal(first, m.ssd_fp8_matmul(a, sa, b, sb, out_dtype=F32))


# ------------------------------------------------------------------------------------- streams, graphs, refusals

@gpu
def test_calls_on_another_stream():
    """With stream= the call runs there, behind the work that made its inputs, and its outputs stay its own."""
    t = scan_inputs(1, 300, 64, 16, seed=41)
    y0, f0 = run_scan(t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, f = m.ssd_selective_scan(**t, stream=side)
    o, c = m.ssd_conv(t["x"], torch.ones(64, 4, device="cuda"), stream=side)
    n = m.ssd_group_norm(y, stream=side)
    q, s = m.ssd_fp8_quantize(y, stream=side)
    del o, c
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y0) and torch.equal(f, f0)
    assert torch.equal(n, m.ssd_group_norm(y0)) and torch.equal(q.view(torch.uint8),
                                                                m.ssd_fp8_quantize(y0)[0].view(torch.uint8))


@gpu
@pytest.mark.parametrize("L,Dc", [(1, 256), (3, 2560), (700, 512), (5000, 1536)])
def test_calls_in_a_row_without_waiting(L, Dc):
    """A kernel may start while the one before it still runs: chains through the same buffers, with work of other
    kinds in between, give the same bits as with a wait after every call."""
    t = scan_inputs(2, L, Dc, 16, seed=47)
    w = torch.randn(Dc, 4, generator=gen(3)).cuda()
    wq, ws = m.ssd_fp8_quantize(torch.randn(Dc, Dc, generator=gen(4)).cuda() / Dc ** 0.5, 128)

    def chain(wait):
        x, st, cache = t["x"].clone(), t["init_states"].clone(), torch.zeros(2, Dc, 3, dtype=BF16, device="cuda")
        u, y = torch.empty_like(x), torch.empty_like(x)
        done = torch.cuda.synchronize if wait else (lambda: None)
        for i in range(6):
            m.ssd_conv(x, w, None, cache, out=u, conv_state_out=cache)
            done()
            m.ssd_selective_scan(u, t["dt_raw"], t["dt_bias"], t["A"], t["B"], t["C"], t["D"], t["z"],
                                 init_states=st, final_states=st, y=y)
            done()
            m.ssd_group_norm(y, z=u, y=y)
            done()
            if i % 2:
                x.zero_()
                done()
            q, sc = m.ssd_fp8_quantize(y)
            done()
            m.ssd_fp8_matmul(q, sc, wq, ws, out=x)
            done()
            if i % 3 == 2:
                x += u
                done()
        return x, st, cache

    want = chain(True)
    for _ in range(3):
        for a, b in zip(chain(False), want):
            assert torch.equal(a, b)


@gpu
def test_decode_step_in_a_cuda_graph():
    """conv, scan, norm to e4m3 and projection of one token, captured and replayed on new inputs."""
    Dc, N = 256, 16
    t = scan_inputs(2, 6, Dc, N, seed=43)
    w = torch.randn(Dc, 4, generator=gen(1)).cuda()
    wq, ws = m.ssd_fp8_quantize(torch.randn(96, Dc, generator=gen(2)).cuda(), 128)
    keys = ("x", "dt_raw", "B", "C", "z")

    def step(inp, state, cache):
        u, _ = m.ssd_conv(inp["x"], w, None, cache, conv_state_out=cache)
        y, _ = m.ssd_selective_scan(u, inp["dt_raw"], t["dt_bias"], t["A"], inp["B"], inp["C"], t["D"],
                                    init_states=state, final_states=state)
        return m.ssd_fp8_matmul(*m.ssd_group_norm(y, z=inp["z"], quantize=True), wq, ws)

    def cuts(i):
        return {k: t[k][:, i:i + 1].contiguous() for k in keys}

    st, cache = t["init_states"].clone(), torch.zeros(2, Dc, 3, dtype=BF16, device="cuda")
    want = [step(cuts(i), st, cache).clone() for i in range(6)]
    st2, cache2 = t["init_states"].clone(), torch.zeros_like(cache)
    hold = cuts(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(hold, st2.clone(), cache2.clone())  # workspaces exist before the capture
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(hold, st2, cache2)
    torch.cuda.current_stream().wait_stream(side)
    st2.copy_(t["init_states"])
    cache2.zero_()
    for i in range(6):
        for k in keys:
            hold[k].copy_(t[k][:, i:i + 1])
        graph.replay()
        assert torch.equal(out, want[i])


def scan_problem(**kw):
    d = dict(batch=1, seqlen=64, channels=64, dstate=16, ngroups=1, io=1, state=0, packed=0, softplus=1)
    d.update(kw)
    return struct.pack("@5q4i", *d.values())


@pytest.mark.parametrize("bad,status", [(dict(batch=-1), 1), (dict(seqlen=-1), 1), (dict(channels=0), 1),
                                        (dict(dstate=0), 1), (dict(ngroups=5), 1), (dict(ngroups=0), 1),
                                        (dict(io=3), 1), (dict(state=1), 1), (dict(packed=2), 1),
                                        (dict(softplus=-1), 1), (dict(dstate=257), 2),
                                        (dict(packed=1, seqlen=1 << 31), 1), (dict(batch=1 << 40, seqlen=1 << 30), 1)])
def test_scan_refuses_problems(bad, status):
    n = ctypes.c_size_t(0)
    L = m.lib()
    assert L.ssd_selective_scan_workspace_size(scan_problem(**bad), ctypes.byref(n)) == status
    assert L.ssd_selective_scan(scan_problem(**bad), b"\0" * 192, 256, 1 << 30, None) == status


def test_c_entries_refuse_pointers_and_strides():
    L = m.lib()
    a = 1 << 20
    ptr = dict(x=a, dt=a, z=0, B=a, C=a, y=a, A=a, bias=0, D=0, init=0, fin=0, cu=0)
    stride = dict(xs=0, xt=64, ds=0, dt=64, zs=0, zt=0, bs=0, bt=16, cs=0, ct=16, ys=0, yt=64)

    def scan(problem=None, ws=a, n=1 << 30, **kw):
        v = {**{f"p_{k}": x for k, x in ptr.items()}, **stride, **kw}
        return L.ssd_selective_scan(problem or scan_problem(), struct.pack("@12P12q", *v.values()), ws, n, None)

    for kw in (dict(p_x=0), dict(p_dt=0), dict(p_B=0), dict(p_C=0), dict(p_y=0), dict(p_A=0), dict(p_x=a + 1),
               dict(p_A=a + 2), dict(p_init=a + 2), dict(p_cu=a), dict(xt=-1), dict(bs=-64), dict(yt=63),
               dict(xt=1 << 61)):
        assert scan(**kw) == 1, kw
    assert scan(problem=scan_problem(packed=1)) == 1  # no offsets
    assert scan(problem=scan_problem(batch=2), ys=100) == 1  # the sequences' rows of y overlap
    assert scan(ws=0) == 3 and scan(ws=a + 8) == 3 and scan(n=16) == 3
    conv = lambda p, t, ws=None: L.ssd_conv(struct.pack("@3q4i", *p), struct.pack("@7P4q", *t), ws, None)  # noqa: E731
    good = (a, 2 * a, a, 0, 0, 0, 0, 0, 64, 0, 64)
    for p in ((-1, 8, 64, 4, 1, 1, 0), (1, 8, 0, 4, 1, 1, 0), (1, 8, 64, 0, 1, 1, 0), (1, 8, 64, 9, 1, 1, 0),
              (1, 8, 64, 4, 2, 1, 0), (1, 8, 64, 4, 1, 3, 0), (1, 8, 64, 4, 1, 1, 1)):
        assert conv(p, good) == 1, p
    for i, v in ((0, 0), (1, 0), (1, a), (2, 0), (0, a + 1), (4, a + 1), (6, a), (8, -1), (10, 63)):
        t = list(good)
        t[i] = v
        assert conv((1, 8, 64, 4, 1, 1, 0), t) == 1, (i, v)
    assert conv((1, 8, 64, 4, 1, 1, 0), good, 8) == 3
    norm = lambda p, t: L.ssd_group_norm(struct.pack("@3q4ifi", *p), struct.pack("@6P3q", *t), None, None)  # noqa: E731
    t = (a, 0, a, 0, 0, 0, 64, 0, 64)
    for p in ((-1, 64, 1, 1, 1, 0, 0, 0.0, 0), (4, 64, 3, 1, 1, 0, 0, 0.0, 0), (4, 64, 1, 5, 1, 0, 0, 0.0, 0),
              (4, 64, 1, 1, 2, 0, 0, 0.0, 0), (4, 64, 1, 1, 1, 2, 0, 0.0, 0), (4, 64, 1, 1, 1, 0, 1, 0.0, 0),
              (4, 64, 1, 1, 1, 0, 0, -1.0, 0), (4, 64, 1, 1, 1, 0, 0, float("nan"), 0), (4, 64, 1, 1, 1, 0, 0, 0.0, 1)):
        assert norm(p, t) == 1, p
    assert norm((4, 256, 4, 1, 1, 0, 0, 0.0, 0), (a, 0, a, a, 0, 0, 256, 0, 256)) == 2  # scales across groups
    assert norm((4, 64, 1, 1, 1, 0, 0, 0.0, 0), (a, 0, a, 0, 0, 0, 64, 0, 32)) == 1     # rows of y overlap
    assert L.ssd_fp8_quantize(4, 64, 2, 1, a, 64, a, a, None, None) == 1
    assert L.ssd_fp8_quantize(4, 64, 1, 7, a, 64, a, a, None, None) == 1
    assert L.ssd_fp8_quantize(4, 64, 1, 1, None, 64, a, a, None, None) == 1
    mm = lambda p, *t: L.ssd_fp8_matmul(struct.pack("@3q2i", *p), *t, None)  # noqa: E731
    args = (a, a, a, a, None, a, 64, a, 256)
    assert mm((4, 64, 40, 1, 0), *args) == 2       # rows that are no multiple of 16 bytes
    assert mm((4, 64, 48, 3, 0), *args) == 1 and mm((4, 64, 48, 1, 1), *args) == 1 and mm((-1, 64, 48, 1, 0), *args) == 1
    assert mm((4, 64, 48, 1, 0), a + 8, *args[1:]) == 1 and mm((4, 64, 48, 1, 0), None, *args[1:]) == 1
    assert mm((4, 64, 48, 1, 0), *args[:7], None, 256) == 3 and mm((4, 64, 48, 1, 0), *args[:7], a, 16) == 3
    assert mm((4, 64, 48, 1, 0), *args[:6], 63, a, 256) == 1


def test_python_refuses_cpu_tensors():
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        m.ssd_selective_scan(x, x, None, torch.zeros(8, 2), torch.zeros(1, 4, 1, 2), torch.zeros(1, 4, 1, 2))
    with pytest.raises(ValueError, match="CUDA"):
        m.ssd_conv(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        m.ssd_group_norm(x)
    with pytest.raises(ValueError, match="CUDA"):
        m.ssd_fp8_quantize(x)
    with pytest.raises(ValueError, match="CUDA"):
        m.ssd_fp8_matmul(x.to(E4M3), torch.zeros(1, 4, 1), x[0].to(E4M3), torch.zeros(1, 1))


@gpu
def test_python_refuses_wrong_shapes_and_types():
    t = scan_inputs(2, 8, 64, 16)
    for k, v in (("dt_raw", t["dt_raw"][:, :7]), ("A", t["A"][:, :8]), ("A", t["A"].t().contiguous().t()),
                 ("B", t["B"].float()), ("C", t["C"].cpu()), ("D", t["D"].half()), ("z", t["z"][..., :32]),
                 ("init_states", t["init_states"].half()), ("x", t["x"].transpose(1, 2).contiguous().transpose(1, 2)),
                 ("cu_seqlens", torch.zeros(3, dtype=torch.int32, device="cuda")), ("x", t["x"].double())):
        with pytest.raises(ValueError):
            m.ssd_selective_scan(**{**t, k: v}, state_dtype=F32)
    with pytest.raises(ValueError):
        m.ssd_selective_scan(**t, state_dtype=BF16)
    x = t["x"]
    for bad in (dict(conv_weight=torch.ones(64, 9, device="cuda")), dict(conv_weight=torch.ones(63, 4, device="cuda")),
                dict(conv_weight=torch.ones(64, 4, device="cuda"), activation="relu"),
                dict(conv_weight=torch.ones(64, 4, device="cuda"), conv_state=torch.ones(2, 64, 2, device="cuda"))):
        with pytest.raises(ValueError):
            m.ssd_conv(x, **bad)
    for bad in (dict(ngroups=3), dict(gate_first=True), dict(z=x[..., :8]), dict(weight=torch.ones(63, device="cuda")),
                dict(activation="tanh"), dict(y=x.float())):
        with pytest.raises(ValueError):
            m.ssd_group_norm(x, **bad)
    with pytest.raises(m.SsdError) as e:
        m.ssd_group_norm(x, ngroups=2, quantize=True)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        m.ssd_fp8_quantize(x, 64)
    with pytest.raises(ValueError):
        m.ssd_fp8_quantize(x, 128)
    q, s = m.ssd_fp8_quantize(x.reshape(16, 64))
    for bad in ((q.float(), s, q, s[:1]), (q, s.double(), q, s[:1]), (q, s[:3], q, s[:1]), (q, s, q[:, :32], s[:1])):
        with pytest.raises(ValueError):
            m.ssd_fp8_matmul(*bad)


@gpu
def test_bounds_checked_build_reports_no_violation():
    import subprocess
    import sys

    from mamba_ssd_prefill_gb300 import _build

    path = _build.build(checked=True)
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, os.path.join(here, "layer_bounds_cases.py")], capture_output=True, text=True,
                       env={**os.environ, "MAMBA_SSD_LIB": path}, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [ln.split() for ln in r.stdout.splitlines()]
    assert len(lines) > 60 and all(ln[-1] == "0" for ln in lines), r.stdout


@gpu
@pytest.mark.parametrize("kw", [dict(), dict(batch=1, prompt=37, tokens=5, model=64, inner=256, groups=2)],
                         ids=["layer", "odd"])
def test_example_layer_prompt_then_tokens(kw):
    """The example's layer, prompt then tokens, against one long prompt. The library product behind B, C and the steps
    sums in another order for other row counts, so y differs by roundings of bf16 (2^-8 of it), and with a probability
    of 2^-8 over the spacing of e4m3 (2^-4 .. 2^-3 of a value) a value rounds to its neighbour: a row's relative
    2-norm of about sqrt(2^-4) 2^-4 = 2^-6, and below 2^-4, the spacing itself."""
    import importlib.util

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixer_layer.py")
    spec = importlib.util.spec_from_file_location("mixer_layer", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    assert ex.run(**kw) < 2.0 ** -4
