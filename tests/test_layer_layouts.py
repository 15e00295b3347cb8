"""Layouts of the operators around the SSD: leading dimensions and strides that are read and written where they lie, or
refused, and offsets without sequences. The elements around a slice hold NaN where it is read and a guard value where it is written."""
import ctypes
import struct

import pytest
import torch

import mamba_ssd_prefill_gb300 as m
from test_layer_ops import conv_inputs, run_scan, scan_inputs

gpu = pytest.mark.gpu
BF16 = torch.bfloat16
GUARD = 7.0


def cut(base, how):
    return {"heads": lambda t: t[:, :, 2:4], "half": lambda t: t[:, :, 0], "step": lambda t: t[:, :, ::16],
            "last": lambda t: t[:, -1:, 8:104], "one": lambda t: t[:, :, 5:6], "row": lambda t: t[:1, -1:, :96]}[how](base)


def filled(shape, how, dtype=BF16):
    """A tensor of `shape` with values in its slice and NaN around it, and the slice."""
    base = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    view = cut(base, how)
    view.copy_(torch.randn(view.shape, generator=torch.Generator("cpu").manual_seed(len(how))))
    return base, view


# rows at one distance although a dimension of size 1 has another stride: the last token of each prompt, one head of
# one token a sequence, a step longer than its axis, one row
EVEN = [((5, 7, 200), "last"), ((4, 1, 8, 64), "one"), ((4, 1, 8, 64), "step"), ((3, 4, 150), "row")]
# rows at two distances: some heads of one token a sequence, one half of two; of several tokens
UNEVEN = [((4, 1, 8, 64), "heads"), ((4, 1, 2, 8, 64), "half"), ((2, 3, 8, 64), "heads")]


@gpu
@pytest.mark.parametrize("shape,how", EVEN, ids=[h for _, h in EVEN])
def test_rows_of_one_distance_are_read_and_written_where_they_lie(shape, how):
    _, x = filled(shape, how)
    _, z = filled(shape, how)
    xc, zc = x.contiguous(), z.contiguous()
    want = m.ssd_group_norm(xc, z=zc)
    assert bool(torch.isfinite(want).all())
    assert torch.equal(m.ssd_group_norm(x, z=z), want)
    to = torch.full(shape, GUARD, dtype=BF16, device="cuda")
    y = m.ssd_group_norm(x, z=z, y=cut(to, how))
    assert torch.equal(y, want)
    y.fill_(GUARD)
    assert bool((to == GUARD).all())
    q, s = m.ssd_fp8_quantize(x)
    qc, sc = m.ssd_fp8_quantize(xc)
    assert torch.equal(q.view(torch.uint8), qc.view(torch.uint8)) and torch.equal(s, sc)
    w, ws = m.ssd_fp8_quantize(torch.randn(x.shape[-1], x.shape[-1], generator=torch.Generator("cpu").manual_seed(1)).cuda(), 128)
    want = m.ssd_fp8_matmul(qc, sc, w, ws)
    out = m.ssd_fp8_matmul(qc, sc, w, ws, out=cut(to, how))
    assert torch.equal(out, want)
    out.fill_(GUARD)
    assert bool((to == GUARD).all())


@gpu
@pytest.mark.parametrize("shape,how", UNEVEN, ids=[f"{h}{len(s)}-{s[1]}" for s, h in UNEVEN])
def test_rows_of_two_distances_are_refused(shape, how):
    _, x = filled(shape, how)
    xc = x.contiguous()
    to = torch.full(shape, GUARD, dtype=BF16, device="cuda")
    q, s = m.ssd_fp8_quantize(xc)
    w, ws = m.ssd_fp8_quantize(torch.ones(64, 64, device="cuda"), 128)
    for call in (lambda: m.ssd_group_norm(x), lambda: m.ssd_group_norm(xc, z=x),
                 lambda: m.ssd_group_norm(xc, y=cut(to, how)), lambda: m.ssd_fp8_quantize(x),
                 lambda: m.ssd_fp8_matmul(q, s, w, ws, out=cut(to, how))):
        with pytest.raises(ValueError, match="evenly spaced"):
            call()
    assert bool((to == GUARD).all())


@gpu
def test_rows_at_distance_zero():
    x = torch.randn(1, 1, 1, 64, generator=torch.Generator("cpu").manual_seed(3)).to(BF16).cuda()
    for shape in ((2, 6, 1, 64), (2, 1, 6, 64)):
        assert torch.equal(m.ssd_group_norm(x.expand(shape)), m.ssd_group_norm(x).expand(shape))


def test_tokens_of_no_sequence_are_refused():
    L = m.lib()
    n = ctypes.c_size_t(0)
    a = 1 << 20
    scan = lambda seqlen: struct.pack("@5q4i", 0, seqlen, 64, 16, 1, 1, 0, 1, 1)  # noqa: E731
    assert L.ssd_selective_scan_workspace_size(scan(0), ctypes.byref(n)) == 0
    assert L.ssd_selective_scan_workspace_size(scan(5), ctypes.byref(n)) == 1
    tensors = struct.pack("@12P12q", a, a, 0, a, a, a, a, 0, 0, 0, 0, a, 0, 64, 0, 64, 0, 0, 0, 16, 0, 16, 0, 64)
    assert L.ssd_selective_scan(scan(5), tensors, a, 1 << 30, None) == 1
    assert L.ssd_selective_scan(scan(0), tensors, a, 1 << 30, None) == 0
    conv = lambda seqlen: struct.pack("@3q4i", 0, seqlen, 64, 4, 1, 1, 1)  # noqa: E731
    tensors = struct.pack("@7P4q", a, 2 * a, a, 0, 0, 0, a, 0, 64, 0, 64)
    assert L.ssd_conv(conv(5), tensors, None, None) == 1
    assert L.ssd_conv(conv(0), tensors, None, None) == 0


@gpu
def test_offsets_of_no_sequences():
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    w, A = torch.ones(64, 4, device="cuda"), -torch.ones(64, 16, device="cuda")
    for L in (0, 5):
        x, B = torch.ones(1, L, 64, device="cuda"), torch.ones(1, L, 1, 16, device="cuda")
        if L:
            with pytest.raises(ValueError, match="cu_seqlens"):
                m.ssd_selective_scan(x, x, None, A, B, B, cu_seqlens=cu)
            with pytest.raises(ValueError, match="cu_seqlens"):
                m.ssd_conv(x, w, cu_seqlens=cu)
        else:
            y, f = m.ssd_selective_scan(x, x, None, A, B, B, cu_seqlens=cu)
            o, c = m.ssd_conv(x, w, cu_seqlens=cu)
            assert y.shape == o.shape == x.shape and f.shape == (0, 64, 16) and c.shape == (0, 64, 3)


def test_outputs_may_be_token_major_and_must_not_overlap():
    """y [3, 5, 64]: a sequence's rows together, a token's rows together, with gaps; and rows that overlap. What passes the
    checks of the arguments stops here for want of a GPU, or of memory at these addresses: only the checks are asked."""
    L = m.lib()
    if torch.cuda.is_available():
        pytest.skip("addresses that are not the GPU's")
    a = 1 << 20
    problem = struct.pack("@5q4i", 3, 5, 64, 16, 1, 1, 0, 0, 1)
    conv = struct.pack("@3q4i", 3, 5, 64, 4, 1, 1, 0)

    def refused(seq, tok):
        scan = L.ssd_selective_scan(problem, struct.pack("@12P12q", a, a, 0, a, a, a, a, 0, 0, 0, 0, 0, 0, 64, 0, 64, 0, 0,
                                                         0, 16, 0, 16, seq, tok), a, 1 << 30, None)
        assert (scan == 1) == (L.ssd_conv(conv, struct.pack("@7P4q", a, 2 * a, a, 0, 0, 0, 0, 0, 64, seq, tok), None,
                                          None) == 1)
        return scan == 1

    for seq, tok in ((320, 64), (400, 70), (64, 192), (70, 300)):
        assert not refused(seq, tok), (seq, tok)
    for seq, tok in ((319, 64), (320, 63), (64, 191), (63, 192), (0, 64), (64, 64), (100, 150), (64, 0)):
        assert refused(seq, tok), (seq, tok)


@gpu
@pytest.mark.parametrize("L", [1, 2, 75, 900])
def test_token_major_tensors(L):
    """[L, b, ..] tensors, seen as [b, L, ..]: read and written where they lie."""
    t = scan_inputs(3, L, 72, 16, seed=5)
    want = run_scan(t)
    tm = lambda v: v.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    s = {k: tm(v) if k in ("x", "dt_raw", "B", "C", "z") else v for k, v in t.items()}
    to = torch.full((L, 3, 90), GUARD, dtype=BF16, device="cuda")
    y, f = run_scan(s, y=to.transpose(0, 1)[..., 8:80])
    assert torch.equal(y, want[0]) and torch.equal(f, want[1])
    y.fill_(GUARD)
    assert bool((to == GUARD).all())
    x, w, bias, state, _ = conv_inputs(3, L, 72, 4, seed=6)
    want = m.ssd_conv(x, w, bias, state)
    out, c = m.ssd_conv(tm(x), w, bias, state, out=to.transpose(0, 1)[..., 8:80])
    assert torch.equal(out, want[0]) and torch.equal(c, want[1])
    out.fill_(GUARD)
    assert bool((to == GUARD).all())


@gpu
def test_a_product_of_rows_without_elements():
    """K = 0: the scales of no blocks, by rows and by blocks of rows, as the product takes them."""
    for M, N in ((40, 90), (3, 200), (1, 1)):
        a, b = m.ssd_fp8_quantize(torch.zeros(M, 0, device="cuda")), m.ssd_fp8_quantize(torch.zeros(N, 0, device="cuda"), 128)
        assert a[1].shape == (M, 0) and b[1].shape == (-(-N // 128), 0)
        bias = torch.arange(float(N), device="cuda")
        assert torch.equal(m.ssd_fp8_matmul(*a, *b, bias, out_dtype=torch.float32), bias.expand(M, N))


@gpu
def test_bounds_checked_build_reports_no_violation_in_these_layouts():
    import os
    import subprocess
    import sys

    from mamba_ssd_prefill_gb300 import _build

    path = _build.build(checked=True)
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, os.path.join(here, "layer_bounds_layouts.py")], capture_output=True, text=True,
                       env={**os.environ, "MAMBA_SSD_LIB": path}, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [ln.split() for ln in r.stdout.splitlines()]
    at = lines.index(["--", "0"])  # the other list's cases come first
    bad = [ln for ln in lines if ln[-1] != "0"]
    assert len(lines) - at > 200 and not bad, bad


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [4001, 4002, 3996, 4000])
def test_products_into_wider_rows_leave_what_lies_behind(dtype, N):
    """Many rows (the kernel of 128 x 256 tiles), N columns of rows on 16-byte boundaries, whole 16-byte pieces or not."""
    g = torch.Generator("cpu").manual_seed(N)
    a = m.ssd_fp8_quantize(torch.randn(1300, 640, generator=g).cuda())
    b = m.ssd_fp8_quantize(torch.randn(N, 640, generator=g).cuda(), 128)
    want = m.ssd_fp8_matmul(*a, *b, out_dtype=dtype)
    for off, wide in ((0, 4016), (8, 4024), (16, 4032)):
        to = torch.full((1300, wide), GUARD, dtype=dtype, device="cuda")
        out = m.ssd_fp8_matmul(*a, *b, out_dtype=dtype, out=to[:, off:off + N])
        assert torch.equal(out, want)
        out.fill_(GUARD)
        assert bool((to == GUARD).all())
