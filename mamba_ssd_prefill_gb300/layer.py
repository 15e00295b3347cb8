"""The operators around the SSD in a state-space layer, over the C ABI in ``include/ssd.h``: the selective scan, its
causal depthwise convolution, the gated group norm, and the projections in e4m3 with a scale per block of 128.

Like the rest of the binding, these functions check shapes and types, allocate outputs with PyTorch and pass raw
pointers; the computation runs in the library's kernels. Token tensors may be column slices of wider rows (the last
dimension contiguous, any other stride). `stream` (default: the current one) is the stream the kernels run on; with
another than the current stream the outputs are allocated for it, and the inputs are kept until its work is done.
"""
from __future__ import annotations

import ctypes
import struct

import torch

import mamba_ssd_prefill_gb300 as _m

_F32, _I32 = torch.float32, torch.int32
_IO = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_STATE = {torch.float32: 0, torch.float16: 2}
_ACT = {"none": 0, "silu": 1}
E4M3 = torch.float8_e4m3fn

# the C structs of include/ssd.h, in native layout
_SCAN_PROBLEM = struct.Struct("@5q4i").pack
_SCAN_TENSORS = struct.Struct("@12P12q").pack
_CONV_PROBLEM = struct.Struct("@3q4i").pack
_CONV_TENSORS = struct.Struct("@7P4q").pack
_NORM_PROBLEM = struct.Struct("@3q4ifi").pack
_NORM_TENSORS = struct.Struct("@6P3q").pack
_MATMUL_PROBLEM = struct.Struct("@3q2i").pack


_empty = torch.empty
_workspaces: dict = {}  # (use, device, stream) -> (tensor, address, bytes)


def _raw_stream(index):
    """Address of the device's current stream (0: the default one)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _enter(dev, stream, workspace, use, nbytes=256):
    """(stream address, stream if it is not the current one, workspace address, its bytes, the tensor behind it)."""
    index = dev.index
    raw, side = _raw_stream(index), None
    if stream is not None and stream.cuda_stream != raw:
        raw, side = stream.cuda_stream, stream
    if workspace is None:
        key = (use, index, raw)
        have = _workspaces.get(key)
        if have is None or have[2] < nbytes:
            buf = _on(side, lambda: torch.zeros(nbytes, dtype=torch.uint8, device=dev))
            have = _workspaces[key] = (buf, buf.data_ptr(), nbytes)
        return raw, side, have[1], have[2], have[0]
    if isinstance(workspace, _m.Workspace):
        workspace = _on(side, lambda: workspace.get(nbytes))
    return raw, side, workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _on(side, make):
    """make() with stream `side` current (None: as it is), so that what it allocates belongs to that stream."""
    if side is None:
        return make()
    with torch.cuda.stream(side):
        return make()


def _new(side, shape, dtype, dev):
    if side is None:
        return _empty(shape, dtype=dtype, device=dev)
    return _on(side, lambda: _empty(shape, dtype=dtype, device=dev))


def _call(what, fn, dev, *args):
    """fn(*args) on the tensors' device; raises SsdError."""
    if torch._C._cuda_getDevice() != dev.index:
        with torch.cuda.device(dev):
            st = fn(*args)
    else:
        st = fn(*args)
    if st:
        raise _m.SsdError(st, what)


def _keep(side, *used):
    """Memory of other streams is not reused before the work on stream `side` is done with it."""
    for t in used:
        if t is not None:
            t.record_stream(side)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _device(what, t):
    if not t.is_cuda:
        raise ValueError(f"{what} runs on CUDA tensors only (there is no CPU path)")
    return t.device


def _check(name, t, shape, dtype, dev):
    """t has this shape, type and device and contiguous rows (the last dimension)."""
    if t.shape != shape or t.dtype is not dtype or t.device != dev or (t.stride(-1) != 1 and shape[-1] > 1):
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {dev} with a contiguous last dimension, got "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _flat(name, t, shape, dtype, dev):
    """t has this shape, type and device and is contiguous."""
    if t is None:
        return
    if t.shape != shape or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")


def _sequences(what, x, cu_seqlens):
    """(batch, nseq, device) of a regular batch or of packed sequences."""
    if x.dim() != 3:
        raise ValueError("x: expected [batch, seqlen, channels] (packed: [1, T, channels])")
    dev = _device(what, x)
    if cu_seqlens is None:
        return x.shape[0], dev
    if x.shape[0] != 1:
        raise ValueError("x: expected [1, T, channels] with cu_seqlens (sequences packed along T)")
    if cu_seqlens.dtype is not _I32 or cu_seqlens.device != dev or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 \
            or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens: expected a contiguous int32 [nseq + 1] tensor on the device of x")
    return cu_seqlens.numel() - 1, dev


def ssd_selective_scan(x, dt_raw, dt_bias, A, B, C, D=None, z=None, init_states=None, cu_seqlens=None,
                       state_dtype=None, *, softplus=True, y=None, final_states=None, return_final_states=True,
                       workspace=None, stream=None):
    """Selective scan of a state-space layer, for prompts and (seqlen 1) for single tokens.

    x, dt_raw and the optional gate z [b, L, Dc], B and C [b, L, G, N] in one I/O dtype (fp32, bf16, fp16); A [Dc, N],
    dt_bias and D [Dc] fp32 (both optional); init_states [b, Dc, N] in the state dtype (fp32 or fp16). With
    dt = softplus(dt_raw + dt_bias): h = exp(dt A) h + dt x B, y = (h . C + D x) z sigmoid(z), in fp32. cu_seqlens
    (int32 [nseq + 1], on the GPU) packs nseq sequences on the token axis of [1, T, ...] tensors; the states are then
    [nseq, Dc, N]. final_states may be init_states itself (a cache advanced in place). Returns (y, final_states or
    None). Malformed offsets are reported by check() on the workspace."""
    nseq, dev = _sequences("ssd_selective_scan", x, cu_seqlens)
    shape, io = x.shape, x.dtype
    b, L, Dc = shape
    if B.dim() != 4:
        raise ValueError("B: expected [batch, seqlen, ngroups, dstate]")
    G, N = B.shape[2:]
    if state_dtype is None:
        state_dtype = init_states.dtype if init_states is not None else _F32
    if io not in _IO:
        raise ValueError(f"x: unsupported dtype {io}")
    if state_dtype not in _STATE:
        raise ValueError(f"state_dtype: expected fp32 or fp16, got {state_dtype}")
    if Dc < 1 or N < 1 or G < 1 or Dc % G:
        raise ValueError(f"channels {Dc} must be a positive multiple of the {G} groups, with at least one state")
    xs, ds, bs, cs = x.stride(), dt_raw.stride(), B.stride(), C.stride()
    if (dt_raw.shape != shape or dt_raw.dtype is not io or dt_raw.device != dev or xs[2] != 1 or ds[2] != 1
            or B.shape[:2] != shape[:2] or B.dtype is not io or B.device != dev or bs[3] != 1
            or C.shape != B.shape or C.dtype is not io or C.device != dev or cs[3] != 1
            or (G > 1 and (bs[2] != N or cs[2] != N))
            or A.shape != (Dc, N) or A.dtype is not _F32 or A.device != dev or not A.is_contiguous()):
        _check("x", x, shape, io, dev)
        _check("dt_raw", dt_raw, shape, io, dev)
        for name, t in (("B", B), ("C", C)):
            _check(name, t, (b, L, G, N), io, dev)
            if G > 1 and t.stride(2) != N:
                raise ValueError(f"{name}: a token's [ngroups, dstate] must be contiguous")
        _flat("A", A, (Dc, N), _F32, dev)
    for name, t in (("dt_bias", dt_bias), ("D", D)):
        if t is not None and (t.shape != (Dc,) or t.dtype is not _F32 or t.device != dev or not t.is_contiguous()):
            _flat(name, t, (Dc,), _F32, dev)
    zs = (0, 0)
    if z is not None:
        zs = z.stride()
        if z.shape != shape or z.dtype is not io or z.device != dev or zs[2] != 1:
            _check("z", z, shape, io, dev)
    _flat("init_states", init_states, (nseq, Dc, N), state_dtype, dev)
    _flat("final_states", final_states, (nseq, Dc, N), state_dtype, dev)
    lib = _m.lib()
    prob = _SCAN_PROBLEM(nseq, L, Dc, N, G, _IO[io], _STATE[state_dtype], cu_seqlens is not None, bool(softplus))
    nbytes = 256
    if L != 1:  # a single token needs the header only
        n = ctypes.c_size_t(0)
        st = lib.ssd_selective_scan_workspace_size(prob, ctypes.byref(n))
        if st:
            raise _m.SsdError(st, "ssd_selective_scan")
        nbytes = n.value
    raw, side, ws, ws_bytes, ws_buf = _enter(dev, stream, workspace, "scan", nbytes)
    if y is None:
        y = _new(side, shape, io, dev)
    else:
        _check("y", y, shape, io, dev)
    if final_states is None and return_final_states:
        final_states = _new(side, (nseq, Dc, N), state_dtype, dev)
    ys = y.stride()
    tensors = _SCAN_TENSORS(x.data_ptr(), dt_raw.data_ptr(), _ptr(z), B.data_ptr(), C.data_ptr(), y.data_ptr(),
                            A.data_ptr(), _ptr(dt_bias), _ptr(D), _ptr(init_states), _ptr(final_states),
                            _ptr(cu_seqlens), xs[0], xs[1], ds[0], ds[1], zs[0], zs[1], bs[0], bs[1], cs[0], cs[1],
                            ys[0], ys[1])
    _call("ssd_selective_scan", lib.ssd_selective_scan, dev, prob, tensors, ws, ws_bytes, raw)
    if side is not None:
        _keep(side, x, dt_raw, dt_bias, A, B, C, D, z, init_states, cu_seqlens, y, final_states, ws_buf)
    return y, final_states


def ssd_conv(x, conv_weight, conv_bias=None, conv_state=None, cu_seqlens=None, activation="silu", *, out=None,
             conv_state_out=None, return_conv_state=True, workspace=None, stream=None):
    """Causal depthwise convolution over the tokens (ssd_fwd_conv has it in front of the SSD), for prompts and
    (seqlen 1) for single tokens.

    x [b, L, Dc]; conv_weight [Dc, k] (k 1 .. 8, the last tap on the current token) and conv_bias [Dc] fp32;
    conv_state [b, Dc, k-1] in the dtype of x holds the inputs before each sequence (None: zeros). cu_seqlens packs
    sequences as in ssd_selective_scan. Returns (out, conv_state_out or None): the last k-1 inputs, to continue each
    sequence; conv_state_out may be conv_state itself."""
    nseq, dev = _sequences("ssd_conv", x, cu_seqlens)
    b, L, Dc = x.shape
    io = x.dtype
    if io not in _IO:
        raise ValueError(f"x: unsupported dtype {io}")
    if activation not in _ACT:
        raise ValueError(f"activation: expected one of {sorted(_ACT)}, got {activation!r}")
    if conv_weight.dim() != 2 or not 1 <= conv_weight.shape[1] <= 8:
        raise ValueError("conv_weight: expected [channels, k] with k from 1 to 8")
    k = conv_weight.shape[1]
    shape = (b, L, Dc)
    _check("x", x, shape, io, dev)
    _flat("conv_weight", conv_weight, (Dc, k), _F32, dev)
    _flat("conv_bias", conv_bias, (Dc,), _F32, dev)
    _flat("conv_state", conv_state, (nseq, Dc, k - 1), io, dev)
    _flat("conv_state_out", conv_state_out, (nseq, Dc, k - 1), io, dev)
    raw, side, ws, _, ws_buf = _enter(dev, stream, workspace, "conv")
    if out is None:
        out = _new(side, shape, io, dev)
    else:
        _check("out", out, shape, io, dev)
    if conv_state_out is None and return_conv_state:
        conv_state_out = _new(side, (nseq, Dc, k - 1), io, dev)
    xs, os = x.stride(), out.stride()
    prob = _CONV_PROBLEM(nseq, L, Dc, k, _ACT[activation], _IO[io], cu_seqlens is not None)
    tensors = _CONV_TENSORS(x.data_ptr(), out.data_ptr(), conv_weight.data_ptr(), _ptr(conv_bias), _ptr(conv_state),
                            _ptr(conv_state_out), _ptr(cu_seqlens), xs[0], xs[1], os[0], os[1])
    _call("ssd_conv", _m.lib().ssd_conv, dev, prob, tensors, ws, raw)
    if side is not None:
        _keep(side, x, conv_weight, conv_bias, conv_state, cu_seqlens, out, conv_state_out, ws_buf)
    return out, conv_state_out


def _rows(name, t, dtype, dev, shape):
    """t [..., channels] as evenly spaced rows: the row stride."""
    if t.shape == shape and t.dtype is dtype and t.device == dev and t.is_contiguous():
        return shape[-1]
    _check(name, t, shape, dtype, dev)
    if t.dim() == 1 or t.is_contiguous():
        return shape[-1]
    lead, st = shape[:-1], t.stride()
    for i in range(len(lead) - 1):  # leading dimensions collapse into one
        if lead[i] > 1 and st[i] != st[i + 1] * lead[i + 1]:
            raise ValueError(f"{name}: rows must be evenly spaced, got strides {st} for shape {tuple(shape)}")
    return st[len(lead) - 1]


def ssd_group_norm(x, weight=None, bias=None, z=None, ngroups=1, eps=1e-5, *, center=False, activation="silu",
                   gate_first=False, quantize=False, y=None, workspace=None, stream=None):
    """Group norm with an activation, channels last: every token of x [..., Dc] is normalised by itself, its channels
    in `ngroups` groups, with (center) or without the mean taken away, in fp32.

    Without z: act(norm(x) weight + bias). With a gate z of the shape of x: (norm(x) weight + bias) act(z), or with
    gate_first norm(x act(z)) weight + bias. Returns y in the dtype of x (y= may be x itself); with quantize the pair
    (e4m3 values, fp32 scales [..., ceil(Dc / 128)]) that ssd_fp8_matmul takes, rounded once from fp32 (the groups
    must then be multiples of 128 channels, or one)."""
    dev = _device("ssd_group_norm", x)
    io, shape = x.dtype, x.shape
    if io not in _IO:
        raise ValueError(f"x: unsupported dtype {io}")
    if activation not in _ACT:
        raise ValueError(f"activation: expected one of {sorted(_ACT)}, got {activation!r}")
    if x.dim() < 1 or shape[-1] < 1 or ngroups < 1 or shape[-1] % ngroups:
        raise ValueError(f"x: the channels of {tuple(shape)} must be a positive multiple of the {ngroups} groups")
    if gate_first and z is None:
        raise ValueError("gate_first needs a gate z")
    Dc = shape[-1]
    x_row = _rows("x", x, io, dev, shape)
    z_row = _rows("z", z, io, dev, shape) if z is not None else 0
    _flat("weight", weight, (Dc,), _F32, dev)
    _flat("bias", bias, (Dc,), _F32, dev)
    raw, side, ws, _, ws_buf = _enter(dev, stream, workspace, "norm")
    scales = None
    if y is None:
        y = _new(side, shape, E4M3 if quantize else io, dev)
        y_row = Dc
    else:
        y_row = _rows("y", y, E4M3 if quantize else io, dev, shape)
    if quantize:
        scales = _new(side, (*shape[:-1], -(-Dc // 128)), _F32, dev)
    prob = _NORM_PROBLEM(x.numel() // Dc, Dc, ngroups, _IO[io], _ACT[activation], bool(center), bool(gate_first),
                         eps, 0)
    tensors = _NORM_TENSORS(x.data_ptr(), _ptr(z), y.data_ptr(), _ptr(scales), _ptr(weight), _ptr(bias), x_row,
                            z_row, y_row)
    _call("ssd_group_norm", _m.lib().ssd_group_norm, dev, prob, tensors, ws, raw)
    if side is not None:
        _keep(side, x, z, weight, bias, y, scales, ws_buf)
    return (y, scales) if quantize else y


def ssd_fp8_quantize(x, block_rows=1, *, workspace=None, stream=None):
    """e4m3 values and their fp32 scales: one scale per row and 128 columns of x [..., K] (block_rows 1, activations),
    or per 128 x 128 block of a matrix x [N, K] (block_rows 128, weights). With m a block's largest magnitude the
    scale is m / 448 and the values x * (448 / m), rounded to nearest even; a block that holds an infinity or a NaN
    gets the scale NaN. Returns (q, scales), contiguous."""
    dev = _device("ssd_fp8_quantize", x)
    io, shape = x.dtype, x.shape
    if io not in _IO:
        raise ValueError(f"x: unsupported dtype {io}")
    if block_rows not in (1, 128):
        raise ValueError("block_rows: expected 1 or 128")
    if x.dim() < 1 or (block_rows == 128 and x.dim() != 2):
        raise ValueError("x: expected [..., K], or a matrix [N, K] with block_rows=128")
    K = shape[-1]
    x_row = _rows("x", x, io, dev, shape)
    rows = x.numel() // K if K else 0
    raw, side, ws, _, ws_buf = _enter(dev, stream, workspace, "fp8")
    q = _new(side, shape, E4M3, dev)
    kb = -(-K // 128)
    scales = _new(side, (*shape[:-1], kb) if block_rows == 1 else (-(-rows // 128), kb), _F32, dev)
    _call("ssd_fp8_quantize", _m.lib().ssd_fp8_quantize, dev, rows, K, block_rows, _IO[io], x.data_ptr(), x_row,
          q.data_ptr(), scales.data_ptr(), ws, raw)
    if side is not None:
        _keep(side, x, q, scales, ws_buf)
    return q, scales


def ssd_fp8_matmul(a, a_scales, b, b_scales, bias=None, *, out_dtype=torch.bfloat16, out=None, workspace=None,
                   stream=None):
    """a [..., K] times the transpose of the weights b [N, K], both in e4m3 with block scales (a_scales
    [..., ceil(K / 128)], b_scales [ceil(N / 128), ceil(K / 128)], as ssd_fp8_quantize and ssd_group_norm give them),
    accumulated in fp32, plus bias [N] (fp32, optional), in out_dtype (fp32, bf16 or fp16). K is a multiple of 16.
    Returns [..., N]; out= may have rows wider than N."""
    dev = _device("ssd_fp8_matmul", a)
    if a.dim() < 1 or b.dim() != 2 or a.shape[-1] != b.shape[1]:
        raise ValueError(f"expected a [..., K] and b [N, K], got {tuple(a.shape)} and {tuple(b.shape)}")
    if out_dtype not in _IO:
        raise ValueError(f"out_dtype: unsupported dtype {out_dtype}")
    N, K = b.shape
    lead = a.shape[:-1]
    kb = -(-K // 128)
    _flat("a", a, a.shape, E4M3, dev)
    _flat("b", b, b.shape, E4M3, dev)
    _flat("a_scales", a_scales, (*lead, kb), _F32, dev)
    _flat("b_scales", b_scales, (-(-N // 128), kb), _F32, dev)
    _flat("bias", bias, (N,), _F32, dev)
    M = lead.numel()
    raw, side, ws, ws_bytes, ws_buf = _enter(dev, stream, workspace, "fp8")
    if out is None:
        out = _new(side, (*lead, N), out_dtype, dev)
        out_row = N
    else:
        out_row = _rows("out", out, out_dtype, dev, (*lead, N))
    _call("ssd_fp8_matmul", _m.lib().ssd_fp8_matmul, dev, _MATMUL_PROBLEM(M, N, K, _IO[out_dtype], 0), a.data_ptr(),
          a_scales.data_ptr(), b.data_ptr(), b_scales.data_ptr(), _ptr(bias), out.data_ptr(), out_row, ws, ws_bytes,
          raw)
    if side is not None:
        _keep(side, a, a_scales, b, b_scales, bias, out, ws_buf)
    return out
