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


class _Call:
    """Device, stream and workspace of one call."""

    __slots__ = ("device", "stream", "raw", "side", "ws", "guard")

    def __init__(self, device, stream, workspace, kind, nbytes=256):
        import mamba_ssd_prefill_gb300 as m

        self.device = device
        current = torch.cuda.current_stream(device)
        self.side = stream is not None and stream != current
        self.stream = stream if self.side else current
        self.raw = self.stream.cuda_stream
        self.guard = torch.cuda.current_device() != device.index
        if workspace is None:
            key = (kind, device.index, self.raw)
            workspace = m._default_ws.get(key)
            if workspace is None:
                workspace = m._default_ws.setdefault(key, m.Workspace(device))
        if isinstance(workspace, m.Workspace):
            self.ws = self.on(lambda: workspace.get(nbytes))
        else:
            self.ws = workspace

    def on(self, make):
        """make() with the call's stream current, so that what it allocates belongs to that stream."""
        if not self.side:
            return make()
        with torch.cuda.stream(self.stream):
            return make()

    def empty(self, shape, dtype):
        if not self.side:
            return torch.empty(shape, dtype=dtype, device=self.device)
        return self.on(lambda: torch.empty(shape, dtype=dtype, device=self.device))

    def run(self, what, fn, *args, used=()):
        import mamba_ssd_prefill_gb300 as m

        if self.guard:
            with torch.cuda.device(self.device):
                st = fn(*args, self.raw)
        else:
            st = fn(*args, self.raw)
        if st:
            raise m.SsdError(st, what)
        if self.side:  # memory of other streams: not reused before this stream is done with it
            for t in used:
                if t is not None:
                    t.record_stream(self.stream)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _device(what, t):
    if not t.is_cuda:
        raise ValueError(f"{what} runs on CUDA tensors only (there is no CPU path)")
    return t.device


def _lib():
    import mamba_ssd_prefill_gb300 as m

    return m.lib()


def _check(name, t, shape, dtype, dev):
    """t has this shape, type and device and contiguous rows (the last dimension)."""
    if t.shape != shape or t.dtype is not dtype or t.device != dev or (t.stride(-1) != 1 and shape[-1] > 1):
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {dev} with a contiguous last dimension, got "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _flat(name, t, shape, dtype, dev):
    """t has this shape, type and device and is contiguous."""
    if t is not None and (t.shape != shape or t.dtype is not dtype or t.device != dev or not t.is_contiguous()):
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
    b, L, Dc = x.shape
    io = x.dtype
    if io not in _IO:
        raise ValueError(f"x: unsupported dtype {io}")
    if B.dim() != 4:
        raise ValueError("B: expected [batch, seqlen, ngroups, dstate]")
    G, N = B.shape[2], B.shape[3]
    if state_dtype is None:
        state_dtype = init_states.dtype if init_states is not None else _F32
    if state_dtype not in _STATE:
        raise ValueError(f"state_dtype: expected fp32 or fp16, got {state_dtype}")
    if Dc < 1 or N < 1 or G < 1 or Dc % G:
        raise ValueError(f"channels {Dc} must be a positive multiple of the {G} groups, with at least one state")
    shape = (b, L, Dc)
    _check("x", x, shape, io, dev)
    _check("dt_raw", dt_raw, shape, io, dev)
    for name, t in (("B", B), ("C", C)):
        _check(name, t, (b, L, G, N), io, dev)
        if G > 1 and t.stride(2) != N:
            raise ValueError(f"{name}: a token's [ngroups, dstate] must be contiguous")
    _flat("A", A, (Dc, N), _F32, dev)
    _flat("dt_bias", dt_bias, (Dc,), _F32, dev)
    _flat("D", D, (Dc,), _F32, dev)
    _flat("init_states", init_states, (nseq, Dc, N), state_dtype, dev)
    _flat("final_states", final_states, (nseq, Dc, N), state_dtype, dev)
    L_ = _lib()
    prob = _SCAN_PROBLEM(nseq, L, Dc, N, G, _IO[io], _STATE[state_dtype], cu_seqlens is not None, bool(softplus))
    n = ctypes.c_size_t(0)
    st = L_.ssd_selective_scan_workspace_size(prob, ctypes.byref(n))
    if st:
        import mamba_ssd_prefill_gb300 as m

        raise m.SsdError(st, "ssd_selective_scan")
    call = _Call(dev, stream, workspace, "scan", n.value)
    if y is None:
        y = call.empty(shape, io)
    else:
        _check("y", y, shape, io, dev)
    if final_states is None and return_final_states:
        final_states = call.empty((nseq, Dc, N), state_dtype)
    xs, ds, bs, cs, ys = x.stride(), dt_raw.stride(), B.stride(), C.stride(), y.stride()
    if z is not None:
        _check("z", z, shape, io, dev)
        zs = z.stride()
    else:
        zs = (0, 0)
    tensors = _SCAN_TENSORS(x.data_ptr(), dt_raw.data_ptr(), _ptr(z), B.data_ptr(), C.data_ptr(), y.data_ptr(),
                            A.data_ptr(), _ptr(dt_bias), _ptr(D), _ptr(init_states), _ptr(final_states),
                            _ptr(cu_seqlens), xs[0], xs[1], ds[0], ds[1], zs[0], zs[1], bs[0], bs[1], cs[0], cs[1],
                            ys[0], ys[1])
    ws = call.ws
    call.run("ssd_selective_scan", L_.ssd_selective_scan, prob, tensors, ws.data_ptr(),
             ws.numel() * ws.element_size(),
             used=(x, dt_raw, dt_bias, A, B, C, D, z, init_states, cu_seqlens, y, final_states, ws))
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
    call = _Call(dev, stream, workspace, "conv")
    if out is None:
        out = call.empty(shape, io)
    else:
        _check("out", out, shape, io, dev)
    if conv_state_out is None and return_conv_state:
        conv_state_out = call.empty((nseq, Dc, k - 1), io)
    xs, os = x.stride(), out.stride()
    prob = _CONV_PROBLEM(nseq, L, Dc, k, _ACT[activation], _IO[io], cu_seqlens is not None)
    tensors = _CONV_TENSORS(x.data_ptr(), out.data_ptr(), conv_weight.data_ptr(), _ptr(conv_bias), _ptr(conv_state),
                            _ptr(conv_state_out), _ptr(cu_seqlens), xs[0], xs[1], os[0], os[1])
    call.run("ssd_conv", _lib().ssd_conv, prob, tensors, call.ws.data_ptr(),
             used=(x, conv_weight, conv_bias, conv_state, cu_seqlens, out, conv_state_out, call.ws))
    return out, conv_state_out


def _rows(name, t, dtype, dev, shape):
    """t [..., channels] as evenly spaced rows: the row stride."""
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
    call = _Call(dev, stream, workspace, "norm")
    scales = None
    if y is None:
        y = call.empty(shape, E4M3 if quantize else io)
        y_row = Dc
    else:
        y_row = _rows("y", y, E4M3 if quantize else io, dev, shape)
    if quantize:
        scales = call.empty((*shape[:-1], -(-Dc // 128)), _F32)
    prob = _NORM_PROBLEM(x.numel() // Dc, Dc, ngroups, _IO[io], _ACT[activation], bool(center), bool(gate_first),
                         eps, 0)
    tensors = _NORM_TENSORS(x.data_ptr(), _ptr(z), y.data_ptr(), _ptr(scales), _ptr(weight), _ptr(bias), x_row,
                            z_row, y_row)
    call.run("ssd_group_norm", _lib().ssd_group_norm, prob, tensors, call.ws.data_ptr(),
             used=(x, z, weight, bias, y, scales, call.ws))
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
    call = _Call(dev, stream, workspace, "fp8")
    q = call.empty(shape, E4M3)
    scales = call.empty((*shape[:-1], -(-K // 128)) if block_rows == 1 else (-(-rows // 128), -(-K // 128)), _F32)
    call.run("ssd_fp8_quantize", _lib().ssd_fp8_quantize, rows, K, block_rows, _IO[io], x.data_ptr(), x_row,
             q.data_ptr(), scales.data_ptr(), call.ws.data_ptr(), used=(x, q, scales, call.ws))
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
    call = _Call(dev, stream, workspace, "fp8")
    if out is None:
        out = call.empty((*lead, N), out_dtype)
        out_row = N
    else:
        out_row = _rows("out", out, out_dtype, dev, (*lead, N))
    ws = call.ws
    call.run("ssd_fp8_matmul", _lib().ssd_fp8_matmul, _MATMUL_PROBLEM(M, N, K, _IO[out_dtype], 0), a.data_ptr(),
             a_scales.data_ptr(), b.data_ptr(), b_scales.data_ptr(), _ptr(bias), out.data_ptr(), out_row,
             ws.data_ptr(), ws.numel() * ws.element_size(),
             used=(a, a_scales, b, b_scales, bias, out, ws))
    return out
