"""The operators around the SSD in a state-space layer, over the C ABI in ``include/ssd.h``: the selective scan, its
causal depthwise convolution, the gated group norm, and the projections in e4m3 with a scale per block of 128.

Like the rest of the binding, these functions check shapes and types, allocate outputs with PyTorch and pass raw
pointers; the computation runs in the library's kernels. The marshalling itself is C++ (``csrc/layer_binding.cpp``,
built in-tree as ``_layer.so``): for a single token it would take longer than the kernel. Token tensors may be column
slices of wider rows (the last dimension contiguous, any other stride). `stream` (default: the current one) is the
stream the kernels run on; with another than the current stream the outputs are allocated for it, and the inputs are
kept until its work is done. `workspace` (a Workspace) carries the device status that check() reads; it may serve ssd_fwd's
calls too, a plain tensor in its place must not. Without it a call
takes a status header of its device (check() without a workspace reads it) and, for a scan in segments, a buffer of its
device and stream that grows; a graph that is being captured takes such a buffer from its own memory, so that it may be
replayed on any stream whatever is called in between. Graphs captured with one and the same Workspace must not be
replayed at the same time.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

import mamba_ssd_prefill_gb300 as _m

_native = None
_lock = threading.Lock()


def _bind():
    """Load the binding and give it the entries of the library that the package loaded."""
    global _native
    with _lock:
        if _native is None:
            lib = _m.lib()
            path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_layer.so")
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; "
                                   f"g.build()'`.")
            from . import _layer

            entries = (lib.ssd_selective_scan_workspace_size, lib.ssd_selective_scan, lib.ssd_conv,
                       lib.ssd_group_norm, lib.ssd_fp8_quantize, lib.ssd_fp8_matmul)
            _layer.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in entries), _m.SsdError, _m.Workspace)
            _native = _layer
    return _native


def ssd_selective_scan(x, dt_raw, dt_bias, A, B, C, D=None, z=None, init_states=None, cu_seqlens=None,
                       state_dtype=None, *, softplus=True, y=None, final_states=None, return_final_states=True,
                       workspace=None, stream=None):
    """Selective scan of a state-space layer, for prompts and (seqlen 1) for single tokens.

    x, dt_raw and the optional gate z [b, L, Dc], B and C [b, L, G, N] in one I/O dtype (fp32, bf16, fp16); A [Dc, N],
    dt_bias and D [Dc] fp32 (both optional); init_states [b, Dc, N] in the state dtype (fp32 or fp16). With
    dt = softplus(dt_raw + dt_bias): h = exp(dt A) h + dt x B, y = (h . C + D x) z sigmoid(z), in fp32. cu_seqlens
    (int32 [nseq + 1], on the GPU) packs nseq sequences on the token axis of [1, T, ...] tensors; the states are then
    [nseq, Dc, N]. final_states may be init_states itself (a cache advanced in place). Returns (y, final_states or
    None). Malformed offsets are reported by check()."""
    return (_native or _bind()).selective_scan(x, dt_raw, dt_bias, A, B, C, D, z, init_states, cu_seqlens, state_dtype,
                                               softplus, y, final_states, return_final_states, workspace, stream)


def ssd_conv(x, conv_weight, conv_bias=None, conv_state=None, cu_seqlens=None, activation="silu", *, out=None,
             conv_state_out=None, return_conv_state=True, workspace=None, stream=None):
    """Causal depthwise convolution over the tokens (ssd_fwd_conv has it in front of the SSD), for prompts and
    (seqlen 1) for single tokens.

    x [b, L, Dc]; conv_weight [Dc, k] (k 1 .. 8, the last tap on the current token) and conv_bias [Dc] fp32;
    conv_state [b, Dc, k-1] in the dtype of x holds the inputs before each sequence (None: zeros). cu_seqlens packs
    sequences as in ssd_selective_scan. Returns (out, conv_state_out or None): the last k-1 inputs, to continue each
    sequence; conv_state_out may be conv_state itself."""
    return (_native or _bind()).conv(x, conv_weight, conv_bias, conv_state, cu_seqlens, activation, out,
                                     conv_state_out, return_conv_state, workspace, stream)


def ssd_group_norm(x, weight=None, bias=None, z=None, ngroups=1, eps=1e-5, *, center=False, activation="silu",
                   gate_first=False, quantize=False, y=None, workspace=None, stream=None):
    """Group norm with an activation, channels last: every token of x [..., Dc] is normalised by itself, its channels
    in `ngroups` groups, with (center) or without the mean taken away, in fp32.

    Without z: act(norm(x) weight + bias). With a gate z of the shape of x: (norm(x) weight + bias) act(z), or with
    gate_first norm(x act(z)) weight + bias. Returns y in the dtype of x (y= may be x itself); with quantize the pair
    (e4m3 values, fp32 scales [..., ceil(Dc / 128)]) that ssd_fp8_matmul takes, rounded once from fp32 (the groups
    must then be multiples of 128 channels, or one)."""
    return (_native or _bind()).group_norm(x, weight, bias, z, ngroups, eps, center, activation, gate_first, quantize,
                                           y, workspace, stream)


def ssd_fp8_quantize(x, block_rows=1, *, workspace=None, stream=None):
    """e4m3 values and their fp32 scales: one scale per row and 128 columns of x [..., K] (block_rows 1, activations),
    or per 128 x 128 block of a matrix x [N, K] (block_rows 128, weights). With m a block's largest magnitude the
    scale is m / 448 and the values x * (448 / m), rounded to nearest even; a block that holds an infinity or a NaN
    gets the scale NaN. Returns (q, scales), contiguous."""
    return (_native or _bind()).fp8_quantize(x, block_rows, workspace, stream)


def ssd_fp8_matmul(a, a_scales, b, b_scales, bias=None, *, out_dtype=torch.bfloat16, out=None, workspace=None,
                   stream=None):
    """a [..., K] times the transpose of the weights b [N, K], both in e4m3 with block scales (a_scales
    [..., ceil(K / 128)], b_scales [ceil(N / 128), ceil(K / 128)], as ssd_fp8_quantize and ssd_group_norm give them),
    accumulated in fp32, plus bias [N] (fp32, optional), in out_dtype (fp32, bf16 or fp16). K is a multiple of 16.
    Returns [..., N]; out= may have rows wider than N."""
    return (_native or _bind()).fp8_matmul(a, a_scales, b, b_scales, bias, out_dtype, out, workspace, stream)
