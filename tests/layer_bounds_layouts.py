"""More cases of the operators around the SSD for the bounds-checked debug build (run as a script by
test_layer_layouts.py with MAMBA_SSD_LIB pointing at libmamba_ssd_checked.so): slices at odd addresses, token-major
tensors, states and caches in place, packed segments with few states, every kernel that the other list leaves out.
Each slice ends where its buffer ends. Prints one line per case: "<name> <status>" (0 = no violation)."""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "tests"))

import mamba_ssd_prefill_gb300 as m  # noqa: E402
from layer_bounds_cases import run  # noqa: E402
from test_layer_ops import BF16, F16, F32, MODES, conv_inputs, norm_inputs, scan_inputs  # noqa: E402

print("--", 0)
TOKENS = ("x", "dt_raw", "B", "C", "z")


def sliced(t, off):
    """The same values as the last columns of wider rows, `off` elements into them."""
    flat = t.reshape(*t.shape[:2], -1)
    wide = torch.zeros(*flat.shape[:2], flat.shape[2] + off, dtype=t.dtype, device="cuda")
    wide[..., off:] = flat
    return wide[..., off:].unflatten(-1, t.shape[2:]) if t.dim() > 3 else wide[..., off:]


def token_major(t):
    return t.transpose(0, 1).contiguous().transpose(0, 1)


for io in (F32, BF16, F16):
    for b, L, Dc, N in ((3, 1, 70, 16), (19, 1, 64, 7), (9, 1, 40, 200), (2, 75, 66, 16), (2, 1200, 40, 4), (1, 900, 72, 24)):
        for off in (0, 1, 2, 8):
            t = scan_inputs(b, L, Dc, N, io=io)
            s = {k: sliced(v, off) if k in TOKENS else v for k, v in t.items()}
            y = torch.zeros(b, L, Dc + off, dtype=io, device="cuda")[..., off:]
            st = s["init_states"]
            run(f"scan-slice-{io}-{L}x{Dc}x{N}-{off}",
                lambda ws: m.ssd_selective_scan(**s, y=y, final_states=st, workspace=ws))
        s = {k: token_major(v) if k in TOKENS else v for k, v in t.items()}
        run(f"scan-token-major-{io}-{L}x{Dc}x{N}", lambda ws: m.ssd_selective_scan(
            **s, y=token_major(torch.zeros(b, L, Dc, dtype=io, device="cuda")), workspace=ws))
    for b, L, Dc, k in ((5, 1, 130, 4), (2, 45, 72, 4), (2, 45, 66, 8), (1, 700, 33, 2)):
        for off in (0, 1, 2, 8):
            x, w, bias, state, _ = conv_inputs(b, L, Dc, k, io=io)
            out = torch.zeros(b, L, Dc + off, dtype=io, device="cuda")[..., off:]
            run(f"conv-slice-{io}-{L}x{Dc}-{k}-{off}",
                lambda ws: m.ssd_conv(sliced(x, off), w, bias, state, out=out, conv_state_out=state, workspace=ws))
    for rows, Dc, G in ((9, 96, 3), (5, 1538, 1), (4, 1001, 1), (3, 30000, 1), (2, 26000, 2)):
        for off in (0, 1, 8):
            x, kw = norm_inputs(rows, Dc, io, MODES[4], 1)
            kw["z"] = sliced(kw["z"][None], off)[0]
            y = torch.zeros(rows, Dc + off, dtype=io, device="cuda")[:, off:]
            run(f"norm-slice-{io}-{rows}x{Dc}-{off}",
                lambda ws: m.ssd_group_norm(sliced(x[None], off)[0], ngroups=G, y=y, workspace=ws, **kw))
            if G == 1:
                run(f"norm-slice-e4m3-{io}-{rows}x{Dc}-{off}", lambda ws: m.ssd_group_norm(
                    sliced(x[None], off)[0], ngroups=G, quantize=True, workspace=ws, **kw))
    for rows, K, br in ((7, 200, 1), (300, 140, 128), (130, 256, 128)):
        for off in (0, 1, 8):
            x = sliced(torch.randn(1, rows, K, device="cuda").to(io), off)[0]
            run(f"quantize-slice-{io}-{rows}x{K}-{br}-{off}", lambda ws: m.ssd_fp8_quantize(x, br, workspace=ws))
for N in (4, 8, 16, 100):
    for lengths in ([1024, 64, 960, 0, 1, 1023, 512, 512], [0, 4096], [3] * 1000):
        t = scan_inputs(1, sum(lengths), 150, N, lengths=lengths)
        run(f"packed-{N}-{len(lengths)}",
            lambda ws: m.ssd_selective_scan(**t, final_states=t["init_states"], workspace=ws))
x, w, bias, state, cu = conv_inputs(1, 500, 66, 4, lengths=[0, 3, 397, 0, 100])
run("conv-packed-in-place", lambda ws: m.ssd_conv(x, w, bias, state, cu, conv_state_out=state, workspace=ws))
for M, N, K in ((700, 2000, 1296), (500, 1001, 1280), (40, 90, 0), (20, 513, 8192)):
    q = m.ssd_fp8_quantize(torch.randn(M, K, device="cuda"))
    wq = m.ssd_fp8_quantize(torch.randn(N, K, device="cuda"), 128)
    for out in (F32, BF16, F16):
        for off in (0, 3):
            to = torch.zeros(M, N + off, dtype=out, device="cuda")[:, off:]
            run(f"matmul-slice-{M}x{N}x{K}-{out}-{off}", lambda ws: m.ssd_fp8_matmul(
                *q, *wq, torch.zeros(N, device="cuda"), out_dtype=out, out=to, workspace=ws))
