"""Cases of the operators around the SSD for the bounds-checked debug build (run as a script by test_layer_ops.py with
MAMBA_SSD_LIB pointing at libmamba_ssd_checked.so). Prints one line per case: "<name> <status>" (0 = no violation)."""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "tests"))

import mamba_ssd_prefill_gb300 as m  # noqa: E402
from test_layer_ops import BF16, CONV, F16, F32, MODES, NORM, PACKED, SCAN, conv_inputs, norm_inputs, scan_inputs  # noqa: E402

assert m.LIB_PATH.endswith("libmamba_ssd_checked.so"), m.LIB_PATH


def run(name, fn):
    ws = m.Workspace("cuda")
    fn(ws)
    try:
        m.check(ws)
        status = 0
    except m.SsdError as e:
        status = e.status
    print(name, status, flush=True)


for i, (b, L, Dc, N, kw) in enumerate(SCAN):
    t = scan_inputs(b, L, Dc, N, **kw)
    run(f"scan{i}", lambda ws: m.ssd_selective_scan(**t, state_dtype=kw.get("state", F32), workspace=ws))
for i, (lengths, Dc, N, kw) in enumerate(PACKED):
    t = scan_inputs(1, sum(lengths), Dc, N, lengths=lengths, **kw)
    run(f"packed{i}", lambda ws: m.ssd_selective_scan(**t, state_dtype=kw.get("state", F32), workspace=ws))
for i, (b, L, Dc, k, kw) in enumerate(CONV):
    a = conv_inputs(b, L, Dc, k, **kw)
    run(f"conv{i}", lambda ws: m.ssd_conv(*a, workspace=ws))
for i, (rows, Dc, G, io) in enumerate(NORM):
    x, kw = norm_inputs(rows, Dc, io, MODES[i % len(MODES)], i)
    run(f"norm{i}", lambda ws: m.ssd_group_norm(x, ngroups=G, workspace=ws, **kw))
    if G == 1 or Dc // G % 128 == 0:
        run(f"norm{i}-e4m3", lambda ws: m.ssd_group_norm(x, ngroups=G, quantize=True, workspace=ws, **kw))
for rows, K, br, io in ((1, 128, 1, BF16), (37, 2560, 1, F32), (9, 200, 1, F16), (7, 1, 1, BF16), (300, 200, 128, F32),
                        (129, 640, 128, BF16)):
    x = torch.randn(rows, K, device="cuda").to(io)
    run(f"quantize-{rows}x{K}-{br}", lambda ws: m.ssd_fp8_quantize(x, br, workspace=ws))
for M, N, K in ((1, 128, 128), (17, 129, 144), (65, 257, 400), (130, 513, 2560), (300, 2560, 1536), (3, 5, 16)):
    a = m.ssd_fp8_quantize(torch.randn(M, K, device="cuda"))
    w = m.ssd_fp8_quantize(torch.randn(N, K, device="cuda"), 128)
    for out in (F32, BF16):
        run(f"matmul-{M}x{N}x{K}-{out}", lambda ws: m.ssd_fp8_matmul(*a, *w, out_dtype=out, workspace=ws))
