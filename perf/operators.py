"""The operators around the SSD in a state-space layer, as they are measured: the selective scan with its causal
convolution, the gated group norm, and the projections in 8-bit floating point with a scale per block of 128.

Each case is one call of a layer's forward pass (a prompt, packed prompts, or one new token per sequence). With
`own` false `run` computes it from elementary torch operations in 32 bits, with `own` true through this package.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 128      # elements along K that share one scale
E4M3_MAX = 448.0

# The largest listed work of each operator; drawn cases stay below it.
MOST_SCAN = 65536 * 1536 * 16
MOST_CONV = 65536 * 5376
MOST_NORM = 16384 * 5120
MOST_PROJ = 16384 * 2560 * 10576


def listed():
    return [
        # one new token of one conversation, 130M-shaped layer: launch latency
        dict(name="scan-token-1", op="scan", batch=1, seqlen=1, channels=1536, states=16, groups=1, io="bf16",
             state="f32", gate=True, init=True, packed=False),
        # one new token for each of 256 conversations, 2.7B-shaped layer, cached states in fp16
        dict(name="scan-token-256", op="scan", batch=256, seqlen=1, channels=5120, states=16, groups=1, io="bf16",
             state="f16", gate=True, init=True, packed=False),
        # a batch of prompts, 130M-shaped layer, continuing from earlier states
        dict(name="scan-prompts-4k", op="scan", batch=4, seqlen=4096, channels=1536, states=16, groups=1, io="bf16",
             state="f32", gate=True, init=True, packed=False),
        # one prompt through a 2.7B-shaped layer
        dict(name="scan-prompt-16k", op="scan", batch=1, seqlen=16384, channels=5120, states=16, groups=1, io="bf16",
             state="f32", gate=True, init=False, packed=False),
        # one long document through a narrow layer: few channels, a long serial axis
        dict(name="scan-document-64k", op="scan", batch=1, seqlen=65536, channels=1536, states=16, groups=1, io="bf16",
             state="f32", gate=True, init=False, packed=False),
        # prompts of different lengths (one of them empty at times) packed on one axis, odd sizes, two groups
        dict(name="scan-packed-f16", op="scan", batch=37, seqlen=9001, channels=1000, states=24, groups=2, io="f16",
             state="f32", gate=False, init=True, packed=True),
        # the convolution in front, prompts of a 2.7B-shaped layer (x, B and C channels)
        dict(name="conv-prompts-8k", op="conv", batch=8, seqlen=8192, channels=5376, width=4, io="bf16", packed=False),
        # the same for one new token of 64 conversations: the cache is shifted by one
        dict(name="conv-token-64", op="conv", batch=64, seqlen=1, channels=5376, width=4, io="bf16", packed=False),
        # the gated norm before the output projection, 130M-shaped layer
        dict(name="norm-16k", op="norm", rows=16384, channels=1536, groups=1, io="bf16", center=False,
             gate_first=True),
        # norm in 8 groups, its output in 8 bits, and the output projection of a 2.7B-shaped layer; an odd row count
        dict(name="norm-project-8k", op="norm_project", rows=8191, channels=5120, groups=8, outputs=2560, io="bf16",
             center=True, gate_first=False),
        # the input projection of a 2.7B-shaped layer for 16 new tokens: the weights' bytes count
        dict(name="project-16", op="project", rows=16, channels=2560, outputs=10576, io="bf16"),
        # the same for a batch of prompts: the tensor cores' rate counts
        dict(name="project-16k", op="project", rows=16384, channels=2560, outputs=10576, io="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _size(rng, lo, hi, of=1):
    """The same, a multiple of `of`."""
    n = _log(rng, lo, hi) // of * of
    return max(of, n if n != 3072 else n - of)


def draw(rng):
    op = rng.choice(["token", "prompt", "prompt", "packed", "conv", "norm", "norm_project", "project"])
    io = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("token", "prompt", "packed"):
        groups = rng.choice([1, 1, 2, 5])
        states = rng.choice([16, 16, 8, rng.randint(1, 64)])
        channels = _size(rng, 96, 5120, groups)
        if op == "token":
            batch, seqlen = _log(rng, 1, 256), 1
        elif op == "packed":
            batch, seqlen = rng.randint(1, 64), _log(rng, 64, 32768)
        else:
            batch, seqlen = _log(rng, 1, 16), _log(rng, 2, 65536)
        tokens = (1 if op == "packed" else batch) * seqlen
        if tokens * channels * states > MOST_SCAN:
            if op != "packed":
                batch = 1
            seqlen = max(2, min(seqlen, MOST_SCAN // (batch if op != "packed" else 1) // (channels * states)))
        return dict(op="scan", batch=batch, seqlen=seqlen, channels=channels, states=states, groups=groups, io=io,
                    state=rng.choice(["f32", "f32", "f16"]), gate=rng.random() < 0.7, init=rng.random() < 0.5,
                    packed=op == "packed")
    if op == "conv":
        channels, width = _size(rng, 96, 10752), rng.choice([4, 4, 2, 3, 8])
        packed = rng.random() < 0.4
        batch, seqlen = _log(rng, 1, 64), _log(rng, 1, 32768)
        seqlen = max(1, min(seqlen, MOST_CONV // (channels * (1 if packed else batch))))
        return dict(op="conv", batch=batch, seqlen=seqlen, channels=channels, width=width, io=io, packed=packed)
    groups = rng.choice([1, 1, 2, 8])
    if op != "norm":  # 8-bit operands: the layer's own types are 16-bit ones
        io = rng.choice(["bf16", "f16"])
    if op == "norm":
        channels = _size(rng, 96, 8192, groups)
        rows = min(_log(rng, 1, 65536), MOST_NORM // channels)
        return dict(op="norm", rows=rows, channels=channels, groups=groups, io=io, center=rng.random() < 0.5,
                    gate_first=rng.random() < 0.5)
    if op == "norm_project":  # each scale's block lies within one group
        channels = _size(rng, 256, 8192, groups * BLOCK)
    else:
        channels = _size(rng, 256, 8192, 16)
    outputs = _size(rng, 256, 10752)
    rows = max(1, min(_log(rng, 1, 16384), MOST_PROJ // (channels * outputs)))
    c = dict(op=op, rows=rows, channels=channels, outputs=outputs, io=io)
    if op == "norm_project":
        c.update(groups=groups, center=rng.random() < 0.5, gate_first=rng.random() < 0.5)
    return c


# ------------------------------------------------------------------------------------------------------ inputs

def _lengths(case, seed):
    """Lengths of packed sequences: random cuts of the axis, so that some are short and some may be empty."""
    g = torch.Generator("cpu").manual_seed(seed)
    cuts = torch.randint(0, case["seqlen"] + 1, (case["batch"] - 1,), generator=g).sort().values.tolist()
    edges = [0, *cuts, case["seqlen"]]
    return [b - a for a, b in zip(edges, edges[1:])]


def _offsets(lengths):
    cu = torch.zeros(len(lengths) + 1, dtype=torch.int64)
    cu[1:] = torch.tensor(lengths).cumsum(0)
    return cu


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    io = DTYPES[case["io"]]

    def randn(*shape, scale=1.0, dtype=io):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = dict(case=case)
    if case["op"] in ("scan", "conv"):
        if case["packed"]:
            lengths = _lengths(case, seed)
            cu = _offsets(lengths)
            s["cu_seqlens"] = cu.to(torch.int32).cuda()
            s["lengths"], b, L = lengths, 1, case["seqlen"]
        else:
            b, L = case["batch"], case["seqlen"]
            lengths = [L] * b
            s["cu_seqlens"] = None
            s["lengths"] = lengths
            cu = _offsets(lengths)
        # where the plain form puts what enters a sequence and finds what leaves it
        live = [i for i, n in enumerate(lengths) if n > 0]
        s["live"] = torch.tensor(live, device="cuda")
        s["first"] = cu[:-1][live].cuda()
        s["last"] = (cu[1:][live] - 1).cuda()
    if case["op"] == "scan":
        D, N, G, nseq = case["channels"], case["states"], case["groups"], case["batch"]
        # x and the gate are column slices of one projection's rows, as a layer has them
        rows = randn(b, L, 2 * D + 16)
        s["x"], s["z"] = rows[..., :D], (rows[..., D + 16:] if case["gate"] else None)
        s["dt_raw"] = randn(b, L, D)
        s["B"], s["C"] = randn(b, L, G, N), randn(b, L, G, N)
        dt0 = torch.exp(torch.rand(D, generator=g, device="cuda") * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
        s["dt_bias"] = torch.log(torch.expm1(dt0))
        s["A"] = -(torch.arange(1, N + 1, device="cuda") * torch.exp(randn(D, N, scale=0.1, dtype=torch.float32)))
        s["D"] = randn(D, dtype=torch.float32)
        st = DTYPES[case["state"]]
        s["init_states"] = randn(nseq, D, N, scale=0.1, dtype=st) if case["init"] else None
        s["state_dtype"] = st
    elif case["op"] == "conv":
        D, k = case["channels"], case["width"]
        s["x"] = randn(b, L, D)
        s["conv_weight"] = (torch.rand(D, k, generator=g, device="cuda") * 2 - 1) / math.sqrt(k)
        s["conv_bias"] = randn(D, scale=0.1, dtype=torch.float32)
        s["conv_state"] = randn(case["batch"], D, k - 1)
    else:
        M, D = case["rows"], case["channels"]
        s["x"] = randn(M, D)
        if case["op"] != "project":
            s["z"] = randn(M, D)
            s["weight"] = 1 + randn(D, scale=0.1, dtype=torch.float32)
            s["bias"] = randn(D, scale=0.1, dtype=torch.float32)
        if case["op"] != "norm":  # the weights in 8 bits, kept from call to call
            w = randn(case["outputs"], D, scale=D ** -0.5, dtype=torch.float32)
            s["w"], s["w_scales"] = _quantize(w, BLOCK)
    return s


# -------------------------------------------------------------------------------------------------- plain forms

def _blocks(t, rows):
    """t [M, K] padded with zeros to whole blocks: [M / rows, rows, K / BLOCK, BLOCK]."""
    M, K = t.shape
    t = torch.nn.functional.pad(t, (0, -K % BLOCK, 0, -M % rows))
    return t.reshape(t.shape[0] // rows, rows, t.shape[1] // BLOCK, BLOCK)


def _quantize(t, rows):
    """t [M, K] in 32 bits -> e4m3 values [M, K] and the scales of its blocks [ceil(M / rows), ceil(K / BLOCK)]."""
    M, K = t.shape
    blocks = _blocks(t, rows)
    most = blocks.abs().amax(dim=(1, 3))
    top = torch.full_like(most, E4M3_MAX)  # a tensor: a plain number would be multiplied with a rounded reciprocal
    inverse = torch.where(most > 0, top / most, torch.ones_like(most))
    scales = torch.where(most > 0, most / top, torch.ones_like(most))
    q = (blocks * inverse[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.reshape(q.shape[0] * rows, -1)[:M, :K].contiguous(), scales


def _values(q, scales, rows):
    """What 8-bit values and their scales stand for, in 32 bits."""
    M, K = q.shape
    v = _blocks(q.float(), rows) * scales[:, None, :, None]
    return v.reshape(v.shape[0] * rows, -1)[:M, :K]


def _silu(v):
    return v / (1 + torch.exp(-v))


def _plain_conv(s):
    x, k = s["x"].float(), s["case"]["width"]
    L, D = x.shape[0] * x.shape[1], x.shape[2]
    x = x.reshape(L, D)
    cache = s["conv_state"].float()
    # position of each token in its sequence, and its sequence
    start = torch.zeros(L, dtype=torch.int64, device=x.device)
    start[s["first"]] = s["first"]
    start = start.cummax(0).values
    seq = torch.zeros(L, dtype=torch.int64, device=x.device)
    seq[s["first"]] = s["live"]
    seq = seq.cummax(0).values
    t = torch.arange(L, device=x.device)
    back = torch.arange(k - 1, -1, -1, device=x.device)
    rows = t[:, None] - back                     # [L, k] input rows under the taps
    before = rows - start[:, None]               # < 0: from the cache
    # the cached inputs as rows behind the others
    cached = cache.transpose(1, 2).reshape(-1, D)
    rows = torch.where(before >= 0, rows, L + seq[:, None] * (k - 1) + (k - 1) + before)
    every = torch.cat([x, cached])
    acc = (every[rows] * s["conv_weight"].t()).sum(1) + s["conv_bias"]
    out = _silu(acc).to(s["x"].dtype).reshape(s["x"].shape)
    # the last k - 1 inputs of each sequence
    state = s["conv_state"].clone()
    rows = s["last"][:, None] - back[1:]
    before = rows - start[s["last"]][:, None]
    rows = torch.where(before >= 0, rows, L + s["live"][:, None] * (k - 1) + (k - 1) + before)
    state[s["live"]] = every[rows].transpose(1, 2).to(state.dtype)
    return out, state


def _scan(a, b, most):
    """h[t] = a[t] h[t-1] + b[t] along the first axis in place, by doubling; a is 0 where a sequence begins, and no
    sequence is longer than `most`."""
    step = 1
    while step < most:
        b[step:] = b[step:] + a[step:] * b[:-step]
        a[step:] = a[step:] * a[:-step]
        step *= 2
    return b


def _plain_scan(s):
    c = s["case"]
    D, N, G = c["channels"], c["states"], c["groups"]
    x, raw = s["x"].reshape(-1, D).float(), s["dt_raw"].reshape(-1, D).float() + s["dt_bias"]
    T = x.shape[0]
    B, C = s["B"].reshape(T, G, 1, N).float(), s["C"].reshape(T, G, 1, N).float()
    dt = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw)))
    a = torch.exp(dt[:, :, None] * s["A"])
    h = ((dt * x).reshape(T, G, D // G, 1) * B).reshape(T, D, N)
    if s["init_states"] is not None:
        h[s["first"]] += a[s["first"]] * s["init_states"][s["live"]].float()
    a[s["first"]] = 0
    h = _scan(a, h, max(s["lengths"]))
    del a
    y = (h.reshape(T, G, D // G, N) * C).sum(-1).reshape(T, D) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].reshape(T, D).float())
    if s["init_states"] is not None:
        final = s["init_states"].clone()
    else:
        final = torch.zeros(c["batch"], D, N, dtype=s["state_dtype"], device=x.device)
    final[s["live"]] = h[s["last"]].to(s["state_dtype"])
    return y.to(s["x"].dtype).reshape(s["x"].shape), final


def _plain_norm(s):
    """The norm in 32 bits, before any rounding."""
    c = s["case"]
    x, z = s["x"].float(), _silu(s["z"].float())
    M, D = x.shape
    v = x * z if c["gate_first"] else x
    v = v.reshape(M, c["groups"], D // c["groups"])
    if c["center"]:
        v = v - v.mean(-1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5)
    v = v.reshape(M, D) * s["weight"] + s["bias"]
    return v if c["gate_first"] else v * z


def _plain_project(s, v):
    q, scales = _quantize(v, 1)
    return (_values(q, scales, 1) @ _values(s["w"], s["w_scales"], BLOCK).t()).to(s["x"].dtype)


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "scan":
        return _plain_scan(s)
    if op == "conv":
        return _plain_conv(s)
    if op == "norm":
        return _plain_norm(s).to(s["x"].dtype)
    if op == "norm_project":
        return _plain_project(s, _plain_norm(s))
    return _plain_project(s, s["x"].float())


def _own(s, op):
    import mamba_ssd_prefill_gb300 as ssd

    if op == "scan":
        return ssd.ssd_selective_scan(s["x"], s["dt_raw"], s["dt_bias"], s["A"], s["B"], s["C"], s["D"], z=s["z"],
                                      init_states=s["init_states"], cu_seqlens=s["cu_seqlens"],
                                      state_dtype=s["state_dtype"])
    if op == "conv":
        return ssd.ssd_conv(s["x"], s["conv_weight"], s["conv_bias"], s["conv_state"], cu_seqlens=s["cu_seqlens"])
    c = s["case"]
    if op == "norm":
        return ssd.ssd_group_norm(s["x"], s["weight"], s["bias"], z=s["z"], ngroups=c["groups"], center=c["center"],
                                  gate_first=c["gate_first"])
    if op == "norm_project":
        q, scales = ssd.ssd_group_norm(s["x"], s["weight"], s["bias"], z=s["z"], ngroups=c["groups"],
                                       center=c["center"], gate_first=c["gate_first"], quantize=True)
    else:
        q, scales = ssd.ssd_fp8_quantize(s["x"])
    return ssd.ssd_fp8_matmul(q, scales, s["w"], s["w_scales"], out_dtype=s["x"].dtype)


# --------------------------------------------------------------------------------------------------------- work

def work(case):
    e = BYTES[case["io"]]
    if case["op"] == "scan":
        T = case["seqlen"] * (1 if case["packed"] else case["batch"])
        D, N, G = case["channels"], case["states"], case["groups"]
        states = case["batch"] * D * N * BYTES[case["state"]]
        return dict(bytes=e * T * ((4 if case["gate"] else 3) * D + 2 * G * N) + states * (2 if case["init"] else 1)
                    + 4 * D * (N + 2),
                    flops=7 * T * D * N)
    if case["op"] == "conv":
        T, D, k = case["seqlen"] * (1 if case["packed"] else case["batch"]), case["channels"], case["width"]
        return dict(bytes=2 * e * (T * D + case["batch"] * D * (k - 1)) + 4 * D * (k + 1), flops=(2 * k + 4) * T * D)
    M, D = case["rows"], case["channels"]
    if case["op"] == "norm":
        return dict(bytes=3 * e * M * D + 8 * D, flops=12 * M * D)
    F = case["outputs"]
    weights = F * D + 4 * (-(-F // BLOCK)) * (-(-D // BLOCK))
    if case["op"] == "project":
        return dict(bytes=e * M * (D + F) + weights, flops=2 * M * D * F)
    return dict(bytes=e * M * (2 * D + F) + 8 * D + weights, flops=2 * M * D * F + 12 * M * D)


# -------------------------------------------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "scan":
        return _exact_scan(s)
    if op == "conv":
        return _exact_conv(s)
    if op == "project":
        return _exact_project(s, s["x"].double())
    v = _exact_norm(s)
    return v if op == "norm" else _exact_project(s, v)


def _exact_scan(s):
    """The recurrence token by token in 64 bits, the sequences side by side (the longest first)."""
    c = s["case"]
    D, N, G = c["channels"], c["states"], c["groups"]
    lengths = s["lengths"]
    order = sorted(range(len(lengths)), key=lambda i: -lengths[i])
    begin = _offsets(lengths)[:-1][order].cuda()
    x, C = s["x"].reshape(-1, D).double(), s["C"].reshape(-1, G, N).double()
    raw = s["dt_raw"].reshape(-1, D).double() + s["dt_bias"].double()
    dt = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    B, A = s["B"].reshape(-1, G, N).double(), s["A"].double()
    h = torch.zeros(len(lengths), D, N, dtype=torch.float64, device=x.device)
    if s["init_states"] is not None:
        h.copy_(s["init_states"][order])
    y = x * s["D"].double()
    live = len(lengths)
    for t in range(lengths[order[0]]):
        while lengths[order[live - 1]] <= t:
            live -= 1
        at = begin[:live] + t
        d = dt[at]
        e = h[:live]
        e.mul_(torch.exp(d[:, :, None] * A))
        e.view(live, G, D // G, N).add_((d * x[at]).view(live, G, D // G, 1) * B[at][:, :, None])
        y[at] += torch.matmul(e.view(live, G, D // G, N), C[at][..., None]).view(live, D)
    if s["z"] is not None:
        z = s["z"].reshape(-1, D).double()
        y *= z * torch.sigmoid(z)
    final = torch.empty_like(h)
    final[order] = h
    return y.reshape(s["x"].shape), final


def _exact_conv(s):
    """Each sequence by itself: its cached inputs in front of it, one shifted product a tap."""
    k, w = s["case"]["width"], s["conv_weight"].double()
    x, at = s["x"].reshape(-1, s["case"]["channels"]), 0
    outs, states = [], []
    for i, n in enumerate(s["lengths"]):
        row = torch.cat([s["conv_state"][i].double().t(), x[at:at + n].double()])
        acc = s["conv_bias"].double().expand(n, -1)
        for j in range(k):
            acc = acc + w[:, j] * row[j:j + n]
        outs.append(acc * torch.sigmoid(acc))
        states.append(row[n:].t())
        at += n
    return torch.cat(outs).reshape(s["x"].shape), torch.stack(states)


def _exact_norm(s):
    c = s["case"]
    z = s["z"].double()
    gate = z * torch.sigmoid(z)
    groups = []
    for v in (s["x"].double() * gate if c["gate_first"] else s["x"].double()).chunk(c["groups"], 1):
        var, mean = torch.var_mean(v, 1, correction=0, keepdim=True)
        groups.append((v - mean) * torch.rsqrt(var + 1e-5) if c["center"]
                      else v * torch.rsqrt(var + mean * mean + 1e-5))
    v = torch.cat(groups, 1) * s["weight"].double() + s["bias"].double()
    return v if c["gate_first"] else v * gate


def _exact_project(s, v):
    """The activations rounded to e4m3 with one scale per block, the product block by block."""
    K = v.shape[1]
    out = torch.zeros(v.shape[0], s["w"].shape[0], dtype=torch.float64, device=v.device)
    for j in range(0, K, BLOCK):
        part = v[:, j:j + BLOCK]
        scale = part.abs().amax(1, keepdim=True) / E4M3_MAX
        scale[scale == 0] = 1
        part = part / scale
        # spacing of e4m3: 2^(e - 3) in [2^e, 2^(e+1)), 2^-9 below 2^-6
        step = torch.exp2(torch.frexp(part.abs().clamp(min=2.0 ** -6)).exponent.double() - 4)
        part = torch.round(part / step) * step * scale
        scales = s["w_scales"][:, j // BLOCK].double().repeat_interleave(BLOCK)[:out.shape[1], None]
        out += part @ (s["w"][:, j:j + BLOCK].double() * scales).t()
    return out
