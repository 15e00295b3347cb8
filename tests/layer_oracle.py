"""Plain 64-bit forms of the operators around the SSD, with a running bound on the error of a 32-bit computation.

The bounds are derived from the arithmetic, not fitted: u = 2^-24 is half a unit in the last place of fp32, the
hardware's 2^x has a relative error of 2^-22, softplus, the sigmoid and their products a few units (2^-21).
"""
import torch

U = 2.0 ** -24
OUT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # one rounding of an output
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half a subnormal step


def silu(v):
    return v * torch.sigmoid(v)


def lengths_of(cu):
    cu = cu.tolist()
    return [b - a for a, b in zip(cu, cu[1:])]


def scan(x, dt_raw, dt_bias, A, B, C, D=None, z=None, init_states=None, cu_seqlens=None, softplus=True):
    """(y, final states, error bound of y before its rounding, error bound of the states) in 64 bits on the CPU."""
    f = lambda t: None if t is None else t.detach().cpu().double()  # noqa: E731
    io = x.dtype
    x, dt_raw, dt_bias, A, B, C, D, z, init = map(f, (x, dt_raw, dt_bias, A, B, C, D, z, init_states))
    b, L, Dc = x.shape
    G, N = B.shape[2:]
    if cu_seqlens is not None:
        bounds = cu_seqlens.tolist()
        spans = [(0, s, e) for s, e in zip(bounds, bounds[1:])]
    else:
        spans = [(i, 0, L) for i in range(b)]
    y, ey = torch.zeros_like(x), torch.zeros_like(x)
    fin = torch.zeros(len(spans), Dc, N, dtype=torch.float64)
    efin = torch.zeros_like(fin)
    dt = dt_raw if dt_bias is None else dt_raw + dt_bias
    if softplus:
        dt = torch.clamp(dt, min=0) + torch.log1p(torch.exp(-dt.abs()))
    for i, (row, t0, t1) in enumerate(spans):
        h = torch.zeros(Dc, N, dtype=torch.float64) if init is None else init[i].clone()
        e = torch.zeros_like(h)
        for t in range(t0, t1):
            d = dt[row, t][:, None]
            a = torch.exp(d * A)
            Bt = B[row, t].repeat_interleave(Dc // G, 0)
            Ct = C[row, t].repeat_interleave(Dc // G, 0)
            into = d * x[row, t][:, None] * Bt
            # the decay's error: 2^x itself, its argument (dt, the scaled A and their product), the multiplication
            da = 2.0 ** -22 + 2.0 ** -20 * (d * A).abs() + U
            e = a * (e + da * h.abs()) + 2.0 ** -21 * into.abs()
            h = a * h + into
            e = e + U * h.abs()
            ch = (Ct * h).sum(1)
            ech = (Ct.abs() * e).sum(1) + (N + 2) * U * (Ct * h).abs().sum(1)
            if D is not None:
                ech = ech + 2 * U * (D * x[row, t]).abs()
                ch = ch + D * x[row, t]
            ech = ech + 2 * U * ch.abs()
            if z is not None:
                g = silu(z[row, t])
                # the sigmoid's argument: its error grows with |z| while the value stays below |z|
                ech = ech * g.abs() + ch.abs() * (g.abs() * 2.0 ** -21 + z[row, t].abs() * 2.0 ** -126)
                ech = ech + (ch * g).abs() * z[row, t].abs() * 2.0 ** -23
                ch = ch * g
            y[row, t], ey[row, t] = ch, ech
        fin[i], efin[i] = h, e
    return y, fin, ey * 1.01 + TINY[io], efin * 1.01


def conv(x, w, bias=None, state=None, cu_seqlens=None, activation="silu"):
    """(out, cache, error bound of out before its rounding) in 64 bits on the CPU."""
    f = lambda t: None if t is None else t.detach().cpu().double()  # noqa: E731
    io = x.dtype
    x, w, bias, state = map(f, (x, w, bias, state))
    b, L, Dc = x.shape
    k = w.shape[1]
    if cu_seqlens is not None:
        bounds = cu_seqlens.tolist()
        spans = [(0, s, e) for s, e in zip(bounds, bounds[1:])]
    else:
        spans = [(i, 0, L) for i in range(b)]
    out, err = torch.zeros_like(x), torch.zeros_like(x)
    cache = torch.zeros(len(spans), Dc, k - 1, dtype=torch.float64)
    for i, (row, t0, t1) in enumerate(spans):
        before = torch.zeros(k - 1, Dc, dtype=torch.float64) if state is None else state[i].t()
        rows = torch.cat([before, x[row, t0:t1]])
        n = t1 - t0
        acc = torch.zeros(n, Dc, dtype=torch.float64)
        mag = torch.zeros_like(acc)
        for j in range(k):
            acc += w[:, j] * rows[j:j + n]
            mag += (w[:, j] * rows[j:j + n]).abs()
        if bias is not None:
            acc += bias
            mag += bias.abs()
        e = (k + 1) * U * mag
        if activation == "silu":  # |d silu| <= 1.1
            e = 1.1 * e + silu(acc).abs() * (2.0 ** -21 + acc.abs() * 2.0 ** -23)
            acc = silu(acc)
        out[row, t0:t1], err[row, t0:t1] = acc, e
        cache[i] = rows[n:].t()
    return out, cache, err * 1.01 + TINY[io]


def group_norm(x, weight=None, bias=None, z=None, ngroups=1, eps=1e-5, center=False, activation="silu",
               gate_first=False):
    """(y, error bound before its rounding) in 64 bits on the CPU."""
    f = lambda t: None if t is None else t.detach().cpu().double()  # noqa: E731
    io = x.dtype
    x, weight, bias, z = map(f, (x, weight, bias, z))
    Dc = x.shape[-1]
    act = silu if activation == "silu" else (lambda v: v)
    eact = (lambda v: act(v).abs() * (2.0 ** -21 + v.abs() * 2.0 ** -23)) if activation == "silu" else torch.zeros_like
    v, ev = x, torch.zeros_like(x)
    if gate_first:
        ev = x.abs() * eact(z) + (x * act(z)).abs() * U
        v = x * act(z)
    v, ev = (t.reshape(*x.shape[:-1], ngroups, Dc // ngroups) for t in (v, ev))
    # a sum of n values by threads that add n / 32 of them at most and then join: n / 32 + 16 roundings
    c = (Dc // ngroups / 32 + 16) * U
    if center:
        mag = v.abs().mean(-1, keepdim=True)
        v = v - v.mean(-1, keepdim=True)
        ev = ev + c * mag + ev.mean(-1, keepdim=True) + U * v.abs()
    ms = (v * v).mean(-1, keepdim=True)
    r = 1 / torch.sqrt(ms + eps)
    ems = c * ms + 2 * (v.abs() * ev).mean(-1, keepdim=True) + (ev * ev).mean(-1, keepdim=True)
    n = v * r
    en = ev * r + n.abs() * (0.5 * ems / (ms + eps) * 1.1 + 2.0 ** -22 + 2 * U)
    n, en = n.reshape(x.shape), en.reshape(x.shape)
    if weight is not None:
        n, en = n * weight, en * weight.abs()
    if bias is not None:
        n = n + bias
    en = en + 2 * U * n.abs() + (0 if bias is None else U * bias.abs())
    if z is None:
        en = 1.1 * en + eact(n)
        n = act(n)
    elif not gate_first:
        en = en * act(z).abs() + n.abs() * eact(z) + (n * act(z)).abs() * U
        n = n * act(z)
    return n, en * 1.01 + TINY[io]


def quantize(x, block_rows):
    """ssd_fp8_quantize by its definition in fp32 on the CPU: e4m3 values and scales."""
    x = x.detach().cpu().float()
    M, K = x.shape
    pad = torch.nn.functional.pad(x, (0, -K % 128, 0, -M % block_rows))
    blocks = pad.reshape(pad.shape[0] // block_rows, block_rows, pad.shape[1] // 128, 128)
    m = blocks.abs().amax(dim=(1, 3))
    inv = torch.where(m > 0, torch.full_like(m, 448.0) / m, torch.ones_like(m)).clamp(max=torch.finfo(torch.float32).max)
    scales = torch.where(m > 0, m / torch.full_like(m, 448.0), torch.ones_like(m))  # (a number as the divisor would be multiplied as its reciprocal)
    q = (blocks * inv[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.reshape(pad.shape)[:M, :K].contiguous(), scales


def values(q, scales, block_rows):
    """What e4m3 values and their scales stand for, in 64 bits on the CPU."""
    q, scales = q.detach().cpu().float().double(), scales.detach().cpu().double()
    M, K = q.shape
    return q * scales.repeat_interleave(block_rows, 0)[:M].repeat_interleave(128, 1)[:, :K]


def matmul(a, a_scales, b, b_scales, bias=None):
    """(product in 64 bits, error bound before its rounding). The tensor cores align the products of one instruction
    to the largest of them; with no fewer than 13 bits kept below it, and the blocks then added in fp32, 2^-12 of the
    sum of magnitudes covers what is cut off."""
    va, vb = values(a, a_scales, 1), values(b, b_scales, 128)
    y, mag = va @ vb.t(), va.abs() @ vb.abs().t()
    if bias is not None:
        y, mag = y + bias.cpu().double(), mag + bias.cpu().double().abs()
    return y, mag * 2.0 ** -12


def within(got, want, err, dtype):
    """got (of dtype) is want rounded once, up to err; returns the worst excess and whether it holds."""
    got = got.detach().cpu().double()
    bound = err * 1.01 + OUT[dtype] * (want.abs() + err)
    excess = (got - want).abs() - bound
    return bool((excess <= 0).all()), float(excess.max()) if excess.numel() else 0.0
