"""Every kernel of the e4m3 product by itself, forced where the library would choose another: the one of 128 x 256 tiles
over several blocks of K and several tiles a CTA, and the ones for few tokens with K split over 1 to 8 CTAs."""
import pytest
import torch

import layer_oracle as lo
import mamba_ssd_prefill_gb300 as m
from test_layer_ops import gen, ok

gpu = pytest.mark.gpu
F32, BF16, F16, E4M3 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn
WIDE = (0, 1)
NARROW = [(tile, splits) for tile in (16, 32, 64, 128) for splits in (1, 2, 4, 8)]


@pytest.fixture
def force():
    yield m.debug_product
    m.debug_product()


def test_the_hook_takes_what_exists(force):
    for tile, splits in [WIDE, *NARROW, (-1, -1)]:
        force(tile, splits)
    for bad in ((0, 2), (0, -1), (-1, 1), (8, 1), (16, 0), (16, 3), (256, 1), (16, 16), (-2, -1)):
        with pytest.raises(m.SsdError) as e:
            force(*bad)
        assert e.value.status == 1


def whole_numbers(M, N, K, seed):
    """Small whole numbers under scales that are powers of two: every sum is exact whatever its order."""
    g = gen(seed)
    a = torch.randint(-2, 3, (M, K), generator=g).float().to(E4M3)
    b = torch.randint(-2, 3, (N, K), generator=g).float().to(E4M3)
    sa = torch.exp2(torch.randint(-3, 4, (M, -(-K // 128)), generator=g).float())
    sb = torch.exp2(torch.randint(-3, 4, (-(-N // 128), -(-K // 128)), generator=g).float())
    bias = torch.randint(-50, 50, (N,), generator=g).float()
    want = lo.values(a, sa, 1) @ lo.values(b, sb, 128).t()
    return [t.cuda() for t in (a, sa, b, sb, bias)], want, want + bias.double()


def call(args, **kw):
    ws = m.Workspace("cuda")
    out = m.ssd_fp8_matmul(*args, workspace=ws, **kw)
    m.check(ws)
    return out


# tokens, outputs, K: 10 blocks and a part, an odd number of outputs, a part of every tile; more tiles than SMs; one block
SIZES = [(70, 301, 1296), (1300, 4000, 1296), (333, 2561, 1152), (5, 140, 2048)]


@gpu
@pytest.mark.parametrize("M,N,K", SIZES, ids=[f"{a}x{b}x{c}" for a, b, c in SIZES])
@pytest.mark.parametrize("tile,splits", [WIDE, *NARROW], ids=lambda v: str(v))
def test_exact_products(force, tile, splits, M, N, K):
    args, want, biased = whole_numbers(M, N, K, M)
    force(tile, splits)
    assert torch.equal(call(args[:4], out_dtype=F32).cpu().double(), want)
    for dtype in (F32, BF16, F16):
        # [M, N] at an odd distance: no 16-byte rows; and rows on 16-byte boundaries
        for off, wide in ((0, N), (3, N + 8), (8, (N + 23) // 8 * 8)):
            to = torch.full((M, wide), 7.0, dtype=dtype, device="cuda")
            got = call(args, out_dtype=dtype, out=to[:, off:off + N])
            assert torch.equal(got.cpu(), biased.to(dtype)), (dtype, off)
            assert bool((to[:, :off] == 7).all()) and bool((to[:, off + N:] == 7).all())


@gpu
@pytest.mark.parametrize("tile,splits", [WIDE, (16, 8), (32, 1), (32, 4), (64, 2), (128, 1), (128, 8)],
                         ids=lambda v: str(v))
@pytest.mark.parametrize("M,N,K", [(150, 513, 2560), (1000, 5000, 1168)])
def test_values(force, tile, splits, M, N, K):
    g = gen(M)
    a, sa = lo.quantize(torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g)), 1)
    b, sb = lo.quantize(torch.randn(N, K, generator=g) * K ** -0.5, 128)
    bias = torch.randn(N, generator=g)
    y, err = lo.matmul(a, sa, b, sb, bias)
    force(tile, splits)
    args = [t.cuda() for t in (a, sa, b, sb, bias)]
    first = call(args, out_dtype=F32)
    ok(first, y, err, F32)
    ok(call(args, out_dtype=BF16), y, err, BF16)
    for _ in range(3):
        assert torch.equal(call(args, out_dtype=F32), first)


@gpu
@pytest.mark.parametrize("tile,splits", [(-1, -1), WIDE, (16, 1), (16, 4), (64, 2), (128, 8)], ids=lambda v: str(v))
@pytest.mark.parametrize("side", ["a", "b"])
def test_scales_keep_all_their_bits(force, tile, splits, side):
    """Odd whole numbers up to 2^20 as the scales of one side, powers of two as the other's; a single 1 in each block of a
    and -1, 0 or 1 in b: sums of at most 11 terms below 2^24, exact in fp32 and in no shorter type."""
    M, N, K = 200, 500, 1296
    kb, g = -(-K // 128), gen(3)
    a, b = torch.zeros(M, K), torch.randint(-1, 2, (N, K), generator=g).float()
    for j in range(kb):
        at = j * 128 + torch.randint(0, min(128, K - j * 128), (M,), generator=g)
        a[torch.arange(M), at] = 1
    odd = lambda *s: (torch.randint(0, 1 << 19, s, generator=g) * 2 + 1).float()  # noqa: E731
    two = lambda *s: torch.exp2(torch.full(s, -5.0))  # noqa: E731
    nb = -(-N // 128)
    sa, sb = (odd(M, kb), two(nb, kb)) if side == "a" else (two(M, kb), odd(nb, kb))
    a, b = a.to(E4M3), b.to(E4M3)
    force(tile, splits)
    got = call([t.cuda() for t in (a, sa, b, sb)], out_dtype=F32)
    assert torch.equal(got.cpu().double(), lo.values(a, sa, 1) @ lo.values(b, sb, 128).t())


@gpu
def test_forced_kernels_that_do_not_hold_the_problem_are_refused(force):
    args, want, _ = whole_numbers(20, 130, 384, 1)  # three blocks
    for tile, splits in ((16, 4), (128, 8)):
        force(tile, splits)
        with pytest.raises(m.SsdError) as e:
            call(args[:4])
        assert e.value.status == 2
    args, want, _ = whole_numbers(20, 130, 31 * 128, 1)  # 31 blocks of 128 scales
    force(128, 1)
    with pytest.raises(m.SsdError) as e:
        call(args[:4])
    assert e.value.status == 2
    force()
    assert torch.equal(call(args[:4], out_dtype=F32).cpu().double(), want)


@gpu
def test_the_library_s_own_choice_for_many_and_for_few_rows(force):
    """Large products take the 128 x 256 tiles and few tokens do not: the same bits as the forced kernel's, which adds the
    blocks in another order than one that splits K."""
    g = gen(9)
    for M, N, K, same, other in ((2000, 5000, 2560, WIDE, (128, 8)), (16, 2560, 2560, None, WIDE)):
        a, sa = (t.cuda() for t in lo.quantize(torch.randn(M, K, generator=g), 1))
        b, sb = (t.cuda() for t in lo.quantize(torch.randn(N, K, generator=g), 128))
        force()
        own = call((a, sa, b, sb), out_dtype=F32)
        if same:
            force(*same)
            assert torch.equal(call((a, sa, b, sb), out_dtype=F32), own)
        force(*other)
        assert not torch.equal(call((a, sa, b, sb), out_dtype=F32), own)
