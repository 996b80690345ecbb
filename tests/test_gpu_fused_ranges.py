"""Products with a fused epilogue at the ends of their scales' ranges, against
FP64: every kernel (few rows, split-K, tiles, pairs)."""
import math

import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _knobs import knobs
from _layers import F8, randn

pytestmark = pytest.mark.gpu
ROWS = (2, 20, 200, 600)      # rows of A: the warps' product, split-K, tiles, pairs


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def codes_of(seed, *shape, size=1.0):
    return (size * randn(seed, *shape)).to(F8).view(torch.uint8)


def wide(x):
    return x.view(F8).double()


def check_saturating(codes, value, err, sd):
    """E4M3(value / sd) where FP32 knows value to `err`: within half a step below
    448, +-448 with the value's sign above, either in between; NaN as NaN."""
    sd = torch.full_like(value, float(sd))
    q, off = value / sd, (err / sd).nan_to_num(0.0, 0.0, 0.0)
    got = codes.view(F8).double()
    nan = q.isnan()
    assert (codes[nan] == 0x7F).all() and not got[~nan].isnan().any()
    # two roundings of the quotient (2^-22), half a step of the code
    bound = 1.01 * off + q.abs() * 2.0 ** -22
    beyond = torch.where(q.isinf(), value.abs() > err, q.abs() - bound > 448)
    assert (got[beyond] == q[beyond].sign() * 448).all()
    inside = ~nan & ~beyond
    limit = q[inside].clamp(-448, 448)
    step = torch.maximum(limit.abs() * 2.0 ** -4, torch.full_like(limit, 2.0 ** -10))
    assert ((got[inside] - limit).abs() <= step + bound[inside]).all()
    return int(beyond.sum()), int(inside.sum())


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("scale", [1e-40, 2.0 ** -126, 1.0, 2.0 ** 126, 0.0, math.inf, math.nan])
@pytest.mark.parametrize("act", [dg.DG_ACT_NONE, dg.DG_ACT_RELU])
def test_output_scales_saturate(M, scale, act):
    """Tiny scales saturate every value that is not 0, and large ones leave none."""
    N, K = 264, 256
    A, B = codes_of(1, M, K, size=30), codes_of(2, N, K, size=30)
    A[0] = 0
    sa, sb = 0.02 + 0.05 * randn(3, M).abs(), 0.02 + 0.05 * randn(4, N).abs()
    codes = torch.zeros(M, N, dtype=torch.uint8, device="cuda")
    dg.dg_fp8_gemm_fused(A, B, codes, sa, sb, act=act, scale_d=torch.full((1,), scale, device="cuda"), out=dg.DG_E4M3)
    ab = sa.double()[:, None] * sb.double()
    value, size = (wide(A) @ wide(B).T) * ab, (wide(A).abs() @ wide(B).T.abs()) * ab
    if act == dg.DG_ACT_RELU:
        value = value.clamp_min(0)
    beyond, _ = check_saturating(codes, value, size * 2.0 ** -18, scale)
    if 0 <= scale < 1e-30:      # all rows but the first, or what is positive of them
        assert beyond > (0.4 if act == dg.DG_ACT_RELU else 0.9) * (M - 1) * N


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("scale", [1e-40, 2.0 ** -126, 2.0 ** -121, 2.0 ** 100, 2.0 ** 118])
def test_output_scales_of_values_as_small_or_large(M, scale):
    """Values of the scale's own size: their quotients are in range."""
    N, K = 264, 256
    A, B = codes_of(1, M, K, size=2.0 ** -4), codes_of(2, N, K, size=2.0 ** -4)
    A[0] = 0
    half = math.frexp(scale)[1] // 2
    sa = torch.full((M,), 2.0 ** half, device="cuda") * (1 + randn(3, M).abs())
    sb = torch.full((N,), 2.0 ** half, device="cuda") * (1 + randn(4, N).abs())
    codes = torch.zeros(M, N, dtype=torch.uint8, device="cuda")
    dg.dg_fp8_gemm_fused(A, B, codes, sa, sb, scale_d=torch.full((1,), scale, device="cuda"), out=dg.DG_E4M3)
    sd = float(torch.full((1,), scale))      # as FP32 holds it
    ab = sa.double()[:, None] * sb.double()
    value, size = (wide(A) @ wide(B).T) * ab, (wide(A).abs() @ wide(B).T.abs()) * ab
    # FP32's subnormal step once in the value (and once in a subnormal ab times |acc| < 8)
    err = size * 2.0 ** -18 + 2.0 ** -149 * 9
    _, inside = check_saturating(codes, value, err, sd)
    assert inside > 0.9 * M * N


# Powers of two of the rows' and the columns' scales, from a zero row's to the
# largest that a row of BF16 values has; those of ordinary rows among them.
ROW_POWERS = (0, -120, -70, 60, 119, -100, 63, -62, 64, -8)
COLUMN_POWERS = (0, -12, -120, 119, 70, -62, 64, -63, -30, 5)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("N", [264, 1001])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("fp16", [False, True])
def test_products_of_scales_beyond_fp32(M, N, bias, fp16):
    """Scales whose product leaves FP32, though the result does not; empty sums
    are their bias whatever the scales."""
    K = 256
    A, B = (codes_of(i, n, K, size=0.5) for i, n in ((1, M), (2, N)))
    if fp16:
        A, B = wide(A).half(), wide(B).half()
    A[0], A[M // 2] = 0, 0
    power = [torch.tensor([p[i % len(p)] for i in range(n)], device="cuda", dtype=torch.float64)
             for p, n in ((ROW_POWERS, M), (COLUMN_POWERS, N))]
    sa, sb = ((2.0 ** p * (1 + torch.rand(len(p), device="cuda", dtype=torch.float64))).float() for p in power)
    b = randn(5, N) if bias else None
    D = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    if fp16:
        dg.dg_hgemm_fused(A, B, D, bias=b, scale_a=sa, scale_b=sb, out=dg.DG_BF16)
    else:
        dg.dg_fp8_gemm_fused(A, B, D, sa, sb, bias=b)
    acc, size = A.double() if fp16 else wide(A), B.double() if fp16 else wide(B)
    acc, size = acc @ size.T, acc.abs() @ size.T.abs()
    ab = sa.double()[:, None] * sb.double()
    want = acc * ab + (b.double() if bias else 0)
    got = D.double()
    assert not got.isnan().any()
    # accumulation, four roundings more, FP32's subnormal step, and BF16's rounding
    err = size * ab * (2.0 ** -23 * (K / 16 + 24)) + 2.0 ** -149
    bound = err + want.abs() * 2.0 ** -8 + 2.0 ** -134
    top = torch.finfo(torch.bfloat16).max
    beyond = want.abs() > top * (1 + 2.0 ** -9) + err
    assert (got[beyond].isinf() & (got[beyond].sign() == want[beyond].sign())).all()
    near = want.abs() <= top - err
    assert ((got[near] - want[near]).abs() <= bound[near]).all()
    # both kinds are there: a product of scales that FP32 does not hold, and a result that it does
    if M > 10:
        odd = (ab < 2.0 ** -126) | (ab > 2.0 ** 127)
        assert (odd & near & (acc != 0)).sum() > 0.1 * M * N and beyond.any()
    empty = (b.double() if bias else torch.zeros(N, dtype=torch.float64, device="cuda")).bfloat16().double()
    assert torch.equal(got[0], empty) and torch.equal(got[M // 2], empty)


@pytest.mark.parametrize("env", [dict(DG_2CTA="0", DG_FORCE_BLOCK_N="96"), dict(DG_2CTA="0", DG_FORCE_BLOCK_N="256"),
                                 dict(DG_2CTA="1", DG_FORCE_BLOCK_N="160"), dict(DG_2CTA="1", DG_FORCE_BLOCK_N="256"),
                                 dict(DG_2CTA="1", DG_FORCE_BLOCK_N="224", DG_STREAM_K="1")])
@pytest.mark.parametrize("short", [16, 3])
def test_extreme_scales_of_some_tiles(env, short):
    """Several tiles a CTA, of which some have extreme scales and others none;
    bias, residual and ReLU behind them."""
    M, K, bn = 500, 256, int(env["DG_FORCE_BLOCK_N"])
    N = 100 * bn - short
    A, B = (codes_of(i, n, K, size=0.5) for i, n in ((1, M), (2, N)))
    sa, sb = 1 + randn(3, M).abs(), 1 + randn(4, N).abs()
    sa[7], sa[300:310] = 2.0 ** -120, 2.0 ** 80
    sb[5 * bn:6 * bn] *= 2.0 ** -90
    sb[40 * bn + 3], sb[N - 1] = 2.0 ** 100, 2.0 ** -70
    bias, residual = randn(5, N), randn(6, M, N).to(torch.bfloat16)
    D = residual.clone()
    with knobs(**env):
        p = dg.dg_gemm_plan(M, N, K)
        assert p["path"] == 3 and p["block_n"] == bn and p["tiles"] > p["grid"], p
        dg.dg_fp8_gemm_fused(A, B, D, sa, sb, bias=bias, act=dg.DG_ACT_RELU, residual=D)
    ab = sa.double()[:, None] * sb.double()
    acc, size = (wide(A) @ wide(B).T) * ab, (wide(A).abs() @ wide(B).T.abs()) * ab
    want = (acc + bias.double()).clamp_min(0) + residual.double()
    err = (size + bias.double().abs()) * (2.0 ** -23 * (K / 16 + 24)) + want.abs() * 2.0 ** -23
    top = torch.finfo(torch.bfloat16).max
    near = want.abs() <= top - err
    got = D.double()
    assert not got.isnan().any() and near.float().mean() > 0.99
    assert ((got[near] - want[near]).abs() <= (err + want.abs() * 2.0 ** -8 + 2.0 ** -134)[near]).all()
