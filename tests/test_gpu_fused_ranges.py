"""Products with a fused epilogue at the ends of their scales' ranges, against
FP64: every kernel (few rows, split-K, tiles, pairs)."""
import math

import pytest
import torch

import fp16_tensor_core_gb300 as dg
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
