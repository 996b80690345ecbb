"""SiLU and the tanh form of GELU where the logistic function is below FP32's
normal numbers but x times it is not (x from about -87, or -10 for the tanh
form): values and gradients against FP64, alone, gated and in a product."""
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _layers import BF, F8, STEP, TINY, act64, close

pytestmark = pytest.mark.gpu
NORMAL = 2.0 ** -126
# The exponent's argument, at most 2^7.1 in base 2, is off by five roundings of
# 2^-24 (square, polynomial, product, the constants): 5 2^-24 2^7.1 ln 2 < 2^-15;
# the exponential, reciprocal and products add less than 2^-20.
REL = 2.0 ** -14
LOW = {dg.DG_ACT_SILU: (-92.0, -80.0), dg.DG_ACT_GELU_TANH: (-10.35, -9.7)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def gates(act, rows, cols):
    low, high = LOW[act]
    x = torch.linspace(low, high, rows * cols, device="cuda").view(rows, cols).to(BF)
    value, slope, _ = act64(x.double(), act)
    # there are values whose logistic function is not a normal number, but they are
    lost = ((value / x.double()).abs() < NORMAL) & (value.abs() >= NORMAL)
    assert lost.sum() > 20
    return x, value, slope


def near(got, want, step, what):
    """Normal values to REL and their rounding; what lies below may be 0."""
    bound = want.abs() * (step + REL) + torch.where(want.abs() < NORMAL, want.abs(), torch.zeros_like(want))
    close(got, want, bound + TINY[BF], what)
    kept = want.abs() >= NORMAL
    assert (got[kept] != 0).all(), what


@pytest.mark.parametrize("act", LOW)
def test_values(act):
    x, value, _ = gates(act, 40, 264)
    y = torch.zeros_like(x)
    dg.dg_activate(x, act, y=y)
    near(y, value, STEP[BF], "y")
    up = torch.full_like(x, 2.0 ** 100)
    y = torch.zeros_like(x)
    dg.dg_activate(torch.cat((x, up), 1), act, y=y, gated=True)
    close(y, value * 2.0 ** 100, value.abs() * 2.0 ** 100 * (STEP[BF] + REL) + NORMAL * 2.0 ** 100 * (value.abs() < NORMAL),
          "gated")
    assert (y[value.abs() >= NORMAL] != 0).all()


@pytest.mark.parametrize("act", LOW)
@pytest.mark.parametrize("gated", [False, True])
def test_gradients(act, gated):
    x, value, slope = gates(act, 40, 264)
    dy = torch.full_like(x, 2.0 ** 60)
    both = torch.cat((x, torch.ones_like(x)), 1) if gated else x
    dx, dbias = torch.zeros_like(both), torch.zeros(both.shape[1], device="cuda")
    scratch = torch.empty(dg.dg_activate_grad_scratch(40, 264, gated), dtype=torch.uint8, device="cuda")
    dg.dg_activate_grad(dy, act, dx, x=both, gated=gated, dbias=dbias, scratch=scratch)
    want = slope * 2.0 ** 60
    if gated:
        want = torch.cat((want, value * 2.0 ** 60), 1)
    lost = NORMAL * 2.0 ** 60
    close(dx, want, want.abs() * (STEP[BF] + REL) + lost * (want.abs() < lost), "dx")
    assert (dx[want.abs() >= lost] != 0).all()
    close(dbias, want.sum(0), want.abs().sum(0) * (REL + 2.0 ** -17) + (want.abs() * (want.abs() < lost)).sum(0), "dbias")


@pytest.mark.parametrize("act", LOW)
@pytest.mark.parametrize("M", [2, 20, 200, 600])
def test_in_a_product(act, M):
    """Through the bias: an operand of zeros."""
    x, _, _ = gates(act, 8, 136)
    bias = x.float().view(-1)
    N = bias.numel()
    A, B = torch.zeros(M, 64, dtype=torch.uint8, device="cuda"), torch.zeros(N, 64, dtype=torch.uint8, device="cuda")
    one, D = torch.ones(1, device="cuda"), torch.zeros(M, N, dtype=BF, device="cuda")
    dg.dg_fp8_gemm_fused(A, B, D, one, one, bias=bias, act=act)
    near(D, act64(bias.double(), act)[0].expand(M, N), STEP[BF], "D")
    codes = torch.zeros(M, N, dtype=torch.uint8, device="cuda")
    dg.dg_fp8_gemm_fused(A, B, codes, one, one, bias=bias, act=act, out=dg.DG_E4M3,
                         scale_d=torch.full((1,), 2.0 ** -125, device="cuda"))
    want = act64(bias.double(), act)[0] * 2.0 ** 125
    close(codes.view(F8), want.clamp(-448, 448).expand(M, N), (want.abs() * (2.0 ** -4 + REL) + 2.0 ** -1).expand(M, N), "codes")


@pytest.mark.parametrize("act", LOW)
def test_the_rest_of_the_range(act):
    """Large, small and special values are what they were."""
    x = torch.tensor([0.0, 2.0 ** -133, -2.0 ** -133, 2.0 ** -120, -2.0 ** -120, 1.0, -1.0, 3.0e38, -3.0e38, 1e5, -1e5,
                      float("inf"), float("nan"), -0.0, 88.0, 100.0], device="cuda").to(BF).view(2, 8)
    y = torch.zeros_like(x)
    dg.dg_activate(x, act, y=y)
    value = act64(x.double().clamp(-1e6, 3.4e38), act)[0]
    value[x.double() < -1e4] = 0
    value[x == float("inf")] = float("inf")
    value[x.isnan()] = float("nan")
    close(y, value, value.abs() * (STEP[BF] + REL) + TINY[BF], "y")
