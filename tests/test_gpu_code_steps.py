"""E4M3 outputs are the nearest code but for what FP32 cannot tell: within half
a step of the value's own binade (2^-4 of the value is twice that near the
binade's top), and the share of codes that are not the nearest is that of
values next to a tie."""
import math

import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _layers import ACT, BF, DTYPES, F8, ROW, act64, norm64, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def half_step(v):
    """Half the distance of E4M3 numbers around v (448 at most)."""
    power = v.abs().clamp(2.0 ** -6, 448.0).contiguous().view(torch.int64) & (0x7FF << 52)     # FP64's exponent alone
    return power.view(torch.float64) * 2.0 ** -4


def nearest(v):
    """E4M3 of FP64 values, ties to even: FP32 first would round twice."""
    step = 2 * half_step(v)
    return torch.round(v / step) * step


def check_steps(q, v, off):
    """Codes of values v that are known to `off`: the nearest, or for values
    that close to a tie the one beyond it."""
    v = v.clamp(-448, 448)
    got = q.view(F8).double().reshape(v.shape)
    err = (got - v).abs()
    bad = err > half_step(v) + off
    assert not bad.any(), (int(bad.sum()), got[bad][:5], v[bad][:5])
    # a tie lies within `off` of a value once in a half step's length
    share = (got != nearest(v)).double().mean().item()
    expected = (2 * off / half_step(v)).clamp(max=1).mean().item()
    assert share <= expected + 4 * math.sqrt(expected / v.numel()) + 4 / v.numel(), (share, expected)


@pytest.mark.parametrize("rows,cols", [(300, 264), (500, 4096), (40, 11008), (30, 24576)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(rows, cols, dtype, residual):
    x, w = randn(1, rows, cols).to(dtype), (1 + 0.2 * randn(2, cols)).to(dtype)
    r = randn(3, rows, cols).to(dtype) if residual else None
    want = norm64(x.double() + (r.double() if residual else 0), w.double(), 1e-5)
    q, scale = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda"), torch.zeros(rows, device="cuda")
    dg.dg_rmsnorm_e4m3(x, q, scale, weight=w, residual=r, eps=1e-5)
    v = want / scale.double()[:, None]
    check_steps(q, v, v.abs() * 2 * ROW)
    one, amax = torch.full((1,), float(want.abs().amax()) / 300, device="cuda"), torch.zeros(1, device="cuda")
    dg.dg_rmsnorm_e4m3_amax(x, one, q, amax, weight=w, residual=r, eps=1e-5)
    v = want / one.double()
    check_steps(q, v, v.abs() * 2 * ROW)


@pytest.mark.parametrize("rows,cols", [(300, 264), (500, 4096), (40, 14336), (20, 28672)])
@pytest.mark.parametrize("act", [dg.DG_ACT_GELU, dg.DG_ACT_GELU_TANH, dg.DG_ACT_SILU])
@pytest.mark.parametrize("gated", [False, True])
def test_activation(rows, cols, act, gated):
    x = (1.5 * randn(rows + act, rows, (2 if gated else 1) * cols)).to(BF)
    y = act64(x.double()[:, :cols], act)[0]
    if gated:
        y = y * x.double()[:, cols:]
    q, scale = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda"), torch.zeros(rows, device="cuda")
    dg.dg_activate(x, act, q=q, q_scale=scale, gated=gated)
    v = y / scale.double()[:, None]
    check_steps(q, v, v.abs() * 2 * ACT)


@pytest.mark.parametrize("M,N,K", [(4, 4096, 1024), (16, 4096, 4096), (129, 1000, 1040), (640, 1536, 2048)])
@pytest.mark.parametrize("act", [dg.DG_ACT_NONE, dg.DG_ACT_GELU, dg.DG_ACT_SILU])
def test_product(M, N, K, act):
    A, B = ((30 * randn(i, n, K)).to(F8).view(torch.uint8) for i, n in ((1, M), (2, N)))
    sa, sb = 0.02 + 0.05 * randn(3, M).abs(), (0.02 + 0.05 * randn(4, N).abs()) / math.sqrt(K)
    bias = randn(5, N)
    a, b = A.view(F8).double(), B.view(F8).double()
    ab = sa.double()[:, None] * sb.double()
    acc = (a @ b.T) * ab + bias.double()
    err = ((a.abs() @ b.abs().T) * ab + bias.double().abs()) * (2.0 ** -23 * (K / 16 + 24))
    want = act64(acc, act)[0]
    err = 1.2 * err + want.abs() * ACT
    sd = torch.full((1,), float(want.abs().amax()) / 300, device="cuda")
    codes = torch.zeros(M, N, dtype=torch.uint8, device="cuda")
    dg.dg_fp8_gemm_fused(A, B, codes, sa, sb, bias=bias, act=act, scale_d=sd, out=dg.DG_E4M3)
    check_steps(codes, want / sd.double(), 1.1 * err / sd.double())


def test_the_bound_itself():
    """Half steps and nearest codes against PyTorch's conversion of every code and midpoint."""
    codes = torch.arange(0x7F, dtype=torch.uint8).view(F8).double().cuda()     # 0 .. 448
    mid = (codes[1:] + codes[:-1]) / 2
    for v in (codes, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)):
        assert torch.equal(nearest(v), v.float().to(F8).double())
    assert torch.equal(half_step(codes[:-1]), (codes[1:] - codes[:-1]) / 2)
