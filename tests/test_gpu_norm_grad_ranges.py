"""The norm's gradient where a row's sum of g s leaves FP32 though dx does not
(BF16 rows near 2^50 under gradients near 2^80 and beyond), beside ordinary
rows, and where that of s^2 does too."""
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _layers import BF, ROW, close, randn, rounded

pytestmark = pytest.mark.gpu
EPS = 1e-5
# powers of two of (s, dy) of each row in turn; the fourth is ordinary
SIZES = [(50, 80), (63, 66), (20, 112), (0, 0), (80, 60), (100, 100), (120, 40), (126, 110), (10, 116)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


# lanes of a warp, a warp and blocks a row, clusters of two and four blocks
@pytest.mark.parametrize("cols", [8, 64, 256, 1040, 4096, 8192, 11008, 24576])
@pytest.mark.parametrize("rows", [9, 700])
@pytest.mark.parametrize("weight", [False, True])
def test_sums_beyond_fp32(cols, rows, weight):
    # magnitudes below 2, and along s in part, so that mean(g u) is of g's size
    s = randn(cols, rows, cols).clamp(-1.9, 1.9)
    dy = (0.5 * s + randn(cols + 1, rows, cols).clamp(-1, 1)).clamp(-1.9, 1.9)
    power = torch.tensor([SIZES[i % len(SIZES)] for i in range(rows)], device="cuda", dtype=torch.float64)
    s, dy = ((x.double() * 2.0 ** power[:, i:i + 1]).to(BF) for i, x in enumerate((s, dy)))
    w = (0.5 + 0.5 * torch.rand(cols, device="cuda", generator=torch.Generator("cuda").manual_seed(5))).to(BF)
    dx, dw = torch.zeros_like(s), torch.zeros(cols, device="cuda")
    scratch = torch.empty(dg.dg_rmsnorm_grad_scratch(rows, cols), dtype=torch.uint8, device="cuda")
    dg.dg_rmsnorm_grad(s, dy, dx, weight=w if weight else None, dweight=dw, scratch=scratch, eps=EPS)
    size = torch.sqrt((s.double() ** 2).mean(-1, keepdim=True) + EPS)
    u, g = s.double() / size, dy.double() * (w.double() if weight else 1.0)
    grad = (g - u * (g * u).mean(-1, keepdim=True)) / size
    terms = (g.abs() + u.abs() * (g * u).abs().mean(-1, keepdim=True)) / size
    # (a reciprocal of 2^-126 and below keeps 21 bits: within ROW)
    close(dx, grad, rounded(grad, BF) + terms * 4 * ROW, "dx")
    assert dx.isfinite().all()
    # columns' sums: of rows of very different size, in FP32
    close(dw, (dy.double() * u).sum(0), (dy.double() * u).abs().sum(0) * (2 * ROW + 2.0 ** -16), "dweight")
