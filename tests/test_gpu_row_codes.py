"""A row's codes are formed with the scale that is written: E4M3 of the value
times that scale's FP32 reciprocal, both rounded once, bit for bit.  Shown
where the values themselves are exact in FP32: an activation's checkpoint, and
DG_ACT_NONE and DG_ACT_RELU's outputs."""
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _layers import BF, F8, HALF, MIN_SCALE, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def expected(y):
    """(codes, scales) of rows of FP32 values; IEEE division on the host."""
    y = y.cpu()
    scale = (y.abs().amax(-1) / torch.tensor(448.0)).clamp_min(MIN_SCALE)
    by = torch.tensor(1.0) / scale
    return (y * by[..., None]).to(F8).view(torch.uint8), scale


@pytest.mark.parametrize("rows,cols", [(1, 8), (37, 24), (513, 256), (300, 1040), (200, 4096), (90, 11008), (40, 32768)])
@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -12, 2.0 ** 9])
def test_codes_are_of_the_scale_written(rows, cols, dtype, gated, size):
    halves = 2 if gated else 1
    # each row with a size of its own: scales with every mantissa
    x = (randn(rows + cols, rows, halves * cols) * (0.5 + randn(cols, rows, 1).abs()) * size).to(dtype)
    q, x_q = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda"), torch.zeros_like(x, dtype=torch.uint8)
    q_scale, x_scale = torch.zeros(rows, device="cuda"), torch.zeros(rows, halves, device="cuda")
    act = dg.DG_ACT_NONE if size == 1.0 else dg.DG_ACT_RELU
    dg.dg_activate(x, act, q=q, q_scale=q_scale, x_q=x_q, x_scale=x_scale, gated=gated)
    want, scale = expected(x.float().view(rows, halves, cols))
    assert torch.equal(x_scale.cpu(), scale)
    assert torch.equal(x_q.cpu().view(rows, halves, cols), want)
    y = x.float()[:, :cols]
    if act == dg.DG_ACT_RELU:
        y = y.clamp_min(0)
    if gated:
        y = y * x.float()[:, cols:]
    want, scale = expected(y)
    assert torch.equal(q_scale.cpu(), scale)
    # (a zero times a negative factor is -0, whose code is -0's on either side)
    assert torch.equal(q.cpu(), want)
