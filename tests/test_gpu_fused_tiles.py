"""The fused epilogue on every tile that the planner can choose: each width,
one and two K blocks a stage, single CTAs and pairs, one tile a CTA and
several, against FP64.  Widths of an odd number of 32-column chunks give the
two halves of the epilogue warps unequal shares.  The plan is asserted."""
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _knobs import knobs
from _layers import BF, HALF
from test_gpu_fused_gemm import check

pytestmark = pytest.mark.gpu
SINGLE, PAIRS = (64, 96, 128, 160, 192, 224, 256), (128, 160, 192, 224, 256)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def both(M, N, K, plan, fp16):
    p = dg.dg_gemm_plan(M, N, K, dg.DG_FP16 if fp16 else dg.DG_E4M3, dg.DG_BF16)
    assert (p["path"], p["block_m"], p["block_n"], p["block_k"]) == plan, p
    check(M, N, K, fp16, dg.DG_BF16, dg.DG_ACT_SILU, True, True, HALF)
    if fp16:
        check(M, N, K, True, dg.DG_FP16, dg.DG_ACT_NONE, None, False, HALF, in_place=True)
    else:
        check(M, N, K, False, dg.DG_E4M3, dg.DG_ACT_GELU, True, True, BF)
    return p


# Columns short of whole tiles: by a multiple of eight (bulk stores), and odd.
@pytest.mark.parametrize("short", [24, 3])
@pytest.mark.parametrize("fp16", [False, True])
@pytest.mark.parametrize("kps", [1, 2])
@pytest.mark.parametrize("bn", SINGLE)
def test_single_tiles(bn, kps, fp16, short):
    K, block = 1040, 64 if fp16 else 128
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    with knobs(DG_2CTA="0", DG_FORCE_BLOCK_N=str(bn), DG_TC_KPS=str(kps), DG_SPLITK="0"):
        two = kps == 2 and bn <= 128          # one wave only
        p = both(130, 3 * bn - short, K, (3, 128, bn, block * (2 if two else 1)), fp16)
        assert p["tiles"] == 6
        p = both(130, bn * (sms // 2 + 20) - short, K, (3, 128, bn, block), fp16)
        assert p["tiles"] > sms


@pytest.mark.parametrize("short", [24, 3])
@pytest.mark.parametrize("fp16", [False, True])
@pytest.mark.parametrize("kps", [1, 2])
@pytest.mark.parametrize("bn", PAIRS)
def test_pair_tiles(bn, kps, fp16, short):
    K, block = 1040, 64 if fp16 else 128
    slots = torch.cuda.get_device_properties(0).multi_processor_count // 2
    with knobs(DG_2CTA="1", DG_FORCE_BLOCK_N=str(bn), DG_PAIR_KPS=str(kps)):
        p = both(300, 3 * bn - short, K, (3, 256, bn, block * kps), fp16)
        assert p["tiles"] == 6
        p = both(300, bn * (slots // 2 + 12) - short, K, (3, 256, bn, block * kps), fp16)
        assert p["tiles"] > slots
