"""Pair tiles of every width whose last wave is split along K (DG_SPLIT_TAIL=1)
into two, three and four ranges, plain and with a fused epilogue, against
FP64.  One row of tiles, so that their number can be chosen: with P pairs,
P + P // s tiles leave P // s to be cut into s ranges each, for s up to 4.  The
log line of the call says that they were."""
import math
import re

import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _knobs import knobs
from _layers import BF, F8, HALF, STEP, TINY, act64, close, randn

pytestmark = pytest.mark.gpu
WIDTHS = (128, 160, 192, 224, 256)
M = 256


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    with knobs(DG_2CTA="1", DG_SPLIT_TAIL="1", DG_LOG="1"):
        yield
    assert dg.dg_sync_status() == dg.DG_OK


def split_of(capfd):
    """(pairs, tiles left over, K ranges) of the last call, from its log line."""
    found = re.findall(r"on (\d+) pairs, the last (\d+) in (\d+) K ranges", capfd.readouterr().err)
    return tuple(int(v) for v in found[-1]) if found else None


def operands(N, K, fp16, seed):
    a, b = randn(seed, M, K), randn(seed + 1, N, K) / math.sqrt(K)
    if fp16:
        return a.half(), b.half(), None, None
    sa, sb = 0.5 + randn(seed + 2, M).abs(), (0.5 + randn(seed + 3, N).abs()) / math.sqrt(K)
    return a.to(F8).view(torch.uint8), (b * math.sqrt(K)).to(F8).view(torch.uint8), sa, sb


def wide(x):
    return x.view(F8).double() if x.dtype == torch.uint8 else x.double()


def pairs_of(capfd):
    """How many pairs run at once: from a launch that is split whatever it is."""
    slots = torch.cuda.get_device_properties(0).multi_processor_count // 2
    N, K = 256 * (slots + 8), 1024
    A, B, _, _ = operands(N, K, False, 0)
    one, D = torch.ones(1, device="cuda"), torch.empty(M, N, dtype=BF, device="cuda")
    capfd.readouterr()
    with knobs(DG_FORCE_BLOCK_N="256"):
        dg.dg_fp8_gemm(A, B, D, one, one)
    return split_of(capfd)[0]


@pytest.mark.parametrize("ranges", [2, 3, 4])
@pytest.mark.parametrize("bn", WIDTHS)
@pytest.mark.parametrize("kps", [1, 2])
@pytest.mark.parametrize("fp16", [False, True])
def test_widths(ranges, bn, kps, fp16, capfd):
    pairs = pairs_of(capfd)
    left = pairs // ranges
    assert left > 0 and min(pairs // left, 4) == ranges
    for edge in (8, 3):     # rows of whole 16-byte pieces (bulk stores), and others
        N, K = bn * (pairs + left) - edge, 1040
        A, B, sa, sb = operands(N, K, fp16, ranges)
        bias, residual = randn(7, N), randn(8, M, N).to(HALF)
        acc, size = wide(A) @ wide(B).T, wide(A).abs() @ wide(B).T.abs()
        whole = torch.full((M * N + 64,), 77, dtype=HALF, device="cuda")
        D = whole[:M * N].view(M, N)
        # FP32 sums of exact products, 16 or more to an instruction, a few more
        # additions between the ranges
        rel = 2.0 ** -23 * (K / 16 + 24)
        with knobs(DG_FORCE_BLOCK_N=str(bn), DG_PAIR_KPS=str(kps)):
            p = dg.dg_gemm_plan(M, N, K, dg.DG_FP16 if fp16 else dg.DG_E4M3, dg.DG_FP16)
            block = 64 if fp16 else 128
            assert (p["path"], p["block_m"], p["block_n"], p["block_k"]) == (3, 256, bn, block * kps), p
            one = torch.ones(1, device="cuda")
            capfd.readouterr()
            if fp16:
                dg.dg_hgemm(A, B, D, dg.DG_FP16)
            else:
                dg.dg_fp8_gemm(A, B, D, one, one * 0.5, out=dg.DG_FP16)
                acc, size = acc * 0.5, size * 0.5
            assert split_of(capfd) == (pairs, left, ranges)
            close(D, acc, size * rel + acc.abs() * STEP[HALF] + TINY[HALF], "plain")
            assert (whole[M * N:] == 77).all()
            if not fp16:
                acc, size = (t * 2 * sa.double()[:, None] * sb.double() for t in (acc, size))
            D.copy_(residual)
            kw = dict(bias=bias, act=dg.DG_ACT_RELU, out=dg.DG_FP16)
            if fp16:
                dg.dg_hgemm_fused(A, B, D, residual=D, **kw)
            else:
                dg.dg_fp8_gemm_fused(A, B, D, sa, sb, residual=D, **kw)
            assert split_of(capfd) == (pairs, left, ranges)
        acc, size = acc + bias.double(), size + bias.double().abs()
        want = act64(acc, dg.DG_ACT_RELU)[0] + residual.double()
        close(D, want, size * rel + want.abs() * (STEP[HALF] + 2.0 ** -23) + TINY[HALF], "fused")
        assert (whole[M * N:] == 77).all()


@pytest.mark.parametrize("ranges", [2, 4])
@pytest.mark.parametrize("bn", [128, 224])
def test_scales_beyond_fp32_in_a_split_tile(ranges, bn, capfd):
    """Scales that are applied in two steps, of a tile whose parts are added first."""
    pairs = pairs_of(capfd)
    left = pairs // ranges
    N, K = bn * (pairs + left) - 8, 1040
    A, B, sa, sb = operands(N, K, False, ranges)
    sa[::3] *= 2.0 ** -100
    sa[1::3] *= 2.0 ** 90
    sb[::2] *= 2.0 ** -80
    sb[1::4] *= 2.0 ** 30
    D = torch.zeros(M, N, dtype=BF, device="cuda")
    with knobs(DG_FORCE_BLOCK_N=str(bn)):
        capfd.readouterr()
        dg.dg_fp8_gemm_fused(A, B, D, sa, sb)
        assert split_of(capfd) == (pairs, left, ranges)
    ab = sa.double()[:, None] * sb.double()
    want = (wide(A) @ wide(B).T) * ab
    err = (wide(A).abs() @ wide(B).T.abs()) * ab * 2.0 ** -23 * (K / 16 + 24)
    close(D, want, err + want.abs() * STEP[BF] + 2.0 ** -133, "D")
    # rows and columns whose scale is more than its rest, under results that are normal numbers
    for far in ((sa < 2.0 ** -62) | (sa >= 2.0 ** 64)).view(-1, 1), ((sb < 2.0 ** -62) | (sb >= 2.0 ** 64)).view(1, -1):
        assert (far & (want.abs() > 2.0 ** -100)).any()
