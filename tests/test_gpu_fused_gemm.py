"""Products with scales per row, bias, activation and residual in their
epilogue against FP64, on every kernel that the planner can pick."""
import math

import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _knobs import knobs
from _layers import ACT, ACT_TINY, BF, F8, HALF, STEP, TINY, act64, close, randn

pytestmark = pytest.mark.gpu
OUT = {dg.DG_BF16: BF, dg.DG_FP16: HALF, dg.DG_E4M3: torch.uint8}
ACTS = [dg.DG_ACT_NONE, dg.DG_ACT_RELU, dg.DG_ACT_GELU, dg.DG_ACT_GELU_TANH, dg.DG_ACT_SILU]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def operands(M, N, K, fp16, rows, seed):
    a, b = randn(seed, M, K) * 2, randn(seed + 1, N, K)
    if fp16:
        scales = None, None
        if rows is not None:
            scales = (0.5 + randn(seed + 2, M if rows else 1).abs(), (0.5 + randn(seed + 3, N if rows else 1).abs()) /
                      math.sqrt(max(K, 1)))
        return a.half(), (b if rows is not None else b / math.sqrt(max(K, 1))).half(), *scales
    sa = 0.02 + randn(seed + 2, M if rows else 1).abs() * 0.05
    sb = (0.02 + randn(seed + 3, N if rows else 1).abs() * 0.05) / math.sqrt(max(K, 1))
    return (30 * a).to(F8).view(torch.uint8), (30 * b).to(F8).view(torch.uint8), sa, sb


def wide(x):
    return x.view(F8).double() if x.dtype == torch.uint8 else x.double()


def check(M, N, K, fp16=False, out=dg.DG_BF16, act=dg.DG_ACT_NONE, rows=True, bias=True, residual=BF, seed=0,
          in_place=False):
    A, B, sa, sb = operands(M, N, K, fp16, rows, seed)
    b = randn(seed + 4, N) if bias else None
    r = None if residual is None else randn(seed + 5, M, N).to(residual)
    kw = dict(bias=b, act=act, residual=r, out=out)
    acc, size = wide(A) @ wide(B).T, wide(A).abs() @ wide(B).T.abs()
    if sa is not None:
        scale = sa.double().reshape(-1, 1) * sb.double().reshape(1, -1)
        acc, size = acc * scale, size * scale
    if bias:
        acc, size = acc + b.double(), size + b.double().abs()
    # FP32 sums of exact products, at least 16 of them to an instruction: K / 16
    # additions in a row and a few more between warps or CTAs, 2^-23 each
    err = size * (2.0 ** -23 * (K / 16 + 24))
    value = act64(acc, act)[0]
    want = value + (0 if r is None else r.double())
    err = 1.2 * err + value.abs() * ACT + ACT_TINY + want.abs() * 2.0 ** -23    # (|act'| < 1.2)
    whole = torch.full((M * N + 64,), 77, dtype=OUT[out], device="cuda")        # what lies behind D stays
    D = whole[:M * N].view(M, N)
    if out == dg.DG_E4M3:
        sd = torch.full((1,), float(want.abs().amax()) / 300 if want.numel() else 1.0, device="cuda")
        amax = torch.full((1,), -1.0, device="cuda")
        dg.dg_fp8_gemm_fused(A, B, D, sa, sb, scale_d=sd, amax_d=amax, **kw)
        v = (want / sd.double()).clamp(-448, 448)
        close(D.view(F8), v, v.abs() * 2.0 ** -4 + 2.0 ** -10 + 1.1 * err / sd.double(), "codes")
        top = want.abs().amax().reshape(1) if want.numel() else torch.zeros(1, device="cuda")
        close(amax, top, err.amax().reshape(1) if err.numel() else top, "amax")
    else:
        if in_place:
            D.copy_(r)
            kw["residual"] = D
        if fp16:
            dg.dg_hgemm_fused(A, B, D, scale_a=sa, scale_b=sb, **kw)
        else:
            dg.dg_fp8_gemm_fused(A, B, D, sa, sb, **kw)
        close(D, want, err + want.abs() * STEP[OUT[out]] + TINY[OUT[out]], "D")
    assert (whole[M * N:] == 77).all()
    return D


SHAPES = [(1, 1000, 1040), (1, 40000, 256), (4, 4096, 4096), (8, 300, 512), (13, 1000, 1040), (16, 12288, 4096),
          (9, 1000, 4368), (33, 4096, 11008), (64, 999, 2048), (128, 2000, 4096), (129, 1000, 1040), (130, 203, 272),
          (300, 777, 272), (640, 1536, 2048), (1024, 4096, 512), (700, 5000, 1552), (3, 5, 16), (1, 1, 16)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fp16,out,act,residual", [
    (False, dg.DG_BF16, dg.DG_ACT_NONE, BF), (False, dg.DG_E4M3, dg.DG_ACT_GELU, None),
    (False, dg.DG_FP16, dg.DG_ACT_RELU, BF), (True, dg.DG_FP16, dg.DG_ACT_SILU, HALF),
    (True, dg.DG_BF16, dg.DG_ACT_GELU_TANH, None)])
def test_shapes(M, N, K, fp16, out, act, residual):
    check(M, N, K, fp16, out, act, True, True, residual, seed=M)


@pytest.mark.parametrize("M,N,K", [(3, 520, 256), (20, 520, 256), (150, 520, 256), (520, 1040, 1024)])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,bias,residual", [(False, False, None), (False, True, HALF), (True, False, BF)])
@pytest.mark.parametrize("fp16", [False, True])
def test_forms(M, N, K, act, rows, bias, residual, fp16):
    check(M, N, K, fp16, dg.DG_FP16, act, rows, bias, residual)
    if fp16:
        check(M, N, K, True, dg.DG_BF16, act, None, bias, residual)     # no scales
    else:
        check(M, N, K, False, dg.DG_E4M3, act, rows, bias, residual)


@pytest.mark.parametrize("env", [
    dict(DG_STAGED_EPI="0"), dict(DG_SPLITK="1"), dict(DG_SPLITK="0"), dict(DG_MMA_GEMV="0"), dict(DG_2CTA="1"),
    dict(DG_2CTA="0"), dict(DG_2CTA="1", DG_SPLIT_TAIL="1"), dict(DG_2CTA="1", DG_STREAM_K="1"),
    dict(DG_SPLITK="1", DG_SPLITK_ROWS="1"), dict(DG_FORCE_BLOCK_N="96"), dict(DG_FORCE_BLOCK_N="224", DG_2CTA="0")])
@pytest.mark.parametrize("M,N,K", [(2, 1000, 1040), (16, 2000, 2048), (50, 2000, 2048), (128, 1999, 1040),
                                   (300, 3000, 2048), (2500, 5003, 1600)])
def test_every_kernel(env, M, N, K):
    with knobs(**env):
        check(M, N, K, False, dg.DG_BF16, dg.DG_ACT_SILU, True, True, BF)
        check(M, N, K, False, dg.DG_E4M3, dg.DG_ACT_NONE, True, True, HALF)
        check(M, N, K, True, dg.DG_FP16, dg.DG_ACT_RELU, False, False, HALF)


@pytest.mark.parametrize("M,N,K", [(1, 1000, 1040), (16, 4096, 4096), (100, 4096, 4096), (129, 1000, 1040),
                                   (640, 1536, 2048), (300, 777, 272)])
def test_into_the_residual(M, N, K):
    for fp16, out in ((False, dg.DG_BF16), (True, dg.DG_FP16)):
        kw = dict(fp16=fp16, out=out, act=dg.DG_ACT_GELU, residual=OUT[out])
        assert torch.equal(check(M, N, K, **kw), check(M, N, K, in_place=True, **kw))


@pytest.mark.parametrize("M,N", [(1, 40), (70, 1001)])
@pytest.mark.parametrize("out,residual", [(dg.DG_BF16, BF), (dg.DG_FP16, None), (dg.DG_E4M3, HALF)])
def test_empty_sums(M, N, out, residual):
    check(M, N, 0, False, out, dg.DG_ACT_GELU, True, True, residual)
    check(M, N, 0, False, out, dg.DG_ACT_SILU, False, False, BF)
    if out != dg.DG_E4M3:
        check(M, N, 0, True, out, dg.DG_ACT_NONE, None, True, residual)


def test_no_outputs():
    z = torch.zeros(0, 32, dtype=torch.uint8, device="cuda")
    b = torch.zeros(48, 32, dtype=torch.uint8, device="cuda")
    one, amax = torch.ones(1, device="cuda"), torch.ones(1, device="cuda")
    dg.dg_fp8_gemm_fused(z, b, torch.zeros(0, 48, dtype=BF, device="cuda"), one, one, amax_d=amax)
    assert amax == 0


def test_as_the_plain_product():
    """Without more in its epilogue: the plain product, to its last rounding."""
    for M, N, K in ((1, 1000, 1040), (16, 12288, 4096), (129, 1000, 1040), (640, 1536, 2048)):
        A, B, sa, sb = operands(M, N, K, False, False, 3)
        D, E = torch.zeros(M, N, dtype=BF, device="cuda"), torch.zeros(M, N, dtype=BF, device="cuda")
        dg.dg_fp8_gemm(A, B, D, sa, sb)
        dg.dg_fp8_gemm_fused(A, B, E, sa, sb)
        assert torch.equal(D, E)


@pytest.mark.parametrize("M,N,K", [(5, 520, 256), (40, 4096, 4096), (200, 520, 256), (520, 1040, 1024)])
def test_nan_stays_in_its_row(M, N, K):
    """A row of scale NaN (from a norm of a NaN) spoils its row of D and no other."""
    A, B, sa, sb = operands(M, N, K, False, True, 1)
    D, E = torch.zeros(M, N, dtype=BF, device="cuda"), torch.zeros(M, N, dtype=BF, device="cuda")
    dg.dg_fp8_gemm_fused(A, B, D, sa, sb, act=dg.DG_ACT_RELU)
    sa[M // 2] = math.nan
    A[M // 2] = 0x7F
    amax, codes = torch.zeros(1, device="cuda"), torch.zeros(M, N, dtype=torch.uint8, device="cuda")
    dg.dg_fp8_gemm_fused(A, B, E, sa, sb, act=dg.DG_ACT_RELU)
    assert E[M // 2].isnan().all()
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(D[keep], E[keep])
    dg.dg_fp8_gemm_fused(A, B, codes, sa, sb, act=dg.DG_ACT_RELU, scale_d=torch.ones(1, device="cuda"), amax_d=amax,
                         out=dg.DG_E4M3)
    assert (codes[M // 2] == 0x7F).all() and amax.isnan().all()


@pytest.mark.parametrize("scale", [1e-40, 2.0 ** -126, 2.0 ** 126, 0.0, math.inf, math.nan])
def test_output_scales_of_every_size(scale):
    for M in (2, 20, 200, 600):
        A, B, sa, sb = operands(M, 264, 256, False, True, 5)
        A[0] = 0
        codes = torch.zeros(M, 264, dtype=torch.uint8, device="cuda")
        sd = torch.full((1,), scale, device="cuda")
        dg.dg_fp8_gemm_fused(A, B, codes, sa, sb, scale_d=sd, out=dg.DG_E4M3)
        v = (wide(A) @ wide(B).T) * sa.double()[:, None] * sb.double()
        size = (wide(A).abs() @ wide(B).T.abs()) * sa.double()[:, None] * sb.double()
        bound = (size * 2.0 ** -18 / sd.double()).nan_to_num(0, 0, 0)
        want = (v / sd.double()).clamp(-448, 448)
        near = want.abs() < 448        # (a value may saturate on one side only)
        close(codes.view(F8).double()[near | want.isnan()], want[near | want.isnan()],
              (want.abs() * 2.0 ** -4 + 2.0 ** -10 + bound)[near | want.isnan()])


def test_refusals():
    A, B, sa, sb = operands(4, 32, 64, False, True, 0)
    D, one = torch.zeros(4, 32, dtype=BF, device="cuda"), torch.ones(1, device="cuda")
    codes = torch.zeros(4, 32, dtype=torch.uint8, device="cuda")
    for call, match in [
            (lambda: dg.dg_fp8_gemm_fused(A, B[:, :48].contiguous(), D, sa, sb), "must agree"),
            (lambda: dg.dg_fp8_gemm_fused(A, B, D[:3], sa, sb), "must agree"),
            (lambda: dg.dg_fp8_gemm_fused(A, B, codes, sa, sb), "must agree"),
            (lambda: dg.dg_fp8_gemm_fused(A.half(), B.half(), D, sa, sb), "must agree"),
            (lambda: dg.dg_hgemm_fused(A, B, D), "must agree"),
            (lambda: dg.dg_hgemm_fused(A.to(BF), B.to(BF), D, out=dg.DG_BF16), "must agree"),
            (lambda: dg.dg_fp8_gemm_fused(A, B, D, sa, sb, out=dg.DG_FP16), "must agree"),
            (lambda: dg.dg_fp8_gemm_fused(A, B, D, sa[:3], sb), "scale_a must be FP32 with 4"),
            (lambda: dg.dg_fp8_gemm_fused(A, B, D, sa, sb[:5]), "scale_b must be FP32 with 32"),
            (lambda: dg.dg_fp8_gemm_fused(A, B, D, sa, sb, bias=sb.half()), "bias must be FP32"),
            (lambda: dg.dg_fp8_gemm_fused(A, B, D, sa, sb, residual=D.float()), "residual must be BF16 or FP16"),
            (lambda: dg.dg_fp8_gemm_fused(A, B, D, sa, sb, residual=D[:, :16].contiguous()), "shape of D"),
            (lambda: dg.dg_fp8_gemm_fused(A, B.T, D, sa, sb), "contiguous"),
            (lambda: dg.dg_fp8_gemm_fused(A[0], B, D, sa, sb), "two dimensions")]:
        with pytest.raises(ValueError, match=match):
            call()
    for call in (lambda: dg.dg_fp8_gemm_fused(A, B, D, sa, None), lambda: dg.dg_fp8_gemm_fused(A, B, D, sa, sb, act=9),
                 lambda: dg.dg_fp8_gemm_fused(A, B, codes, sa, sb, out=dg.DG_E4M3),
                 lambda: dg.dg_fp8_gemm_fused(A, B, codes, sa, sb, out=dg.DG_E4M3, scale_d=one, amax_d=one),
                 lambda: dg.dg_fp8_gemm_fused(A, B, D, sa, sb, residual=D.view(HALF), out=dg.DG_BF16),
                 lambda: dg.dg_hgemm_fused(A.half(), B.half(), D, scale_a=sa, out=dg.DG_BF16)):
        with pytest.raises(dg.DgError):
            call()


def test_graph_and_streams():
    for M, N, K in ((4, 4096, 4096), (16, 4096, 4096), (200, 1000, 1040), (640, 1536, 2048)):
        A, B, sa, sb = operands(M, N, K, False, True, 2)
        D, b = torch.zeros(M, N, dtype=BF, device="cuda"), randn(1, N)
        codes, amax, sd = torch.zeros(M, N, dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda"), torch.ones(
            1, device="cuda")

        def calls(stream=None):
            dg.dg_fp8_gemm_fused(A, B, D, sa, sb, bias=b, act=dg.DG_ACT_SILU, residual=D, stream=stream)
            dg.dg_fp8_gemm_fused(A, B, codes, sa, sb, bias=b, scale_d=sd, amax_d=amax, out=dg.DG_E4M3, stream=stream)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            calls()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            calls()
        D.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        replayed = [D.clone(), codes.clone(), amax.clone()]
        D.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            calls(stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(replayed, (D, codes, amax)))
        dg.dg_release_stream(side)


@pytest.mark.parametrize("N", [33024, 33001])
def test_offsets_past_32_bits(N):
    """The last rows of an output of more than 2^31 elements, onto a residual."""
    M, K = 66000, 64
    A, B, sa, sb = operands(M, N, K, False, True, 6)
    D, bias, few = torch.empty(M, N, dtype=BF, device="cuda"), randn(1, N), slice(M - 40, M)
    D[few] = randn(2, 40, N).to(BF)
    alone = D[few].clone()
    dg.dg_fp8_gemm_fused(A, B, D, sa, sb, bias=bias, act=dg.DG_ACT_SILU, residual=D)
    want = (wide(A[few]) @ wide(B).T) * sa[few].double()[:, None] * sb.double() + bias.double()
    size = (wide(A[few]).abs() @ wide(B).T.abs()) * sa[few].double()[:, None] * sb.double() + bias.double().abs()
    want = act64(want, dg.DG_ACT_SILU)[0] + alone.double()
    close(D[few], want, 1.2 * size * 2.0 ** -18 + want.abs() * (STEP[BF] + 2.0 ** -22) + size * ACT + ACT_TINY, "D")
