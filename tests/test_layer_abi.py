"""Refusals of the entry points around a layer's products (norm, activation,
fused products) at the C ABI and in Python: every argument error comes back
before anything touches a device.  CPU only."""
import ctypes
import math

import pytest
import torch

import fp16_tensor_core_gb300 as dg
from fp16_tensor_core_gb300 import build as dg_build

FAKE = 0x7F0000000000   # aligned, never dereferenced: every call below fails validation
BAD, OFF = dg.DG_ERR_INVALID_VALUE, dg.DG_ERR_MISALIGNED
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    dg_build.build()
    return dg.lib()


def rows(data=FAKE, stride=64):
    return dg._Rows(data, stride)


COMMON = [
    (dict(rows=-1), BAD), (dict(rows=1 << 31), BAD), (dict(cols=0), BAD), (dict(cols=32776), BAD),
    (dict(cols=60), OFF), (dict(dtype=dg.DG_E4M3), BAD), (dict(dtype=9), BAD),
]
NORM = COMMON + [
    (dict(x=None), BAD), (dict(x=rows(None)), BAD), (dict(x=rows(FAKE + 8)), OFF), (dict(x=rows(stride=68)), OFF),
    (dict(x=rows(stride=-64)), BAD), (dict(residual=rows(FAKE + 2)), OFF), (dict(residual=rows(None)), BAD),
    (dict(sum=rows(FAKE, 4)), OFF), (dict(sum=rows(FAKE, 56)), BAD), (dict(weight=FAKE + 8), OFF),
    (dict(eps=0.0), BAD), (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD), (dict(eps=math.inf), BAD),
    (dict(eps=2.0 ** -127), BAD), (dict(sum=rows(FAKE, 128)), BAD),
    (dict(residual=rows(FAKE + 4096, 0), sum=rows(FAKE + 4096, 64)), BAD),
]


def norm_args(kw):
    a = dict(x=rows(), residual=None, sum=None, weight=None, rows=4, cols=64, eps=1e-6, dtype=dg.DG_BF16)
    a.update({k: v for k, v in kw.items() if k in a})
    return [a[k] for k in ("x", "residual", "sum", "weight", "rows", "cols", "eps", "dtype")]


@pytest.mark.parametrize("kw,expect", NORM + [
    (dict(y=None), BAD), (dict(y=rows(FAKE + 4)), OFF), (dict(y=rows(stride=32)), BAD),
    (dict(sum=rows(FAKE), y=rows(FAKE)), BAD), (dict(y=rows(FAKE, 72)), BAD),
    (dict(residual=rows(FAKE + 64, 0), y=rows(FAKE + 64)), BAD),
])
def test_rmsnorm(L, kw, expect):
    assert L.dg_rmsnorm(*norm_args(kw), kw.get("y", rows(FAKE + 4096)), None) == expect


@pytest.mark.parametrize("kw,expect", NORM + [
    (dict(q=None), BAD), (dict(scale=None), BAD), (dict(q=FAKE + 8), OFF), (dict(scale=FAKE + 2), OFF),
])
def test_rmsnorm_e4m3(L, kw, expect):
    assert L.dg_rmsnorm_e4m3(*norm_args(kw), kw.get("q", FAKE), kw.get("scale", FAKE), None) == expect


@pytest.mark.parametrize("kw,expect", NORM + [
    (dict(q=None), BAD), (dict(scale=None), BAD), (dict(amax=None), BAD), (dict(q=FAKE + 8), OFF),
    (dict(scale=FAKE + 2), OFF), (dict(amax=FAKE + 1), OFF), (dict(next=FAKE + 2), OFF), (dict(amax=FAKE), BAD),
    (dict(next=FAKE + 64), BAD),
])
def test_rmsnorm_e4m3_amax(L, kw, expect):
    assert L.dg_rmsnorm_e4m3_amax(*norm_args(kw), kw.get("scale", FAKE), kw.get("q", FAKE),
                                  kw.get("amax", FAKE + 64), kw.get("next", FAKE + 128), None) == expect


@pytest.mark.parametrize("kw,expect", COMMON + [
    (dict(x=None), BAD), (dict(x=rows(FAKE + 8)), OFF), (dict(dy=None), BAD), (dict(dy=rows(stride=12)), OFF),
    (dict(dsum=rows(FAKE + 2)), OFF), (dict(dx=None), BAD), (dict(dx=rows(stride=0)), BAD), (dict(eps=0.0), BAD),
    (dict(dy=rows(FAKE, 0)), BAD), (dict(x=rows(FAKE, 72)), BAD), (dict(dsum=rows(FAKE, 72)), BAD),
    (dict(weight=FAKE + 8), OFF), (dict(dweight=FAKE, scratch=None), BAD), (dict(dweight=FAKE + 4), OFF),
    (dict(dweight=FAKE, scratch=FAKE + 4), OFF),
])
def test_rmsnorm_grad(L, kw, expect):
    a = dict(x=rows(), weight=None, dy=rows(), dsum=None, rows=4, cols=64, eps=1e-6, dtype=dg.DG_FP16, dx=rows(),
             dweight=None, scratch=FAKE, bytes=BIG)
    a.update(kw)
    assert L.dg_rmsnorm_grad(*a.values(), None) == expect


@pytest.mark.parametrize("kw,expect", COMMON + [
    (dict(act=-1), BAD), (dict(act=5), BAD), (dict(x=None), BAD), (dict(x=rows(stride=4)), OFF),
    (dict(y=rows(FAKE + 8)), OFF), (dict(y=rows(stride=40)), BAD), (dict(q=FAKE), BAD), (dict(q_scale=FAKE), BAD),
    (dict(x_q=FAKE), BAD), (dict(q=FAKE + 8, q_scale=FAKE), OFF), (dict(x_q=FAKE, x_scale=FAKE + 2), OFF),
    (dict(gated=1, x=rows(FAKE, 128), y=rows(FAKE, 128)), BAD), (dict(x=rows(FAKE, 0), y=rows(FAKE)), BAD),
])
def test_activate(L, kw, expect):
    a = dict(x=rows(), gated=0, act=dg.DG_ACT_SILU, rows=4, cols=64, dtype=dg.DG_BF16, y=rows(FAKE + 4096), q=None,
             q_scale=None, x_q=None, x_scale=None)
    a.update(kw)
    assert L.dg_activate(*a.values(), None) == expect


@pytest.mark.parametrize("kw,expect", COMMON + [
    (dict(act=7), BAD), (dict(dy=None), BAD), (dict(x=None), BAD), (dict(x=None, x_q=FAKE), BAD),
    (dict(x_q=FAKE, x_scale=FAKE), BAD), (dict(x=None, x_q=FAKE + 4, x_scale=FAKE), OFF), (dict(dx=None), BAD),
    (dict(dx=rows(stride=40)), BAD), (dict(gated=1), BAD), (dict(dbias=FAKE, scratch=None), BAD),
    (dict(gated=1, x=rows(FAKE, 128), dx=rows(FAKE, 128)), BAD), (dict(dy=rows(FAKE, 0)), BAD),
    (dict(x=rows(FAKE, 72)), BAD), (dict(gated=1, dy=rows(FAKE + 64), x=rows(FAKE, 0), dx=rows(FAKE, 128)), BAD),
    (dict(dbias=FAKE + 4), OFF), (dict(scratch=FAKE + 8), OFF),
])
def test_activate_grad(L, kw, expect):
    a = dict(dy=rows(), x=rows(), x_q=None, x_scale=None, gated=0, act=dg.DG_ACT_GELU, rows=4, cols=64,
             dtype=dg.DG_BF16, dx=rows(), dbias=None, scratch=FAKE, bytes=BIG)
    a.update(kw)
    assert L.dg_activate_grad(*a.values(), None) == expect


def test_scratch_sizes(L):
    n = ctypes.c_int64()
    assert L.dg_rmsnorm_grad_scratch(4, 64, 152, None) == BAD
    assert L.dg_rmsnorm_grad_scratch(-1, 64, 152, ctypes.byref(n)) == BAD
    assert L.dg_activate_grad_scratch(4, 60, 0, 152, ctypes.byref(n)) == OFF
    assert L.dg_rmsnorm_grad_scratch(0, 64, 152, ctypes.byref(n)) == dg.DG_OK and n.value == 0
    # a partial sum of the columns a block, and no block without a row
    assert L.dg_rmsnorm_grad_scratch(3, 64, 152, ctypes.byref(n)) == dg.DG_OK and 64 * 4 <= n.value <= 3 * 64 * 4
    assert L.dg_activate_grad_scratch(3, 64, 1, 152, ctypes.byref(n)) == dg.DG_OK and 128 * 4 <= n.value <= 3 * 128 * 4
    # no more than the SMs need, however many rows
    assert L.dg_rmsnorm_grad_scratch(1 << 30, 4096, 152, ctypes.byref(n)) == dg.DG_OK and n.value < 1 << 25


def epilogue(**kw):
    a = dict(scale_a=FAKE, scale_b=FAKE, scale_a_rows=0, scale_b_rows=0, bias=None, act=0, residual=None,
             residual_type=dg.DG_BF16, scale_d=None, amax_d=None)
    a.update(kw)
    return dg._Epilogue(*a.values())


EPILOGUE = [
    (dict(e=None), BAD), (dict(e=epilogue(act=5)), BAD), (dict(e=epilogue(scale_a=None)), BAD),
    (dict(e=epilogue(scale_a=FAKE + 2)), OFF), (dict(e=epilogue(scale_a=FAKE + 4, scale_a_rows=1)), OFF),
    (dict(e=epilogue(scale_b=FAKE + 8, scale_b_rows=1)), OFF), (dict(e=epilogue(bias=FAKE + 4)), OFF),
    (dict(e=epilogue(residual=FAKE + 8)), OFF), (dict(e=epilogue(residual=FAKE + 64, residual_type=1)), BAD),
    (dict(e=epilogue(residual=FAKE, residual_type=dg.DG_FP16)), BAD), (dict(e=epilogue(amax_d=FAKE + 1)), OFF),
    (dict(e=epilogue(amax_d=FAKE)), BAD), (dict(e=epilogue(scale_b_rows=1, amax_d=FAKE + 4 * 31)), BAD),
    (dict(e=epilogue(scale_a_rows=1, amax_d=FAKE + 12)), BAD), (dict(e=epilogue(bias=FAKE + 256, amax_d=FAKE + 260)), BAD),
    (dict(M=-1), BAD), (dict(N=1 << 31), BAD), (dict(A=None), BAD), (dict(D=None), BAD), (dict(A=FAKE + 8), OFF),
    (dict(K=36), OFF), (dict(out=7), BAD),
]


@pytest.mark.parametrize("kw,expect", EPILOGUE + [
    (dict(e=epilogue(scale_a=None, scale_b=None)), BAD), (dict(out=dg.DG_E4M3), BAD),
    (dict(out=dg.DG_E4M3, e=epilogue(scale_d=FAKE + 2)), OFF),
    (dict(out=dg.DG_E4M3, e=epilogue(scale_d=FAKE, amax_d=FAKE)), BAD),
    (dict(out=dg.DG_E4M3, e=epilogue(scale_d=FAKE, residual=FAKE)), BAD),
    (dict(K=0, out=dg.DG_E4M3), BAD), (dict(K=8), OFF),
])
def test_fp8_gemm_fused(L, kw, expect):
    a = dict(A=FAKE, B=FAKE, D=FAKE, M=4, N=32, K=64, e=epilogue(), out=dg.DG_BF16)
    a.update(kw)
    assert L.dg_fp8_gemm_fused(*a.values(), None) == expect


@pytest.mark.parametrize("kw,expect", EPILOGUE + [
    (dict(out=dg.DG_E4M3, e=epilogue(scale_d=FAKE)), BAD),
    (dict(e=epilogue(scale_a=None, scale_b=None, scale_a_rows=1)), BAD),
])
def test_hgemm_fused(L, kw, expect):
    a = dict(A=FAKE, B=FAKE, D=FAKE, M=4, N=32, K=64, e=epilogue(), out=dg.DG_BF16)
    a.update(kw)
    assert L.dg_hgemm_fused(*a.values(), None) == expect


BF = torch.bfloat16


@pytest.mark.parametrize("call", [
    lambda x, q, s: dg.dg_rmsnorm(x, x), lambda x, q, s: dg.dg_rmsnorm_e4m3(x, q, s),
    lambda x, q, s: dg.dg_rmsnorm_e4m3_amax(x, s, q, s), lambda x, q, s: dg.dg_rmsnorm_grad(x, x, x),
    lambda x, q, s: dg.dg_activate(x, dg.DG_ACT_SILU, y=x), lambda x, q, s: dg.dg_activate_grad(x, 4, x, x=x),
    lambda x, q, s: dg.dg_fp8_gemm_fused(q, q, x, s, s), lambda x, q, s: dg.dg_hgemm_fused(x, x, x)])
def test_host_tensors(L, call):
    with pytest.raises(ValueError, match="CUDA device memory"):
        call(torch.zeros(4, 64, dtype=BF), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4))


def test_shapes_and_types_in_python(L):
    for x in (torch.zeros(4, 64), torch.zeros(64, dtype=BF), torch.zeros(4, 128, dtype=BF)[:, ::2],
              torch.zeros(2, 4, 64, dtype=BF)):
        with pytest.raises(ValueError, match="x must be BF16 or FP16"):
            dg.dg_rmsnorm(x, x)
    with pytest.raises(AttributeError):
        dg.dg_rmsnorm(None, None)
    with pytest.raises(TypeError):
        dg.dg_activate(torch.zeros(4, 64, dtype=BF), "silu")


def test_the_native_functions_count_their_arguments(L):
    native = dg._load_native()
    for f in (native.rmsnorm, native.rmsnorm_e4m3, native.rmsnorm_e4m3_amax, native.rmsnorm_grad, native.activate,
              native.activate_grad, native.fp8_gemm_fused, native.hgemm_fused, native.bind_layer):
        with pytest.raises(TypeError, match="arguments wanted"):
            f()
        with pytest.raises(TypeError, match="arguments wanted"):
            f(*range(20))
