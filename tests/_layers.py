"""FP64 definitions of the operators around a layer's products (norm,
activation, product with an epilogue) and the error bounds that their tests
share."""
from __future__ import annotations

import math

import torch

import fp16_tensor_core_gb300 as dg

BF, HALF = torch.bfloat16, torch.float16
DTYPES = [BF, HALF]
F8 = torch.float8_e4m3fn
MIN_SCALE = 2.0 ** -120

# FP32 arithmetic of a row: a sum of squares takes at most 64 serial additions
# a thread and 10 in the tree, half of which relative error a square root
# passes on, and a handful of roundings follow: 2^-24 (74 / 2 + 10) < 2^-18.
ROW = 2.0 ** -18
# A value rounded once: half a step, relative, and half the smallest subnormal.
STEP = {BF: 2.0 ** -8, HALF: 2.0 ** -11}
TINY = {BF: 2.0 ** -134, HALF: 2.0 ** -25}


def close(got, want, bound, what=""):
    got = got.double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= bound))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:5], want[bad][:5])


def rounded(want, dtype, rel=ROW):
    """Bound on a value of relative FP32 error `rel`, rounded to dtype."""
    return want.abs() * (STEP[dtype] + 2 * rel) + TINY[dtype]


def check_codes(q, scale, y, rel=ROW):
    """Codes and scales (per row of y, the last dimension) of FP64 values y that
    the kernel knows to a relative error `rel`."""
    want = torch.clamp_min(y.abs().amax(-1) / 448, MIN_SCALE)
    close(scale, want, want * (rel + 2.0 ** -23), "scale")
    v = y / want[..., None]
    # half a step of E4M3 (2^-4 relative, 2^-10 below its normal numbers)
    close(q.view(F8).reshape(y.shape), v, v.abs() * (2.0 ** -4 + 4 * rel) + 2.0 ** -10, "codes")


def act64(x, act):
    """The activation and its derivative, and the size of the derivative's terms."""
    one = torch.ones_like(x)
    if act == dg.DG_ACT_NONE:
        return x, one, one
    if act == dg.DG_ACT_RELU:
        return x.clamp_min(0), (x > 0).double(), one
    if act == dg.DG_ACT_GELU:
        phi = 0.5 * torch.special.erfc(-x / math.sqrt(2))
        pdf = torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        return x * phi, phi + x * pdf, phi + x.abs() * (pdf + 2.0 ** -7)
    if act == dg.DG_ACT_GELU_TANH:
        k = math.sqrt(8 / math.pi)
        u, du = k * (x + 0.044715 * x ** 3), k * (1 + 3 * 0.044715 * x ** 2)
    else:
        u, du = x, one
    g = torch.sigmoid(u)
    # 1 - g is formed from g: 2^-24 of 1, whatever is left
    return x * g, g + x * g * torch.sigmoid(-u) * du, g + x.abs() * du * g * (torch.sigmoid(-u) + 2.0 ** -7)


# The logistic forms: an exponential whose argument u is off by 2^-23 |u|, a
# reciprocal and products; |u| stays below 32 in the tests (x below 12, where
# the tanh form's u is larger but its value is x or 0 to FP32's last bits), so
# 2^-23 32 + 2^-20 < 2^-17.  GELU: exp(-x^2 / 2)
# with x^2 / 2 <= 72 of two roundings, 2^-23 72 < 2^-16.8, a polynomial of
# relative error 5.2e-7 < 2^-20.8 and a few roundings more: below 2^-16.
ACT = 2.0 ** -16
# Reciprocals below 2^-126 are 0: values below that times |x| <= 12 are lost.
ACT_TINY = 2.0 ** -122


def norm64(s, weight, eps):
    r = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return s * r * (1.0 if weight is None else weight)


def randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def view(x, pad):
    """x in rows `pad` elements longer, the rest NaN; and what lies behind the rows."""
    if pad == 0:
        return x, None
    whole = torch.full((x.shape[0], x.shape[1] + pad), math.nan, dtype=x.dtype, device="cuda")
    whole[:, :x.shape[1]] = x
    return whole[:, :x.shape[1]], whole[:, x.shape[1]:]
