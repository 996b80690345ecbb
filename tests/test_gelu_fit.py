"""The polynomial behind GELU's tail, with the coefficients as the kernels hold
them: FP32 steps, and a reciprocal off by its instruction's 2^-23 either way,
against the scaled complementary error function.  CPU only."""
import os
import re

import numpy as np
import pytest

from fp16_tensor_core_gb300 import build as dg_build

special = pytest.importorskip("scipy.special")
BOUND = 2.0 ** -20      # what activation.cuh states


def coefficients():
    with open(os.path.join(dg_build.CSRC, "activation.cuh")) as f:
        body = f.read().split("gelu_tail(pair magnitude", 1)[1].split("return", 1)[0]
    values = [np.float32(v) for v in re.findall(r"pair_of\((-?[0-9.e-]+)f\)", body)]
    slope, one, *poly = values
    assert one == 1.0 and len(poly) == 8
    return slope, poly


@pytest.mark.parametrize("off", [-2.0 ** -23, 0.0, 2.0 ** -23])
def test_relative_error(off):
    slope, poly = coefficients()
    a = np.linspace(0, 14, 2_000_001).astype(np.float32).astype(np.float64)
    step = lambda x: x.astype(np.float32).astype(np.float64)     # noqa: E731
    t = step((1 + off) / step(a * np.float64(slope) + 1))
    p = step(t * np.float64(poly[0]) + np.float64(poly[1]))
    for c in poly[2:]:
        p = step(p * t + np.float64(c))
    want = special.erfcx(a / np.sqrt(2)) / 2
    worst = np.abs(p / want - 1).max()
    assert worst < BOUND, worst
