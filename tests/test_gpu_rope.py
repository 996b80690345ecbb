"""dg_rope_table and dg_rope against FP64.

Table: one rounding to FP32 of an FP64 value whose angle is off by at most
p f 2^-52, so within 2^-24 + p 2^-50 of the exact cosine and sine.
Rotation: two FP32 products and a sum (3 * 2^-24 of |a| + |b|, times the
table's magnitude), then one rounding to the 16-bit type."""
import numpy as np
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _serving import ROUND, TORCH, f64, rope64, table64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def make_table(positions, rotary, **kw):
    t = torch.empty(positions, rotary // 2, 2, device="cuda")
    dg.dg_rope_table(t, **kw)
    return t


@pytest.mark.parametrize("positions,rotary,base", [(1, 16, 10000.0), (1000, 128, 10000.0),
                                                   (200_003, 64, 500_000.0), (77, 256, 10000.0)])
def test_table(positions, rotary, base):
    t = f64(make_table(positions, rotary, base=base))
    want = table64(positions, rotary, base)
    p = np.arange(positions)[:, None, None]
    assert np.all(np.abs(t - want) <= 2.0 ** -24 + p * 2.0 ** -50)


def test_table_scalings():
    r, L, s = 64, 4096.0, 8.0
    i = np.arange(r // 2)
    f = 10000.0 ** (-2.0 * i / r)
    p = np.arange(30_000, dtype=np.float64)[:, None]

    def check(freq, magnitude=1.0, **kw):
        t = f64(make_table(p.size, r, magnitude=magnitude, **kw))
        want = magnitude * np.stack((np.cos(p * freq), np.sin(p * freq)), axis=-1)
        assert np.all(np.abs(t - want) <= magnitude * (2.0 ** -23 + p[..., None] * 2.0 ** -48))

    check(f / s, scaling=dg.DG_ROPE_LINEAR, factor=s)
    check((10000.0 * s ** (r / (r - 2.0))) ** (-2.0 * i / r), scaling=dg.DG_ROPE_NTK, factor=s)
    turns = L * f / (2 * np.pi)
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    assert 0 < np.count_nonzero(keep == 1.0) < keep.size and np.any((keep > 0) & (keep < 1))
    check((1 - keep) * f / s + keep * f, scaling=dg.DG_ROPE_BY_PARTS, factor=s, original_positions=L,
          slow_rotations=1.0, fast_rotations=32.0, magnitude=1.2079441541679836)


def bound(x, table, positions, layout, inverse, dtype):
    want = rope64(x, table, positions, layout, inverse)
    half = table.shape[1]
    mag = np.abs(x)
    i = np.arange(half)
    a, b = (i, i + half) if layout == dg.DG_ROPE_HALF else (2 * i, 2 * i + 1)
    both = np.zeros_like(x)
    both[..., a] = both[..., b] = mag[..., a] + mag[..., b]
    top = max(1.0, np.abs(table).max())
    return want, ROUND[dtype] * 1.001 * np.abs(want) + 2.0 ** -22 * top * both + 2.0 ** -25


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
@pytest.mark.parametrize("layout", [dg.DG_ROPE_HALF, dg.DG_ROPE_INTERLEAVED])
@pytest.mark.parametrize("tokens,heads,dim,rotary,inverse", [
    (1, 1, 16, 16, False), (1, 40, 128, 128, False), (7, 3, 80, 32, True), (33, 5, 96, 96, False),
    (500, 32, 128, 64, True), (19, 8, 256, 256, False), (3, 70, 256, 48, False),
    (2000, 40, 64, 64, False),
])
def test_rope(tokens, heads, dim, rotary, inverse, layout, dtype):
    g = torch.Generator(device="cuda").manual_seed(tokens + dim)
    table = make_table(9000, rotary)
    x = torch.randn(tokens, heads, dim, generator=g, device="cuda").to(TORCH[dtype])
    pos = torch.randint(0, 9000, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 8999
    out = torch.full_like(x, 77.0)
    rotary_handle = dg.DgRotary(table, layout)
    dg.dg_rope(x, out, pos, rotary_handle, inverse=inverse)
    want, tol = bound(f64(x), f64(table), pos.cpu().numpy(), layout, inverse, dtype)
    assert np.all(np.abs(f64(out) - want) <= tol)
    assert torch.equal(out[..., rotary:], x[..., rotary:])      # the rest is copied
    dg.dg_rope(x, x, pos, rotary_handle, inverse=inverse)       # in place: the same bits
    assert torch.equal(x, out)


def test_strided_views_touch_nothing_else():
    """Queries inside a packed row turn in place; a transposed output."""
    t, h, d = 37, 6, 64
    table = make_table(100, 64)
    rows = torch.randn(t, 3 * h + 1, d, device="cuda").half()
    before = rows.clone()
    pos = torch.arange(t, device="cuda", dtype=torch.int32)
    r = dg.DgRotary(table)
    q = rows[:, h:2 * h]
    out = torch.zeros(h, t, d, device="cuda", dtype=torch.float16).transpose(0, 1)
    dg.dg_rope(q, out, pos, r)
    dg.dg_rope(q, q, pos, r)
    want, tol = bound(f64(before[:, h:2 * h]), f64(table), np.arange(t), dg.DG_ROPE_HALF, False, dg.DG_FP16)
    assert np.all(np.abs(f64(out) - want) <= tol)
    assert torch.equal(q, out)
    assert torch.equal(rows[:, :h], before[:, :h]) and torch.equal(rows[:, 2 * h:], before[:, 2 * h:])


@pytest.mark.parametrize("layout", [dg.DG_ROPE_HALF, dg.DG_ROPE_INTERLEAVED])
def test_gradient(layout):
    """inverse is the transposed map: checked against differences of the
    forward map (exact for a linear map but for its output rounding)."""
    t, h, d, r = 5, 2, 32, 32
    table = make_table(64, r, magnitude=1.5)
    rot = dg.DgRotary(table, layout)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(t, h, d, generator=g, device="cuda").half()
    grad = torch.randn(t, h, d, generator=g, device="cuda").half()
    pos = torch.tensor([0, 1, 7, 31, 63], dtype=torch.int32, device="cuda")
    y, gx = torch.empty_like(x), torch.empty_like(x)
    dg.dg_rope(x, y, pos, rot)
    dg.dg_rope(grad, gx, pos, rot, inverse=True)
    want, tol = bound(f64(grad), f64(table), pos.cpu().numpy(), layout, True, dg.DG_FP16)
    assert np.all(np.abs(f64(gx) - want) <= tol)
    for j in range(0, d, 5):
        moved, ym = x.clone(), torch.empty_like(x)
        moved[..., j] += 4.0
        step = f64(moved)[..., j] - f64(x)[..., j]
        dg.dg_rope(moved, ym, pos, rot)
        diff = np.sum((f64(ym) - f64(y)) * f64(grad), axis=-1) / step
        # two roundings of y per element that moved (a pair), values up to 1.5 * (|x| + 4)
        slack = 2 * 2.0 ** -11 * 12.0 * 2 * np.abs(f64(grad)).max() / 3.9
        assert np.all(np.abs(diff - f64(gx)[..., j]) <= slack)


def test_position_outside_the_table():
    table = make_table(10, 16)
    x = torch.randn(4, 2, 16, device="cuda").half()
    out = torch.full_like(x, 5.0)
    pos = torch.tensor([3, 10, -1, 9], dtype=torch.int32, device="cuda")
    dg.dg_rope(x, out, pos, dg.DgRotary(table))
    assert dg.dg_sync_status() == dg.DG_ERR_INVALID_VALUE
    assert torch.all(out[1:3] == 5.0)
    want, tol = bound(f64(x)[[0, 3]], f64(table), np.array([3, 9]), dg.DG_ROPE_HALF, False, dg.DG_FP16)
    assert np.all(np.abs(f64(out)[[0, 3]] - want) <= tol)


def test_infinities_and_nan_stay_in_their_pair():
    table = make_table(50, 32)
    x = torch.randn(2, 1, 32, device="cuda").to(torch.bfloat16)
    ref = torch.empty_like(x)
    pos = torch.tensor([4, 17], dtype=torch.int32, device="cuda")
    r = dg.DgRotary(table, dg.DG_ROPE_INTERLEAVED)
    dg.dg_rope(x, ref, pos, r)
    y = x.clone()
    y[0, 0, 6], y[1, 0, 9] = float("nan"), float("inf")
    out = torch.empty_like(y)
    dg.dg_rope(y, out, pos, r)
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[0, 0, 6:8] = touched[1, 0, 8:10] = True
    assert torch.equal(out[~touched], ref[~touched])
    assert not torch.isfinite(out[touched]).any()
