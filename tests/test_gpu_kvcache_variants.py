"""dg_kv_append over the widths, rotated parts and sizes at which its split
over lanes and blocks changes; checks and bounds of test_gpu_kvcache."""
import numpy as np
import pytest
import torch

import fp16_tensor_core_gb300 as dg
import test_gpu_kvcache as kv
from _serving import TORCH, cached, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
@pytest.mark.parametrize("layout", [dg.DG_ROPE_HALF, dg.DG_ROPE_INTERLEAVED])
@pytest.mark.parametrize("tokens,q_heads,heads,dim,rotary,page,pages", [
    (5, 2, 1, 16, 16, 8, 1), (9, 3, 2, 256, 16, 4, 4), (33, 1, 3, 208, 112, 16, 3), (70, 4, 5, 256, 256, 32, 3),
    (3000, 4, 8, 128, 128, 64, 48), (5000, 2, 2, 64, 32, 16, 400), (2500, 3, 3, 240, 160, 8, 400),
    (1300, 40, 20, 128, 64, 128, 11), (6001, 1, 1, 32, 32, 16, 400),
])
def test_rotated_rows(tokens, q_heads, heads, dim, rotary, page, pages, layout, dtype):
    kv.test_append_packed_rows_with_rotation(tokens, q_heads, heads, dim, rotary, page, pages, layout, dtype)


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
@pytest.mark.parametrize("tokens,heads,dim,page,pages", [
    (7, 1, 16, 4, 2), (4000, 1, 48, 16, 260), (2600, 5, 128, 32, 90), (5000, 2, 64, 64, 80), (1500, 9, 256, 16, 100),
    (700, 64, 112, 8, 90),
])
def test_plain_rows(tokens, heads, dim, page, pages, dtype):
    kv.test_append_without_rotation_is_bit_exact(tokens, heads, dim, page, pages, dtype)


@pytest.mark.parametrize("layout", [dg.DG_ROPE_HALF, dg.DG_ROPE_INTERLEAVED])
@pytest.mark.parametrize("tokens", [6, 4000])
def test_a_special_value_spoils_its_row_alone(tokens, layout):
    """NaN and infinity in any lane, turned or not, of small and large calls."""
    heads, dim, rotary = 3, 96, 64
    k = torch.randn(tokens, heads, dim, device="cuda").to(TORCH[dg.DG_BF16])
    v = k.clone()
    t = torch.empty(tokens + 1, rotary // 2, 2, device="cuda")
    dg.dg_rope_table(t)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    rot = dg.DgRotary(t, layout)
    cache, bad = (make_cache(-(-tokens // 16), heads, 16, dim) for _ in range(2))
    dg.dg_kv_append(k, v, pos, cache, positions=pos, rotary=rot)
    spots = [(1, 0, 5, "nan"), (2, 1, 40, "inf"), (4, 2, 95, "-inf"), (tokens - 1, 0, 64, "nan")]
    for token, head, d, what in spots:
        k[token, head, d] = float(what)
        v[token, 2 - head, d] = float(what)
    dg.dg_kv_append(k, v, pos, bad, positions=pos, rotary=rot)
    slots = np.arange(tokens)
    for i in (2, 3):                                        # codes of keys and of values
        want, got = cached(cache, slots)[i], cached(bad, slots)[i]
        for token, head, _, _ in spots:
            h = head if i == 2 else 2 - head
            assert not got[token, h].any()
            got[token, h] = want[token, h]
        assert np.array_equal(want, got)
    for i in (4, 5):                                        # scales
        want, got = cached(cache, slots)[i], cached(bad, slots)[i]
        for token, head, _, _ in spots:
            h = head if i == 4 else 2 - head
            assert np.isnan(got[token, h])
            got[token, h] = want[token, h]
        assert np.array_equal(want, got)
