"""Sizes of dg_attn_decode whose products pass 32 bits."""
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _serving import make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def test_an_empty_request_of_more_elements_than_32_bits_count():
    """2^25 + 64 rows of 256 under a table too wide for whole units: zeros and
    -infinity in every one (17 GB of outputs; the queries are one row)."""
    q_len, heads, dim, page = (1 << 19) + 1, 64, 256, 1024
    cache = make_cache(9, 1, page, dim)
    q = torch.ones(1, heads, dim, dtype=torch.bfloat16, device="cuda").expand(q_len, -1, -1)
    out = torch.full((q_len, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q_len, heads), 7.0, device="cuda")
    table = torch.arange(9, dtype=torch.int32, device="cuda")[None]
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    scratch = torch.empty(dg.dg_attn_decode_scratch(1, q_len, heads, cache), dtype=torch.uint8, device="cuda")
    dg.dg_attn_decode(q, out, cache, table, lens, scratch, lse=lse)
    assert torch.isneginf(lse).all()
    assert not any(part.any().item() for part in out.view(torch.int16).split(1 << 16))
