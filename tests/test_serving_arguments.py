"""Arguments that the Python serving calls must refuse although each tensor by
itself is well formed.  CPU only: refused before anything reaches the library."""
import pytest

import fp16_tensor_core_gb300 as dg
from fp16_tensor_core_gb300 import build as dg_build
from test_serving_binding import CACHE, I32, FakeHeads


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dg_build.build()


class FakeTable:
    """What dg_attn_decode reads of a device page table."""

    dtype, is_cuda = I32, True

    def __init__(self, shape, stride):
        self.shape, self._stride = shape, stride

    def stride(self):
        return self._stride

    def data_ptr(self):
        return 0x7F0000000000


@pytest.mark.parametrize("stride", [(0, 1), (1, 1), (4, 1)])
def test_page_table_rows_that_share_entries(stride):
    """An expanded table, and overlapping windows: a row's pages are looked up
    a row's width apart, past the end of what such a table holds."""
    q = FakeHeads()
    with pytest.raises(ValueError, match="page_table must have a row of its own"):
        dg.dg_attn_decode(q, q, CACHE, FakeTable((3, 5), stride), None, None)


def test_a_prefix_without_its_length_and_the_other_way_round():
    q, table = FakeHeads(), FakeTable((3, 5), (5, 1))
    for kw in (dict(prefix_pages=FakeTable((5,), (1,))), dict(prefix_len=20), dict(prefix_len=-1)):
        with pytest.raises(ValueError, match="prefix_pages and prefix_len must be given together"):
            dg.dg_attn_decode(q, q, CACHE, table, None, None, **kw)


def test_queries_without_their_output_and_the_other_way_round():
    k = FakeHeads()
    for kw in (dict(q=k), dict(q_out=k)):
        with pytest.raises(ValueError, match="q and q_out must be given together"):
            dg.dg_kv_append(k, k, None, CACHE, **kw)
