"""The Python serving calls on tensors that are views, and on arguments that
do not go together."""
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from test_gpu_attn_decode import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def test_page_table_views():
    """One row's stride means nothing; rows of a wider table are taken as they
    lie; rows that share entries are refused, and nothing is written."""
    c = Case([100], q_heads=4, kv_heads=2, dim=64)
    want = c.run()
    for stride in (1, 3, 100):
        got = c.run(page_table=c.table.as_strided(c.table.shape, (stride, 1)))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c = Case([100, 40, 64], q_heads=4, kv_heads=2, dim=64)
    want = c.run()
    big = torch.full((3, c.table.shape[1] + 5), 2 ** 30, dtype=torch.int32, device="cuda")
    big[:, 2:-3] = c.table
    got = c.run(page_table=big[:, 2:-3])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = torch.full_like(c.q, 3.0)
    for table in (c.table[0].expand(3, -1), c.table.flatten().unfold(0, 5, 4)[:3]):
        with pytest.raises(ValueError, match="page_table must have a row of its own"):
            c.run(page_table=table, out=out)
    assert torch.all(out == 3.0)


def test_a_length_of_zero_is_no_prefix():
    """A buffer of pages that is kept while nothing is shared."""
    c = Case([100, 40], q_heads=4, kv_heads=2, dim=64)
    want = c.run(prefix_pages=None, prefix_len=None)
    for pages in (None, c.table[0], c.table[0, :0]):
        got = c.run(prefix_pages=pages, prefix_len=0)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
