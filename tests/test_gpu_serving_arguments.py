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


def test_the_stride_of_a_single_token_or_head():
    """A view of one row of a pitch that no second row could have."""
    rows = torch.randn(5, 132, device="cuda").bfloat16()
    one = rows[:, :128].view(5, 2, 64)[:1]
    table = torch.empty(50, 32, 2, device="cuda")
    dg.dg_rope_table(table)
    rot, at = dg.DgRotary(table), torch.tensor([7], dtype=torch.int32, device="cuda")
    want = torch.empty(1, 2, 64, dtype=one.dtype, device="cuda")
    dg.dg_rope(one.contiguous(), want, at, rot)
    before = rows.clone()
    dg.dg_rope(one, one, at, rot)
    assert torch.equal(one, want)
    before[0, :128] = want.flatten()
    assert torch.equal(rows, before)
    x = torch.randn(5, 1, 64, device="cuda").half()
    want, got = torch.empty_like(x), torch.zeros_like(x)
    at = torch.arange(5, dtype=torch.int32, device="cuda")
    dg.dg_rope(x, want, at, rot)
    dg.dg_rope(x.as_strided((5, 1, 64), (64, 7, 1)), got.as_strided((5, 1, 64), (64, 3, 1)), at, rot)
    assert torch.equal(got, want)
    with pytest.raises(dg.DgError, match="MISALIGNED"):
        dg.dg_rope(rows[:, :128].view(5, 2, 64), torch.empty(5, 2, 64, dtype=rows.dtype, device="cuda"), at, rot)
