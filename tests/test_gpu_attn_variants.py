"""The variants of dg_attn_decode that a call's sizes choose between: page
tables wide enough that equal runs of tiles cross requests and blocks (and the
same requests under a narrow table), the shared prefix in one share and in
many, and the order of the kernels of successive calls.  Bounds as derived in
test_gpu_attn_decode."""
import numpy as np
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _serving import TORCH
from test_gpu_attn_decode import LENS, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def wide(lens, page=16, tokens=6000, **kw):
    """A table of many more pages than the lengths need."""
    return Case(lens, page=page, width=tokens // page, **kw)


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (6, 6), (8, 2), (20, 1), (32, 8)])
def test_wide_tables(q_heads, kv_heads, dim, dtype):
    c = wide(LENS, q_heads=q_heads, kv_heads=kv_heads, dim=dim, dtype=dtype)
    c.check(*c.run())


@pytest.mark.parametrize("q_len", [2, 5, 40])
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(4, 4, 64), (8, 2, 128), (14, 2, 128), (6, 2, 256)])
def test_several_new_tokens(q_len, q_heads, kv_heads, dim):
    c = wide([0, 1, 3, 33, 64, 2300], q_len=q_len, q_heads=q_heads, kv_heads=kv_heads, dim=dim)
    c.check(*c.run(), requests=[0, 1, 2, 3, 4] if q_len == 40 else None)


@pytest.mark.parametrize("page", [1, 8, 64, 2048])
def test_page_sizes(page):
    c = wide([3, 1500, 0, 65], page=page, tokens=4096, q_heads=4, kv_heads=2, dim=64, dtype=dg.DG_FP16)
    c.check(*c.run())


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_tables_around_the_switch(dim):
    """The last table that gives every request a block of its own, the first
    that does not, and the same requests under both."""
    limit = 512 if dim == 256 else 1024
    lens = [limit, 0, 1, limit - 1, 200, limit // 2 + 5]
    for width in (limit // 16, limit // 16 + 1):
        c = Case(lens, width=width, q_heads=8, kv_heads=2, dim=dim, seed=4)
        c.check(*c.run())


@pytest.mark.parametrize("lens", [[0] * 5 + [3000] + [0] * 5, [1] * 300 + [5000], [32] * 64, [0, 0, 0]])
def test_uneven_batches(lens):
    c = wide(lens, q_heads=4, kv_heads=2, dim=128, dtype=dg.DG_FP16)
    c.check(*c.run(), requests=sorted({0, len(lens) // 2, len(lens) - 1}))


@pytest.mark.parametrize("batch,q_len,q_heads,kv_heads,dim,prefix", [
    (7, 1, 8, 2, 128, 5000),        # prefix over all SMs, joined by its own kernels
    (3, 2, 6, 2, 256, 3000),
    (12, 2, 8, 8, 64, 1025),
    (50, 1, 8, 4, 128, 3000),       # on the tensor cores, in shares
    (40, 1, 4, 2, 64, 100),         # one tile: one share
    (600, 1, 32, 32, 64, 300),      # more units than SMs: one share
])
def test_prefix_and_wide_tables(batch, q_len, q_heads, kv_heads, dim, prefix):
    lens = [(613 * i) % 1500 if i % 7 else 0 for i in range(batch)]
    c = wide(lens, q_len=q_len, q_heads=q_heads, kv_heads=kv_heads, dim=dim, prefix=prefix)
    c.check(*c.run(), requests=sorted({0, 1, batch // 2, batch - 1}))


PREFIXES = [(5, 200), (5, 3000), (60, 100), (60, 3000)]   # batch, prefix: 4 rows per token and key head


@pytest.mark.parametrize("batch,prefix", PREFIXES)
def test_strided_outputs_behind_a_prefix(batch, prefix):
    c = Case([(37 * i) % 200 for i in range(batch)], q_heads=8, kv_heads=2, dim=128, prefix=prefix)
    want = c.run()
    c.check(*want, requests=[0, 1, batch - 1])
    packed = torch.randn(batch, 12, 128, device="cuda").bfloat16()
    packed[:, :8] = c.q
    rows = torch.full((batch, 9, 136), 5.0, device="cuda").bfloat16()
    out, lse = c.run(q=packed[:, :8], out=rows[:, :8, :128])
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.all(rows[:, 8] == 5.0) and torch.all(rows[..., 128:] == 5.0)
    assert torch.equal(c.run(lse=None)[0], want[0])


@pytest.mark.parametrize("tokens", [400, 6000])
@pytest.mark.parametrize("batch,prefix", [(5, 0)] + PREFIXES)
def test_steps_without_a_pause(batch, prefix, tokens):
    """Cache writes and attention one behind the other, as a decode loop
    launches them, give what each step gives by itself."""
    c = Case([1 + (37 * i) % 200 for i in range(batch)], q_heads=8, kv_heads=2, dim=128, prefix=prefix,
             width=tokens // 16)
    steps = 12
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(steps, batch + 1, 2, 128, generator=g, device="cuda").to(TORCH[c.dtype])
    q = torch.randn(steps, *c.q.shape, generator=g, device="cuda").to(TORCH[c.dtype])
    # every request's first token, and one of the prefix, are written anew
    shared = [int(c.prefix_slots[-1])] if prefix else [-1]
    at = torch.tensor([int(s[0]) for s in c.slots] + shared, dtype=torch.int32, device="cuda")
    outs = torch.zeros(2, *q.shape, dtype=c.q.dtype, device="cuda")
    lses = torch.zeros(2, steps, *c.q.shape[:2], device="cuda")
    for pause in (0, 1):
        torch.cuda.synchronize()
        for i in range(steps):
            dg.dg_kv_append(x[i], x[i], at, c.cache)
            if pause:
                torch.cuda.synchronize()
            c.run(q=q[i], out=outs[pause, i], lse=lses[pause, i])
            if pause:
                torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(lses[0], lses[1])
    c.q = q[-1]
    c.check(outs[0, -1], lses[0, -1], requests=[0, batch - 1])


@pytest.mark.parametrize("batch,prefix", PREFIXES)
def test_nan_in_the_prefix_reaches_every_row(batch, prefix):
    c = Case([(37 * i) % 50 for i in range(batch)], q_heads=8, kv_heads=2, dim=128, prefix=prefix)
    k = torch.randn(1, 2, 128, device="cuda").bfloat16()
    v = k.clone()
    v[0, 1, 3] = float("nan")                                # the second key head's
    ref = c.run()[0]
    dg.dg_kv_append(k, v, torch.tensor([int(c.prefix_slots[7])], dtype=torch.int32, device="cuda"), c.cache)
    out = c.run()[0]
    assert torch.isnan(out[:, 4:]).all() and torch.isfinite(out[:, :4]).all() and torch.isfinite(ref).all()


@pytest.mark.parametrize("batch,prefix", PREFIXES)
def test_bad_prefix_pages_are_reported(batch, prefix):
    c = Case([(37 * i) % 50 for i in range(batch)], q_heads=8, kv_heads=2, dim=128, prefix=prefix)
    for bad in (c.cache.c.pages, -1, 2 ** 31 - 1):
        c.pp[2] = bad
        c.run()
        assert dg.dg_sync_status() == dg.DG_ERR_INVALID_VALUE
    c.pp[2] = int(c.prefix_pages[2])
    c.check(*c.run(), requests=[0, batch - 1])


@pytest.mark.parametrize("dim", [64, 128])
def test_uneven_scores_in_a_prefix_of_many_rows(dim):
    """Maxima that move from tile to tile: late tokens with the largest keys."""
    c = Case([5] * 40, q_heads=4, kv_heads=1, dim=dim, prefix=1500, q_size=8.0, spread=2.0, seed=11,
             dtype=dg.DG_FP16)
    k = torch.randn(1500, 1, dim, device="cuda") * torch.linspace(0.05, 6.0, 1500, device="cuda")[:, None, None]
    v = torch.randn(1500, 1, dim, device="cuda")
    dg.dg_kv_append(k.half(), v.half(), torch.from_numpy(c.prefix_slots.astype(np.int32)).cuda(), c.cache)
    c.check(*c.run(), requests=[0, 17, 39])


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (6, 6), (8, 2), (20, 1), (32, 8)])
def test_tables_for_equal_runs(q_heads, kv_heads, dim, dtype):
    """Tables too wide for a cluster per request."""
    c = wide(LENS, tokens=9000, q_heads=q_heads, kv_heads=kv_heads, dim=dim, dtype=dtype)
    c.check(*c.run())


@pytest.mark.parametrize("q_len", [1, 3, 40])
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(4, 4, 64), (8, 2, 128), (14, 2, 128), (6, 2, 256)])
def test_equal_runs_of_uneven_requests(q_len, q_heads, kv_heads, dim):
    c = wide([0, 1, 3, 2300, 33, 0, 64, 700], tokens=9000, q_len=q_len, q_heads=q_heads, kv_heads=kv_heads, dim=dim)
    c.check(*c.run(), requests=[0, 1, 2, 4, 5, 6] if q_len == 40 else None)


@pytest.mark.parametrize("batch", [1, 2, 5, 10, 20, 39, 77])
@pytest.mark.parametrize("dim,q_heads", [(64, 4), (64, 60), (128, 8), (128, 40), (256, 4)])
def test_clusters_of_every_size(batch, dim, q_heads):
    """From a cluster of eight blocks per (request, key head) to one block;
    requests shorter than the cluster's first block among them."""
    lens = [(1500, 0, 1, 32, 33, 64, 65, 256, 257, 900)[i % 10] for i in range(batch)]
    c = wide(lens, tokens=1600, q_heads=q_heads, kv_heads=4, dim=dim)
    c.check(*c.run(), requests=sorted({0, batch // 2, batch - 1} | set(range(min(batch, 9)))))


@pytest.mark.parametrize("tokens", [1600, 9000])
def test_graph_of_back_to_back_calls(tokens):
    """Calls that follow one another in a graph, each reading the last one's output."""
    c = wide([1500, 40, 0, 700], tokens=tokens, q_heads=8, kv_heads=2, dim=128)
    outs = [torch.zeros_like(c.q) for _ in range(4)]

    def chain():
        q = c.q
        for o in outs:
            c.run(q=q, out=o)
            q = o

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain()
    s.synchronize()
    want = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        chain()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
