"""dg_attn_decode where one token outweighs thousands of others: what the
others add together must not be lost with the weight of each.

Bounds as in test_gpu_attn_decode, but for the weights' subnormals in FP16:
weights reach 2^15 over a row's own tokens (and a prefix of few rows), and at
least 2^7 (less one rounding of the reference) over a prefix on the tensor
cores, so that a weight below 2^-14, off by 2^-25, is off by at most 2^-32 *
1.001 of the row's largest weight-times-value-scale."""
import numpy as np
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _serving import ROUND, TORCH, f64
from test_gpu_attn_decode import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def fill(c, slots, sink, bits):
    """Tokens of score 0 with values in the second half of the dims; token
    `sink` has 2^bits times their weight, and values in the first half."""
    n, heads, dim = len(slots), c.cache.kv_heads, c.dim
    k = torch.zeros(n, heads, dim, device="cuda")
    v = torch.zeros_like(k)
    v[..., dim // 2:] = 0.5 + 0.5 * torch.rand(n, heads, dim // 2, device="cuda")
    v[..., -1] = 1.0
    if sink is not None:
        k[sink] = bits * np.log(2.0) / dim ** 0.5
        v[sink] = 0.0
        v[sink, :, :dim // 2] = 1.0
    at = torch.from_numpy(np.asarray(slots, dtype=np.int32)).cuda()
    dg.dg_kv_append(k.to(TORCH[c.dtype]), v.to(TORCH[c.dtype]), at, c.cache)


def check(c, requests):
    out, lse = c.run()
    ref, ref_lse, pv, qk, top = c.reference(requests)
    rows = np.concatenate([np.arange(b * c.q_len, (b + 1) * c.q_len) for b in requests])
    out, lse, d, n = f64(out)[rows], f64(lse)[rows], 2.0 ** -20 * qk, max(c.lens) + c.prefix
    tol = (2.0 ** -11 + 4 * d + 2.0 ** -19)[..., None] * pv + (n * 1.001 * 2.0 ** -32 * top)[..., None] + \
        ROUND[c.dtype] * np.abs(ref) + 2.0 ** -25
    tail = ref[-1, :, c.dim // 2:]
    assert np.all(np.abs(tail) > 3 * tol[-1, :, c.dim // 2:])   # a lost tail would show
    assert np.all(np.abs(out - ref) <= tol), np.max(np.abs(out - ref) / tol)
    assert np.all(np.abs(lse - ref_lse) <= 2 * d + 2.0 ** -19 * (1 + np.abs(ref_lse)))


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,width,q_len,sink", [
    (250, None, 1, 0),          # a block a request
    (4000, None, 1, 0),         # a cluster
    (4000, 2000, 1, 0),         # equal runs
    (4000, 2000, 5, 1234),      # more rows than a unit of eight, a late sink
])
def test_own_tokens(n, width, q_len, sink, dim, dtype):
    c = Case([n, 3], q_len=q_len, q_heads=4, kv_heads=1, dim=dim, page=16, dtype=dtype, width=width)
    c.q.fill_(1.0)
    fill(c, c.slots[0], sink, 28)
    check(c, [0])


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("batch,prefix,sink", [
    (2, 4000, 0),               # few rows
    (40, 120, 0),               # one tile, one share
    (40, 4000, 0),              # shares
    (40, 4000, 3300),           # a late sink
    (700, 2500, 0),             # more row tiles than SMs per key head: one share of many tiles
])
def test_prefix(batch, prefix, sink, dim, dtype):
    q_heads = 4 if batch < 700 else 32
    c = Case([1 + i % 3 for i in range(batch)], q_heads=q_heads, kv_heads=1, dim=dim, page=16, prefix=prefix, dtype=dtype)
    c.q.fill_(1.0)
    for s in c.slots:
        fill(c, s, None, 0)
    fill(c, c.prefix_slots, sink, 28)
    check(c, [0, batch - 1])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_sink_among_own_tokens_of_a_long_prefix(dim):
    """The tail is the whole prefix: joined, it keeps what it adds."""
    c = Case([40] * 40, q_heads=4, kv_heads=1, dim=dim, page=16, prefix=4000, dtype=dg.DG_FP16)
    c.q.fill_(1.0)
    for s in c.slots:
        fill(c, s, 7, 28)
    fill(c, c.prefix_slots, None, 0)
    check(c, [0, 39])
