"""dg_attn_decode with BF16 queries whose elements differ by many powers of
two, and with queries and keys near the ends of BF16's range.

Bounds as in test_gpu_attn_decode: a BF16 element that is not below 2^-32 of
its row's largest enters the products exactly."""
import numpy as np
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from test_gpu_attn_decode import Case

pytestmark = pytest.mark.gpu

PATHS = [   # batch, prefix, tokens of the table
    (2, 0, None), (2, 0, 9000), (2, 200, None), (40, 200, None), (40, 3000, None),
]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def make(batch, prefix, tokens, dim, seed):
    return Case([(61 * i) % 150 + 20 for i in range(batch)], q_heads=8, kv_heads=2, dim=dim, prefix=prefix,
                width=None if tokens is None else tokens // 16, seed=seed)


def write(c, keys):
    """Keys (a function of (tokens, heads, dim)) and normal values everywhere."""
    every = np.concatenate(c.slots + [c.prefix_slots]).astype(np.int32)
    k = keys(every.size, c.cache.kv_heads, c.dim).to(torch.bfloat16)
    v = torch.randn(k.shape, device="cuda").to(torch.bfloat16)
    dg.dg_kv_append(k, v, torch.from_numpy(every).cuda(), c.cache)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("batch,prefix,tokens", PATHS)
def test_small_elements_beside_large_ones(batch, prefix, tokens, dim):
    """One dim of the queries is 2^28 times the others, and no key has it:
    the scores are the others'."""
    c = make(batch, prefix, tokens, dim, 21)
    torch.manual_seed(3)

    def keys(*shape):
        k = torch.randn(*shape, device="cuda")
        k[..., 5] = 0.0
        return k

    write(c, keys)
    c.q = torch.where(c.q.abs() < 0.25, 0.25, c.q)
    c.q[..., 5] = 2.0 ** 28
    c.check(*c.run(), requests=[0, batch - 1])


@pytest.mark.parametrize("key_size,query_size", [(2.0 ** 104, 2.0 ** -100), (2.0 ** -50, 2.0 ** 52),
                                                 (2.0 ** 6, 2.0 ** -122), (2.0 ** -20, 2.0 ** 123)])
@pytest.mark.parametrize("batch,prefix,tokens", PATHS)
def test_sizes_near_the_ends_of_the_range(batch, prefix, tokens, key_size, query_size):
    """Queries and keys whose products are ordinary (or nothing, or, by a
    small scale, made ordinary): no factor of a score leaves FP32 before it."""
    c = make(batch, prefix, tokens, 128, 22)
    torch.manual_seed(4)
    write(c, lambda *shape: torch.randn(*shape, device="cuda") * key_size)
    c.q = (torch.randn(c.q.shape, device="cuda") * query_size).to(torch.bfloat16)
    scale = min(1.0, 1.0 / (key_size * query_size)) * c.dim ** -0.5
    c.check(*c.run(scale=scale), requests=[0, batch - 1], scale=scale)
