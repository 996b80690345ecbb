"""The decode loop's last step against FP64 attention over what dg_kv_read
gives back.

The block's queries are BF16 and exact in FP64; keys and values read as FP16
are off by 2^-11 of themselves (their codes times scale).  With u = sum |q k|
scale the largest over a row's tokens, a score is off by 2^-11 u + 2^-20 u, a
weight relative to their sum by twice that (e^x <= 1 + 1.01 x here), and the
output by that of sum p |v| in all, plus its FP16 weights' and values' 2^-11
each and the BF16 rounding of the result; a weight below 2^-14 of the largest
is off by 2^-25 of it, at most n of them."""
import os
import sys

import numpy as np
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _serving import attention64, f64, rope64

pytestmark = pytest.mark.gpu


def test_last_step_and_moved_tokens():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decode_loop

    server, y = decode_loop.run()
    block = server.block
    assert torch.isfinite(y).all()
    q, out = block.last
    for b in (0, 5, server.batch - 1):
        n = int(server.lens[b])
        own = server.slots(b, torch.arange(n, dtype=torch.int32, device="cuda"))
        slots = torch.cat((torch.arange(server.shared, dtype=torch.int32, device="cuda"), own))
        k = torch.empty(slots.numel(), block.kv_heads, block.dim, dtype=torch.float16, device="cuda")
        v = torch.empty_like(k)
        dg.dg_kv_read(block.cache, slots, k, v)
        seen = np.ones((1, slots.numel()), dtype=bool)
        ref, _, pv, qk, _ = attention64(f64(q[b:b + 1]), f64(k), f64(v), np.ones((slots.numel(), block.kv_heads)),
                                        block.dim ** -0.5, seen)
        d = (2.0 ** -11 + 2.0 ** -20) * 1.01 * qk
        top = np.abs(f64(v)).max()
        tol = (2 * d[..., None] + 2.0 ** -10) * 1.01 * pv + 2.0 ** -25 * slots.numel() * top + \
            2.0 ** -8 * 1.01 * np.abs(ref) + 2.0 ** -25
        assert np.all(np.abs(f64(out[b:b + 1]) - ref) <= tol)


def test_dropping_the_oldest_tokens_turns_the_kept_keys():
    """The kept keys, turned to their new positions: two FP16 roundings of
    the row and two quantisations (2^-4 of an element, at least 2^-10 scales)
    apart."""
    from fp16_tensor_core_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decode_loop

    block = decode_loop.Attention(seed=3)
    server = decode_loop.Server(block, torch.randn(70, 1024, device="cuda"), 2)
    server.prompt(1, torch.randn(200, 1024, device="cuda"))
    at = torch.arange(200, dtype=torch.int32, device="cuda")

    def read(slots):
        k = torch.empty(slots.numel(), block.kv_heads, block.dim, dtype=torch.float16, device="cuda")
        v = torch.empty_like(k)
        dg.dg_kv_read(block.cache, slots, k, v)
        return f64(k), f64(v)

    k0, v0 = read(server.slots(1, at[60:]))
    server.drop_oldest(1, 60)
    assert int(server.lens[1]) == 140
    k1, v1 = read(server.slots(1, at[:140]))
    table = f64(block.rotary.table)
    back = rope64(k0, table, np.arange(130, 270), dg.DG_ROPE_HALF, inverse=True)
    want = rope64(back, table, np.arange(70, 210), dg.DG_ROPE_HALF)
    # the row's largest pair bounds what a rotation carries from one element to another
    scale = np.abs(want).max(-1, keepdims=True) / 448.0
    assert np.all(np.abs(k1 - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * scale + 2.0 ** -9 * np.abs(k0).max(-1, keepdims=True))
    assert np.all(np.abs(v1 - v0) <= 2.0 ** -4 * np.abs(v0) + 2.0 ** -10 * np.abs(v0).max(-1, keepdims=True) / 448.0 +
                  2.0 ** -10 * np.abs(v0))
    assert dg.dg_sync_status() == dg.DG_OK
