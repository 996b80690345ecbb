"""A decoder's attention block served from a paged E4M3 cache.

FP8 projections (dg_quantize_e4m3, dg_fp8_gemm) around the serving operators:
a system prompt is run once and its pages shared; every request runs its own
prompt behind it; then all requests decode together, one token a step
(dg_kv_append turns and writes the step's keys and values and turns its
queries, dg_attn_decode answers them).  At the end one request drops its oldest
tokens: the kept keys are read back (dg_kv_read), turned back to position
zero (dg_rope, inverse) and written again at their new places.

    python examples/decode_loop.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp16_tensor_core_gb300 as dg


def int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Linear:
    """y = x W^T with W quantised once and x at every call."""

    def __init__(self, weight):
        self.codes, self.scale = self.quantize(weight)

    @staticmethod
    def quantize(x):
        amax, scale = torch.zeros(2, 1, device="cuda")
        codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
        dg.dg_amax(x, amax, scale)
        dg.dg_quantize_e4m3(x, scale, codes)
        return codes, scale

    def __call__(self, x):
        codes, scale = self.quantize(x.float().contiguous())
        y = torch.empty(x.shape[0], self.codes.shape[0], dtype=torch.bfloat16, device="cuda")
        dg.dg_fp8_gemm(codes, self.codes, y, scale, self.scale, None, dg.DG_BF16)
        return y


class Attention:
    """QKV projection, rotary positions, cache, attention, output projection."""

    def __init__(self, hidden=1024, q_heads=16, kv_heads=4, dim=64, pages=256, page=32, positions=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.dim, self.page = q_heads, kv_heads, dim, page
        self.qkv = Linear(torch.randn((q_heads + 2 * kv_heads) * dim, hidden, generator=g, device="cuda") * hidden ** -0.5)
        self.out = Linear(torch.randn(hidden, q_heads * dim, generator=g, device="cuda") * hidden ** -0.5)
        table = torch.empty(positions, dim // 2, 2, device="cuda")
        dg.dg_rope_table(table)
        self.rotary = dg.DgRotary(table, dg.DG_ROPE_HALF)
        shape = (pages, kv_heads, page, dim)
        self.cache = dg.DgKvCache(*(torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)),
                                  *(torch.ones(shape[:3], device="cuda") for _ in range(2)))
        self.scratch = torch.empty(0, dtype=torch.uint8, device="cuda")

    def __call__(self, x, batch, positions, slots, page_table, kv_lens, prefix_pages=None, prefix_len=0):
        """x [batch * q_len, hidden]: the newest tokens of each request."""
        qkv = self.qkv(x).view(x.shape[0], self.q_heads + 2 * self.kv_heads, self.dim)
        q, k, v = qkv.split((self.q_heads, self.kv_heads, self.kv_heads), dim=1)
        dg.dg_kv_append(k, v, slots, self.cache, positions=positions, rotary=self.rotary, q=q, q_out=q)
        need = dg.dg_attn_decode_scratch(batch, x.shape[0] // batch, self.q_heads, self.cache, prefix_len)
        if self.scratch.numel() < need:
            self.scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
        y = torch.empty(x.shape[0], self.q_heads, self.dim, dtype=torch.bfloat16, device="cuda")
        dg.dg_attn_decode(q, y, self.cache, page_table, kv_lens, self.scratch, prefix_pages=prefix_pages,
                          prefix_len=prefix_len)
        self.last = (q, y)
        return self.out(y.view(x.shape[0], -1))


class Server:
    """Requests behind one system prompt; pages are handed out in order."""

    def __init__(self, block, system, requests, max_tokens=512):
        self.block, self.shared, self.batch = block, system.shape[0], requests
        page = block.page
        prefix, own = -(-self.shared // page), -(-max_tokens // page)
        self.prefix_pages = torch.arange(prefix, dtype=torch.int32, device="cuda")
        self.table = prefix + torch.arange(requests * own, dtype=torch.int32, device="cuda").view(requests, own)
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        at = torch.arange(self.shared, dtype=torch.int32, device="cuda")
        block(system, 1, at, at, self.prefix_pages[None], int32([self.shared]))   # pages in order: slot = position

    def slots(self, request, at):
        return (self.table[request, (at // self.block.page).long()] * self.block.page + at % self.block.page).int()

    def prompt(self, request, x):
        """A request's own prompt, behind the shared one."""
        n = x.shape[0]
        at = torch.arange(n, dtype=torch.int32, device="cuda")
        self.lens[request] = n
        return self.block(x, 1, self.shared + at, self.slots(request, at), self.table[request:request + 1],
                          self.lens[request:request + 1], self.prefix_pages, self.shared)

    def step(self, x):
        """One new token for every request."""
        every = torch.arange(self.batch, device="cuda")
        at = self.lens.clone()
        self.lens += 1
        return self.block(x, self.batch, self.shared + at, self.slots(every, at), self.table, self.lens,
                          self.prefix_pages, self.shared)

    def drop_oldest(self, request, n):
        """Forgets a request's first n own tokens; the others move up."""
        b, have = self.block, int(self.lens[request])
        kept = torch.arange(n, have, dtype=torch.int32, device="cuda")
        k = torch.empty(have - n, b.kv_heads, b.dim, dtype=torch.float16, device="cuda")
        v = torch.empty_like(k)
        dg.dg_kv_read(b.cache, self.slots(request, kept), k, v)
        dg.dg_rope(k, k, self.shared + kept, b.rotary, inverse=True)
        dg.dg_kv_append(k, v, self.slots(request, kept - n), b.cache, positions=self.shared + kept - n, rotary=b.rotary)
        self.lens[request] = have - n


def run(requests=12, shared=300, steps=8, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    block = Attention(seed=seed)
    hidden = block.out.codes.shape[0]

    def tokens(n):
        return torch.randn(n, hidden, generator=g, device="cuda")

    server = Server(block, tokens(shared), requests)
    x = torch.stack([server.prompt(i, tokens(1 + 11 * i))[-1] for i in range(requests)]).float()
    for _ in range(steps):
        y = server.step(x).float()
        x = torch.nn.functional.rms_norm(x + y, (hidden,))
    server.drop_oldest(requests - 1, 40)
    y = server.step(x)
    assert dg.dg_sync_status() == dg.DG_OK
    return server, y


if __name__ == "__main__":
    dg.dg_init()
    server, y = run()
    x = y.float()
    server.step(x)
    torch.cuda.synchronize()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(20):
        y = server.step(x)
    end.record()
    torch.cuda.synchronize()
    print(f"{server.batch} requests behind {server.shared} shared tokens, own lengths {server.lens.tolist()}: "
          f"{start.elapsed_time(end) / 20 * 1e3:.0f} us a step, outputs finite: {bool(torch.isfinite(y).all())}")
