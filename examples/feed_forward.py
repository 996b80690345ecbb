"""A gated feed-forward block on E4M3 products, forward and backward.

The residual stream and the last block's output meet in the norm
(dg_rmsnorm_e4m3), whose codes and row scales feed the first product
(dg_fp8_gemm_fused, bias); its output passes the gate (dg_activate), whose
codes feed the second product, which adds its result to the stream in place.
Weights are quantised by rows (dg_activate without an activation).  In
training the gate keeps its input in 8 bits; backward, the products are FP16
(dg_hgemm), and the gate and the norm take dg_activate_grad and
dg_rmsnorm_grad.

    python examples/feed_forward.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp16_tensor_core_gb300 as dg

FP16 = torch.float16


def empty(*shape, dtype=FP16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Weight:
    """A weight [out, in]: codes with a scale a row, and its transpose in FP16 for the backward pass."""

    def __init__(self, w):
        self.codes, self.scale = empty(*w.shape, dtype=torch.uint8), empty(w.shape[0], 1, dtype=torch.float32)
        dg.dg_activate(w, dg.DG_ACT_NONE, x_q=self.codes, x_scale=self.scale)
        value = self.codes.view(torch.float8_e4m3fn).float() * self.scale
        self.transposed = value.T.to(FP16).contiguous()

    def __call__(self, codes, scale, **kw):
        out = kw.pop("out", None)
        if out is None:
            out = empty(codes.shape[0], self.codes.shape[0])
        dg.dg_fp8_gemm_fused(codes, self.codes, out, scale, self.scale, out=dg.DG_FP16, **kw)
        return out

    def backward(self, dy):
        dx = empty(dy.shape[0], self.transposed.shape[0])
        dg.dg_hgemm(dy, self.transposed, dx)
        return dx


class FeedForward:
    """x + down(silu(gate(y)) * up(y)), y = norm(x), with x the stream after its addition of `delta`."""

    def __init__(self, hidden=1024, inner=2816, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.norm = (1 + 0.1 * randn(hidden)).to(FP16)
        self.gate_up = Weight((randn(2 * inner, hidden) * hidden ** -0.5).to(FP16))
        self.bias = 0.1 * randn(2 * inner)
        self.down = Weight((randn(hidden, inner) * inner ** -0.5).to(FP16))
        self.hidden, self.inner = hidden, inner

    def __call__(self, x, delta=None, training=False):
        """The new stream (a buffer of its own); delta is added to x first."""
        n = x.shape[0]
        stream = empty(n, self.hidden)
        codes, scale = empty(n, self.hidden, dtype=torch.uint8), empty(n, dtype=torch.float32)
        dg.dg_rmsnorm_e4m3(x, codes, scale, weight=self.norm, residual=delta, sum=stream)
        both = self.gate_up(codes, scale, bias=self.bias)
        h, h_scale = empty(n, self.inner, dtype=torch.uint8), empty(n, dtype=torch.float32)
        kept = (empty(n, 2 * self.inner, dtype=torch.uint8), empty(n, 2, dtype=torch.float32)) if training else (None, None)
        dg.dg_activate(both, dg.DG_ACT_SILU, q=h, q_scale=h_scale, x_q=kept[0], x_scale=kept[1], gated=True)
        self.saved = dict(stream=stream.clone() if training else None, codes=codes, scale=scale, both=both, h=h,
                          h_scale=h_scale, kept=kept)
        return self.down(h, h_scale, residual=stream, out=stream)

    def backward(self, d_out):
        """Gradients of x (and of delta alike), of the norm's weight and of the bias."""
        s, n = self.saved, d_out.shape[0]
        dh = self.down.backward(d_out)
        d_both, d_bias = empty(n, 2 * self.inner), empty(2 * self.inner, dtype=torch.float32)
        scratch = empty(max(dg.dg_activate_grad_scratch(n, self.inner, gated=True),
                            dg.dg_rmsnorm_grad_scratch(n, self.hidden)), dtype=torch.uint8)
        dg.dg_activate_grad(dh, dg.DG_ACT_SILU, d_both, x_q=s["kept"][0], x_scale=s["kept"][1], gated=True,
                            dbias=d_bias, scratch=scratch)
        dy = self.gate_up.backward(d_both)
        dx, d_norm = empty(n, self.hidden), empty(self.hidden, dtype=torch.float32)
        dg.dg_rmsnorm_grad(s["stream"], dy, dx, weight=self.norm, dsum=d_out, dweight=d_norm, scratch=scratch)
        self.partial = dict(dh=dh, d_both=d_both, dy=dy)
        return dx, d_norm, d_bias


def run(tokens=200, seed=1, **sizes):
    g = torch.Generator(device="cuda").manual_seed(seed)
    block = FeedForward(seed=seed, **sizes)
    x, delta, d_out = (torch.randn(tokens, block.hidden, generator=g, device="cuda").to(FP16) for _ in range(3))
    out = block(x, delta, training=True)
    grads = block.backward(d_out)
    assert dg.dg_sync_status() == dg.DG_OK
    return block, (x, delta, d_out), out, grads


if __name__ == "__main__":
    dg.dg_init()
    block, (x, delta, d_out), _, _ = run(4096, hidden=4096, inner=11008)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(x, delta, training=True)
        block.backward(d_out)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    graph.replay()
    start.record()
    for _ in range(10):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"4096 tokens, 4096 x 11008: {start.elapsed_time(end) / 10 * 1e3:.0f} us forward and backward")
