"""The feed-forward block, each step of it against FP64 from what the step was
given, forward and backward; its single-token form captured and replayed."""
import os
import sys

import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _layers import ACT, ACT_TINY, F8, HALF, ROW, act64, check_codes, close, norm64, rounded

pytestmark = pytest.mark.gpu
SILU = dg.DG_ACT_SILU


@pytest.fixture(scope="module")
def example():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import feed_forward
    yield feed_forward
    assert dg.dg_sync_status() == dg.DG_OK


def value(codes, scale):
    return codes.view(F8).double() * scale.double().reshape(scale.shape[0], -1)


def product(a, b):
    """a b^T and the bound of FP32 sums of it (16 products to an instruction, 2^-23 an addition)."""
    return a @ b.T, (a.abs() @ b.abs().T) * 2.0 ** -23 * (a.shape[1] / 16 + 24)


@pytest.mark.parametrize("tokens", [1, 7, 200, 700])
def test_every_step(example, tokens):
    block, (x, delta, d_out), out, (dx, d_norm, d_bias) = example.run(tokens)
    s, p, f = block.saved, block.partial, block.inner
    # forward
    stream = x.double() + delta.double()
    close(s["stream"], stream, rounded(stream, HALF, 2.0 ** -24), "stream")
    check_codes(s["codes"], s["scale"], norm64(stream, block.norm.double(), 1e-6))
    both, err = product(value(s["codes"], s["scale"]), value(block.gate_up.codes, block.gate_up.scale))
    both = both + block.bias.double()
    close(s["both"], both, rounded(both, HALF) + err, "gate and up")
    gate, up = s["both"].double().chunk(2, dim=1)
    check_codes(s["h"], s["h_scale"], act64(gate, SILU)[0] * up, ACT)
    halves = s["both"].double().view(tokens, 2, f)
    check_codes(s["kept"][0], s["kept"][1], halves, 2.0 ** -22)
    y, err = product(value(s["h"], s["h_scale"]), value(block.down.codes, block.down.scale))
    y = y + s["stream"].double()
    close(out, y, rounded(y, HALF) + err, "out")
    # backward
    dh, err = product(d_out.double(), block.down.transposed.double())
    close(p["dh"], dh, rounded(dh, HALF) + err, "dh")
    kept = (s["kept"][0].view(F8).double().view(tokens, 2, f) * s["kept"][1].double()[..., None]).view(tokens, -1)
    gate, up = kept.chunk(2, dim=1)
    act, slope, terms = act64(gate, SILU)
    g = p["dh"].double()
    want = torch.cat((g * up * slope, g * act), dim=1)
    bound = torch.cat(((g * up).abs() * terms, (g * act).abs()), dim=1) * ACT + g.abs().repeat(1, 2) * 2.0 ** -20
    close(p["d_both"], want, rounded(want, HALF) + bound + ACT_TINY, "d gate and up")
    close(d_bias, want.sum(0), bound.sum(0) + want.abs().sum(0) * 2.0 ** -16, "dbias")
    dy, err = product(p["d_both"].double(), block.gate_up.transposed.double())
    close(p["dy"], dy, rounded(dy, HALF) + err, "dy")
    size = torch.sqrt((s["stream"].double() ** 2).mean(-1, keepdim=True) + 1e-6)
    u, g = s["stream"].double() / size, p["dy"].double() * block.norm.double()
    want = (g - u * (g * u).mean(-1, keepdim=True)) / size + d_out.double()
    bound = (g.abs() + u.abs() * (g * u).abs().mean(-1, keepdim=True)) / size + d_out.double().abs()
    close(dx, want, rounded(want, HALF) + bound * 4 * ROW, "dx")
    dyu = p["dy"].double() * u
    close(d_norm, dyu.sum(0), dyu.abs().sum(0) * (2 * ROW + 2.0 ** -16), "dweight")


def test_decode_step_captured(example):
    block = example.FeedForward(seed=3)
    x = torch.randn(3, block.hidden, device="cuda").to(HALF)
    delta = torch.randn(3, block.hidden, device="cuda").to(HALF)
    block(x, delta)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(x, delta)
    for _ in range(2):
        x.mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, block(x, delta))
