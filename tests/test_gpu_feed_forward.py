"""The feed-forward block, each step of it against FP64 from what the step was
given, forward and backward; its single-token form captured and replayed."""
import os
import sys

import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _layers import ACT, ACT_TINY, BF, F8, HALF, ROW, act64, check_codes, close, norm64, rounded

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


def test_operands_written_just_before():
    """Weights, bias and scales that the kernel before still writes when the
    launches overlap it: read as they are then, not as they were."""
    M, N, K = 200, 1040, 1024
    g = torch.Generator(device="cuda").manual_seed(5)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    x, r = randn(M, K).to(BF), randn(M, K).to(BF)
    codes = randn(N, K).to(torch.float8_e4m3fn).view(torch.uint8)
    new = [randn(K).to(BF), randn(N), 0.1 + randn(N).abs(), torch.full((1,), 0.02, device="cuda")]
    zeros = [torch.zeros_like(t) for t in new]
    weight, bias, scale_b, scale = at = [t.clone() for t in zeros]
    q, row_scale = torch.zeros(M, K, dtype=torch.uint8, device="cuda"), torch.zeros(M, device="cuda")
    amax, D = torch.zeros(1, device="cuda"), [torch.zeros(m, N, dtype=BF, device="cuda") for m in (4, 60, M)]
    q_x, scale_x = torch.zeros(M, N, dtype=torch.uint8, device="cuda"), torch.zeros(M, device="cuda")
    y, dx = torch.zeros_like(x), torch.zeros_like(D[2])
    dy, dw = randn(M, N).to(BF), torch.zeros(K, device="cuda")
    scratch = torch.empty(dg.dg_rmsnorm_grad_scratch(M, K), dtype=torch.uint8, device="cuda")
    outputs = [q, row_scale, amax, *D, y, dx, dw]

    def one(i):
        if i == 0:
            dg.dg_rmsnorm_e4m3_amax(x, scale, q, amax, weight=weight, residual=r)
        elif i == 1:
            dg.dg_rmsnorm(x, y, weight=weight)
        elif i == 2:
            dg.dg_rmsnorm_grad(x, r, y, weight=weight, dweight=dw, scratch=scratch)
        elif i < 6:
            d = D[i - 3]
            dg.dg_fp8_gemm_fused(codes[:len(d)], codes, d, scale_b[:len(d)], scale_b, bias=bias, amax_d=amax)
        else:
            dg.dg_activate(D[2], dg.DG_ACT_SILU, x_q=q_x, x_scale=scale_x)
            dg.dg_activate_grad(dy, dg.DG_ACT_SILU, dx, x_q=q_x, x_scale=scale_x)

    def run(i, late):
        for a, b in zip(at, zeros if late else new):
            a.copy_(b)
        for t in outputs if i < 6 else [dx, q_x, scale_x]:
            t.zero_()
        torch.cuda.synchronize()
        if late:
            torch.cuda._sleep(100000)
            for a, b in zip(at, new):
                a.copy_(b)
        one(i)
        torch.cuda.synchronize()
        return [t.clone() for t in outputs]

    for i in range(7):
        want = run(i, False)
        for _ in range(3):
            for a, b in zip(run(i, True), want):
                assert torch.equal(a, b), i
