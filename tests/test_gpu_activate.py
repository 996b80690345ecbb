"""The activation between two products (gated or not, E4M3 output, 8-bit
checkpoint of its input) and its gradient against FP64."""
import math

import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _layers import ACT, ACT_TINY, BF, DTYPES, F8, HALF, act64, check_codes, close, randn, rounded, view

pytestmark = pytest.mark.gpu
ACTS = [dg.DG_ACT_NONE, dg.DG_ACT_RELU, dg.DG_ACT_GELU, dg.DG_ACT_GELU_TANH, dg.DG_ACT_SILU]
SHAPES = [(1, 8), (1, 11008), (3, 1040), (7, 64), (129, 1000), (33, 8192), (3, 16384), (2, 28672), (2, 32768),
          (1300, 256), (31, 11008), (64, 2000)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def bytes_(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda")


def halves(x, gated):
    return x.reshape(x.shape[0], 2 if gated else 1, -1)


def forward64(x, act, gated):
    if not gated:
        return act64(x, act)[0]
    gate, up = x.chunk(2, dim=1)
    return act64(gate, act)[0] * up


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("gated", [False, True])
def test_forward(rows, cols, act, dtype, gated):
    width = 2 * cols if gated else cols
    x, _ = view((2.5 * randn(rows + cols, rows, width)).clamp(-12, 12).to(dtype), 8)
    want = forward64(x.double(), act, gated)
    y, rest = view(torch.zeros(rows, cols, dtype=dtype, device="cuda"), 16)
    q, qs, xq, xs = bytes_(rows, cols), torch.zeros(rows, device="cuda"), bytes_(rows, width), torch.zeros(
        rows, width // cols, device="cuda")
    dg.dg_activate(x, act, y=y, q=q, q_scale=qs, x_q=xq, x_scale=xs, gated=gated)
    # (a gate that vanishes is multiplied by up)
    close(y, want, rounded(want, dtype, ACT) + ACT_TINY * x.double().abs().clamp_min(1)[:, -cols:], "y")
    assert rest.isnan().all()
    check_codes(q, qs, want, ACT)
    check_codes(halves(xq, gated), xs, halves(x.double(), gated), 2.0 ** -23)
    alone = [torch.zeros_like(y), bytes_(rows, cols), torch.zeros_like(qs), bytes_(rows, width), torch.zeros_like(xs)]
    dg.dg_activate(x, act, y=alone[0], gated=gated)
    dg.dg_activate(x, act, q=alone[1], q_scale=alone[2], gated=gated)
    dg.dg_activate(x, act, x_q=alone[3], x_scale=alone[4], gated=gated)
    for a, b in zip(alone, (y, q, qs, xq, xs)):
        assert torch.equal(a, b)


def gradient64(dy, x, act, gated):
    """dx and the size of its terms."""
    if not gated:
        _, slope, terms = act64(x, act)
        return dy * slope, dy.abs() * terms
    gate, up = x.chunk(2, dim=1)
    value, slope, terms = act64(gate, act)
    return (torch.cat((dy * up * slope, dy * value), dim=1),
            torch.cat(((dy * up).abs() * terms, (dy * value).abs()), dim=1))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("checkpoint", [False, True])
def test_gradient(rows, cols, act, dtype, gated, checkpoint):
    width = 2 * cols if gated else cols
    x = (2.5 * randn(rows + cols, rows, width)).clamp(-12, 12).to(dtype)
    dy, _ = view(randn(rows, rows, cols).to(dtype), 8)
    kw = dict(gated=gated)
    x64 = x.double()
    if checkpoint:
        xq, xs = bytes_(rows, width), torch.zeros(rows, width // cols, device="cuda")
        dg.dg_activate(x, act, x_q=xq, x_scale=xs, gated=gated)
        x64 = (halves(xq, gated).view(F8).double() * xs.double()[..., None]).reshape(rows, width)
        kw.update(x_q=xq, x_scale=xs)
    else:
        kw.update(x=view(x, 24)[0])
    want, terms = gradient64(dy.double(), x64, act, gated)
    dx, rest = view(torch.zeros_like(x), 8)
    dbias = torch.full((width,), math.nan, device="cuda")
    scratch = torch.empty(dg.dg_activate_grad_scratch(rows, cols, gated), dtype=torch.uint8, device="cuda")
    dg.dg_activate_grad(dy, act, dx, dbias=dbias, scratch=scratch, **kw)
    # (a checkpoint's codes times scale are rounded once more: x is off by 2^-24
    # of itself, and act' changes by at most |x| |act''| <= 2 times that)
    close(dx, want, rounded(want, dtype) + terms * ACT + dy.double().abs().repeat(1, width // cols) * 2.0 ** -20, "dx")
    assert rest.isnan().all()
    # at most 1300 terms a column, fewer than 200 additions in a row: 2^-24 200 < 2^-16
    close(dbias, want.sum(0), (terms * (ACT + 2.0 ** -16)).sum(0) + dy.double().abs().sum(0).repeat(width // cols) *
          2.0 ** -20, "dbias")
    again = torch.zeros_like(x)
    dg.dg_activate_grad(dy, act, again, **kw)
    assert torch.equal(again, dx)


@pytest.mark.parametrize("act", [dg.DG_ACT_GELU, dg.DG_ACT_GELU_TANH, dg.DG_ACT_SILU])
def test_gradient_against_differences(act):
    rows, cols = 5, 264
    x, c = (2 * randn(1, rows, 2 * cols)).half(), randn(2, rows, cols).half()
    dx, dbias = torch.zeros_like(x), torch.zeros(2 * cols, device="cuda")
    scratch = torch.empty(dg.dg_activate_grad_scratch(rows, cols, True), dtype=torch.uint8, device="cuda")
    dg.dg_activate_grad(c, act, dx, x=x, gated=True, dbias=dbias, scratch=scratch)
    bias = randn(3, 2 * cols).double()     # a bias in front of the activation: the same for every row
    h = 1e-4
    slope = sum(sign * (forward64(x.double() + sign * h * bias, act, True) * c.double()).sum() for sign in (1, -1)) / (2 * h)
    got = (dbias.double() * bias).sum()
    # FP32 sums (2^-16 of the terms); differences to h^2
    assert abs(got - slope) <= 2.0 ** -16 * (dx.double() * bias).abs().sum() + 1e-4


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
def test_extremes(act, dtype):
    """The type's largest and smallest values, zeros, infinities and NaN."""
    big = torch.finfo(dtype).max
    x = torch.tensor([[0.0, -0.0, big, -big, 2.0 ** -14, -30.0, 30.0, 1000.0],
                      [math.nan, 1.0, -1.0, 2.0, 3.0, -2.0, 0.5, 0.25],
                      [math.inf, 1.0, -1.0, 2.0, 3.0, -2.0, 0.5, 0.25]], dtype=dtype, device="cuda")
    y, q, qs = torch.ones_like(x), bytes_(3, 8), torch.zeros(3, device="cuda")
    xq, xs = bytes_(3, 8), torch.zeros(3, 1, device="cuda")
    dg.dg_activate(x, act, y=y, q=q, q_scale=qs, x_q=xq, x_scale=xs)
    want = act64(x.double(), act)[0]
    want = torch.where(want.abs() > big, want.sign() * math.inf, want)
    close(y, want, rounded(want, dtype, 2.0 ** -10) + 2.0 ** -30, "y")   # at -30: exp's argument, 2^-18, and beyond
    for codes, scale in ((q, qs[:, None]), (xq, xs)):
        value = codes.view(F8).double() * scale.double()
        assert value[1].isnan().all() and value[2].isnan().any()
    # rows whose scale's reciprocal is near FP32's ends
    check_codes(xq[:1], xs[:1, 0], x[:1].double(), 2.0 ** -22)
    small = x[:1, :2].repeat(1, 4) + 2.0 ** (-130 if dtype == BF else -24) * torch.arange(8, device="cuda").to(dtype)
    dg.dg_activate(small, act, x_q=xq[:1], x_scale=xs[:1])
    check_codes(xq[:1], xs[:1, 0], small.double(), 2.0 ** -22)
    dx = torch.zeros_like(x)
    dg.dg_activate_grad(torch.ones_like(x), act, dx, x=x)
    slope = act64(x[0].double(), act)[1]
    slope[2], slope[3] = 1, 1 if act == dg.DG_ACT_NONE else 0
    close(dx[0], slope, rounded(slope, dtype) + 2.0 ** -20, "slope")
    assert dx[1, 0].isnan() or act == dg.DG_ACT_NONE
    assert dx[2, 0] == 1 if act in (dg.DG_ACT_NONE, dg.DG_ACT_RELU) else dx[2, 0].isnan()   # 0 times infinity
    zero = torch.zeros(2, 8, dtype=dtype, device="cuda")
    dg.dg_activate(zero, act, q=q[:2], q_scale=qs[:2])
    assert (q[:2] & 0x7F == 0).all() and (qs[:2] == 2.0 ** -120).all()


def test_in_place():
    x, dy = randn(1, 200, 2048).to(BF), randn(2, 200, 2048).to(BF)
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    dg.dg_activate(x, dg.DG_ACT_SILU, y=y)
    dg.dg_activate_grad(dy, dg.DG_ACT_SILU, dx, x=x)
    z = x.clone()
    dg.dg_activate(z, dg.DG_ACT_SILU, y=z)
    assert torch.equal(z, y)
    for i in range(2):
        args = [dy.clone(), x.clone()]
        dg.dg_activate_grad(args[0], dg.DG_ACT_SILU, args[i], x=args[1])
        assert torch.equal(args[i], dx)
    gate, g = x.clone(), dy[:, :1024].contiguous()
    want = torch.zeros_like(x)
    dg.dg_activate_grad(g, dg.DG_ACT_SILU, want, x=x, gated=True)
    dg.dg_activate_grad(g, dg.DG_ACT_SILU, gate, x=gate, gated=True)
    assert torch.equal(gate, want)


def test_empty_calls():
    x = torch.zeros(0, 64, dtype=BF, device="cuda")
    dg.dg_activate(x, dg.DG_ACT_SILU, y=x)
    dg.dg_activate(torch.zeros(2, 64, dtype=BF, device="cuda"), dg.DG_ACT_SILU)     # nothing asked for
    dbias = torch.ones(64, device="cuda")
    dg.dg_activate_grad(x, dg.DG_ACT_SILU, x, x=x, dbias=dbias, scratch=torch.empty(16, device="cuda"))
    assert (dbias == 0).all()


def test_refusals():
    x = randn(0, 4, 64).to(BF)
    q, s = bytes_(4, 64), torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="given together"):
        dg.dg_activate(x, dg.DG_ACT_SILU, q=q)
    with pytest.raises(ValueError, match="q_scale must be FP32 with 4"):
        dg.dg_activate(x, dg.DG_ACT_SILU, q=q, q_scale=s[:2])
    with pytest.raises(ValueError, match="two halves"):
        dg.dg_activate(randn(0, 4, 65).to(BF), dg.DG_ACT_SILU, y=x, gated=True)
    with pytest.raises(ValueError, match="must be given"):
        dg.dg_activate_grad(x, dg.DG_ACT_SILU, x)
    with pytest.raises(ValueError, match="must be given"):
        dg.dg_activate_grad(x, dg.DG_ACT_SILU, x, x=x, x_q=q, x_scale=s)
    with pytest.raises(ValueError, match="counterpart"):
        dg.dg_activate_grad(x, dg.DG_ACT_SILU, x, x=x, gated=True)
    with pytest.raises(TypeError):
        dg.dg_activate(x, "silu", y=x)
    for call in (lambda: dg.dg_activate(x, 5, y=x), lambda: dg.dg_activate(x, dg.DG_ACT_SILU, y=x[:, :32], gated=True),
                 lambda: dg.dg_activate(x, dg.DG_ACT_SILU, y=x[:1].expand(4, 64)),
                 lambda: dg.dg_activate_grad(x, dg.DG_ACT_SILU, x, x=x, dbias=torch.zeros(64, device="cuda"))):
        with pytest.raises(dg.DgError):
            call()


def test_graph():
    x, dy = randn(1, 50, 2048).to(HALF), randn(2, 50, 1024).to(HALF)
    out = [bytes_(50, 1024), torch.zeros(50, device="cuda"), bytes_(50, 2048), torch.zeros(50, 2, device="cuda"),
           torch.zeros_like(x), torch.zeros(2048, device="cuda")]
    scratch = torch.empty(dg.dg_activate_grad_scratch(50, 1024, True), dtype=torch.uint8, device="cuda")

    def calls():
        dg.dg_activate(x, dg.DG_ACT_SILU, q=out[0], q_scale=out[1], x_q=out[2], x_scale=out[3], gated=True)
        dg.dg_activate_grad(dy, dg.DG_ACT_SILU, out[4], x_q=out[2], x_scale=out[3], gated=True, dbias=out[5],
                            scratch=scratch)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls()
    for _ in range(2):
        x.mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in out]
        calls()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, out))


def test_offsets_past_32_bits():
    """Rows behind element 2^32 of a gated input, their codes behind 2^31, as the
    same rows alone."""
    rows, cols = 70000, 32768
    x = torch.zeros(rows, 2 * cols, dtype=BF, device="cuda")
    few, dy = randn(41, 2, 2 * cols).to(BF), randn(42, 2, cols).to(BF)
    x[-2:] = few
    q, scale = torch.empty(rows, cols, dtype=torch.uint8, device="cuda"), torch.empty(rows, device="cuda")
    x_q, x_scale = torch.empty(rows, 2 * cols, dtype=torch.uint8, device="cuda"), torch.empty(rows, 2, device="cuda")
    dg.dg_activate(x, dg.DG_ACT_SILU, q=q, q_scale=scale, x_q=x_q, x_scale=x_scale, gated=True)
    alone = [torch.empty_like(t[:2]) for t in (q, scale, x_q, x_scale)]
    dg.dg_activate(few, dg.DG_ACT_SILU, q=alone[0], q_scale=alone[1], x_q=alone[2], x_scale=alone[3], gated=True)
    for got, want in zip((q, scale, x_q, x_scale), alone):
        assert torch.equal(got[-2:], want)
    up = torch.zeros(rows, cols, dtype=BF, device="cuda")
    up[-2:] = dy
    dg.dg_activate_grad(up, dg.DG_ACT_SILU, x, x_q=x_q, x_scale=x_scale, gated=True)
    want = torch.empty_like(few)
    dg.dg_activate_grad(dy, dg.DG_ACT_SILU, want, x_q=alone[2], x_scale=alone[3], gated=True)
    assert torch.equal(x[-2:], want) and (x[0] == 0).all()
