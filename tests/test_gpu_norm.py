"""Root-mean-square norm (16-bit and E4M3 output, residual, recorded scale)
and its gradient against FP64."""
import math

import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _layers import BF, DTYPES, F8, HALF, ROW, STEP, check_codes, close, norm64, randn, rounded, view

pytestmark = pytest.mark.gpu
EPS = 1e-6
SHAPES = [(1, 8), (1, 4096), (3, 1040), (7, 64), (129, 1000), (65, 8192), (5, 11008), (3, 16384), (2, 24576),
          (2, 32768), (1300, 256), (5000, 512), (400, 8200), (500, 16384), (400, 32768)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def inputs(rows, cols, dtype, seed=0):
    x = (randn(seed, rows, cols) * torch.exp(randn(seed + 1, rows, 1))).to(dtype)
    return x, randn(seed + 2, rows, cols).to(dtype), (1 + 0.3 * randn(seed + 3, cols)).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("residual,weight,pad", [(True, True, 0), (False, True, 8), (True, False, 24)])
def test_norm(rows, cols, dtype, residual, weight, pad):
    x, r, w = inputs(rows, cols, dtype, seed=rows + cols)
    s64 = x.double() + r.double() if residual else x.double()
    want = norm64(s64, w.double() if weight else None, EPS)
    x, _ = view(x, pad)
    total, total_rest = view(torch.zeros_like(r), pad)
    y, y_rest = view(torch.zeros_like(r), pad)
    kw = dict(weight=w if weight else None, residual=view(r, pad)[0] if residual else None, sum=total, eps=EPS)
    dg.dg_rmsnorm(x, y, **kw)
    close(y, want, rounded(want, dtype), "y")
    close(total, s64, rounded(s64, dtype, 2.0 ** -24), "sum")
    for rest in (total_rest, y_rest):
        assert rest is None or rest.isnan().all()
    q, scale = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda"), torch.zeros(rows, device="cuda")
    dg.dg_rmsnorm_e4m3(x, q, scale, **{**kw, "sum": None})
    check_codes(q, scale, want)
    given = torch.full((1,), float(want.abs().amax()) / 300, device="cuda")   # the largest saturate
    amax, following = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    q.zero_()
    dg.dg_rmsnorm_e4m3_amax(x, given, q, amax, next_scale_out=following, **kw)
    top = want.abs().amax().reshape(1)
    close(amax, top, top * ROW, "amax")
    assert torch.equal(following, (amax.double() / 448).float())   # correctly rounded
    v = (want / given.double()).clamp(-448, 448)
    close(q.view(F8), v, v.abs() * (2.0 ** -4 + 4 * ROW) + 2.0 ** -10, "codes of the given scale")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dsum,weight,pad", [(True, True, 0), (False, False, 8)])
def test_gradient(rows, cols, dtype, dsum, weight, pad):
    s, dy, w = inputs(rows, cols, dtype, seed=rows + 2 * cols)
    extra = randn(9, rows, cols).to(dtype) if dsum else None
    size = torch.sqrt((s.double() ** 2).mean(-1, keepdim=True) + EPS)
    u = s.double() / size
    g = dy.double() * (w.double() if weight else 1.0)
    want = (g - u * (g * u).mean(-1, keepdim=True)) / size
    terms = (g.abs() + u.abs() * (g * u).abs().mean(-1, keepdim=True)) / size
    if dsum:
        want, terms = want + extra.double(), terms + extra.double().abs()
    dx, rest = view(torch.zeros_like(s), pad)
    dw = torch.full((cols,), math.nan, device="cuda")
    scratch = torch.empty(dg.dg_rmsnorm_grad_scratch(rows, cols), dtype=torch.uint8, device="cuda")
    dg.dg_rmsnorm_grad(view(s, pad)[0], view(dy, pad)[0], dx, weight=w if weight else None, dsum=extra, dweight=dw,
                       scratch=scratch, eps=EPS)
    close(dx, want, rounded(want, dtype) + terms * 4 * ROW, "dx")
    assert rest is None or rest.isnan().all()
    # a column: `rows` terms, each of relative error 2 ROW, fewer than 200 additions
    # in a row: 200 2^-24 < 2^-16
    close(dw, (dy.double() * u).sum(0), (dy.double() * u).abs().sum(0) * (2 * ROW + 2.0 ** -16), "dweight")
    again = torch.zeros_like(dx)
    dg.dg_rmsnorm_grad(s, dy, again, weight=w if weight else None, dsum=extra, eps=EPS)   # without dweight
    assert torch.equal(again, dx)


def test_gradient_against_differences():
    """dx and dweight predict the change of sum(y c) along a direction."""
    rows, cols = 6, 520
    x, c, w = inputs(rows, cols, HALF, seed=4)
    d, dwt = randn(11, rows, cols).double(), randn(12, cols).double()
    dx, dw = torch.zeros_like(x), torch.zeros(cols, device="cuda")
    scratch = torch.empty(dg.dg_rmsnorm_grad_scratch(rows, cols), dtype=torch.uint8, device="cuda")
    dg.dg_rmsnorm_grad(x, c, dx, weight=w, dweight=dw, scratch=scratch, eps=EPS)

    def loss(h):
        return (norm64(x.double() + h * d, w.double() + h * dwt, EPS) * c.double()).sum()

    h = 1e-4
    slope = (loss(h) - loss(-h)) / (2 * h)
    got = (dx.double() * d).sum() + (dw.double() * dwt).sum()
    # dx is rounded to FP16 (2^-11 of each term); the difference is off by h^2
    # times third derivatives of order 1
    assert abs(got - slope) <= 2.0 ** -10 * (dx.double() * d).abs().sum() + 1e-5 * abs(slope) + 1e-4


@pytest.mark.parametrize("dtype", DTYPES)
def test_special_rows(dtype):
    """Zero rows, rows with a NaN or an infinity, the rows beside them, and
    values whose squares FP32 does not hold."""
    x, _, w = inputs(6, 4096, dtype, seed=3)
    x[0] = 0
    x[1, 7] = math.nan
    x[2, 5] = -math.inf
    x[3] *= 2.0 ** 100 if dtype == BF else 1.0
    x[4] *= 2.0 ** -100 if dtype == BF else 2.0 ** -14
    want = norm64(x.double(), w.double(), EPS)
    y = torch.zeros_like(x)
    dg.dg_rmsnorm(x, y, weight=w, eps=EPS)
    close(y, want, rounded(want, dtype) + 2.0 ** -126, "y")     # FP32 flushes nothing above its subnormals
    assert (y[0] == 0).all() and y[1].isnan().all() and y[2, 5].isnan() and (y[2, :5] == 0).all()
    q, scale = torch.zeros(6, 4096, dtype=torch.uint8, device="cuda"), torch.zeros(6, device="cuda")
    dg.dg_rmsnorm_e4m3(x, q, scale, weight=w, eps=EPS)
    value = q.view(F8).double() * scale.double()[:, None]
    assert (q[0] & 0x7F == 0).all() and scale[0] == 2.0 ** -120    # (a negative weight's zero is -0)
    assert value[1].isnan().all() and value[2].isnan().all()
    check_codes(q[3:4], scale[3:4], want[3:4])
    check_codes(q[5:], scale[5:], want[5:])
    dy = randn(8, 6, 4096).to(dtype)
    dx = torch.zeros_like(x)
    dg.dg_rmsnorm_grad(x, dy, dx, weight=w, eps=EPS)
    size = torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + EPS)
    u, g = x.double() / size, dy.double() * w.double()
    grad = (g - u * (g * u).mean(-1, keepdim=True)) / size
    terms = (g.abs() + u.abs() * (g * u).abs().mean(-1, keepdim=True)) / size
    for i in (0, 3, 4, 5):
        close(dx[i], grad[i], rounded(grad[i], dtype) + terms[i] * 4 * ROW, f"dx of row {i}")
    assert dx[1].isnan().all()


@pytest.mark.parametrize("cols", [8, 256, 4096, 16384])
def test_rows_at_the_top_of_the_range(cols):
    """Elements up to BF16's largest, whose squares' sum leaves FP32 by far,
    beside elements down to 2^-60."""
    x = randn(21, 5, cols).clamp(-3, 3).mul(2.0 ** 126).to(BF)      # below 1.5 2^127
    x[1] = torch.finfo(BF).max
    x[2] = -torch.finfo(BF).max
    x[2, 1::2] = 2.0 ** -60
    x[3, 1:] = 2.0 ** 58
    w = randn(22, cols).to(BF)
    want = norm64(x.double(), w.double(), EPS)
    y = torch.zeros_like(x)
    dg.dg_rmsnorm(x, y, weight=w, eps=EPS)
    # a reciprocal of 2^-128 keeps 21 bits: 2^-22, within `rounded`'s ROW
    close(y, want, rounded(want, BF) + 2.0 ** -126, "y")
    q, scale = torch.zeros(5, cols, dtype=torch.uint8, device="cuda"), torch.zeros(5, device="cuda")
    dg.dg_rmsnorm_e4m3(x, q, scale, weight=w, eps=EPS)
    check_codes(q, scale, want)
    dy = randn(23, 5, cols).to(BF)
    dx, dw = torch.zeros_like(x), torch.zeros(cols, device="cuda")
    scratch = torch.empty(dg.dg_rmsnorm_grad_scratch(5, cols), dtype=torch.uint8, device="cuda")
    dg.dg_rmsnorm_grad(x, dy, dx, weight=w, dweight=dw, scratch=scratch, eps=EPS)
    size = torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + EPS)
    u, g = x.double() / size, dy.double() * w.double()
    grad = (g - u * (g * u).mean(-1, keepdim=True)) / size
    terms = (g.abs() + u.abs() * (g * u).abs().mean(-1, keepdim=True)) / size
    close(dx, grad, rounded(grad, BF) + terms * 4 * ROW, "dx")
    close(dw, (dy.double() * u).sum(0), (dy.double() * u).abs().sum(0) * (2 * ROW + 2.0 ** -16), "dweight")


@pytest.mark.parametrize("scale", [1e-40, 2.0 ** -130, 2.0 ** -100, 2.0 ** 125, 0.0, math.inf, math.nan])
def test_recorded_scales_of_every_size(scale):
    x, _, w = inputs(3, 256, HALF, seed=6)
    x[0] = 0
    given, amax = torch.full((1,), scale, device="cuda"), torch.zeros(1, device="cuda")
    q = torch.zeros(3, 256, dtype=torch.uint8, device="cuda")
    dg.dg_rmsnorm_e4m3_amax(x, given, q, amax, weight=w)
    want = (norm64(x.double(), w.double(), 1e-6) / given.double()).clamp(-448, 448)
    close(q.view(F8), want, want.abs() * (2.0 ** -4 + 4 * ROW) + 2.0 ** -10)


def test_recorded_scale_in_place_and_nan():
    x, _, _ = inputs(5, 512, BF, seed=2)
    scale, amax = torch.ones(1, device="cuda"), torch.zeros(1, device="cuda")
    q = torch.zeros(5, 512, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        dg.dg_rmsnorm_e4m3_amax(x, scale, q, amax, next_scale_out=scale)
    assert torch.equal(scale, (amax.double() / 448).float()) and (q.view(F8).float().abs().amax() == 448)
    x[3, 3] = math.nan
    dg.dg_rmsnorm_e4m3_amax(x, scale, q, amax)
    assert amax.isnan().all() and q[3].view(F8).float().isnan().all()
    dg.dg_rmsnorm_e4m3_amax(x[:0], scale, q[:0], amax, next_scale_out=scale)
    assert amax == 0 and scale == 1


@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place(dtype):
    x, r, w = inputs(300, 4096, dtype, seed=5)
    y, total = torch.zeros_like(x), torch.zeros_like(x)
    dg.dg_rmsnorm(x, y, weight=w, residual=r, sum=total)
    for sum_at, y_at in (("x", "r"), ("r", "x")):
        at = {"x": x.clone(), "r": r.clone()}
        dg.dg_rmsnorm(at["x"], at[y_at], weight=w, residual=at["r"], sum=at[sum_at])
        assert torch.equal(at[sum_at], total) and torch.equal(at[y_at], y)
    dx = torch.zeros_like(x)
    dg.dg_rmsnorm_grad(x, r, dx, weight=w, dsum=total)
    for i in range(3):
        args = [x.clone(), r.clone(), total.clone()]
        dg.dg_rmsnorm_grad(args[0], args[1], args[i], weight=w, dsum=args[2])
        assert torch.equal(args[i], dx)


def test_no_rows():
    x = torch.zeros(0, 64, dtype=BF, device="cuda")
    dg.dg_rmsnorm(x, x)
    dg.dg_rmsnorm_e4m3(x, torch.zeros(0, 64, dtype=torch.uint8, device="cuda"), torch.zeros(0, device="cuda"))
    dw = torch.ones(64, device="cuda")
    scratch = torch.empty(dg.dg_rmsnorm_grad_scratch(0, 64) + 16, dtype=torch.uint8, device="cuda")
    dg.dg_rmsnorm_grad(x, x, x, dweight=dw, scratch=scratch)
    assert (dw == 0).all()


def test_refusals():
    x = randn(0, 4, 64).to(BF)
    y, q, s = torch.zeros_like(x), torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), torch.zeros(4, device="cuda")
    scale, dw = torch.ones(1, device="cuda"), torch.zeros(64, device="cuda")
    with pytest.raises(ValueError, match="counterpart"):
        dg.dg_rmsnorm(x, y[:3])
    with pytest.raises(ValueError, match="counterpart"):
        dg.dg_rmsnorm(x, y.half())
    with pytest.raises(ValueError, match="contiguous rows"):
        dg.dg_rmsnorm(x[:, ::2], y[:, ::2])
    with pytest.raises(ValueError, match="weight must be of x's type with 64"):
        dg.dg_rmsnorm(x, y, weight=torch.ones(64, device="cuda"))
    with pytest.raises(ValueError, match="row_scale must be FP32 with 4"):
        dg.dg_rmsnorm_e4m3(x, q, s[:3])
    with pytest.raises(ValueError, match="q must be uint8 with 256"):
        dg.dg_rmsnorm_e4m3(x, q[:2], s)
    for call in (lambda: dg.dg_rmsnorm(x, y, eps=0.0), lambda: dg.dg_rmsnorm(x, y, sum=y),
                 lambda: dg.dg_rmsnorm(x, y[:1].expand(4, 64)), lambda: dg.dg_rmsnorm(x[:, :60], y[:, :60]),
                 lambda: dg.dg_rmsnorm_e4m3_amax(x, scale, q, scale),
                 lambda: dg.dg_rmsnorm_grad(x, x, y, dweight=dw),
                 lambda: dg.dg_rmsnorm_grad(x, x, y, dweight=dw, scratch=torch.empty(16, device="cuda"))):
        with pytest.raises(dg.DgError):
            call()
    shared = x[:1].expand(4, 64)      # an input may name the same row several times
    dg.dg_rmsnorm(shared, y)
    assert torch.equal(y[0], y[3])


def test_streams_and_graphs():
    """A captured call, replayed on new inputs, and calls on another stream."""
    x, r, w = inputs(40, 2048, BF, seed=7)
    q, s = torch.zeros(40, 2048, dtype=torch.uint8, device="cuda"), torch.zeros(40, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros(2048, device="cuda")
    scratch = torch.empty(dg.dg_rmsnorm_grad_scratch(40, 2048), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()

    def calls(stream=None):
        dg.dg_rmsnorm_e4m3(x, q, s, weight=w, residual=r, stream=stream)
        dg.dg_rmsnorm_grad(x, r, dx, weight=w, dweight=dw, scratch=scratch, stream=stream)

    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    first = [t.clone() for t in (q, s, dx, dw)]
    with torch.cuda.graph(graph, stream=side):
        calls()
    for t in (q, s, dx, dw):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (q, s, dx, dw)))
    x.mul_(2.0)
    r.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in (q, s, dx, dw)]
    calls(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(replayed, (q, s, dx, dw)))


@pytest.mark.parametrize("cols", [12000, 32768])
def test_wide_gradient_captured(cols):
    """Rows that several blocks share, several of them to each; captured, and
    two calls on two streams at once."""
    x, r, w = inputs(333, cols, BF, seed=9)
    dx, dw = [torch.zeros_like(x) for _ in range(3)], [torch.zeros(cols, device="cuda") for _ in range(3)]
    size = dg.dg_rmsnorm_grad_scratch(333, cols)
    scratch = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(3)]

    def call(i, stream=None):
        dg.dg_rmsnorm_grad(x, r, dx[i], weight=w, dsum=r, dweight=dw[i], scratch=scratch[i], stream=stream)

    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    call(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=sides[0]):
        call(1)
    for _ in range(3):
        graph.replay()
        call(2, sides[1])
    torch.cuda.synchronize()
    for i in (1, 2):
        assert torch.equal(dx[0], dx[i]) and torch.equal(dw[0], dw[i])


def test_offsets_past_32_bits():
    """Rows behind element 2^32 (as views of a wide buffer, with dense E4M3
    codes behind 2^31) as the same rows alone."""
    rows, cols, stride = 70000, 32768, 65536
    assert rows * cols > 2 ** 31 and rows * stride > 2 ** 32
    wide = torch.empty(rows, stride, dtype=BF, device="cuda")
    x, y = wide[:, :cols], wide[:, cols:]
    few, w = randn(31, 2, cols).to(BF), randn(32, cols).to(BF)
    x[:2], x[-2:] = few, few
    dg.dg_rmsnorm(x, y, weight=w)
    alone = torch.zeros_like(few)
    dg.dg_rmsnorm(few, alone, weight=w)
    assert torch.equal(y[:2], alone) and torch.equal(y[-2:], alone)
    q, scale = torch.empty(rows, cols, dtype=torch.uint8, device="cuda"), torch.empty(rows, device="cuda")
    dg.dg_rmsnorm_e4m3(x, q, scale, weight=w)
    assert torch.equal(q[:2], q[-2:]) and torch.equal(scale[:2], scale[-2:])
    check_codes(q[-2:], scale[-2:], norm64(few.double(), w.double(), 1e-6))
    y[-2:] = few
    dg.dg_rmsnorm_grad(x, y, y, weight=w)
    dg.dg_rmsnorm_grad(few, few, alone, weight=w)
    assert torch.equal(y[-2:], alone)
