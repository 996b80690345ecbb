"""Measured cases of the operators around a layer's products.

Root-mean-square norm with the residual's addition and an E4M3 output
(``dg_rmsnorm_e4m3``, ``dg_rmsnorm_e4m3_amax``, ``dg_rmsnorm``) and its gradient
(``dg_rmsnorm_grad``), the matrix product with scales per row, bias, activation
and residual in its epilogue (``dg_fp8_gemm_fused``, ``dg_hgemm_fused``), and
the activation between two products with an E4M3 output and an 8-bit
checkpoint of its input (``dg_activate``), which its gradient reads
(``dg_activate_grad``).  With ``own`` false, ``run`` computes them in plain
torch operations in FP32.
"""
from __future__ import annotations

import math

import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -120
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of a small batch in front of the QKV projection: latency counts.
        dict(name="norm_step", op="norm", rows=8, cols=4096, dtype="bf16", out="rows", residual=True),
        # A prompt's tokens on their way into an E4M3 product, the residual stream updated on the way.
        dict(name="norm_prompt", op="norm", rows=16001, cols=4096, dtype="bf16", out="rows", residual=True),
        # Wide rows with the scale that the last call recorded (one scale for the tensor).
        dict(name="norm_recorded", op="norm", rows=6001, cols=8192, dtype="fp16", out="tensor", residual=False),
        # A small ragged fine-tuning batch, and a training batch with the residual stream's own gradient.
        dict(name="norm_grad_small", op="norm_grad", rows=129, cols=1040, dtype="fp16", dsum=False),
        dict(name="norm_grad_large", op="norm_grad", rows=16384, cols=4096, dtype="bf16", dsum=True),
        # The attention's output projection for four tokens, into the residual stream.
        dict(name="product_step", op="product", M=4, N=4096, K=4096, operands="e4m3", out="bf16", act="none",
             bias=True, residual=True, rows=True),
        # An odd FP16 product with everything in its epilogue.
        dict(name="product_odd", op="product", M=129, N=1000, K=1040, operands="fp16", out="fp16", act="silu",
             bias=True, residual=True, rows=False),
        # A prompt's first feed-forward product, whose output is the next one's E4M3 operand.
        dict(name="product_prompt", op="product", M=4096, N=11008, K=4096, operands="e4m3", out="e4m3",
             act="gelu", bias=True, residual=False, rows=True),
        # The gate between two products of a decode step.
        dict(name="gate_step", op="act", rows=16, cols=11008, dtype="bf16", act="silu", gated=True,
             y=False, q=True, checkpoint=False),
        # The same in training: output for the next product, input kept in 8 bits for the backward pass.
        dict(name="gate_checkpoint", op="act", rows=8192, cols=11008, dtype="bf16", act="silu", gated=True,
             y=False, q=True, checkpoint=True),
        # The backward pass of a small ungated activation from its input, and of the gate from the checkpoint.
        dict(name="act_grad_small", op="act_grad", rows=63, cols=2000, dtype="fp16", act="gelu_tanh",
             gated=False, checkpoint=False, dbias=True),
        dict(name="gate_grad", op="act_grad", rows=8192, cols=11008, dtype="bf16", act="silu", gated=True,
             checkpoint=True, dbias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "product", "product", "product", "act", "act_grad"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "product":
        operands = rng.choice(["e4m3", "e4m3", "fp16"])
        m = _log(rng, 1, 4096)
        n = _log(rng, 16, 11008)
        step = 16 if operands == "e4m3" else 8
        k = max(1, _log(rng, 16, 12288) // step) * step
        out = rng.choice(["bf16", "fp16", "e4m3"] if operands == "e4m3" else ["bf16", "fp16"])
        return dict(op=op, M=m, N=n, K=k, operands=operands, out=out,
                    act=rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu"]),
                    bias=rng.random() < 0.6, residual=out != "e4m3" and rng.random() < 0.6,
                    rows=operands == "e4m3" and rng.random() < 0.7)
    if op in ("norm", "norm_grad"):
        cols = max(1, _log(rng, 16, 20000) // 16) * 16
        rows = _log(rng, 1, min(40000, 60_000_000 // cols))
        if op == "norm":
            return dict(op=op, rows=rows, cols=cols, dtype=dtype, out=rng.choice(["rows", "rows", "tensor", "half"]),
                        residual=rng.random() < 0.7)
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, dsum=rng.random() < 0.5)
    gated = rng.random() < 0.6
    cols = max(1, _log(rng, 16, 16384) // 16) * 16
    rows = _log(rng, 1, min(40000, 80_000_000 // (2 * cols if gated else cols)))
    act = rng.choice(["relu", "gelu", "gelu_tanh", "silu", "silu"])
    if op == "act":
        q = rng.random() < 0.6
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, act=act, gated=gated, y=not q or rng.random() < 0.3,
                    q=q, checkpoint=rng.random() < 0.5)
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, act=act, gated=gated, checkpoint=rng.random() < 0.6,
                dbias=rng.random() < 0.6)


def work(case):
    op = case["op"]
    if op == "product":
        m, n, k = case["M"], case["N"], case["K"]
        e = 1 if case["operands"] == "e4m3" else 2
        o = 1 if case["out"] == "e4m3" else 2
        scales = 4 * (m + n) if case["rows"] else 8 if e == 1 else 0
        return {"bytes": (m + n) * k * e + m * n * o * (2 if case["residual"] else 1) + scales +
                (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    r, c = case["rows"], case["cols"]
    if op == "norm":
        out = {"rows": r * (c + 4), "tensor": r * c + 12, "half": 2 * r * c}[case["out"]]
        return {"bytes": 2 * r * c * (3 if case["residual"] else 1) + 2 * c + out, "flops": 5 * r * c}
    if op == "norm_grad":
        return {"bytes": 2 * r * c * (4 if case["dsum"] else 3) + 6 * c, "flops": 9 * r * c}
    w = 2 * c if case["gated"] else c          # columns of the input
    halves = 2 if case["gated"] else 1
    if op == "act":
        return {"bytes": 2 * r * w + (2 * r * c if case["y"] else 0) + (r * (c + 4) if case["q"] else 0) +
                (r * (w + 4 * halves) if case["checkpoint"] else 0), "flops": 8 * r * w}
    return {"bytes": 2 * r * c + (r * (w + 4 * halves) if case["checkpoint"] else 2 * r * w) + 2 * r * w +
            (4 * w if case["dbias"] else 0), "flops": 12 * r * w}


# ------------------------------------------------------------------ inputs

def _quantise(x):
    """E4M3 codes and FP32 scales of the rows of x."""
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp_min(MIN_SCALE)
    return (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(F8), scale


def _halves(x, gated):
    """[rows, halves, columns of a half]: each half of a gated input has scales of its own."""
    return x.reshape(x.shape[0], 2 if gated else 1, -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case}

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "product":
        m, n, k = case["M"], case["N"], case["K"]
        dt = torch.uint8 if case["out"] == "e4m3" else DTYPES[case["out"]]
        if case["operands"] == "e4m3":
            # tokens of different magnitude, a weight of about 1 / sqrt(K)
            a = randn(m, k) * torch.exp(randn(m, 1))
            b = randn(n, k) * k ** -0.5
            if case["rows"]:
                a, s["scale_a"] = _quantise(a)
                b, s["scale_b"] = _quantise(b)
            else:
                s["scale_a"], s["scale_b"] = (x.abs().amax().reshape(1) / E4M3_MAX for x in (a, b))
                a, b = (x / y for x, y in ((a, s["scale_a"]), (b, s["scale_b"])))
                a, b = (x.clamp(-E4M3_MAX, E4M3_MAX).to(F8) for x in (a, b))
            s["A"], s["B"] = a.view(torch.uint8), b.view(torch.uint8)
        else:
            s["A"], s["B"] = randn(m, k).half(), (randn(n, k) * k ** -0.5).half()
            s["scale_a"] = s["scale_b"] = None
        s["bias"] = randn(n) if case["bias"] else None
        s["residual"] = randn(m, n).to(dt) if case["residual"] else None
        s["scale_d"] = torch.full((1,), 16.0 / E4M3_MAX, device="cuda") if case["out"] == "e4m3" else None
        s["amax_d"] = empty((1,), torch.float32) if case["out"] == "e4m3" else None
        s["D"] = empty((m, n), dt)
        return s
    r, c, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    if op in ("norm", "norm_grad"):
        # tokens of different magnitude; the stream grows past the layers' outputs
        s["x"] = (randn(r, c) * torch.exp(randn(r, 1))).to(dt)
        s["weight"] = (1 + 0.2 * randn(c)).to(dt)
    if op == "norm":
        s["residual"] = (3 * randn(r, c)).to(dt) if case["residual"] else None
        s["sum"] = empty((r, c), dt) if case["residual"] else None
        if case["out"] == "half":
            s["y"] = empty((r, c), dt)
        else:
            s["q"] = empty((r, c), torch.uint8)
            s["row_scale"] = empty((r,), torch.float32)
        if case["out"] == "tensor":
            s["scale"] = torch.full((1,), 9.0 / E4M3_MAX, device="cuda")
            s["amax"], s["next_scale"] = empty((1,), torch.float32), empty((1,), torch.float32)
    elif op == "norm_grad":
        s["dy"] = randn(r, c).to(dt)
        s["dsum"] = randn(r, c).to(dt) if case["dsum"] else None
        s["dx"] = empty((r, c), dt)
        s["dweight"] = empty((c,), torch.float32)
    else:
        w = 2 * c if case["gated"] else c
        x = (randn(r, w) * 1.5).to(dt)
        if op == "act":
            s["x"] = x
            s["y"] = empty((r, c), dt) if case["y"] else None
            s["q"] = empty((r, c), torch.uint8) if case["q"] else None
            s["q_scale"] = empty((r,), torch.float32) if case["q"] else None
            s["x_q"] = empty((r, w), torch.uint8) if case["checkpoint"] else None
            s["x_scale"] = empty((r, w // c), torch.float32) if case["checkpoint"] else None
        else:
            s["x"] = s["x_q"] = s["x_scale"] = None
            if case["checkpoint"]:
                codes, s["x_scale"] = _quantise(_halves(x.float(), case["gated"]))
                s["x_q"] = codes.reshape(r, w).view(torch.uint8)
            else:
                s["x"] = x
            s["dy"] = randn(r, c).to(dt)
            s["dx"] = empty((r, w), dt)
            s["dbias"] = empty((w,), torch.float32) if case["dbias"] else None
    return s


# ------------------------------------------------------------------- passes

def _act(x, kind):
    if kind == "relu":
        return torch.where(x > 0, x, 0.0)
    if kind == "gelu":
        return 0.5 * x * torch.erfc(-x * math.sqrt(0.5))
    if kind == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    if kind == "silu":
        return x / (1 + torch.exp(-x))
    return x


def _act_slope(x, kind):
    if kind == "relu":
        return (x > 0).to(x.dtype)
    if kind == "gelu":
        return 0.5 * torch.erfc(-x * math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x * x * x))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)
    if kind == "silu":
        g = 1 / (1 + torch.exp(-x))
        return g * (1 + x * (1 - g))
    return torch.ones_like(x)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "product":
        wide = (lambda x: x.view(F8).float()) if case["operands"] == "e4m3" else (lambda x: x.float())
        d = wide(s["A"]) @ wide(s["B"]).T
        if s["scale_a"] is not None:
            d = d * s["scale_a"][:, None] * s["scale_b"][None, :]
        if case["bias"]:
            d = d + s["bias"]
        d = _act(d, case["act"])
        if case["residual"]:
            d = d + s["residual"].float()
        if case["out"] != "e4m3":
            return d.to(DTYPES[case["out"]])
        return [(d / s["scale_d"]).clamp(-E4M3_MAX, E4M3_MAX).to(F8), d.abs().amax().reshape(1)]
    if op == "norm":
        v, dt = s["x"].float(), s["x"].dtype
        outs = []
        if case["residual"]:
            v = v + s["residual"].float()
            outs = [v.to(dt)]
        y = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["weight"].float()
        if case["out"] == "rows":
            return outs + list(_quantise(y))
        if case["out"] == "tensor":
            amax = y.abs().amax().reshape(1)
            return outs + [(y / s["scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(F8), amax, amax / E4M3_MAX]
        return outs + [y.to(dt)]
    if op == "norm_grad":
        x, dy = s["x"].float(), s["dy"].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        unit = x * r
        g = dy * s["weight"].float()
        dx = r * (g - unit * (g * unit).mean(-1, keepdim=True))
        if case["dsum"]:
            dx = dx + s["dsum"].float()
        return [dx.to(s["x"].dtype), (dy * unit).sum(0)]
    c, kind = case["cols"], case["act"]
    if op == "act":
        x = s["x"].float()
        y = _act(x[:, :c], kind) * x[:, c:] if case["gated"] else _act(x, kind)
        outs = [y.to(s["x"].dtype)] if case["y"] else []
        if case["q"]:
            outs += list(_quantise(y))
        if case["checkpoint"]:
            codes, scale = _quantise(_halves(x, case["gated"]))
            outs += [codes.reshape(x.shape), scale]
        return outs
    if case["checkpoint"]:
        x = (_halves(s["x_q"], case["gated"]).view(F8).float() * s["x_scale"][..., None]).reshape(s["x_q"].shape)
    else:
        x = s["x"].float()
    dy = s["dy"].float()
    if case["gated"]:
        gate, up = x[:, :c], x[:, c:]
        dx = torch.cat((dy * up * _act_slope(gate, kind), dy * _act(gate, kind)), dim=1)
    else:
        dx = dy * _act_slope(x, kind)
    return [dx.to(s["dy"].dtype)] + ([dx.sum(0)] if case["dbias"] else [])


def run(state):
    if not own:
        return _plain(state)
    import fp16_tensor_core_gb300 as dg

    s, case = state, state["case"]
    op = case["op"]
    if op == "norm":
        outs = [s["sum"]] if case["residual"] else []
        kw = dict(weight=s["weight"], residual=s["residual"], sum=s["sum"], eps=EPS)
        if case["out"] == "half":
            dg.dg_rmsnorm(s["x"], s["y"], **kw)
            return outs + [s["y"]]
        if case["out"] == "rows":
            dg.dg_rmsnorm_e4m3(s["x"], s["q"], s["row_scale"], **kw)
            return outs + [s["q"].view(F8), s["row_scale"]]
        dg.dg_rmsnorm_e4m3_amax(s["x"], s["scale"], s["q"], s["amax"], next_scale_out=s["next_scale"], **kw)
        return outs + [s["q"].view(F8), s["amax"], s["next_scale"]]
    if op == "norm_grad":
        if "scratch" not in s:
            s["scratch"] = torch.empty(dg.dg_rmsnorm_grad_scratch(case["rows"], case["cols"]), dtype=torch.uint8,
                                       device="cuda")
        dg.dg_rmsnorm_grad(s["x"], s["dy"], s["dx"], weight=s["weight"], dsum=s["dsum"], dweight=s["dweight"],
                           scratch=s["scratch"], eps=EPS)
        return [s["dx"], s["dweight"]]
    act = getattr(dg, "DG_ACT_" + case["act"].upper())
    if op == "product":
        out = getattr(dg, "DG_" + case["out"].upper())
        if case["operands"] == "fp16":
            dg.dg_hgemm_fused(s["A"], s["B"], s["D"], bias=s["bias"], act=act, residual=s["residual"], out=out)
            return s["D"]
        dg.dg_fp8_gemm_fused(s["A"], s["B"], s["D"], s["scale_a"], s["scale_b"], bias=s["bias"], act=act,
                             residual=s["residual"], scale_d=s["scale_d"], amax_d=s["amax_d"], out=out)
        return [s["D"].view(F8), s["amax_d"]] if case["out"] == "e4m3" else s["D"]
    if op == "act":
        dg.dg_activate(s["x"], act, y=s["y"], q=s["q"], q_scale=s["q_scale"], x_q=s["x_q"], x_scale=s["x_scale"],
                       gated=case["gated"])
        return (([s["y"]] if case["y"] else []) + ([s["q"].view(F8), s["q_scale"]] if case["q"] else []) +
                ([s["x_q"].view(F8), s["x_scale"]] if case["checkpoint"] else []))
    if case["dbias"] and "scratch" not in s:
        n = dg.dg_activate_grad_scratch(case["rows"], case["cols"], gated=case["gated"])
        s["scratch"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    dg.dg_activate_grad(s["dy"], act, s["dx"], x=s["x"], x_q=s["x_q"], x_scale=s["x_scale"], gated=case["gated"],
                        dbias=s["dbias"], scratch=s.get("scratch"))
    return [s["dx"]] + ([s["dbias"]] if case["dbias"] else [])


# -------------------------------------------------------------- definitions

def _exact_codes(y):
    """What rows of y are before their rounding to E4M3, and their scales."""
    scale = torch.linalg.vector_norm(y, ord=math.inf, dim=-1) / 448
    scale = torch.maximum(scale, torch.full_like(scale, 2.0 ** -120))
    return [y / scale.unsqueeze(-1), scale]


def _exact_act(x, kind):
    """The activation and its derivative in FP64, from x times a distribution function."""
    if kind == "none":
        return x, torch.ones_like(x)
    if kind == "relu":
        return x.clamp_min(0), torch.heaviside(x, torch.zeros_like(x))
    if kind == "gelu":
        phi = torch.special.ndtr(x)
        return x * phi, phi + x * torch.exp(-x.square() / 2) * (2 * math.pi) ** -0.5
    if kind == "gelu_tanh":    # (1 + tanh u) / 2 is the logistic function of 2 u
        k = 2 * (2 / math.pi) ** 0.5
        u, du = k * (x + 0.044715 * x ** 3), k * (1 + 0.134145 * x ** 2)
    else:
        u, du = x, torch.ones_like(x)
    p = torch.sigmoid(u)
    return x * p, p + x * p * torch.sigmoid(-u) * du


def exact(case, seed):
    """The operators' definitions in FP64."""
    s = prepare(case, seed)
    op = case["op"]

    def wide(x):
        return x.view(F8).double() if x.dtype == torch.uint8 else x.double()

    if op == "product":
        n = case["N"]
        sa = torch.ones(1, device="cuda") if s["scale_a"] is None else s["scale_a"]
        sb = torch.ones(1, device="cuda") if s["scale_b"] is None else s["scale_b"]
        b = (wide(s["B"]) * sb.double().reshape(-1, 1)).T.contiguous()
        out = torch.empty(case["M"], n, dtype=torch.float64, device="cuda")
        for i in range(0, case["M"], 1024):
            part = wide(s["A"][i:i + 1024]) @ b
            part *= sa.double().reshape(-1, 1)[i:i + 1024] if sa.numel() > 1 else sa.double()
            if case["bias"]:
                part += s["bias"].double()
            part = _exact_act(part, case["act"])[0]
            if case["residual"]:
                part += s["residual"][i:i + 1024].double()
            out[i:i + 1024] = part
        if case["out"] != "e4m3":
            return out
        return [(out / s["scale_d"].double()).clamp(-448, 448), torch.max(out.max(), -out.min()).reshape(1)]
    if op in ("norm", "norm_grad"):
        v = s["x"].double()
        if op == "norm" and case["residual"]:
            v = v + s["residual"].double()
        size = (torch.linalg.vector_norm(v, dim=-1, keepdim=True).square() / case["cols"] + EPS).sqrt()
        unit, w = v / size, s["weight"].double()
        if op == "norm_grad":
            # the gradient is g / size without its part along x, but for eps's share
            g = s["dy"].double() * w
            dx = (g - unit * (torch.einsum("rc,rc->r", g, unit) / case["cols"])[:, None]) / size
            if case["dsum"]:
                dx += s["dsum"].double()
            return [dx, torch.einsum("rc,rc->c", s["dy"].double(), unit)]
        y = unit * w
        outs = [v] if case["residual"] else []
        if case["out"] == "rows":
            return outs + _exact_codes(y)
        if case["out"] == "tensor":
            top = torch.max(y.max(), -y.min()).reshape(1)
            return outs + [(y / s["scale"].double()).clamp(-448, 448), top, top / 448]
        return outs + [y]
    c = case["cols"]
    if op == "act":
        x = s["x"].double()
        y = _exact_act(x[:, :c], case["act"])[0]
        if case["gated"]:
            y *= x[:, c:]
        outs = ([y] if case["y"] else []) + (_exact_codes(y) if case["q"] else [])
        if case["checkpoint"]:
            codes, scale = _exact_codes(x.view(case["rows"], -1, c))
            outs += [codes.view_as(x), scale]
        return outs
    x = s["x"].double() if s["x"] is not None else (
        wide(s["x_q"]).view(case["rows"], -1, c) * s["x_scale"].double().unsqueeze(-1)).view(case["rows"], -1)
    value, slope = _exact_act(x[:, :c], case["act"])
    dy = s["dy"].double()
    dx = torch.empty_like(x)
    if case["gated"]:
        torch.mul(dy * x[:, c:], slope, out=dx[:, :c])
        torch.mul(dy, value, out=dx[:, c:])
    else:
        torch.mul(dy, slope, out=dx)
    return [dx] + ([torch.einsum("rc->c", dx)] if case["dbias"] else [])
