"""Measured cases of the serving operators next to the QKV projection.

Rotary positions (``dg_rope``), the E4M3 key/value cache written and read back
(``dg_kv_append``, ``dg_kv_read``) and attention over that cache with or
without a prefix that the whole batch shares (``dg_attn_decode``).  With
``own`` false, ``run`` computes them in plain torch operations in FP32.
"""
from __future__ import annotations

import math

import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -60
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step's queries and keys of a small batch: latency counts.
        dict(name="rope_step", op="rope", tokens=8, heads=40, dim=128, rotary=128, layout="half",
             dtype="bf16", inverse=False, table=8192),
        # The gradient of a training batch's rotation: interleaved pairs, half of each head, a ragged token count.
        dict(name="rope_gradient", op="rope", tokens=16385, heads=32, dim=128, rotary=64,
             layout="interleaved", dtype="fp16", inverse=True, table=32768),
        # One decode step's cache write behind the 12288-wide QKV projection (32 heads of each).
        dict(name="append_step", op="append", tokens=16, q_heads=32, kv_heads=32, dim=128, rotary=128,
             layout="half", dtype="bf16", page=64, pages=512, table=8192),
        # A prompt's cache write with grouped heads, odd length, small pages, part of the head rotated.
        dict(name="append_prompt", op="append", tokens=16001, q_heads=32, kv_heads=8, dim=128, rotary=64,
             layout="interleaved", dtype="fp16", page=16, pages=1280, table=32768),
        # Reading one request's keys and values back, small and large.
        dict(name="read_short", op="read", tokens=100, kv_heads=32, dim=128, dtype="fp16", page=64, pages=64),
        dict(name="read_long", op="read", tokens=40001, kv_heads=8, dim=128, dtype="bf16", page=64, pages=700),
        # One request's decode step with a short cache, one key head per query head: the smallest call.
        dict(name="attn_single", op="attn", batch=1, q_len=1, q_heads=32, kv_heads=32, dim=128, max_len=300,
             page=64, prefix=0, dtype="bf16"),
        # A ragged serving batch with grouped heads (some requests empty, some of one token).
        dict(name="attn_batch", op="attn", batch=64, q_len=1, q_heads=32, kv_heads=8, dim=128, max_len=4099,
             page=64, prefix=0, dtype="bf16"),
        # Few requests with long caches.
        dict(name="attn_long", op="attn", batch=3, q_len=1, q_heads=32, kv_heads=8, dim=128, max_len=120001,
             page=128, prefix=0, dtype="fp16"),
        # Several new tokens per request (draft verification), 64-wide heads, small pages.
        dict(name="attn_draft", op="attn", batch=24, q_len=5, q_heads=16, kv_heads=4, dim=64, max_len=2500,
             page=16, prefix=0, dtype="fp16"),
        # A batch behind one long system prompt, short own caches.
        dict(name="attn_prefix", op="attn", batch=96, q_len=1, q_heads=32, kv_heads=8, dim=128, max_len=400,
             page=64, prefix=12000, dtype="bf16"),
        # A small batch behind a medium prompt, one key head per query head.
        dict(name="attn_prefix_small", op="attn", batch=12, q_len=1, q_heads=32, kv_heads=32, dim=128,
             max_len=200, page=32, prefix=2000, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n == 3072 else n


HEADS = [(32, 32), (32, 8), (40, 8), (16, 4), (12, 2), (8, 1), (7, 7)]


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attn", "attn", "prefix"])
    dim = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    q_heads, kv_heads = rng.choice(HEADS)
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        heads = rng.choice([1, 3, 8, 32, 40])
        return dict(op=op, tokens=_log(rng, 1, (1 << 26) // (heads * dim) if heads > 3 else 20000),
                    heads=heads, dim=dim, rotary=dim // rng.choice([1, 1, 2, 4]), layout=layout,
                    dtype=dtype, inverse=rng.random() < 0.5, table=32768)
    if op == "append":
        tokens = _log(rng, 1, min(16000, 90_000_000 // ((q_heads + 2 * kv_heads) * dim)))
        page = rng.choice([16, 32, 64, 128])
        return dict(op=op, tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    rotary=dim // rng.choice([1, 1, 2]), layout=layout, dtype=dtype, page=page,
                    pages=tokens // page + rng.randint(2, 40), table=32768)
    if op == "read":
        tokens = _log(rng, 1, 40_000_000 // (kv_heads * dim))
        page = rng.choice([16, 32, 64, 128])
        return dict(op=op, tokens=tokens, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page,
                    pages=tokens // page + rng.randint(2, 40))
    if op == "attn":
        batch = _log(rng, 1, 128)
        most = min(120_000, 250_000_000 // (batch * kv_heads * dim))
        return dict(op=op, batch=batch, q_len=rng.choice([1, 1, 1, 2, 4, 7]), q_heads=q_heads,
                    kv_heads=kv_heads, dim=dim, max_len=_log(rng, 1, most),
                    page=rng.choice([16, 32, 64, 128]), prefix=0, dtype=dtype)
    batch = _log(rng, 2, 96)
    return dict(op="attn", batch=batch, q_len=rng.choice([1, 1, 2]), q_heads=q_heads, kv_heads=kv_heads,
                dim=dim, max_len=_log(rng, 1, 600), page=rng.choice([16, 32, 64, 128]),
                prefix=_log(rng, 16, min(16000, 600_000_000 // (batch * q_heads * dim))), dtype=dtype)


def lens_of(case):
    """The requests' own token counts: spread over 0..max_len, the longest always there."""
    n, most = case["batch"], case["max_len"]
    lens = [most]
    for i in range(1, n):
        lens.append(int(most * ((i * 0.6180339887) % 1.0)))
    if n >= 8:
        lens[3], lens[5] = 0, 1
    return lens


def visible(case):
    """Per request and query: how many of the request's own tokens it sees."""
    q = case["q_len"]
    return [[max(0, n - q + 1 + i) for i in range(q)] for n in lens_of(case)]


def work(case):
    d, op = case["dim"], case["op"]
    if op == "rope":
        t, h = case["tokens"], case["heads"]
        return {"bytes": 4 * t * h * d + t * (4 + 4 * case["rotary"]), "flops": 3 * t * h * case["rotary"]}
    if op == "append":
        t, hq, hk = case["tokens"], case["q_heads"], case["kv_heads"]
        return {"bytes": t * (4 * hq * d + hk * (6 * d + 8) + 8 + 4 * case["rotary"]),
                "flops": t * (3 * (hq + hk) * case["rotary"] + 4 * hk * d)}
    if op == "read":
        t, hk = case["tokens"], case["kv_heads"]
        return {"bytes": t * (hk * (6 * d + 8) + 4), "flops": 2 * t * hk * d}
    b, hq, hk, p = case["batch"], case["q_heads"], case["kv_heads"], case["prefix"]
    cached = sum(max(v) for v in visible(case)) + p
    rows = b * case["q_len"] * hq
    pairs = sum(sum(v) for v in visible(case)) * hq + rows * p
    return {"bytes": cached * hk * 2 * (d + 4) + rows * (4 * d + 4) + 4 * (cached // case["page"] + b),
            "flops": 4 * d * pairs}


# ------------------------------------------------------------------ inputs

def _rotary_table(positions, rotary, device):
    f = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=device) / rotary)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * f
    return torch.stack((a.cos(), a.sin()), dim=-1).float().contiguous()


def _quantise(x):
    """E4M3 codes (as bytes) and FP32 scales of the rows of x."""
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp_min(MIN_SCALE)
    codes = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), scale


def _filled_cache(case, pages, gen):
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    out = []
    for _ in range(2):
        codes, scale = _quantise(torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16).float())
        out += [codes, scale]
    return {"k": out[0], "v": out[2], "k_scale": out[1], "v_scale": out[3]}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dt)

    def permutation(n):
        return torch.randperm(n, generator=gen, device="cuda")

    if op in ("rope", "append"):
        s["table"] = _rotary_table(case["table"], case["rotary"], "cuda")
        # a prompt's positions run on from some start; a step's are each request's own
        t = case["tokens"]
        if t > 256:
            first = int(torch.randint(0, case["table"] - t, (1,), generator=gen, device="cuda").item())
            pos = torch.arange(first, first + t, device="cuda")
        else:
            pos = torch.randint(0, case["table"], (t,), generator=gen, device="cuda")
        s["positions"] = pos.to(torch.int32)
    if op == "rope":
        s["x"] = randn(case["tokens"], case["heads"], case["dim"])
        s["out"] = torch.empty_like(s["x"])
    elif op == "append":
        hq, hk, d, t = case["q_heads"], case["kv_heads"], case["dim"], case["tokens"]
        qkv = randn(t, hq + 2 * hk, d)   # the projection's packed rows
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q_out"] = torch.empty(t, hq, d, dtype=dt, device="cuda")
        shape = (case["pages"], hk, case["page"], d)
        s["cache"] = {"k": torch.zeros(shape, dtype=torch.uint8, device="cuda"),
                      "v": torch.zeros(shape, dtype=torch.uint8, device="cuda"),
                      "k_scale": torch.ones(shape[:3], device="cuda"),
                      "v_scale": torch.ones(shape[:3], device="cuda")}
        if t > 256:   # a prompt fills whole pages of a scattered list
            pages = permutation(case["pages"])[:, None] * case["page"]
            s["slots"] = (pages + torch.arange(case["page"], device="cuda")).reshape(-1)[:t].to(torch.int32)
        else:         # a step writes one slot of each request
            s["slots"] = permutation(case["pages"] * case["page"])[:t].to(torch.int32)
    elif op == "read":
        s["cache"] = _filled_cache(case, case["pages"], gen)
        pages = permutation(case["pages"])[:, None] * case["page"]
        t = case["tokens"]
        s["slots"] = (pages + torch.arange(case["page"], device="cuda")).reshape(-1)[:t].to(torch.int32)
        s["k_out"] = torch.empty(t, case["kv_heads"], case["dim"], dtype=dt, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        b, page = case["batch"], case["page"]
        width = max(1, -(-case["max_len"] // page))
        shared = -(-case["prefix"] // page)
        need = sum(-(-n // page) for n in lens_of(case)) + shared
        order = permutation(need + 3).to(torch.int32)
        s["cache"] = _filled_cache(case, need + 3, gen)
        s["kv_lens"] = torch.tensor(lens_of(case), dtype=torch.int32, device="cuda")
        table = torch.zeros(b, width, dtype=torch.int32)
        order_cpu, at = order.cpu(), shared
        for i, n in enumerate(lens_of(case)):
            k = -(-n // page)
            table[i, :k] = order_cpu[at:at + k]
            at += k
        s["page_table"] = table.cuda()
        s["prefix_pages"] = order[:shared].contiguous() if shared else None
        s["q"] = randn(b * case["q_len"], case["q_heads"], case["dim"]) * 2
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(b * case["q_len"], case["q_heads"], device="cuda")
    return s


# ------------------------------------------------------------------- passes

def _values(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale[..., None]


def _rotate(x, table, positions, layout, inverse=False):
    """x (FP32) with the first 2 * table.shape[1] dims of each head rotated."""
    half = table.shape[1]
    cs = table[positions.long()]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    if inverse:
        s = -s
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    if layout == "half":
        a, b = head[..., :half], head[..., half:]
        turned = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    return torch.cat((turned, rest), dim=-1)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "rope":
        return _rotate(s["x"].float(), s["table"], s["positions"], case["layout"], case["inverse"]).to(s["x"].dtype)
    if op == "append":
        c, page = s["cache"], case["page"]
        slots = s["slots"].long()
        at = (slots // page, slice(None), slots % page)
        q = _rotate(s["q"].float(), s["table"], s["positions"], case["layout"]).to(s["q"].dtype)
        c["k"][at], c["k_scale"][at] = _quantise(_rotate(s["k"].float(), s["table"], s["positions"], case["layout"]))
        c["v"][at], c["v_scale"][at] = _quantise(s["v"].float())
        return _append_outputs(q, c)
    if op == "read":
        c, page = s["cache"], case["page"]
        slots = s["slots"].long()
        at = (slots // page, slice(None), slots % page)
        return [_values(c["k"][at], c["k_scale"][at]).to(s["k_out"].dtype),
                _values(c["v"][at], c["v_scale"][at]).to(s["k_out"].dtype)]
    b, n, hk, d = case["batch"], case["q_len"], case["kv_heads"], case["dim"]
    g = case["q_heads"] // hk
    c, pages = s["cache"], s["page_table"].long()

    def cached(codes, scale, pages):   # pages [..., P] -> [..., heads, tokens, dim]
        return _values(codes[pages], scale[pages]).movedim(-3, -4).flatten(-3, -2)

    q = s["q"].float().view(b, n, hk, g, d) / math.sqrt(d)
    k, v = cached(c["k"], c["k_scale"], pages), cached(c["v"], c["v_scale"], pages)
    score = torch.einsum("bnhgd,bhtd->bhngt", q, k)
    token = torch.arange(score.shape[-1], device="cuda")
    last = s["kv_lens"][:, None] - n + torch.arange(n, device="cuda")
    score = score.masked_fill((token > last[..., None])[:, None, :, None, :], -math.inf)
    if case["prefix"]:
        pages = s["prefix_pages"].long()
        pk = cached(c["k"], c["k_scale"], pages)[:, :case["prefix"]]
        pv = cached(c["v"], c["v_scale"], pages)[:, :case["prefix"]]
        score = torch.cat((torch.einsum("bnhgd,htd->bhngt", q, pk), score), dim=-1)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    p = p / torch.where(total == 0.0, 1.0, total)
    out = torch.einsum("bhngt,bhtd->bnhgd", p[..., case["prefix"]:], v)
    if case["prefix"]:
        out = out + torch.einsum("bhngt,htd->bnhgd", p[..., :case["prefix"]], pv)
    return [out.reshape(b * n, hk * g, d).to(s["q"].dtype), lse.permute(0, 2, 1, 3).reshape(b * n, hk * g)]


def _append_outputs(q, cache):
    """The rotated queries and the whole cache, codes as the values they stand for."""
    return [q, cache["k"].view(torch.float8_e4m3fn), cache["k_scale"],
            cache["v"].view(torch.float8_e4m3fn), cache["v_scale"]]


def _handles(s, dg):
    """What a serving program makes once: its cache and rotary handles and the attention's scratch."""
    if "handles" not in s:
        case, h = s["case"], {}
        if "cache" in s:
            c = s["cache"]
            h["cache"] = dg.DgKvCache(c["k"], c["v"], c["k_scale"], c["v_scale"])
        if "table" in s:
            h["rotary"] = dg.DgRotary(s["table"], layout=dg.DG_ROPE_HALF if case["layout"] == "half"
                                      else dg.DG_ROPE_INTERLEAVED)
        if case["op"] == "attn":
            n = dg.dg_attn_decode_scratch(case["batch"], case["q_len"], case["q_heads"], h["cache"], case["prefix"])
            h["scratch"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        s["handles"] = h
    return s["handles"]


def run(state):
    if not own:
        return _plain(state)
    import fp16_tensor_core_gb300 as dg

    s, case, h = state, state["case"], _handles(state, dg)
    if case["op"] == "rope":
        dg.dg_rope(s["x"], s["out"], s["positions"], h["rotary"], inverse=case["inverse"])
        return s["out"]
    if case["op"] == "append":
        dg.dg_kv_append(s["k"], s["v"], s["slots"], h["cache"], positions=s["positions"], rotary=h["rotary"],
                        q=s["q"], q_out=s["q_out"])
        return _append_outputs(s["q_out"], s["cache"])
    if case["op"] == "read":
        dg.dg_kv_read(h["cache"], s["slots"], s["k_out"], s["v_out"])
        return [s["k_out"], s["v_out"]]
    dg.dg_attn_decode(s["q"], s["out"], h["cache"], s["page_table"], s["kv_lens"], h["scratch"], lse=s["lse"],
                      prefix_pages=s["prefix_pages"], prefix_len=case["prefix"])
    return [s["out"], s["lse"]]


# -------------------------------------------------------------- definitions

def exact(case, seed):
    """The operators' definitions in FP64, one request (or one pair of a rotation) at a time."""
    s = prepare(case, seed)
    op, f8 = case["op"], torch.float8_e4m3fn

    def turned(x, inverse=False):
        half = case["rotary"] // 2
        z = torch.view_as_complex(s["table"].double())[s["positions"].long()][:, None]
        if inverse:
            z = z.conj()
        y = x.double().clone()
        i = torch.arange(half, device="cuda")
        a, b = (2 * i, 2 * i + 1) if case["layout"] == "interleaved" else (i, i + half)
        w = torch.complex(y[..., a], y[..., b]) * z
        y[..., a], y[..., b] = w.real, w.imag
        return y

    if op == "rope":
        return turned(s["x"], case["inverse"])
    if op == "append":
        # a code's value before its rounding to E4M3 is the element over its row's scale
        outs = [turned(s["q"])]
        for x in (turned(s["k"]), s["v"].double()):
            codes = torch.zeros(s["cache"]["k"].shape, dtype=torch.float64, device="cuda")
            scale = torch.ones(codes.shape[:3], dtype=torch.float64, device="cuda")
            rows = torch.maximum(x.abs().amax(-1) / 448, torch.tensor(2.0 ** -60, device="cuda", dtype=torch.float64))
            page, at = s["slots"].long() // case["page"], s["slots"].long() % case["page"]
            codes[page, :, at] = x / rows[..., None]
            scale[page, :, at] = rows
            outs += [codes, scale]
        return outs
    c = s["cache"]
    if op == "read":
        flat = {n: c[n].transpose(1, 2).flatten(0, 1)[s["slots"].long()] for n in c}
        return [flat[n].view(f8).double() * flat[n + "_scale"].double()[..., None] for n in ("k", "v")]
    n, hk, d = case["q_len"], case["kv_heads"], case["dim"]
    g = case["q_heads"] // hk

    def tokens(name, pages, count):   # the first `count` tokens of a list of pages: [heads, count, dim]
        x = c[name][pages].view(f8).double() * c[name + "_scale"][pages].double()[..., None]
        return x.transpose(0, 1).reshape(hk, -1, d)[:, :count]

    empty = torch.zeros(hk, 0, d, dtype=torch.float64, device="cuda")
    pk = pv = empty
    if case["prefix"]:
        pk, pv = (tokens(x, s["prefix_pages"].long(), case["prefix"]) for x in ("k", "v"))
    outs, lses = [], []
    for b, own_len in enumerate(lens_of(case)):
        pages = s["page_table"][b].long()
        k = torch.cat((pk, tokens("k", pages, own_len)), dim=1)
        v = torch.cat((pv, tokens("v", pages, own_len)), dim=1)
        for i in range(n):
            seen = case["prefix"] + max(0, own_len - n + 1 + i)
            q = s["q"][b * n + i].double().view(hk, g, d)
            if seen == 0:
                outs.append(torch.zeros(hk * g, d, dtype=torch.float64, device="cuda"))
                lses.append(torch.full((hk * g,), -math.inf, dtype=torch.float64, device="cuda"))
                continue
            score = q @ k[:, :seen].transpose(1, 2) / d ** 0.5
            outs.append((torch.softmax(score, -1) @ v[:, :seen]).reshape(hk * g, d))
            lses.append(torch.logsumexp(score, -1).reshape(hk * g))
    return [torch.stack(outs), torch.stack(lses)]
