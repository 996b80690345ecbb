"""FP64 definitions of the serving operators (rotary positions, E4M3
key/value cache, attention over it) and helpers shared by their tests."""
from __future__ import annotations

import numpy as np
import torch

import fp16_tensor_core_gb300 as dg
import oracle

TORCH = {dg.DG_BF16: torch.bfloat16, dg.DG_FP16: torch.float16}
ROUND = {dg.DG_BF16: 2.0 ** -8, dg.DG_FP16: 2.0 ** -11}   # unit roundoff: 8 and 11 significant bits
MIN_SCALE = np.float32(2.0 ** -60)


def f64(t):
    return t.detach().double().cpu().numpy()


def decode(codes):
    """E4M3 codes (any shape, uint8) -> float64 values."""
    return np.asarray(oracle.e4m3_decode(np.arange(256, dtype=np.uint8)), dtype=np.float64)[codes]


def table64(positions, rotary_dim, base=10000.0):
    f = base ** (-np.arange(0, rotary_dim, 2, dtype=np.float64) / rotary_dim)
    a = np.arange(positions, dtype=np.float64)[:, None] * f
    return np.stack((np.cos(a), np.sin(a)), axis=-1)


def rope64(x, table, positions, layout, inverse=False):
    """x float64 [tokens, heads, dim]; table float64 [positions, half, 2]."""
    half = table.shape[1]
    c, s = table[positions][:, None, :, 0], table[positions][:, None, :, 1]
    if inverse:
        s = -s
    i = np.arange(half)
    a, b = (i, i + half) if layout == dg.DG_ROPE_HALF else (2 * i, 2 * i + 1)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def make_cache(pages, kv_heads, page, dim, fill=None):
    shape = (pages, kv_heads, page, dim)
    k = torch.zeros(shape, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.ones(shape[:3], device="cuda")
    vs = torch.ones(shape[:3], device="cuda")
    if fill is not None:
        k.fill_(fill)
        v.fill_(fill)
        ks.fill_(float("nan"))
        vs.fill_(float("nan"))
    return dg.DgKvCache(k, v, ks, vs)


def cached(cache, slots):
    """Float64 keys and values [tokens, kv_heads, dim] of cache slots (host),
    and the codes and scales they come from."""
    page = cache.c.page_size
    p, o = torch.as_tensor(slots).long().cuda() // page, torch.as_tensor(slots).long().cuda() % page
    kc, vc = cache.k[p, :, o].cpu().numpy(), cache.v[p, :, o].cpu().numpy()
    ks, vs = cache.k_scale[p, :, o].cpu().numpy(), cache.v_scale[p, :, o].cpu().numpy()
    return (decode(kc) * ks[..., None].astype(np.float64),
            decode(vc) * vs[..., None].astype(np.float64), kc, vc, ks, vs)


def attention64(q, k, v, vs, scale, seen):
    """One request's rows: q [rows, heads, dim]; k, v [tokens, kv_heads, dim];
    row i sees the tokens where seen[i] is true.  Returns out, lse and, per
    element, the bounds' ingredients: sum of p |v|, the largest sum of |q k|
    scale, and 448 * the largest p * value scale."""
    rows, heads, dim = q.shape
    group = heads // k.shape[1]
    out = np.zeros((rows, heads, dim))
    lse = np.full((rows, heads), -np.inf)
    pv, qk, top = np.zeros_like(out), np.zeros_like(lse), np.zeros_like(lse)
    for i in range(rows):
        idx = np.flatnonzero(seen[i])
        if idx.size == 0:
            continue
        for h in range(heads):
            kk, vv = k[idx, h // group], v[idx, h // group]
            x = kk @ q[i, h] * scale
            m = x.max()
            e = np.exp(x - m)
            p = e / e.sum()
            out[i, h] = p @ vv
            lse[i, h] = m + np.log(e.sum())
            pv[i, h] = p @ np.abs(vv)
            qk[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
            top[i, h] = 448.0 * (p * vs[idx, h // group]).max()
    return out, lse, pv, qk, top
