"""Refusals of the serving entry points (rotary table and positions, cache
writes and reads, attention): every argument error comes back as a status
before anything touches a device.  CPU only."""
import ctypes
import math

import pytest

import fp16_tensor_core_gb300 as dg
from fp16_tensor_core_gb300 import build as dg_build

FAKE = 0x7F0000000000   # aligned, never dereferenced: every call below fails validation
BAD, OFF = dg.DG_ERR_INVALID_VALUE, dg.DG_ERR_MISALIGNED


@pytest.fixture(scope="module")
def L():
    dg_build.build()
    return dg.lib()


def heads(data=FAKE, ts=1024, hs=128):
    return dg._Heads(data, ts, hs)


def rotary(table=FAKE, positions=100, dim=128, layout=0):
    return dg._Rotary(table, positions, dim, layout)


def cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=10, kv_heads=2, page=16, dim=128):
    return dg._KvCache(k, v, ks, vs, pages, kv_heads, page, dim)


def scaling(base=10000.0, kind=0, factor=2.0, original=4096.0, slow=1.0, fast=32.0, magnitude=1.0):
    return dg._RopeScaling(base, kind, factor, original, slow, fast, magnitude)


@pytest.mark.parametrize("kw,expect", [
    (dict(positions=-1), BAD), (dict(dim=24), BAD), (dict(dim=0), BAD), (dict(dim=272), BAD),
    (dict(table=None), BAD), (dict(table=FAKE + 8), OFF), (dict(sc=None), BAD),
    (dict(sc=scaling(base=0.0)), BAD), (dict(sc=scaling(base=math.nan)), BAD),
    (dict(sc=scaling(magnitude=0.0)), BAD), (dict(sc=scaling(kind=4)), BAD),
    (dict(sc=scaling(kind=1, factor=0.0)), BAD), (dict(sc=scaling(kind=3, original=0.0)), BAD),
    (dict(sc=scaling(kind=3, slow=8.0, fast=8.0)), BAD),
])
def test_rope_table(L, kw, expect):
    a = dict(table=FAKE, positions=10, dim=64, sc=scaling())
    a.update(kw)
    sc = None if a["sc"] is None else ctypes.byref(a["sc"])
    assert L.dg_rope_table(a["table"], a["positions"], a["dim"], sc, None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(tokens=-1), BAD), (dict(tokens=1 << 31), BAD), (dict(heads=-1), BAD), (dict(heads=65537), BAD),
    (dict(dim=24), BAD), (dict(dim=272), BAD), (dict(dim=64), BAD), (dict(dtype=dg.DG_E4M3), BAD),
    (dict(x=None), BAD), (dict(x=heads(data=None)), BAD), (dict(x=heads(data=FAKE + 2)), OFF),
    (dict(out=heads(ts=1020)), OFF), (dict(out=heads(hs=4)), OFF), (dict(x=heads(ts=-1024)), BAD),
    (dict(pos=None), BAD), (dict(pos=FAKE + 2), OFF), (dict(rot=None), BAD),
    (dict(rot=rotary(table=None)), BAD), (dict(rot=rotary(table=FAKE + 4)), OFF),
    (dict(rot=rotary(dim=136)), BAD), (dict(rot=rotary(layout=2)), BAD), (dict(rot=rotary(positions=0)), BAD),
])
def test_rope(L, kw, expect):
    a = dict(x=heads(), out=heads(), tokens=4, heads=8, dim=128, pos=FAKE, rot=rotary(), dtype=dg.DG_BF16)
    a.update(kw)
    assert L.dg_rope(a["x"], a["out"], a["tokens"], a["heads"], a["dim"], a["pos"], a["rot"], 0,
                     a["dtype"], None) == expect


CACHE_ERRORS = [
    (dict(cache=None), BAD), (dict(cache=cache(k=None)), BAD), (dict(cache=cache(v=FAKE + 8)), OFF),
    (dict(cache=cache(ks=FAKE + 2)), OFF), (dict(cache=cache(vs=None)), BAD),
    (dict(cache=cache(pages=0)), BAD), (dict(cache=cache(page=48)), BAD), (dict(cache=cache(page=0)), BAD),
    (dict(cache=cache(page=131072)), BAD), (dict(cache=cache(pages=1 << 28)), BAD),
    (dict(cache=cache(kv_heads=0)), BAD), (dict(cache=cache(dim=72)), BAD), (dict(cache=cache(dim=512)), BAD),
    (dict(dtype=7), BAD),
]


@pytest.mark.parametrize("kw,expect", CACHE_ERRORS + [
    (dict(tokens=-3), BAD), (dict(slots=None), BAD), (dict(slots=FAKE + 1), OFF), (dict(k=None), BAD),
    (dict(v=heads(data=FAKE + 8)), OFF), (dict(q=None), BAD), (dict(q_out=None), BAD), (dict(q_heads=0), BAD),
    (dict(rot=None), BAD), (dict(pos=None), BAD), (dict(rot=rotary(dim=144)), BAD), (dict(q=heads(hs=100)), OFF),
])
def test_kv_append(L, kw, expect):
    a = dict(q=heads(), q_out=heads(), q_heads=8, k=heads(), v=heads(), tokens=4, pos=FAKE, rot=rotary(),
             slots=FAKE, cache=cache(), dtype=dg.DG_FP16)
    a.update(kw)
    assert L.dg_kv_append(a["q"], a["q_out"], a["q_heads"], a["k"], a["v"], a["tokens"], a["pos"], a["rot"],
                          a["slots"], a["cache"], a["dtype"], None) == expect


@pytest.mark.parametrize("kw,expect", CACHE_ERRORS + [
    (dict(tokens=-3), BAD), (dict(slots=None), BAD), (dict(slots=FAKE + 1), OFF),
    (dict(v=heads(data=FAKE + 8)), OFF), (dict(k=heads(ts=9)), OFF),
])
def test_kv_read(L, kw, expect):
    a = dict(k=heads(), v=heads(), tokens=4, slots=FAKE, cache=cache(), dtype=dg.DG_FP16)
    a.update(kw)
    assert L.dg_kv_read(a["cache"], a["slots"], a["tokens"], a["k"], a["v"], a["dtype"], None) == expect


@pytest.mark.parametrize("kw,expect", CACHE_ERRORS + [
    (dict(batch=-1), BAD), (dict(batch=2049), BAD), (dict(q_len=0), BAD), (dict(q_heads=0), BAD),
    (dict(q_heads=7), BAD), (dict(cache=cache(dim=96)), BAD), (dict(max_pages=-1), BAD),
    (dict(stride=3), BAD), (dict(max_pages=1 << 28, stride=1 << 28), BAD), (dict(lens=None), BAD),
    (dict(lens=FAKE + 1), OFF), (dict(table=None), BAD), (dict(table=FAKE + 2), OFF),
    (dict(prefix_len=-1), BAD), (dict(prefix_len=5, prefix=None), BAD), (dict(scale=math.inf), BAD),
    (dict(scale=math.nan), BAD), (dict(scratch=None), BAD), (dict(scratch=FAKE + 8), OFF),
    (dict(q=None), BAD), (dict(out=heads(data=None)), BAD), (dict(out=heads(ts=12)), OFF), (dict(lse=FAKE + 2), OFF),
])
def test_attn_decode(L, kw, expect):
    a = dict(q=heads(), out=heads(), lse=FAKE, batch=3, q_len=1, q_heads=8, cache=cache(), table=FAKE, stride=4,
             max_pages=4, lens=FAKE, prefix=FAKE, prefix_len=0, scale=0.1, dtype=dg.DG_BF16, scratch=FAKE,
             size=1 << 40)
    a.update(kw)
    assert L.dg_attn_decode(a["q"], a["out"], a["lse"], a["batch"], a["q_len"], a["q_heads"], a["cache"],
                            a["table"], a["stride"], a["max_pages"], a["lens"], a["prefix"], a["prefix_len"],
                            a["scale"], a["dtype"], a["scratch"], a["size"], None) == expect


def test_scratch_size(L):
    n = ctypes.c_int64()
    get = lambda *a: (L.dg_attn_decode_scratch(*a, 152, ctypes.byref(n)), n.value)  # noqa: E731
    rc, plain = get(8, 1, 32, 128, 0)
    assert rc == dg.DG_OK and plain > 0
    rc, shared = get(8, 1, 32, 128, 100)
    assert rc == dg.DG_OK and shared >= plain + 8 * 32 * 128 * 4
    assert get(8, 1, 32, 96, 0)[0] == BAD and get(-1, 1, 32, 128, 0)[0] == BAD
    assert L.dg_attn_decode_scratch(8, 1, 32, 128, 0, 152, None) == BAD
    # an empty batch needs no pointers
    assert L.dg_attn_decode(None, None, None, 0, 1, 8, cache(), None, 0, 0, None, None, 0, 1.0, dg.DG_BF16,
                            None, 0, None) == dg.DG_OK
