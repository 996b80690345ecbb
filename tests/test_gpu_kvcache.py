"""dg_kv_append and dg_kv_read.

Without rotation codes and scales are the quantiser's rule on each (token,
head) row, bit for bit.  With it the scale is within 2^-21 of the FP64 one
(two products, a sum and a division in FP32), and each code is a nearest
E4M3 value of the FP64 quotient up to the same relative error.  Reading back
is one FP32 product rounded once, bit for bit."""
import numpy as np
import pytest
import torch

import fp16_tensor_core_gb300 as dg
import oracle
from _serving import MIN_SCALE, ROUND, TORCH, cached, decode, f64, make_cache, rope64, table64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def quantise_rows(x32):
    """The rule on the last axis: FP32 scales and codes."""
    top = np.abs(x32).max(-1)
    scale = np.maximum((top / np.float32(448.0)).astype(np.float32), MIN_SCALE)
    codes = np.stack([oracle.quantize_e4m3(r, s) for r, s in
                      zip(x32.reshape(-1, x32.shape[-1]), scale.reshape(-1))])
    return scale, codes.reshape(x32.shape)


def inputs(tokens, heads, dim, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, heads, dim, generator=g, device="cuda")
    x *= 10.0 ** (torch.rand(tokens, heads, 1, generator=g, device="cuda") * 4 - 3)   # rows of all sizes
    return x.to(TORCH[dtype])


SHAPES = [  # tokens, kv_heads, dim, page, pages
    (1, 1, 16, 1, 3), (5, 3, 64, 16, 2), (1, 32, 128, 64, 1), (40, 2, 80, 8, 9), (300, 4, 96, 16, 20),
    (17, 1, 256, 32, 2), (2000, 8, 128, 64, 33), (9, 2, 208, 2, 6),
]


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
@pytest.mark.parametrize("tokens,heads,dim,page,pages", SHAPES)
def test_append_without_rotation_is_bit_exact(tokens, heads, dim, page, pages, dtype):
    k, v = inputs(tokens, heads, dim, dtype, 1), inputs(tokens, heads, dim, dtype, 2)
    slots = torch.randperm(pages * page)[:tokens]
    cache = make_cache(pages, heads, page, dim, fill=0x55)
    dg.dg_kv_append(k, v, slots.int().cuda(), cache)
    assert dg.dg_sync_status() == dg.DG_OK
    _, _, kc, vc, ks, vs = cached(cache, slots)
    for x, codes, scale in ((k, kc, ks), (v, vc, vs)):
        ref_scale, ref = quantise_rows(x.float().cpu().numpy())
        assert np.array_equal(scale.view(np.uint32), ref_scale.view(np.uint32))
        assert np.array_equal(codes, ref)
    free = np.setdiff1d(np.arange(pages * page), slots.numpy())      # the other slots are untouched
    if free.size:
        _, _, kc, vc, ks, vs = cached(cache, free)
        assert np.all(kc == 0x55) and np.all(vc == 0x55) and np.isnan(ks).all() and np.isnan(vs).all()


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
@pytest.mark.parametrize("layout", [dg.DG_ROPE_HALF, dg.DG_ROPE_INTERLEAVED])
@pytest.mark.parametrize("tokens,q_heads,heads,dim,rotary,page,pages", [
    (1, 32, 32, 128, 128, 64, 2), (3, 5, 1, 80, 32, 4, 2), (60, 0, 2, 96, 96, 16, 5),
    (31, 8, 4, 256, 64, 32, 1), (1100, 32, 8, 128, 128, 64, 20), (700, 12, 12, 64, 48, 16, 60),
])
def test_append_packed_rows_with_rotation(tokens, q_heads, heads, dim, rotary, page, pages, layout, dtype):
    qkv = inputs(tokens, q_heads + 2 * heads, dim, dtype, 3)
    before = qkv.clone()
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:]
    table = torch.from_numpy(table64(5000, rotary)).float().cuda()
    pos = torch.randint(0, 5000, (tokens,), dtype=torch.int32, device="cuda")
    slots = torch.randperm(pages * page)[:tokens]
    drop = tokens // 3
    dev_slots = slots.int().cuda()
    if tokens > 3:
        dev_slots[drop] = -1
    cache = make_cache(pages, heads, page, dim, fill=0x11)
    rot = dg.DgRotary(table, layout)
    kw = dict(q=q, q_out=torch.empty_like(q)) if q_heads else {}
    dg.dg_kv_append(k, v, dev_slots, cache, positions=pos, rotary=rot, **kw)
    assert dg.dg_sync_status() == dg.DG_OK
    assert torch.equal(qkv, before)
    keep = np.array([i for i in range(tokens) if not (tokens > 3 and i == drop)])
    _, _, kc, vc, ks, vs = cached(cache, slots.numpy()[keep])
    p = pos.cpu().numpy()
    turned = rope64(f64(before)[:, q_heads:q_heads + heads], f64(table), p, layout)[keep]
    want = np.maximum(np.abs(turned).max(-1) / 448.0, 2.0 ** -60)
    assert np.all(np.abs(ks - want) <= 2.0 ** -21 * want)
    y = turned / ks[..., None].astype(np.float64)
    # an element's FP32 rotation is off by 2^-22 of its pair, which is at most 2 * 448 scales
    slack = 2.0 ** -22 * 900.0 + 2.0 ** -22 * np.abs(y)
    assert np.all(np.abs(decode(kc) - np.clip(y, -448, 448)) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) + slack)
    ref_scale, ref = quantise_rows(v.float().cpu().numpy()[keep])
    assert np.array_equal(vs.view(np.uint32), ref_scale.view(np.uint32)) and np.array_equal(vc, ref)
    if tokens > 3:
        _, _, kc, _, ks, _ = cached(cache, slots.numpy()[[drop]])
        assert np.all(kc == 0x11) and np.isnan(ks).all()
    if q_heads:   # the same bits as the rotation alone, also in place
        alone = torch.empty_like(kw["q_out"])
        dg.dg_rope(q, alone, pos, rot)
        assert torch.equal(kw["q_out"], alone)
        dg.dg_kv_append(k, v, dev_slots, cache, positions=pos, rotary=rot, q=q, q_out=q)
        assert torch.equal(q, alone) and torch.equal(qkv[:, q_heads:], before[:, q_heads:])


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
def test_special_rows(dtype):
    """Rows of zeros, of the smallest values, with a NaN or an infinity."""
    dim, n = 64, 6
    x = inputs(n, 1, dim, dtype, 5)
    x[0] = 0.0
    x[1] = 0.0
    x[1, 0, 3] = 2.0 ** -126 if dtype == dg.DG_BF16 else 2.0 ** -24
    x[2, 0, 63] = float("nan")
    x[3, 0, 0] = float("-inf")
    x[4] = 65504.0
    cache = make_cache(1, 1, 8, dim)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    dg.dg_kv_append(x, x, slots, cache)
    _, _, kc, vc, ks, _ = cached(cache, np.arange(n))
    assert ks[0, 0] == MIN_SCALE and not kc[0].any()
    assert ks[1, 0] == max(np.float32(x[1, 0, 3].item()) / np.float32(448.0), MIN_SCALE)
    for i in (2, 3):
        assert np.isnan(ks[i, 0]) and not kc[i].any() and not vc[i].any()
    assert np.all(kc[4] == 0x7E)
    k, v = torch.empty_like(x), torch.empty_like(x)
    dg.dg_kv_read(cache, slots, k, v)
    assert torch.isnan(k[2:4]).all() and not k[0].any() and torch.equal(torch.isnan(k), torch.isnan(v))


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
@pytest.mark.parametrize("tokens,heads,dim,page,pages", SHAPES)
def test_read_back(tokens, heads, dim, page, pages, dtype):
    cache = make_cache(pages, heads, page, dim)
    cache.k.copy_(torch.randint(0, 0x7F, cache.k.shape, dtype=torch.uint8))
    cache.v.copy_(torch.randint(0x80, 0xFF, cache.v.shape, dtype=torch.uint8))
    for s in (cache.k_scale, cache.v_scale):
        s.copy_(10.0 ** (torch.rand(s.shape) * 6 - 6))
    slots = torch.randperm(pages * page)[:tokens]
    if tokens > 4:
        slots[1] = slots[0]     # a slot may be read twice
    k64, v64, kc, vc, ks, vs = cached(cache, slots)
    want = [torch.from_numpy((decode(c).astype(np.float32) * s[..., None])).to(TORCH[dtype])
            for c, s in ((kc, ks), (vc, vs))]
    dev_slots = slots.int().cuda()
    both = torch.full((tokens, 2 * heads + 1, dim), 9.0, dtype=TORCH[dtype], device="cuda")
    dg.dg_kv_read(cache, dev_slots, both[:, :heads], both[:, heads:2 * heads])
    assert torch.equal(both[:, :heads].cpu(), want[0]) and torch.equal(both[:, heads:2 * heads].cpu(), want[1])
    assert torch.all(both[:, 2 * heads] == 9.0)
    one = torch.empty(tokens, heads, dim, dtype=TORCH[dtype], device="cuda")
    dg.dg_kv_read(cache, dev_slots, v=one)
    assert torch.equal(one.cpu(), want[1])
    dg.dg_kv_read(cache, dev_slots, k=one)
    assert torch.equal(one.cpu(), want[0])
    dev_slots[0] = -1
    dg.dg_kv_read(cache, dev_slots, k=one)
    assert not one[0].any() and torch.equal(one[1:].cpu(), want[0][1:])
    assert dg.dg_sync_status() == dg.DG_OK


def test_round_trip_error():
    """Written and read back: off by at most half an E4M3 step of the row."""
    k = inputs(50, 4, 128, dg.DG_FP16, 8)
    cache = make_cache(4, 4, 16, 128)
    slots = torch.randperm(64)[:50].int().cuda()
    dg.dg_kv_append(k, k, slots, cache)
    back = torch.empty_like(k)
    dg.dg_kv_read(cache, slots, v=back)
    x, top = f64(k), np.abs(f64(k)).max(-1, keepdims=True)
    half_step = np.maximum(2.0 ** -4 * np.abs(x), top / 448.0 * 2.0 ** -10)
    assert np.all(np.abs(f64(back) - x) <= half_step * (1 + 2.0 ** -20) + ROUND[dg.DG_FP16] * np.abs(x) + 2.0 ** -24)


def test_slots_and_positions_outside():
    table = torch.from_numpy(table64(10, 16)).float().cuda()
    x = inputs(4, 1, 16, dg.DG_FP16, 9)
    cache = make_cache(2, 1, 4, 16, fill=0x22)
    slots = torch.tensor([0, 8, 1, 2], dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 1, 10, 9], dtype=torch.int32, device="cuda")
    q_out = torch.full_like(x, 3.0)
    dg.dg_kv_append(x, x, slots, cache, positions=pos, rotary=dg.DgRotary(table), q=x, q_out=q_out)
    assert dg.dg_sync_status() == dg.DG_ERR_INVALID_VALUE
    assert torch.all(q_out[1:3] == 3.0) and not torch.any(q_out[0] == 3.0)
    written = (~torch.isnan(cache.k_scale)).flatten().nonzero().flatten().tolist()
    assert written == [0, 2]
    out = torch.full_like(x, 3.0)
    dg.dg_kv_read(cache, slots, k=out)
    assert dg.dg_sync_status() == dg.DG_ERR_INVALID_VALUE
    assert torch.all(out[1] == 3.0)


def test_offsets_past_32_bits():
    """The last page of a cache whose codes pass 4 GiB."""
    heads, page, dim = 8, 64, 128
    pages = (1 << 32) // (heads * page * dim) + 3
    cache = dg.DgKvCache(*(torch.empty(pages, heads, page, dim, dtype=torch.uint8, device="cuda") for _ in range(2)),
                         *(torch.empty(pages, heads, page, device="cuda") for _ in range(2)))
    k = inputs(3, heads, dim, dg.DG_BF16, 4)
    slots = torch.tensor([pages * page - 1, 5, (pages - 1) * page], dtype=torch.int32, device="cuda")
    dg.dg_kv_append(k, k, slots, cache)
    _, _, kc, vc, ks, _ = cached(cache, slots.cpu().numpy())
    scale, codes = quantise_rows(k.float().cpu().numpy())
    assert np.array_equal(kc, codes) and np.array_equal(vc, codes) and np.array_equal(ks, scale)
    back = torch.empty_like(k)
    dg.dg_kv_read(cache, slots, v=back)
    assert torch.equal(back.cpu(), torch.from_numpy(decode(codes).astype(np.float32) * scale[..., None]).bfloat16())
