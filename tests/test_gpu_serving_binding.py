"""Refusals of the Python serving calls on device tensors, the errors the
library gives back, and the streams that calls go to."""
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _serving import make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


def heads(tokens=6, n=2, dim=64, dtype=torch.bfloat16):
    return torch.randn(tokens, n, dim, device="cuda").to(dtype)


def ints(n, dtype=torch.int32):
    return torch.arange(n, dtype=dtype, device="cuda")


def rotary(dim=64):
    t = torch.empty(50, dim // 2, 2, device="cuda")
    dg.dg_rope_table(t)
    return dg.DgRotary(t)


def test_rope():
    x, rot = heads(), rotary()
    for kw, match in [(dict(out=heads(dtype=torch.float16)), "counterpart"), (dict(out=heads(n=3)), "counterpart"),
                      (dict(positions=ints(5)), "positions must be int32 with 6"),
                      (dict(positions=ints(6, torch.int64)), "positions must be int32"),
                      (dict(positions=ints(12)[::2]), "contiguous"), (dict(positions=ints(6).cpu()), "device memory")]:
        args = dict(x=x, out=torch.empty_like(x), positions=ints(6), rotary=rot)
        args.update(kw)
        with pytest.raises(ValueError, match=match):
            dg.dg_rope(**args)
    with pytest.raises(dg.DgError):                       # a rotation wider than the head
        dg.dg_rope(x, x, ints(6), rotary(128))
    with pytest.raises(AttributeError):
        dg.dg_rope(x, x, ints(6), None)
    dg.dg_rope(x[:0], x[:0], ints(0), rot)


def test_kv_append_and_read():
    cache, k = make_cache(2, 2, 16, 64), heads()
    for kw, match in [(dict(v=heads(5)), "v must have the shape"), (dict(k=heads(n=3), v=heads(n=3)), "cache's heads"),
                      (dict(k=heads(dim=32), v=heads(dim=32)), "cache's heads"),
                      (dict(slots=ints(7)), "slots must be int32 with 6"),
                      (dict(positions=ints(7), rotary=rotary()), "positions must be"),
                      (dict(q=heads(5), q_out=heads(5)), "q must have the tokens"),
                      (dict(q=heads(), q_out=heads(n=4)), "q_out must have the shape"),
                      (dict(q=heads(dtype=torch.float16), q_out=heads(dtype=torch.float16)), "type of k")]:
        args = dict(k=k, v=k, slots=ints(6), cache=cache)
        args.update(kw)
        with pytest.raises(ValueError, match=match):
            dg.dg_kv_append(**args)
    with pytest.raises(dg.DgError):                       # positions without a table
        dg.dg_kv_append(k, k, ints(6), cache, positions=ints(6))
    dg.dg_kv_append(k, k, ints(6), cache)
    for kw, match in [(dict(k=heads(5)), "slots must be int32 with 5"), (dict(k=heads(), v=heads(5)), "v must have"),
                      (dict(v=heads(dim=128)), "cache's heads")]:
        with pytest.raises(ValueError, match=match):
            dg.dg_kv_read(cache, ints(6), **kw)
    a, b = heads(dtype=torch.float16), heads(dtype=torch.float16)
    dg.dg_kv_read(cache, ints(6), a, b)
    only = torch.empty_like(b)
    dg.dg_kv_read(cache, ints(6), v=only)
    assert torch.equal(a, b) and torch.equal(b, only)


def test_attn_decode():
    cache, q = make_cache(4, 2, 16, 64), heads(n=4)
    dg.dg_kv_append(heads(40), heads(40), ints(40), cache)
    base = dict(q=q, out=torch.empty_like(q), cache=cache, page_table=ints(6)[:, None] % 4,
                kv_lens=torch.full((6,), 9, dtype=torch.int32, device="cuda"),
                scratch=torch.empty(dg.dg_attn_decode_scratch(6, 1, 4, cache, 20), dtype=torch.uint8, device="cuda"))
    for kw, match in [(dict(out=heads(n=2)), "counterpart"), (dict(page_table=ints(6)), "page_table"),
                      (dict(page_table=ints(6, torch.int64)[:, None]), "page_table must be int32"),
                      (dict(page_table=ints(6).cpu()[:, None]), "page_table"),
                      (dict(page_table=ints(24).view(6, 4)[:, ::2]), "contiguous rows"),
                      (dict(page_table=ints(4)[:, None]), "same number of tokens"),
                      (dict(kv_lens=ints(5)), "kv_lens must be int32 with 6"),
                      (dict(lse=torch.empty(6, 3, device="cuda")), "lse must be FP32 with 24"),
                      (dict(lse=torch.empty(6, 4, device="cuda").half()), "lse must be FP32"),
                      (dict(prefix_pages=ints(1), prefix_len=17), "every page of the prefix"),
                      (dict(prefix_pages=ints(2, torch.int64), prefix_len=17), "prefix_pages must be int32"),
                      (dict(q=heads(n=4, dim=128), out=heads(n=4, dim=128)), "head_dim")]:
        args = dict(base)
        args.update(kw)
        with pytest.raises(ValueError, match=match):
            dg.dg_attn_decode(**args)
    for kw in (dict(scale=float("nan")), dict(scratch=base["scratch"][:16]), dict(q=heads(n=3), out=heads(n=3)),
               dict(prefix_pages=ints(1), prefix_len=-1)):
        with pytest.raises(dg.DgError):
            dg.dg_attn_decode(**{**base, **kw})
    dg.dg_attn_decode(**base)
    want = base["out"].clone()
    dg.dg_attn_decode(**{**base, "scale": 64 ** -0.5})    # the default scale
    assert torch.equal(base["out"], want)


def test_streams():
    """The current stream, a Stream and a handle."""
    x, rot = heads(), rotary()
    want = torch.empty_like(x)
    dg.dg_rope(x, want, ints(6), rot)
    s, at = torch.cuda.Stream(), ints(6)
    torch.cuda.synchronize()
    for call in (lambda o: dg.dg_rope(x, o, at, rot, stream=s), lambda o: dg.dg_rope(x, o, at, rot, stream=s.cuda_stream)):
        out = torch.zeros_like(x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call(out)                                     # a call on another stream would not be captured
        torch.cuda.synchronize()
        assert not out.any()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    out = torch.zeros_like(x)
    with torch.cuda.stream(s):
        dg.dg_rope(x, out, at, rot)
    s.synchronize()
    assert torch.equal(out, want)
