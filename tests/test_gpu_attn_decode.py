"""dg_attn_decode against FP64 attention over the decoded cache.

Bounds, per row with weights p (FP64), u the output type's unit roundoff:
* a score is an FP32 sum of dim products (each exact in FP32: 11 and 4
  significant bits; FP32 accumulation of a tensor-core MMA, 2^-21 of the sum
  of their magnitudes), scaled three times, so off by d = 2^-20 * max_t
  sum |q k| scale; together with the exponential (2^-21) a weight is off by a
  factor 1 + 2 d + 2^-20, in numerator and denominator;
* a weight enters the second product as FP16: 2^-11 of itself, or 2^-25 of
  the row's largest weight-times-value-scale when that is more (for each of
  the n tokens, times a code of at most 448);
* so |out - ref| <= (2^-11 + 4 d + 2^-19) sum p |v| + n 2^-25 top + u |ref|
  (+ 2^-25: FP16 subnormals), and |lse - ref| <= 2 d + 2^-19 (1 + |ref|)."""
import numpy as np
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from _serving import ROUND, TORCH, attention64, cached, f64, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp16_tensor_core_gb300 import build
    build.build()
    dg.dg_init()
    yield
    assert dg.dg_sync_status() == dg.DG_OK


class Case:
    """A filled cache, requests with scattered pages, a shared prefix."""

    def __init__(self, lens, q_len=1, q_heads=8, kv_heads=2, dim=128, page=16, prefix=0, dtype=dg.DG_BF16,
                 seed=0, q_size=2.0, spread=0.5, extra_pages=2, width=None):
        rng = np.random.default_rng(seed)
        self.lens, self.q_len, self.prefix, self.dtype = list(lens), q_len, prefix, dtype
        self.q_heads, self.dim, self.page = q_heads, dim, page
        b = len(self.lens)
        need = [-(-n // page) for n in self.lens]
        shared = -(-prefix // page)
        total = sum(need) + shared + extra_pages
        self.cache = make_cache(total, kv_heads, page, dim, fill=0x7F)   # unused slots: NaN codes and scales
        order = rng.permutation(total)
        self.prefix_pages = order[:shared]
        width = max(need + [1]) if width is None else width
        table = np.full((b, width), 2 ** 30, dtype=np.int32)             # entries past a length are not read
        at = shared
        self.slots = []
        for i, n in enumerate(self.lens):
            pages = order[at:at + need[i]]
            table[i, :need[i]] = pages
            at += need[i]
            self.slots.append((pages[:, None] * page + np.arange(page)).reshape(-1)[:n])
        self.prefix_slots = (self.prefix_pages[:, None] * page + np.arange(page)).reshape(-1)[:prefix]
        every = np.concatenate(self.slots + [self.prefix_slots]).astype(np.int32)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)

        def rows():
            x = torch.randn(every.size, kv_heads, dim, generator=g, device="cuda")
            return (x * torch.exp(spread * torch.randn(every.size, kv_heads, 1, generator=g, device="cuda"))).to(TORCH[dtype])

        if every.size:
            dg.dg_kv_append(rows(), rows(), torch.from_numpy(every).cuda(), self.cache)
        self.q = (torch.randn(b * q_len, q_heads, dim, generator=g, device="cuda") * q_size).to(TORCH[dtype])
        self.table = torch.from_numpy(table).cuda()
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.pp = torch.from_numpy(self.prefix_pages.astype(np.int32)).cuda() if prefix else None
        n = dg.dg_attn_decode_scratch(b, q_len, q_heads, self.cache, prefix)
        self.scratch = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, **kw):
        out = torch.full_like(self.q, 7.0)
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        args = dict(q=self.q, out=out, cache=self.cache, page_table=self.table, kv_lens=self.kv_lens,
                    scratch=self.scratch, lse=lse, prefix_pages=self.pp, prefix_len=self.prefix)
        args.update(kw)
        dg.dg_attn_decode(**args)
        return args["out"], args["lse"]

    def reference(self, requests=None, scale=None):
        scale = self.dim ** -0.5 if scale is None else scale
        got = []
        for b in requests if requests is not None else range(len(self.lens)):
            n, slots = self.lens[b], np.concatenate([self.prefix_slots, self.slots[b]])
            k, v, _, _, _, vs = cached(self.cache, slots)
            tok = np.arange(slots.size)
            seen = np.stack([tok < self.prefix + max(0, n - self.q_len + 1 + i) for i in range(self.q_len)])
            q = f64(self.q[b * self.q_len:(b + 1) * self.q_len])
            got.append(attention64(q, k, v, vs.astype(np.float64), scale, seen))
        return [np.concatenate(x) for x in zip(*got)]

    def check(self, out, lse, requests=None, scale=None):
        ref, ref_lse, pv, qk, top = self.reference(requests, scale)
        if requests is not None:
            rows = np.concatenate([np.arange(b * self.q_len, (b + 1) * self.q_len) for b in requests])
            out, lse = out[rows], lse[rows]
        out, lse = f64(out), f64(lse)
        d = 2.0 ** -20 * qk
        n = max(self.lens) + self.prefix
        tol = (2.0 ** -11 + 4 * d + 2.0 ** -19)[..., None] * pv + (n * 2.0 ** -25 * top)[..., None] + \
            ROUND[self.dtype] * np.abs(ref) + 2.0 ** -25
        assert np.all(np.abs(out - ref) <= tol), np.max(np.abs(out - ref) / tol)
        empty = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(lse), empty) and not out[empty].any()
        err = np.abs(lse[~empty] - ref_lse[~empty])
        assert np.all(err <= 2 * d[~empty] + 2.0 ** -19 * (1 + np.abs(ref_lse[~empty]))), err.max()


LENS = [0, 1, 31, 32, 33, 63, 64, 65, 200, 511]


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (6, 6), (8, 2), (20, 1), (32, 8)])
def test_lengths_and_head_layouts(q_heads, kv_heads, dim, dtype):
    c = Case(LENS, q_heads=q_heads, kv_heads=kv_heads, dim=dim, dtype=dtype)
    c.check(*c.run())


@pytest.mark.parametrize("page", [1, 2, 8, 32, 64, 1024])
@pytest.mark.parametrize("prefix", [0, 70])
def test_page_sizes(page, prefix):
    c = Case([3, 100, 0, 65], page=page, prefix=prefix, q_heads=4, kv_heads=2, dim=64, dtype=dg.DG_FP16)
    c.check(*c.run())


@pytest.mark.parametrize("q_len", [2, 5, 16, 40])
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(4, 4, 64), (8, 2, 128), (14, 2, 128), (6, 2, 256)])
def test_several_new_tokens(q_len, q_heads, kv_heads, dim):
    """Causal among the new tokens; requests shorter than the new tokens
    leave rows that see nothing."""
    c = Case([0, 1, 3, 33, 64, 300], q_len=q_len, q_heads=q_heads, kv_heads=kv_heads, dim=dim)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
@pytest.mark.parametrize("prefix", [1, 32, 33, 1000])
@pytest.mark.parametrize("batch,q_len,q_heads,kv_heads,dim", [
    (1, 1, 4, 4, 64), (7, 1, 8, 2, 128), (40, 1, 16, 2, 128), (9, 3, 10, 1, 64), (5, 2, 4, 2, 256),
])
def test_shared_prefix(batch, q_len, q_heads, kv_heads, dim, prefix, dtype):
    lens = [(37 * i) % 90 for i in range(batch)]
    c = Case(lens, q_len=q_len, q_heads=q_heads, kv_heads=kv_heads, dim=dim, prefix=prefix, dtype=dtype)
    c.check(*c.run())


@pytest.mark.parametrize("batch,q_len,q_heads,kv_heads,dim,prefix", [
    (70, 1, 16, 4, 128, 2100), (33, 4, 8, 2, 64, 777), (130, 1, 8, 8, 128, 515), (64, 2, 8, 1, 128, 4097),
])
def test_prefix_of_many_rows(batch, q_len, q_heads, kv_heads, dim, prefix):
    lens = [(53 * i) % 70 for i in range(batch)]
    c = Case(lens, q_len=q_len, q_heads=q_heads, kv_heads=kv_heads, dim=dim, prefix=prefix, page=32)
    c.check(*c.run(), requests=[0, 1, batch // 2, batch - 1])


def test_prefix_is_the_same_as_own_pages():
    """A prefix split off a request's own pages: the same attention."""
    c = Case([500, 500], q_heads=8, kv_heads=2, dim=128, page=16, dtype=dg.DG_FP16)
    c.table[1] = c.table[0]
    c.slots[1] = c.slots[0]
    want = c.run()
    shared = 320
    c2_lens = torch.tensor([180, 180], dtype=torch.int32, device="cuda")
    scratch = torch.empty(dg.dg_attn_decode_scratch(2, 1, 8, c.cache, shared), dtype=torch.uint8, device="cuda")
    got = c.run(page_table=c.table[:, shared // 16:], kv_lens=c2_lens, scratch=scratch,
                prefix_pages=c.table[0, :shared // 16].contiguous(), prefix_len=shared)
    c.check(*want)
    c.check(*got)


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
def test_long_cache_over_all_sms(dtype):
    c = Case([40_001, 7], q_heads=8, kv_heads=4, dim=128, page=64, dtype=dtype)
    c.check(*c.run())


def test_many_short_requests():
    lens = [(i * 29) % 150 for i in range(700)]
    c = Case(lens, q_heads=8, kv_heads=8, dim=64, page=32, dtype=dg.DG_FP16)
    c.check(*c.run(), requests=list(range(0, 700, 23)) + [699])


@pytest.mark.parametrize("dtype", [dg.DG_BF16, dg.DG_FP16])
def test_sharp_and_uneven_scores(dtype):
    """Scores of hundreds and value rows of very different sizes."""
    c = Case([700, 90], q_heads=4, kv_heads=1, dim=128, dtype=dtype, q_size=30.0, spread=2.5, seed=5)
    c.check(*c.run())


def test_scale_argument_and_tiny_queries():
    c = Case([300], q_heads=4, kv_heads=1, dim=64, dtype=dg.DG_BF16, q_size=1e-30)
    c.check(*c.run(scale=1e29), scale=1e29)
    c.check(*c.run(scale=-3e29), scale=-3e29)
    c.check(*c.run(scale=0.0), scale=0.0)


def test_values_of_zero_and_of_the_smallest_scale():
    """A row of zeros has the smallest scale: it takes its share of the
    softmax and does not spoil the others' precision."""
    c = Case([100], q_heads=2, kv_heads=1, dim=64, dtype=dg.DG_FP16)
    x = torch.randn(100, 1, 64, device="cuda").half()
    v = torch.randn(100, 1, 64, device="cuda").half() * 1e-2
    v[::3] = 0.0
    dg.dg_kv_append(x, v, torch.from_numpy(c.slots[0].astype(np.int32)).cuda(), c.cache)
    c.check(*c.run())


def poison(c, slot, key):
    """A key (or value) row written with a NaN."""
    x = torch.randn(1, c.cache.kv_heads, c.dim, device="cuda").to(TORCH[c.dtype])
    y = x.clone()
    y[0, :, 1] = float("nan")
    at = torch.tensor([slot], dtype=torch.int32, device="cuda")
    dg.dg_kv_append(y if key else x, x if key else y, at, c.cache)


@pytest.mark.parametrize("key", [True, False])
def test_nan_reaches_only_rows_that_see_it(key):
    c = Case([80, 81, 82], q_len=3, q_heads=4, kv_heads=2, dim=64, dtype=dg.DG_FP16)
    ref = c.run()
    poison(c, int(c.slots[1][79]), key)      # the middle query's own token of request 1 (of 81)
    out, lse = c.run()
    hit = torch.zeros(9, dtype=torch.bool)
    hit[4:6] = True
    assert torch.isnan(out[hit]).all()
    assert torch.equal(out[~hit], ref[0][~hit]) and torch.equal(lse[~hit], ref[1][~hit])


def test_infinite_query():
    c = Case([50, 50], q_heads=4, kv_heads=2, dim=64, dtype=dg.DG_BF16)
    ref = c.run()[0]
    c.q[0, 1, 5] = float("inf")
    out = c.run()[0]
    assert torch.isnan(out[0, 1]).all()
    out[0, 1] = ref[0, 1]
    assert torch.equal(out, ref)


def test_strided_queries_and_outputs():
    """Queries inside packed QKV rows; outputs in rows of another pitch."""
    c = Case([100, 3, 257], q_heads=8, kv_heads=2, dim=128, dtype=dg.DG_BF16)
    want = c.run()
    packed = torch.randn(3, 12, 128, device="cuda").bfloat16()
    packed[:, :8] = c.q
    wide = torch.full((3, 9, 136), 5.0, device="cuda").bfloat16()
    out, lse = c.run(q=packed[:, :8], out=wide[:, :8, :128])
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.all(wide[:, 8] == 5.0) and torch.all(wide[..., 128:] == 5.0)
    assert torch.equal(c.run(lse=None)[0], want[0])


def test_repeatable_and_on_streams():
    """The same bits each time, on another stream, and replayed as a graph."""
    c = Case([5000, 1, 0, 333], q_heads=16, kv_heads=4, dim=128, prefix=900)
    want = c.run()
    for _ in range(3):
        got = c.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = torch.zeros_like(c.q), torch.zeros_like(want[1])
    with torch.cuda.stream(s):
        c.run(out=out, lse=lse)
    s.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        c.run(out=out, lse=lse)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_bad_lengths_and_pages_are_reported():
    """No access leaves the cache; the other requests are right."""
    c = Case([70, 40, 90], q_heads=4, kv_heads=2, dim=64, page=16, dtype=dg.DG_FP16)
    c.kv_lens[1] = 10_000
    out, lse = c.run()
    assert dg.dg_sync_status() == dg.DG_ERR_INVALID_VALUE
    c.check(out, lse, requests=[0, 2])
    assert not out[1].any() and torch.isneginf(lse[1]).all()
    c.kv_lens[1] = -4
    c.run()
    assert dg.dg_sync_status() == dg.DG_ERR_INVALID_VALUE
    c.kv_lens[1] = 40
    c.table[1, 1] = c.cache.c.pages
    out, lse = c.run()
    assert dg.dg_sync_status() == dg.DG_ERR_INVALID_VALUE
    c.check(out, lse, requests=[0, 2])


def test_offsets_past_32_bits():
    """Pages past 4 GiB of codes."""
    heads, page, dim = 8, 64, 128
    pages = (1 << 32) // (heads * page * dim) + 40
    c = Case([130, 1000], q_heads=8, kv_heads=heads, dim=dim, page=page, dtype=dg.DG_BF16)
    far = make = dg.DgKvCache(*(torch.empty(pages, heads, page, dim, dtype=torch.uint8, device="cuda") for _ in range(2)),
                              *(torch.empty(pages, heads, page, device="cuda") for _ in range(2)))
    n, move = c.cache.c.pages, pages - c.cache.c.pages
    for a, b in ((make.k, c.cache.k), (make.v, c.cache.v), (make.k_scale, c.cache.k_scale), (make.v_scale, c.cache.v_scale)):
        a[move:move + n] = b
    want = c.run()
    out, lse = c.run(cache=far, page_table=torch.where(c.table < n, c.table + move, c.table))
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_empty_batch_and_all_empty_requests():
    c = Case([0, 0, 0], q_len=2, q_heads=4, kv_heads=2, dim=128)
    out, lse = c.run()
    assert not out.any() and torch.isneginf(lse).all()
    c = Case([0, 0], q_heads=4, kv_heads=2, dim=128, prefix=40)
    c.check(*c.run())
    dg.dg_attn_decode(c.q[:0], c.q[:0], c.cache, c.table[:0], c.kv_lens[:0], c.scratch)
