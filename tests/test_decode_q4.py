"""flux_attn_decode_q4 against softmax attention in 64 bits over the stored values."""
import math

import numpy as np
import pytest
import torch

import q4_reference as ref
from sparse_attention_flux_b200.flux import (FLUX_ERR_DEVICE_CHECK, FLUX_ERR_INVALID_ARG, FLUX_ERR_SHAPE,
                                             FLUX_ERR_UNSUPPORTED, Context, FluxError, kv_q4_pool_shape)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    with Context(0, 64 << 20) as c:
        yield c


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


class Cache:
    """Requests of given lengths in a cache whose free bytes are 0xFF (NaN scales) and whose
    table holds nonsense behind each request's pages."""

    def __init__(self, ctx, lens, Hkv, d, page, seed=0, std=1.0, width=None, vstd=1.0, edit=None):
        self.lens, self.Hkv, self.d, self.page = lens, Hkv, d, page
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        ids = np.random.default_rng(seed).permutation(pages)
        self.pool = torch.full(kv_q4_pool_shape(pages, Hkv, page, d), 0xFF, dtype=torch.uint8, device="cuda")
        table = np.full((len(lens), width or max(1, max(need))), 10 ** 9)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        self.table = torch.tensor(table, dtype=torch.int32, device="cuda")
        self.sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.k = [normal((n, Hkv, d), seed + 10 + b, std) for b, n in enumerate(lens)]
        self.v = [normal((n, Hkv, d), seed + 500 + b, vstd) for b, n in enumerate(lens)]
        if edit:
            edit(self)
        for b, n in enumerate(lens):
            if n:
                u = torch.arange(n, device="cuda")
                slots = self.table[b].long()[u // page] * page + u % page
                ctx.kv_write_q4(self.k[b], self.v[b], slots, self.pool)

    def decode(self, ctx, q, fa=True, sink=1, window=16, block=128, scale=None, stream=None):
        o = torch.full_like(q, 9)
        lse = torch.full(q.shape[:2], 9.0, device="cuda")
        lm = torch.tensor([1, 0, 1 if fa else 0], dtype=torch.uint8, device="cuda")
        ctx.attn_decode_q4(q, self.pool, self.table, self.sl, o, scale or 1 / math.sqrt(self.d), layer_mode=lm,
                           layer=2, sink_blocks=sink, window_blocks=window, block=block, lse=lse, stream=stream)
        return o, lse

    def check(self, q, o, lse, fa=True, sink=1, window=16, block=128, scale=None, skip=()):
        scale = scale or 1 / math.sqrt(self.d)
        G = q.shape[1] // self.Hkv
        o, lse, q = ref.f64(o), ref.f64(lse), ref.f64(q)
        for b, n in enumerate(self.lens):
            u = ref.live_tokens(n, fa, sink, window, block)
            u = u[~np.isin(u // self.page, [j for bb, j in skip if bb == b])]
            k, v = ref.values(ref.f64(self.k[b]))[u], ref.values(ref.f64(self.v[b]))[u]
            for h in range(q.shape[1]):
                want, wl, tol, ltol = ref.decode_row(q[b, h], k[:, h // G], v[:, h // G], scale)
                err = np.abs(o[b, h] - want)
                assert np.all(err <= tol), (b, h, float((err - tol).max()))
                assert lse[b, h] == wl if np.isinf(wl) else abs(lse[b, h] - wl) <= ltol, (b, h, lse[b, h], wl)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (10, 2), (6, 1), (7, 1), (16, 2), (32, 8)])
@pytest.mark.parametrize("lens,page", [([1], 16), ([0, 5, 0], 16), ([15, 16, 17, 31, 32, 33], 16),
                                       ([47, 48, 49, 300], 48), ([129, 1, 64, 1000], 64)])
def test_short_requests(ctx, d, Hq, Hkv, lens, page):
    c = Cache(ctx, lens, Hkv, d, page, seed=len(lens))
    q = normal((len(lens), Hq, d), 1)
    o, lse = c.decode(ctx, q)
    ctx.check()
    c.check(q, o, lse)


@pytest.mark.parametrize("d,Hq,Hkv,page,lens", [
    (128, 8, 2, 64, [9000]), (128, 4, 1, 128, [20000, 3]), (64, 8, 1, 16, [7001, 0, 1, 4096]),
    (128, 8, 8, 32, [2500] * 6), (64, 6, 2, 80, [1, 33, 5000, 777, 64, 2, 0, 1500])])
@pytest.mark.parametrize("fa", [True, False])
def test_long_and_ragged_requests(ctx, d, Hq, Hkv, page, lens, fa):
    c = Cache(ctx, lens, Hkv, d, page, seed=3)
    q = normal((len(lens), Hq, d), 2)
    o, lse = c.decode(ctx, q, fa)
    ctx.check()
    c.check(q, o, lse, fa)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 4, 2), (128, 8, 2), (128, 7, 7)])
@pytest.mark.parametrize("fa", [True, False])
@pytest.mark.parametrize("alike", [True, False])
def test_more_rows_than_sms(ctx, d, Hq, Hkv, fa, alike):
    """Up to three times as many (request, kv head) rows as SMs; all of one length, or ragged
    with empty ones and a long one."""
    B = 80 if Hkv == 2 else 50
    lens = [333] * B if alike else np.random.default_rng(d).integers(0, 400, B).tolist()
    if not alike:
        lens[3], lens[40] = 6000, 0
    c = Cache(ctx, lens, Hkv, d, 32, seed=24)
    q = normal((B, Hq, d), 25)
    o, lse = c.decode(ctx, q, fa, 1, 2, 64)
    ctx.check()
    c.check(q, o, lse, fa, 1, 2, 64)
    again = c.decode(ctx, q, fa, 1, 2, 64)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("B,n", [(300, 1), (700, 40), (129, 200), (4096, 3)])
def test_many_short_requests(ctx, B, n):
    g = np.random.default_rng(B)
    c = Cache.__new__(Cache)
    lens = g.integers(0, n + 1, B).tolist()
    c.lens, c.Hkv, c.d, c.page = lens, 2, 64, 16
    need = [-(-x // 16) for x in lens]
    c.pool = torch.full(kv_q4_pool_shape(sum(need) + 1, 2, 16, 64), 0xFF, dtype=torch.uint8, device="cuda")
    width = max(need) + 1
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :need[b]] = np.arange(at, at + need[b])
        at += need[b]
    c.table = torch.tensor(table, dtype=torch.int32, device="cuda")
    c.sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    slots = np.concatenate([np.zeros(0, np.int64)] + [table[b, np.arange(x) // 16] * 16 + np.arange(x) % 16
                                                     for b, x in enumerate(lens)])
    k, v = normal((len(slots), 2, 64), 1), normal((len(slots), 2, 64), 2)
    ctx.kv_write_q4(k, v, torch.tensor(slots, dtype=torch.int64, device="cuda"), c.pool)
    cu = np.concatenate([[0], np.cumsum(lens)])
    c.k = [k[cu[b]:cu[b + 1]] for b in range(B)]
    c.v = [v[cu[b]:cu[b + 1]] for b in range(B)]
    q = normal((B, 4, 64), 3)
    o, lse = c.decode(ctx, q)
    ctx.check()
    c.check(q, o, lse)


@pytest.mark.parametrize("sink,window,block", [(0, 1, 64), (1, 1, 128), (0, 3, 100), (2, 2, 33), (3, 50, 16),
                                               (1, 1, 1), (0, 1, 1 << 20), (1 << 20, 1, 1 << 20), (1, 16, 128)])
def test_sa_masks(ctx, sink, window, block):
    """Blocks that are no multiple of the 16-token records, sinks that meet the window, a
    window or a sink longer than the request."""
    c = Cache(ctx, [1, 130, 999, 2600, 0, 257], 2, 128, 48, seed=4)
    q = normal((6, 8, 128), 5)
    o, lse = c.decode(ctx, q, False, sink, window, block)
    ctx.check()
    c.check(q, o, lse, False, sink, window, block)


def test_sa_reads_only_its_pages(ctx):
    """Table entries outside the sink and the window may hold anything."""
    c = Cache(ctx, [3000, 2000], 2, 128, 64, seed=6)
    q = normal((2, 8, 128), 6)
    for b, n in enumerate(c.lens):
        first = (-(-n // 128) - 4) * 128 // 64
        c.table[b, 2:first] = -1
    o, lse = c.decode(ctx, q, False, 1, 4, 128)
    ctx.check()
    c.check(q, o, lse, False, 1, 4, 128)


@pytest.mark.parametrize("std,scale", [(40.0, None), (1.0, 3.0), (1e-6, None), (1.0, 1e-8)])
def test_sharp_and_flat_scores(ctx, std, scale):
    """One key takes all the weight; running maxima that grow by hundreds; equal weights."""
    c = Cache(ctx, [3000, 17], 2, 128, 64, seed=7, std=std)
    q = normal((2, 8, 128), 7)
    o, lse = c.decode(ctx, q, scale=scale)
    c.check(q, o, lse, scale=scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qstd,kstd,vstd", [(1e-30, 1.0, 1.0), (1e30, 1e-30, 1.0), (1e-30, 1e30, 1.0),
                                            (1.0, 1.0, 1e-25), (1.0, 1.0, 3e6), (1.0, 1.0, 1e25),
                                            (1e10, 1e-20, 1e12), (0.0, 1.0, 1.0)])
def test_magnitudes(ctx, d, qstd, kstd, vstd):
    """Queries, keys and values far from 1: the largest and smallest that the 4-bit form holds
    well within, values around the size at which the kernel changes its arithmetic."""
    c = Cache(ctx, [700, 45], 2, d, 32, seed=20, std=kstd, vstd=vstd)
    q = normal((2, 8, d), 21, qstd)
    o, lse = c.decode(ctx, q)
    ctx.check()
    c.check(q, o, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_a_few_large_values_and_channels(ctx, d):
    """Single tokens of 1e9 among values of 1, one channel of the query 1e6 times the others
    and one of the keys, a head of the query zero."""
    def edit(c):
        c.v[0][::37] *= 1e9
        c.v[0][5, 0, 32:64] = 0
        c.k[0][..., 7] *= 1e6
        c.k[1][..., 40] *= 1e-6
    c = Cache(ctx, [900, 33], 2, d, 16, seed=22, edit=edit)
    q = normal((2, 8, d), 23)
    q[..., 7] *= 1e-6
    q[:, 1, 40] *= 1e6
    q[1, 3] = 0
    o, lse = c.decode(ctx, q)
    c.check(q, o, lse)


def test_nan_stays_with_its_request_and_head(ctx):
    c = Cache(ctx, [500, 40], 2, 64, 16, seed=8)
    c.k[0][123, 1, 3] = float("nan")
    c.v[1][7, 0, 40] = float("inf")
    for b in (0, 1):
        u = torch.arange(c.lens[b], device="cuda")
        ctx.kv_write_q4(c.k[b], c.v[b], c.table[b].long()[u // 16] * 16 + u % 16, c.pool)
    q = normal((2, 4, 64), 8)
    o, lse = c.decode(ctx, q)
    assert torch.isnan(o[0, 2:]).all() and torch.isfinite(o[0, :2]).all()
    assert torch.isnan(o[1, :2, 32:]).all() and torch.isfinite(o[1, :2, :32]).all()
    assert torch.isfinite(o[1, 2:]).all() and torch.isnan(lse[0, 2:]).all() and torch.isfinite(lse[1]).all()


def test_shared_pages(ctx):
    """Two requests with a common prefix use the same pages."""
    c = Cache(ctx, [200, 200], 1, 128, 64, seed=9)
    c.table[1] = c.table[0]
    q = normal((1, 4, 128), 9).repeat(2, 1, 1)
    o, lse = c.decode(ctx, q)
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])


def test_bad_lengths_and_pages(ctx):
    c = Cache(ctx, [100, 90, 80, 70], 2, 64, 16, seed=10)
    q = normal((4, 4, 64), 10)
    c.sl[0], c.sl[2] = -1, c.table.shape[1] * 16 + 1
    o, lse = c.decode(ctx, q)
    with pytest.raises(FluxError) as e:
        ctx.check()
    assert e.value.code == FLUX_ERR_DEVICE_CHECK
    assert (o[[0, 2]] == 0).all() and torch.isneginf(lse[[0, 2]]).all()
    c.lens = [0, 90, 0, 70]
    c.check(q, o, lse)
    for bad in (-1, c.pool.shape[0], 2 ** 31 - 1):
        c = Cache(ctx, [100, 90], 2, 64, 16, seed=11)
        c.table[0, 2] = bad
        o, lse = c.decode(ctx, q[:2])
        with pytest.raises(FluxError) as e:
            ctx.check()
        assert e.value.code == FLUX_ERR_DEVICE_CHECK
        c.check(q[:2], o, lse, skip=[(0, 2)])          # that page's tokens are left out
    ctx.check()


def test_cache_beyond_32_bits(ctx):
    Hkv, page, d = 8, 64, 128
    pages = (9 << 29) // (Hkv * 4 * 18 * d)
    pool = torch.empty(kv_q4_pool_shape(pages, Hkv, page, d), dtype=torch.uint8, device="cuda")
    c = Cache(ctx, [700], Hkv, d, page, seed=12)
    n = c.table.shape[1]
    far = torch.arange(pages - n, pages, device="cuda")
    pool[far] = c.pool[c.table[0].long()]
    q = normal((1, 8, d), 12)
    want, wl = c.decode(ctx, q)
    c.pool, c.table = pool, far.int()[None].contiguous()
    o, lse = c.decode(ctx, q)
    assert torch.equal(o, want) and torch.equal(lse, wl)


def test_two_contexts_on_two_streams(ctx):
    c = Cache(ctx, [5000, 64, 3000, 1], 2, 128, 64, seed=13)
    q = normal((4, 8, 128), 13)
    want = c.decode(ctx, q)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    with Context(0, 16 << 20) as other:
        got = []
        for _ in range(8):
            for st, cx in zip(streams, (ctx, other)):
                with torch.cuda.stream(st):
                    got.append(c.decode(cx, q, stream=st))
        torch.cuda.synchronize()
        for o, lse in got:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_same_call_same_bits(ctx):
    c = Cache(ctx, [30000, 500, 7], 2, 128, 64, seed=14)
    q = normal((3, 16, 128), 14)
    first = c.decode(ctx, q)
    for _ in range(5):
        again = c.decode(ctx, q)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_refusals(ctx):
    c = Cache(ctx, [100, 90], 2, 64, 16, seed=15)
    q = normal((2, 4, 64), 15)
    o = torch.empty_like(q)
    call = lambda **kw: ctx.attn_decode_q4(*[kw.pop(n, v) for n, v in (  # noqa: E731
        ("q", q), ("pool", c.pool), ("table", c.table), ("sl", c.sl), ("o", o), ("scale", 0.125))], **kw)
    for kw, match in ((dict(o=o[:1]), "inconsistent"), (dict(sl=c.sl[:1]), "inconsistent"),
                      (dict(table=c.table[:1]), "inconsistent"), (dict(table=c.table.long()), "must be"),
                      (dict(q=q.float()), "must be"), (dict(pool=c.pool[..., :-1].contiguous()), "kv_pool"),
                      (dict(lse=torch.empty(7, device="cuda")), "lse"),
                      (dict(layer_mode=torch.ones(1, dtype=torch.uint8, device="cuda"), layer=1), "layer")):
        with pytest.raises(ValueError, match=match):
            call(**kw)
    for kw, code in ((dict(scale=0.0), FLUX_ERR_INVALID_ARG), (dict(scale=float("nan")), FLUX_ERR_INVALID_ARG),
                     (dict(window_blocks=0), FLUX_ERR_INVALID_ARG), (dict(block=0), FLUX_ERR_INVALID_ARG),
                     (dict(sink_blocks=-1), FLUX_ERR_INVALID_ARG)):
        with pytest.raises(FluxError) as e:
            call(**kw)
        assert e.value.code == code
    for Hq in (3, 18):                                 # no whole group; 9 query heads per kv head
        x = normal((2, Hq, 64), 1)
        with pytest.raises(FluxError) as e:
            call(q=x, o=torch.empty_like(x))
        assert e.value.code == FLUX_ERR_UNSUPPORTED
    need = ctx.decode_q4_workspace_bytes(64)
    if need > 256:
        with Context(0, 256) as small, pytest.raises(FluxError) as e:
            small.attn_decode_q4(q, c.pool, c.table, c.sl, o, 0.125)
        assert e.value.code == FLUX_ERR_SHAPE
