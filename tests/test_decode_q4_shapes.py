"""flux_attn_decode_q4 in the shape that batches of up to one row per SM take when their table has
room for long requests (one CTA of 16 warps per SM), rows laid end to end and cut anywhere, and
with tables far wider than the lengths."""
import math
import random

import numpy as np
import pytest
import torch

import q4_bounds
import q4_reference as ref
from sparse_attention_flux_b200.flux import FLUX_ERR_DEVICE_CHECK, Context, FluxError
from test_decode_q4 import Cache, normal

pytestmark = pytest.mark.gpu

SA = dict(sink=2, window=60, block=128)      # long enough for rows to be cut


@pytest.fixture(scope="module")
def ctx():
    with Context(0, 64 << 20) as c:
        yield c


def spread(n, top, seed=0, empty=()):
    """n lengths, even over the logarithm up to top, shuffled; the `empty` ones 0."""
    lens = [int(round(top ** ((k + 1) / n))) for k in range(n)]
    random.Random(seed).shuffle(lens)
    for b in empty:
        lens[b] = 0
    return lens


def check(c, q, o, lse, fa, mask, scale=None):
    scale = scale or 1 / math.sqrt(c.d)
    G = q.shape[1] // c.Hkv
    o, lse, q = ref.f64(o), ref.f64(lse), ref.f64(q)
    for b, n in enumerate(c.lens):
        u = ref.live_tokens(n, fa, **mask)
        for h in range(c.Hkv):
            rows = slice(h * G, h * G + G)
            k, v = (ref.values(ref.f64(x[b][:, h]))[u] for x in (c.k, c.v))
            want, wl, tol, ltol = q4_bounds.decode_rows(q[b, rows], k, v, scale)
            err = np.abs(o[b, rows] - want)
            assert np.all(err <= tol), (b, h, float((err / np.maximum(tol, 1e-300)).max()))
            if n:
                assert np.all(np.abs(lse[b, rows] - wl) <= ltol), (b, h)
            else:
                assert np.all(np.isneginf(lse[b, rows]))


@pytest.mark.parametrize("lens,Hq,Hkv,d,page", [
    (spread(33, 9000, 1, [4, 20]), 4, 1, 64, 16),            # 33 rows
    (spread(24, 12000, 2), 16, 2, 128, 64),
    (spread(16, 10000, 3, [0, 15]), 16, 8, 64, 32),          # 128 rows
    (spread(37, 4000, 4), 12, 4, 128, 48),                   # a row per SM
    ([6000] * 26, 3, 3, 64, 128), ([6000] * 20, 8, 4, 128, 64),   # alike, but no whole number of rows per CTA
    (spread(70, 9000, 5, [69]), 14, 2, 64, 16),
])
@pytest.mark.parametrize("fa", [True, False])
def test_rows_cut_across_ctas(ctx, lens, Hq, Hkv, d, page, fa):
    c = Cache(ctx, lens, Hkv, d, page, seed=41, width=-(-20000 // page))
    q = normal((len(lens), Hq, d), 42)
    o, lse = c.decode(ctx, q, fa, **SA)
    ctx.check()
    check(c, q, o, lse, fa, SA)
    again = c.decode(ctx, q, fa, **SA)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("lens,Hkv", [([131072], 1), ([40000, 1, 0], 2), (spread(24, 30000, 6, [7]), 2),
                                      (spread(16, 32768, 7), 8), ([8000] * 10, 8), ([9000] * 80, 2),
                                      (spread(100, 3000, 8, range(0, 100, 3)), 4), ([33], 1), ([700] * 5, 4)])
@pytest.mark.parametrize("fa", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("width", [None, 140000])
def test_every_live_token_counts_once(ctx, lens, Hkv, fa, d, width):
    """With a query of zeros every weight is one and their sum exact: the logarithm of the number
    of live tokens, to a rounding of log2, of its factor and of their product, tells one token."""
    page = 32
    c = Cache(ctx, lens, Hkv, d, page, seed=43, width=width and width // page)
    q = torch.zeros((len(lens), 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
    o, lse = c.decode(ctx, q, fa, **SA)
    ctx.check()
    lse, o = ref.f64(lse), o.double()
    for b, n in enumerate(lens):
        u = ref.live_tokens(n, fa, **SA)
        if n == 0:
            assert np.all(np.isneginf(lse[b])) and (o[b] == 0).all()
            continue
        want = math.log(len(u))
        assert np.all(np.abs(lse[b] - want) <= 4 * q4_bounds.FP32 * want), (b, n, lse[b], want)
        live = torch.as_tensor(u, device="cuda")
        k, v = torch.empty_like(c.k[b]), torch.empty_like(c.v[b])
        u = torch.arange(n, device="cuda")
        ctx.kv_read_q4(c.pool, c.table[b].long()[u // page] * page + u % page, k, v)
        v = v.double()[live]
        mean, size = v.mean(0), v.abs().mean(0)
        tol = q4_bounds.BF16 * mean.abs() + (len(live) / 16 + 32) * 2 * q4_bounds.FP32 * size
        err = (o[b].unflatten(0, (Hkv, 2)) - mean[:, None]).abs()
        assert (err <= tol[:, None]).all(), (b, n)


@pytest.mark.parametrize("sink,window,block", [(0, 1, 64), (1, 1, 128), (0, 3, 100), (2, 2, 33), (3, 50, 16),
                                               (1, 1, 1), (0, 1, 1 << 20), (1 << 20, 1, 1 << 20), (1, 16, 128)])
def test_masks_with_a_wide_table(ctx, sink, window, block):
    mask = dict(sink=sink, window=window, block=block)
    c = Cache(ctx, [1, 130, 999, 2600, 0, 257], 2, 128, 48, seed=44, width=400)
    q = normal((6, 8, 128), 45)
    o, lse = c.decode(ctx, q, False, **mask)
    ctx.check()
    check(c, q, o, lse, False, mask)


@pytest.mark.parametrize("lens,Hkv", [([100], 8), ([1200] * 8, 1), ([100] * 16, 8), ([4000, 33], 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_the_width_of_the_table_says_nothing(ctx, lens, Hkv, d):
    c = Cache(ctx, lens, Hkv, d, 64, seed=46)
    q = normal((len(lens), 4 * Hkv, d), 47)
    narrow = c.table
    wide = torch.full((len(lens), 2048), 10 ** 9, dtype=torch.int32, device="cuda")
    wide[:, :narrow.shape[1]] = narrow
    for table in (narrow, wide):
        c.table = table
        o, lse = c.decode(ctx, q)
        ctx.check()
        check(c, q, o, lse, True, {})


def test_large_values_and_channels_with_a_wide_table(ctx):
    def edit(c):
        for b in range(40):
            c.v[b][::37] *= 1e9
            c.k[b][..., 7] *= 1e6
    lens = spread(40, 5000, 9)
    c = Cache(ctx, lens, 2, 64, 16, seed=48, width=700, edit=edit)
    q = normal((40, 8, 64), 49)
    q[..., 7] *= 1e-6
    o, lse = c.decode(ctx, q)
    ctx.check()
    check(c, q, o, lse, True, {})


def test_nan_stays_with_its_row_where_rows_are_cut(ctx):
    lens = spread(40, 9000, 10)
    at = max(range(40), key=lambda b: lens[b])
    clean = Cache(ctx, lens, 2, 64, 16, seed=50, width=700)
    q = normal((40, 4, 64), 51)
    want, wl = clean.decode(ctx, q)

    def edit(c):
        c.k[at][lens[at] // 2, 1, 3] = float("nan")
    c = Cache(ctx, lens, 2, 64, 16, seed=50, width=700, edit=edit)
    o, lse = c.decode(ctx, q)
    ctx.check()
    assert torch.isnan(o[at, 2:]).all() and torch.isnan(lse[at, 2:]).all()
    rest = torch.ones((40, 4), dtype=torch.bool, device="cuda")
    rest[at, 2:] = False
    assert torch.equal(o[rest], want[rest]) and torch.equal(lse[rest], wl[rest])


def test_missing_pages_with_a_wide_table(ctx):
    lens = spread(40, 5000, 11)
    q = normal((40, 4, 64), 52)
    for bad in (-1, 10 ** 9, 2 ** 31 - 1):
        c = Cache(ctx, lens, 2, 64, 16, seed=53, width=700)
        b = max(range(40), key=lambda i: lens[i])
        c.table[b, 2] = bad
        o, lse = c.decode(ctx, q)
        with pytest.raises(FluxError) as e:
            ctx.check()
        assert e.value.code == FLUX_ERR_DEVICE_CHECK
        u = torch.arange(lens[b], device="cuda")
        keep = u // 16 != 2                            # that page's tokens are left out
        c.k[b], c.v[b] = c.k[b][keep], c.v[b][keep]
        c.lens = [*lens[:b], lens[b] - 16, *lens[b + 1:]]
        check(c, q, o, lse, True, {})
    ctx.check()


def test_many_empty_requests(ctx):
    """Empty requests before, between and behind the others, in both shapes."""
    for B, Hkv, width in ((60, 2, 700), (1000, 2, 20)):
        lens = [0] * B
        for b in range(B // 7, B - B // 5, 11):
            lens[b] = 1 + 37 * b % 310
        c = Cache(ctx, lens, Hkv, 64, 16, seed=54, width=width)
        q = normal((B, 2 * Hkv, 64), 55)
        o, lse = c.decode(ctx, q)
        ctx.check()
        check(c, q, o, lse, True, {})
