"""Rows into and out of the paged 4-bit cache: bit-exact against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import q4_reference as ref
from sparse_attention_flux_b200.flux import (FLUX_ERR_DEVICE_CHECK, FLUX_ERR_INVALID_ARG,
                                             FLUX_ERR_UNSUPPORTED, Context, FluxError, kv_q4_pool_shape)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    with Context(0, 16 << 20) as c:
        yield c


def pool_of(pages, Hkv, page, d, fill=0xFF):
    return torch.full(kv_q4_pool_shape(pages, Hkv, page, d), fill, dtype=torch.uint8, device="cuda")


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def there_and_back(ctx, k, v, slots, pool):
    ctx.kv_write_q4(k, v, slots, pool)
    ko, vo = torch.full_like(k, 3).contiguous(), torch.full_like(v, 3).contiguous()
    ctx.kv_read_q4(pool, slots, ko, vo)
    return ko, vo


def same_values(got, x):
    want = ref.values(ref.f64(x))
    got = ref.f64(got)
    return np.array_equal(got, want, equal_nan=True)


def run_slots(N, page, offset, pages, seed=0):
    """A request's slots from token `offset` of its first page on, pages in random order."""
    ids = np.random.default_rng(seed).permutation(pages)
    u = offset + np.arange(N)
    return torch.tensor(ids[u // page] * page + u % page, dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("N,page,offset", [(1, 16, 0), (1, 64, 63), (15, 16, 3), (16, 16, 0),
                                           (17, 48, 15), (33, 32, 31), (500, 64, 7), (1000, 128, 0),
                                           (2049, 16, 5)])
def test_runs(ctx, d, Hkv, N, page, offset):
    pages = (N + offset) // page + 2
    pool = pool_of(pages, Hkv, page, d)
    k, v = normal((N, Hkv, d), 1, 2.0), normal((N, Hkv, d), 2, 0.3)
    ko, vo = there_and_back(ctx, k, v, run_slots(N, page, offset, pages), pool)
    ctx.check()
    assert same_values(ko, k) and same_values(vo, v)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 16, 63, 300])
def test_scattered_tokens_leave_the_others(ctx, d, N):
    """Single tokens in any order: every other slot keeps its bytes' meaning."""
    Hkv, page, pages = 2, 48, 20
    pool = pool_of(pages, Hkv, page, d)
    every = torch.arange(pages * page, device="cuda")
    k0, v0 = normal((pages * page, Hkv, d), 3), normal((pages * page, Hkv, d), 4)
    ctx.kv_write_q4(k0, v0, every, pool)
    slots = torch.randperm(pages * page, device="cuda", generator=torch.Generator("cuda").manual_seed(N))[:N]
    k, v = normal((N, Hkv, d), 5), normal((N, Hkv, d), 6)
    ctx.kv_write_q4(k, v, slots.contiguous(), pool)
    k0[slots], v0[slots] = k, v
    ko, vo = torch.empty_like(k0), torch.empty_like(v0)
    ctx.kv_read_q4(pool, every, ko, vo)
    assert same_values(ko, k0) and same_values(vo, v0)


def test_prompt_equals_token_by_token(ctx):
    """The bytes do not depend on how many tokens a call brings or where it starts."""
    N, Hkv, d, page = 200, 2, 128, 64
    k, v = normal((N, Hkv, d), 7), normal((N, Hkv, d), 8)
    slots = run_slots(N, page, 0, 4)
    one, many = pool_of(4, Hkv, page, d, 0), pool_of(4, Hkv, page, d, 0)
    ctx.kv_write_q4(k, v, slots, one)
    at = 0
    for n in (1, 1, 5, 16, 9, 64, 3, 101):
        ctx.kv_write_q4(k[at:at + n], v[at:at + n], slots[at:at + n].contiguous(), many)
        at += n
    assert at == N and torch.equal(one, many)


def test_stored_values_store_again_as_the_same_bits(ctx):
    N, Hkv, d, page = 333, 4, 128, 32
    k, v = normal((N, Hkv, d), 9, 5.0), normal((N, Hkv, d), 10, 1e-5)
    slots = run_slots(N, page, 3, 12)
    a, b = pool_of(12, Hkv, page, d, 0), pool_of(12, Hkv, page, d, 0)
    ko, vo = there_and_back(ctx, k, v, slots, a)
    there_and_back(ctx, ko, vo, slots, b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128])
def test_borders_of_the_rounding(ctx, d):
    """Groups built so that elements sit on rounding borders and beside them, for every
    5-bit scale, and the largest element on every 8-bit value (its quotient by 7 on and
    beside the scale's own border)."""
    rows = []
    for m in range(128, 256):                      # amax = m 2^-4
        s = ref.quantise(np.full(32, m / 16.0))[1][0]
        g = np.zeros(32)
        g[0] = m / 16.0
        for i, n in enumerate(range(-7, 7)):
            tie = torch.tensor((n + 0.5) * s, dtype=torch.float64).to(torch.bfloat16).double().item()
            g[1 + 2 * i] = np.clip(tie, -g[0], g[0])
            near = torch.tensor(tie).to(torch.bfloat16)
            near = torch.nextafter(near, torch.tensor(0.0, dtype=torch.bfloat16)) if i % 2 else near
            g[2 + 2 * i] = np.clip(near.double().item(), -g[0], g[0])
        rows.append(g)
    x = ref.bf16(np.array(rows).reshape(-1, 1, d)).cuda()
    pool = pool_of(20, 1, 16, d)
    slots = run_slots(len(x), 16, 0, 20)
    ko, vo = there_and_back(ctx, x, -x, slots, pool)
    assert same_values(ko, x) and same_values(vo, -x)


@pytest.mark.parametrize("d", [64, 128])
def test_extreme_groups(ctx, d):
    """Zeros, minus zeros, values at and under 2^-100, at and over 2^120, infinities and NaN:
    each only in its own group."""
    specials = [0.0, -0.0, 2.0 ** -133, 2.0 ** -100, -(2.0 ** -100), 2.0 ** -101, 2.0 ** 120, -(2.0 ** 120),
                2.0 ** 121, np.inf, -np.inf, np.nan, 3.0e38, 1.0]
    x = normal((len(specials), 1, d), 11)
    for i, sp in enumerate(specials):
        x[i, 0, :32] = 0 if abs(sp) < 1 else x[i, 0, :32]
        x[i, 0, 5 + i] = sp
    pool = pool_of(2, 1, 16, d)
    slots = torch.arange(len(specials), device="cuda") + 1
    ko, vo = there_and_back(ctx, x, x.flip(-1).contiguous(), slots, pool)
    assert same_values(ko, x) and same_values(vo, x.flip(-1))
    assert torch.isnan(ko[8:13, 0, :32]).all() and torch.isfinite(ko[:, :, 32:]).all()


def test_views_of_a_packed_projection(ctx):
    N, Hq, Hkv, d, page = 77, 6, 2, 128, 16
    x = normal((N, (Hq + 2 * Hkv) * d), 12)
    k = x[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    v = x[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
    pool = pool_of(7, Hkv, page, d)
    ko, vo = there_and_back(ctx, k, v, run_slots(N, page, 9, 7), pool)
    assert same_values(ko, k) and same_values(vo, v)


def test_skipped_and_bad_slots(ctx):
    N, Hkv, d, page, pages = 40, 2, 64, 16, 4
    pool = pool_of(pages, Hkv, page, d, 0)
    k, v = normal((N, Hkv, d), 13), normal((N, Hkv, d), 14)
    slots = torch.arange(N, device="cuda")
    slots[5:9] = -1
    slots[39] = -(2 ** 62)
    ko, vo = there_and_back(ctx, k, v, slots, pool)
    ctx.check()
    skipped = (slots < 0).nonzero().flatten()
    fine = (slots >= 0).nonzero().flatten()
    assert (ko[skipped] == 3).all() and (vo[skipped] == 3).all()      # as they were
    assert same_values(ko[fine], k[fine]) and same_values(vo[fine], v[fine])
    before = pool.clone()
    for bad in (pages * page, 2 ** 40):
        slots = torch.full((1,), bad, dtype=torch.int64, device="cuda")
        ctx.kv_write_q4(k[:1], v[:1], slots, pool)
        with pytest.raises(FluxError) as e:
            ctx.check()
        assert e.value.code == FLUX_ERR_DEVICE_CHECK
        ctx.kv_read_q4(pool, slots, ko[:1], vo[:1])
        with pytest.raises(FluxError):
            ctx.check()
    assert torch.equal(pool, before) and same_values(ko[fine], k[fine])


def test_cache_beyond_32_bits(ctx):
    """Slots whose bytes lie past 2^32 in the cache."""
    Hkv, page, d = 8, 64, 128
    pages = (9 << 29) // (Hkv * 4 * 18 * d)          # 4.8 GB
    pool = torch.empty(kv_q4_pool_shape(pages, Hkv, page, d), dtype=torch.uint8, device="cuda")
    assert pool.numel() > 1 << 32
    k, v = normal((70, Hkv, d), 15), normal((70, Hkv, d), 16)
    slots = torch.arange(pages * page - 70, pages * page, device="cuda")
    slots[:3] = torch.tensor([0, 5, 1 << 19], device="cuda")
    ko, vo = there_and_back(ctx, k, v, slots, pool)
    ctx.check()
    assert same_values(ko, k) and same_values(vo, v)


@pytest.mark.parametrize("d", [64, 128])
def test_read_into_rows_that_start_at_16_bytes(ctx, d):
    N, Hkv, page = 700, 8, 32
    pool = pool_of(24, Hkv, page, d)
    k, v = normal((N, Hkv, d), 17), normal((N, Hkv, d), 18)
    slots = run_slots(N, page, 5, 24)
    ctx.kv_write_q4(k, v, slots, pool)
    out = [torch.zeros(N * Hkv * d + 8, dtype=torch.bfloat16, device="cuda")[8:].view(N, Hkv, d) for _ in range(2)]
    assert out[0].data_ptr() % 32 == 16
    ctx.kv_read_q4(pool, slots, *out)
    assert same_values(out[0], k) and same_values(out[1], v)


def test_refusals(ctx):
    pool = pool_of(3, 2, 16, 64)
    k = normal((4, 2, 64), 1)
    slots = torch.arange(4, device="cuda")
    for args, match in (((k, k[:3], slots, pool), "inconsistent"), ((k, k, slots[:3], pool), "inconsistent"),
                        ((k, k, slots.int(), pool), "slots must be"), ((k.float(), k, slots, pool), "must be"),
                        ((k, k, slots, pool[:, :1].contiguous()), "kv_pool"),
                        ((k, k, slots, pool[..., :-16].contiguous()), "kv_pool"),
                        ((k, k, slots, pool[:, :, :, ::2]), "contiguous"),
                        ((k.transpose(1, 2), k, slots, pool), "contiguous")):
        with pytest.raises(ValueError, match=match):
            ctx.kv_write_q4(*args)
    with pytest.raises(ValueError, match="contiguous"):
        ctx.kv_read_q4(pool, slots, k.expand(4, 2, 64)[:, :1].expand(4, 2, 64), k)
    with pytest.raises(FluxError) as e:
        ctx.kv_write_q4(normal((4, 2, 72), 1)[..., :].contiguous(), normal((4, 2, 72), 1), slots,
                        torch.zeros(3, 2, 1, 18 * 72, dtype=torch.uint8, device="cuda"))
    assert e.value.code == FLUX_ERR_UNSUPPORTED
    buf = torch.zeros(3 * 2 * 18 * 64 + 8, dtype=torch.uint8, device="cuda")[8:].view(3, 2, 1, 18 * 64)
    with pytest.raises(FluxError) as e:
        ctx.kv_write_q4(k, k, slots, buf)
    assert e.value.code == FLUX_ERR_INVALID_ARG
    for bad in (0, 8, 24, 65552):
        with pytest.raises(ValueError):
            kv_q4_pool_shape(1, 1, bad, 64)
    with pytest.raises(ValueError):
        kv_q4_pool_shape(1, 1, 16, 96)
