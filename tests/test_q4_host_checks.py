"""The paged 4-bit cache calls reject bad arguments on the host before any launch (no GPU)."""
import ctypes

import pytest

from sparse_attention_flux_b200 import build, flux

P = ctypes.c_void_p(256)                       # aligned, never dereferenced
ODD = ctypes.c_void_p(264)
CTX = ctypes.c_void_p(4096)                    # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    build.build(quiet=True)
    return flux.lib()


def call(f, base, **change):
    args = dict(base, **change)
    return f(*args.values())


def test_page_table(lib):
    base = dict(ctx=CTX, old=P, new=P, B=4, page=16, sink=0, window=0, free=P, n_free=4, cur=P, cur_out=P,
                table=P, max_pages=4, slots=P, pos=P, n_slots=4, cu=None, stream=None)
    f = lib.flux_build_page_table
    for name in ("ctx", "old", "new", "free", "cur", "cur_out", "table", "slots", "pos"):
        assert call(f, base, **{name: None}) == flux.FLUX_ERR_INVALID_ARG
    for name in ("B", "n_free", "max_pages", "n_slots"):
        assert call(f, base, **{name: 0}) == flux.FLUX_ERR_SHAPE
    assert call(f, base, B=8193) == flux.FLUX_ERR_UNSUPPORTED
    for page in (0, -16, 8, 24, 65552):
        assert call(f, base, page=page) == flux.FLUX_ERR_UNSUPPORTED
    for kw in (dict(sink=1), dict(sink=-1, window=2), dict(window=-1), dict(sink=0, window=1 << 30)):
        assert call(f, base, **kw) == flux.FLUX_ERR_INVALID_ARG


def test_norm_rope(lib):
    base = dict(ctx=CTX, q=P, qs=512, k=P, ks=256, qo=P, qos=512, ko=P, kos=256, N=2, Hq=4, Hkv=2, d=128,
                qw=None, kw=None, eps=1e-6, pos=P, inv=P, rot=128, inter=0, stream=None)
    f = lib.flux_qk_norm_rope
    for name in ("ctx", "q", "k", "qo", "ko", "pos", "inv"):
        assert call(f, base, **{name: None}) == flux.FLUX_ERR_INVALID_ARG
    assert call(f, base, qw=P) == flux.FLUX_ERR_INVALID_ARG
    for kw in (dict(d=96), dict(rot=0), dict(rot=136), dict(rot=24), dict(rot=8)):
        assert call(f, base, **kw) == flux.FLUX_ERR_UNSUPPORTED
    for kw in (dict(N=0), dict(Hq=0), dict(Hkv=-1), dict(N=1 << 30, Hq=4, qs=1 << 20)):
        assert call(f, base, **kw) == flux.FLUX_ERR_SHAPE
    for kw in (dict(eps=float("nan")), dict(eps=-1.0), dict(eps=float("inf")), dict(inter=2), dict(q=ODD),
               dict(qs=511), dict(qs=504), dict(ks=128), dict(ko=ODD), dict(kos=-256)):
        assert call(f, base, **kw) == flux.FLUX_ERR_INVALID_ARG


def test_cache_write_and_read(lib):
    base = dict(ctx=CTX, k=P, ks=256, v=P, vs=256, slots=P, N=3, Hkv=2, d=128, pool=P, pages=4, page=16, stream=None)
    f = lib.flux_kv_write_q4
    for name in ("ctx", "k", "v", "slots", "pool"):
        assert call(f, base, **{name: None}) == flux.FLUX_ERR_INVALID_ARG
    for kw in (dict(N=0), dict(Hkv=0), dict(pages=0), dict(N=(1 << 31) - 1)):
        assert call(f, base, **kw) == flux.FLUX_ERR_SHAPE
    for kw in (dict(d=96), dict(page=8), dict(page=40), dict(page=0)):
        assert call(f, base, **kw) == flux.FLUX_ERR_UNSUPPORTED
    for kw in (dict(k=ODD), dict(pool=ODD), dict(ks=252), dict(vs=128)):
        assert call(f, base, **kw) == flux.FLUX_ERR_INVALID_ARG
    base = dict(ctx=CTX, pool=P, pages=4, page=16, slots=P, N=3, Hkv=2, d=128, k=P, v=P, stream=None)
    f = lib.flux_kv_read_q4
    for name in ("ctx", "k", "v", "slots", "pool"):
        assert call(f, base, **{name: None}) == flux.FLUX_ERR_INVALID_ARG
    assert call(f, base, N=0) == flux.FLUX_ERR_SHAPE
    assert call(f, base, d=32) == flux.FLUX_ERR_UNSUPPORTED
    assert call(f, base, v=ODD) == flux.FLUX_ERR_INVALID_ARG


def test_decode(lib):
    base = dict(ctx=CTX, q=P, pool=P, pages=4, page=16, table=P, max_pages=4, sl=P, o=P, lse=None, B=2, Hq=4,
                Hkv=2, d=128, lm=None, layer=0, sink=1, window=1, block=128, scale=0.1, stream=None)
    f = lib.flux_attn_decode_q4
    for name in ("ctx", "q", "pool", "table", "sl", "o"):
        assert call(f, base, **{name: None}) == flux.FLUX_ERR_INVALID_ARG
    for kw in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(max_pages=0), dict(pages=0), dict(B=40000)):
        assert call(f, base, **kw) == flux.FLUX_ERR_SHAPE
    for kw in (dict(d=80), dict(page=20), dict(Hq=3), dict(Hq=18)):
        assert call(f, base, **kw) == flux.FLUX_ERR_UNSUPPORTED
    for kw in (dict(block=0), dict(sink=-1), dict(window=0), dict(scale=0.0), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(lm=P, layer=-1), dict(q=ODD), dict(pool=ODD)):
        assert call(f, base, **kw) == flux.FLUX_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    assert lib.flux_decode_q4_workspace_bytes(None, 128, ctypes.byref(n)) == flux.FLUX_ERR_INVALID_ARG
