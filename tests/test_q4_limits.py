"""Limits of the decode over the 4-bit cache: those kept on the host (no GPU), and the scale's."""
import ctypes
import math

import numpy as np

import pytest
import torch

import q4_bounds
import q4_reference as ref
from sparse_attention_flux_b200 import build, flux


@pytest.fixture(scope="module")
def lib():
    build.build(quiet=True)
    return flux.lib()


@pytest.mark.parametrize("d", [64, 128])
def test_no_more_ctas_than_the_merge_buffer_has_weights(lib, d):
    """The last merge of a row keeps a weight for each part and head in a part of shared memory that
    holds 320 parts; the launcher makes no more CTAs than that, and the workspace follows."""
    workspace = lib._ZN4flux25decode_q4_workspace_bytesEii     # by head_dim and SMs, as the launcher counts
    workspace.argtypes, workspace.restype = [ctypes.c_int, ctypes.c_int], ctypes.c_size_t
    a_cta = workspace(d, 148) // 296
    assert workspace(d, 148) == 296 * a_cta and workspace(d, 160) == 320 * a_cta
    assert workspace(d, 161) == workspace(d, 1000) == 320 * a_cta


def test_a_scale_beyond_the_factors_range_is_refused(lib):
    p, ctx = ctypes.c_void_p(256), ctypes.create_string_buffer(4096)      # p is never dereferenced
    for scale in (math.nextafter(2.0 ** 120, 1e300) * (1 + 2.0 ** -20), 2.0 ** 121, 3e38):
        assert lib.flux_attn_decode_q4(ctypes.addressof(ctx), p, p, 4, 16, p, 4, p, p, None, 2, 4, 2, 128, None, 0, 1,
                                       1, 128, scale, None) == flux.FLUX_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("q_exp,k_exp,scale_exp", [(117, -97, 1.0), (60, -97, 58.0), (0, -97, 117.0), (-90, -20, 120.0),
                                                   (-83, -38, 120.0), (117, -97, -120.0), (-100, 100, 0.0)])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_and_queries_up_to_the_limits(d, q_exp, k_exp, scale_exp):
    """Normal queries and keys times powers of two: their products with the scale up to 2^120."""
    from test_decode_q4 import Cache, normal

    def edit(c):
        for b, n in enumerate(c.lens):
            c.k[b].mul_(2.0 ** k_exp)
    with flux.Context(0, 16 << 20) as ctx:
        lens = [1, 1, 1, 200]
        c = Cache(ctx, lens, 2, d, 16, seed=71, edit=edit)
        q = normal((4, 8, d), 72).clamp(-4, 4) * 2.0 ** q_exp
        scale = 2.0 ** scale_exp
        o, lse = c.decode(ctx, q, scale=scale)
        ctx.check()
        o, lse, q = ref.f64(o), ref.f64(lse), ref.f64(q)
        assert np.isfinite(o).all() and np.isfinite(lse).all()
        for b, n in enumerate(lens):
            k, v = ref.values(ref.f64(c.k[b])), ref.values(ref.f64(c.v[b]))
            for h in range(2):
                rows = slice(4 * h, 4 * h + 4)
                want, wl, tol, ltol = q4_bounds.decode_rows(q[b, rows], k[:, h], v[:, h], scale)
                assert np.all(np.abs(o[b, rows] - want) <= tol), (b, h)
                assert np.all(np.abs(lse[b, rows] - wl) <= ltol), (b, h)
