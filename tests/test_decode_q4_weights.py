"""flux_attn_decode_q4: the probabilities enter the value product with 16 bits, whatever the group.

Values of alternating sign make the output small beside its terms, so that the roundings of the
probabilities stand out from the one of the output."""
import math

import numpy as np
import pytest
import torch

import q4_bounds
import q4_reference as ref
from sparse_attention_flux_b200.flux import Context
from test_decode_q4 import Cache, normal

pytestmark = pytest.mark.gpu

LENS = [2, 2, 3, 5, 8, 40, 0, 300, 1700]


@pytest.fixture(scope="module")
def ctx():
    with Context(0, 64 << 20) as c:
        yield c


def alternate(c):
    for b, n in enumerate(c.lens):
        if n:
            sign = 1 - 2 * (torch.arange(n, device="cuda") % 2)
            c.v[b] = c.v[b][:1] * sign[:, None, None].to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", range(1, 9))
@pytest.mark.parametrize("vstd", [1.0, 1e8])
@pytest.mark.parametrize("width", [None, 300])
def test_probabilities_keep_16_bits(ctx, d, G, vstd, width):
    """Values below and above the size at which the kernel changes its arithmetic; a table of
    the requests' length and a wide one, which the kernel serves in its two shapes."""
    c = Cache(ctx, LENS, 2, d, 32, seed=31, vstd=vstd, width=width, edit=alternate)
    q = normal((len(LENS), 2 * G, d), 32, 0.05)
    o, lse = c.decode(ctx, q)
    ctx.check()
    o, lse, q = ref.f64(o), ref.f64(lse), ref.f64(q)
    for b, n in enumerate(LENS):
        k, v = ref.values(ref.f64(c.k[b])), ref.values(ref.f64(c.v[b]))
        for h in range(2):
            rows = slice(h * G, h * G + G)
            want, wl, tol, ltol = q4_bounds.decode_rows(q[b, rows], k[:, h], v[:, h], 1 / math.sqrt(d))
            err = np.abs(o[b, rows] - want)
            assert np.all(err <= tol), (b, h, float((err / np.maximum(tol, 1e-300)).max()))
            if n:
                assert np.all(np.abs(lse[b, rows] - wl) <= ltol), (b, h)
            else:
                assert np.all(np.isneginf(lse[b, rows]))
