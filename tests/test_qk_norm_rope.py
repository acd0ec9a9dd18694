"""flux_qk_norm_rope against the formula in 64 bits, within the roundings it makes."""
import numpy as np
import pytest
import torch

import q4_reference as ref
from sparse_attention_flux_b200.flux import FLUX_ERR_INVALID_ARG, FLUX_ERR_UNSUPPORTED, Context, FluxError

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    with Context(0, 16 << 20) as c:
        yield c


def packed(N, Hq, Hkv, d, seed=0, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((N, (Hq + 2 * Hkv) * d), generator=g, device="cuda") * std).to(torch.bfloat16)
    return x, x[:, :Hq * d].unflatten(1, (Hq, d)), x[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))


def freqs(rot, theta=1e6):
    return torch.tensor(theta ** (-np.arange(0, rot, 2) / rot), dtype=torch.float32, device="cuda")


def weights(d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]


def check(got, x, w, eps, pos, inv, inter):
    y, bound = ref.norm_rope(ref.f64(x), None if w is None else ref.f64(w), eps,
                             pos.cpu().numpy(), ref.f64(inv), inter)
    err = np.abs(ref.f64(got) - y)
    assert np.all(np.isfinite(ref.f64(got)))
    assert np.all(err <= bound), float((err - bound).max())


@pytest.mark.parametrize("N,Hq,Hkv", [(1, 1, 1), (1, 32, 8), (7, 3, 1), (16, 32, 8), (129, 8, 2),
                                      (1000, 14, 2), (3001, 5, 5)])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 32), (64, 64), (64, 48), (128, 112), (64, 16)])
@pytest.mark.parametrize("norm,inter", [(True, False), (False, False), (True, True), (False, True)])
def test_matches_the_formula(ctx, N, Hq, Hkv, d, rot, norm, inter):
    _, q, k = packed(N, Hq, Hkv, d, N + d)
    inv = freqs(rot)
    g = np.random.default_rng(N)
    pos = torch.tensor(g.integers(0, 131072, N), dtype=torch.int32, device="cuda")
    qw, kw = weights(d, 5) if norm else (None, None)
    qo, ko = torch.full_like(q, 7).contiguous(), torch.full_like(k, 7).contiguous()
    ctx.qk_norm_rope(q, k, qo, ko, pos, inv, qw, kw, eps=1e-6, interleaved=inter)
    check(qo, q, qw, 1e-6, pos, inv, inter)
    check(ko, k, kw, 1e-6, pos, inv, inter)


@pytest.mark.parametrize("positions", [[0, 1, 131071, 262143], [2 ** 31 - 1, 2 ** 24 + 1, -1, -77777]])
def test_far_and_negative_positions(ctx, positions):
    _, q, k = packed(4, 4, 2, 128)
    inv = freqs(128, 1e4)
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    ctx.qk_norm_rope(q, k, qo, ko, pos, inv)
    check(qo, q, None, 0, pos, inv, False)
    check(ko, k, None, 0, pos, inv, False)


@pytest.mark.parametrize("std", [0.0, 1e-20, 1e-3, 1e15])
def test_norm_of_small_and_large_rows(ctx, std):
    """Zero rows stay zero, rows whose squares vanish under eps shrink with it, and rows of 1e15
    have a sum of squares that fp32 still holds."""
    _, q, k = packed(9, 4, 2, 128, std=std)
    inv = freqs(128)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    qw, kw = weights(128, 1)
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    ctx.qk_norm_rope(q, k, qo, ko, pos, inv, qw, kw, eps=1e-6)
    check(qo, q, qw, 1e-6, pos, inv, False)
    check(ko, k, kw, 1e-6, pos, inv, False)


@pytest.mark.parametrize("inter", [False, True])
def test_in_place_in_a_packed_projection(ctx, inter):
    x, q, k = packed(37, 6, 2, 128, 3)
    before = x.clone()
    inv = freqs(64)
    pos = torch.arange(100, 137, dtype=torch.int32, device="cuda")
    qw, kw = weights(128, 2)
    q0, k0 = q.clone(), k.clone()
    ctx.qk_norm_rope(q, k, q, k, pos, inv, qw, kw, interleaved=inter)
    check(q, q0, qw, 1e-6, pos, inv, inter)
    check(k, k0, kw, 1e-6, pos, inv, inter)
    assert torch.equal(x[:, 8 * 128:], before[:, 8 * 128:])       # v is not touched


def test_rows_do_not_depend_on_the_batch(ctx):
    """A token's row is the same bits alone and in a batch (prompt and decode agree)."""
    _, q, k = packed(2000, 8, 2, 128, 4)
    inv = freqs(128)
    pos = torch.arange(2000, dtype=torch.int32, device="cuda")
    qw, kw = weights(128, 2)
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    ctx.qk_norm_rope(q, k, qo, ko, pos, inv, qw, kw)
    for n in (0, 1, 777, 1999):
        a, b = torch.empty_like(qo[:1]), torch.empty_like(ko[:1])
        ctx.qk_norm_rope(q[n:n + 1], k[n:n + 1], a, b, pos[n:n + 1].contiguous(), inv, qw, kw)
        assert torch.equal(a[0], qo[n]) and torch.equal(b[0], ko[n])


def test_non_finite_rows_stay_in_their_row(ctx):
    _, q, k = packed(5, 4, 2, 64, 6)
    q[2, 1, 3] = float("nan")
    k[4, 0, 0] = float("inf")
    inv = freqs(64)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    qw, kw = weights(64, 2)
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    ctx.qk_norm_rope(q, k, qo, ko, pos, inv, qw, kw)
    fine = torch.isfinite(qo).all(-1)
    assert not fine[2, 1] and fine.sum() == 19
    fine = torch.isfinite(ko).all(-1)
    assert not fine[4, 0] and fine.sum() == 9


def test_refusals(ctx):
    _, q, k = packed(4, 4, 2, 128)
    inv = freqs(128)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    qw, kw = weights(128, 1)
    for args, match in (((q, k[:3], qo, ko, pos, inv), "inconsistent"),
                        ((q, k, qo[:, :3], ko, pos, inv), "inconsistent"),
                        ((q.float(), k, qo, ko, pos, inv), "must be"),
                        ((q.transpose(1, 2), k, qo, ko, pos, inv), "contiguous"),
                        ((q, k, qo, ko, pos[:3], inv), "inconsistent"),
                        ((q, k, qo, ko, pos.long(), inv), "must be"),
                        ((q, k, qo.cpu(), ko, pos, inv), "is on"),
                        ((q, k, qo, ko, pos, inv.double()), "must be")):
        with pytest.raises(ValueError, match=match):
            ctx.qk_norm_rope(*args)
    with pytest.raises(ValueError, match="head_dim"):
        ctx.qk_norm_rope(q, k, qo, ko, pos, inv, qw[:64].contiguous(), kw)
    for kw_, code in ((dict(q_weight=qw), FLUX_ERR_INVALID_ARG), (dict(eps=float("nan")), FLUX_ERR_INVALID_ARG)):
        with pytest.raises(FluxError) as e:
            ctx.qk_norm_rope(q, k, qo, ko, pos, inv, **kw_)
        assert e.value.code == code
    with pytest.raises(FluxError) as e:                            # 130 channels of 128
        ctx.qk_norm_rope(q, k, qo, ko, pos, torch.ones(65, device="cuda"))
    assert e.value.code == FLUX_ERR_UNSUPPORTED
    odd = torch.zeros(4, 4 * 128 + 4, dtype=torch.bfloat16, device="cuda")[:, 4:].unflatten(1, (4, 128))
    with pytest.raises(FluxError) as e:                            # 8-byte offset
        ctx.qk_norm_rope(odd, k, qo, ko, pos, inv)
    assert e.value.code == FLUX_ERR_INVALID_ARG
