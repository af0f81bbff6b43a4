"""Scores beside caches with block scales where their sums are hardest: queries of one sign beside small stored numbers and
zeros, and scores of minus infinity."""
import math

import pytest
import torch

from oracle import kv_cache as K
from tests.test_block_cache_gpu import _check, _filled
from tests.test_kv_cache_gpu import BF16_HALF, F32_HALF, F64
from tests.test_window_gpu import _visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


def _stored(pool, x):
    """x [d or 1] into every row of the pool, as whole numbers."""
    pool.view(torch.uint8).copy_(x.to(pool.dtype).view(torch.uint8).expand(pool.shape))


def check_far(kind, cache, table, q, o, lse, scale, visible):
    """_check where scores span 2^30 and more, so that most weights are far below the largest.  Beside 2^-11 of itself a weight
    (with its value's scale) is off by half of fp16's smallest number, 2^-25; the row's largest is 2^7 at least, so by 2^-32 of
    that, times a stored number of at most 127 or 448, for each of n keys."""
    k, v, ks, vs, host, q = (x.cpu() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale, table, q))
    o, lse, d, P, group = o.double().cpu(), lse.double().cpu(), cache.d, cache.page_size, q.shape[1] // cache.H_kv
    for b in range(q.shape[0]):
        for g in range(cache.H_kv):
            pos, hs = visible(b, g), slice(group * g, group * (g + 1))
            if len(pos) == 0:
                assert not o[b, hs].any() and (lse[b, hs] == -math.inf).all(), (b, g)
                continue
            kk, vv = K.block_rows(k, ks, host[b], g, pos), K.block_rows(v, vs, host[b], g, pos)
            want, wl, size, mag = K.decode(q[b, hs], kk, vv, scale)
            ds = (d + 8) * 2 * F32_HALF * size + 128 * F32_HALF
            sums = len(pos) / 8 * 2 * F32_HALF + 2.0 ** -18
            assert ((lse[b, hs] - wl).abs() <= ds + sums + 2.0 ** -20 * (1 + wl.abs())).all(), (b, g)
            p = torch.exp(scale * q[b, hs].to(F64) @ kk.T - wl[:, None])
            by = vs[host[b, pos // P].long(), g, pos % P // 16].to(F64)
            lost = 2.0 ** -32 * (p * by).amax(1, keepdim=True) * (127 if kind == "int8" else 448) * len(pos)
            bound = BF16_HALF * want.abs() + (2.0 ** -11 + 2 * ds + sums) * mag + lost
            assert ((o[b, hs] - want).abs() <= bound).all(), (b, g, ((o[b, hs] - want).abs() / bound).max())


def _one_sign(shape, gen):
    """Sizes spread over 2^-12 .. 2^6, so that sums of them do not come out even."""
    return (2.0 ** (18 * torch.rand(shape, generator=gen) - 12)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("kind,d,P,group", [("int8", 128, 32, 4), ("int8", 64, 16, 12), ("e4m3", 128, 16, 3)])
def test_keys_of_zeros_score_zero(B, kind, d, P, group):
    """Every product is 0, so every score is, beside queries of one sign and any size: with the bound of the other tests,
    which for a sum of zeros leaves the weights' rounding alone."""
    gen = torch.Generator().manual_seed(91)
    lens, H = [90, 33, 700], 2
    cache, table, n = _filled(B, lens, H, P, d, kind, gen)
    _stored(cache.k, torch.zeros(1, device="cuda"))
    cache.k_scale.copy_(torch.where(cache.k_scale.isnan(), cache.k_scale, 4.0))
    q = _one_sign((3, H * group, d), gen)
    for sign in (1, -1):
        o, lse = B.decode_attention(cache, table, n, sign * q)
        _check(cache, table, sign * q, o, lse, 1 / math.sqrt(d), lambda b, g: torch.arange(lens[b]))


@pytest.mark.parametrize("kind,d,P,group", [("int8", 128, 64, 4), ("int8", 64, 16, 16), ("e4m3", 64, 32, 2)])
def test_small_numbers_beside_queries_of_one_sign(B, kind, d, P, group):
    """Stored keys of 0 and now and then -1 or 1, as in a block whose scale an outlier set: a score is off by its own sum's rounding, which
    goes by the magnitudes of its products."""
    gen = torch.Generator().manual_seed(92)
    lens, H = [300, 1, 77], 2
    cache, table, n = _filled(B, lens, H, P, d, kind, gen)
    small = (torch.randint(-8, 9, cache.k.shape, generator=gen) / 8).trunc().cuda()
    cache.k.view(torch.uint8).copy_(small.to(cache.k.dtype).view(torch.uint8))
    cache.k_scale.copy_(torch.where(cache.k_scale.isnan(), cache.k_scale, 4.0))
    q = _one_sign((3, H * group, d), gen)
    o, lse = B.decode_attention(cache, table, n, q)
    check_far(kind, cache, table, q, o, lse, 1 / math.sqrt(d), lambda b, g: torch.arange(lens[b]))


@pytest.mark.parametrize("kind,d,P,group", [("e4m3", 64, 16, 3), ("e4m3", 128, 64, 8), ("e4m3", 64, 32, 16), ("int8", 64, 16, 3), ("int8", 128, 128, 8)])
def test_rows_whose_keys_all_score_minus_infinity(B, kind, d, P, group):
    """An infinite query beside keys that are negative in its channel: the row gets o = 0 and lse = -inf, alone in its group
    and with all of it, in one tile and in many; the other heads are what they were."""
    gen = torch.Generator().manual_seed(93)
    lens, H, at = [20, 700, 65], 2, 9
    cache, table, n = _filled(B, lens, H, P, d, kind, gen)
    below = torch.randint(1, 100, cache.k.shape[:-1], generator=gen).neg().float().cuda()
    cache.k.view(torch.uint8)[..., at] = below.to(cache.k.dtype).view(torch.uint8)
    q = torch.randn(3, H * group, d, generator=gen).to(torch.bfloat16).cuda()
    hit = torch.zeros(3, H * group, dtype=torch.bool)
    hit[0, 0] = hit[1, 1] = hit[1, group + 2] = hit[2, group:] = True
    bad = q.clone()
    bad[hit.cuda(), at] = math.inf
    for more in ({}, {"window": 50, "sinks": 3}):
        want = B.decode_attention(cache, table, n, q, **more)
        o, lse = B.decode_attention(cache, table, n, bad, **more)
        assert not o[hit.cuda()].any() and (lse[hit.cuda()] == -math.inf).all()
        # a warp's heads renew their references together, so the other heads keep their bounds, not their bits
        o[hit.cuda()], lse[hit.cuda()] = want[0][hit.cuda()], want[1][hit.cuda()]
        _check(cache, table, q, o, lse, 1 / math.sqrt(d),
               lambda b, g: _visible(lens[b], 50, 3) if more else torch.arange(lens[b]))
