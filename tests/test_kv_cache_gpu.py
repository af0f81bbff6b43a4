"""Paged key-value cache on the GPU: append, single-token attention and page selection against plain
64-bit forms (oracle/kv_cache.py), at the sizes, masks and layouts where they can go wrong.

All cache memory that no token was written to holds NaN, so that a key past a length or behind a mask
that reached an output would show.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kv_cache as K
from oracle import masks as M

pytestmark = pytest.mark.gpu

BF16_HALF, E4M3_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -4, 2.0 ** -24
F64 = torch.float64


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


def _table(need, spare, gen):
    """Page table of sequences that need so many pages each, in random order; unused entries name no page."""
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen, device="cpu").to(torch.int32)
    t = torch.full((len(need), max(max(need), 1)), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, max(pages, 1)


def _pools(pages, H, P, d, kv, gen, scale=1.0, joint=False):
    """NaN-filled pools; joint: K and V halves of one tensor, so that pages lie apart."""
    dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    if joint:
        both = torch.full((pages, 2, H, P, d), math.nan, device="cuda").to(dtype)
        return both[:, 0], both[:, 1]
    return tuple(torch.full((pages, H, P, d), math.nan, device="cuda").to(dtype) for _ in range(2))


def _filled(B, lens, H, P, d, kv, gen, joint=False, spare=2):
    """A cache whose sequences hold lens tokens of random values; everything else is NaN."""
    need = [(n + P - 1) // P for n in lens]
    table, pages = _table(need, spare, gen)
    k, v = _pools(pages, H, P, d, kv, gen, joint=joint)
    scales = {}
    if kv == "e4m3":
        scales = {n: (0.01 + 0.02 * torch.rand(H, generator=gen)).cuda() for n in ("k_scale", "v_scale")}
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pos = torch.arange(n)
        at, row = table[b, pos // P].long().cuda(), (pos % P).cuda()
        for pool, name in ((k, "k_scale"), (v, "v_scale")):
            x = torch.randn(n, H, d, generator=gen).cuda()
            if kv == "e4m3":
                x = (x / scales[name][:, None]).clamp(-448, 448).to(pool.dtype).view(torch.uint8)
                pool.view(torch.uint8)[at, :, row] = x
            else:
                pool[at, :, row] = x.to(pool.dtype)
    cache = B.KVCache(k, v, **scales)
    return cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def _host(cache):
    k, v = cache.k.cpu(), cache.v.cpu()
    ks, vs = ((None, None) if cache.k_scale is None else (cache.k_scale.cpu(), cache.v_scale.cpu()))
    return k, v, ks, vs


def _check_decode(cache, table, lens, q, o, lse, scale, visible):
    """visible(b, h_kv) -> ascending positions.  Bounds: a score is off by the fp32 sum of d exact
    products (the tensor core may cut each addition: one step a term) and its scaling; p by that and by its rounding to
    bf16 (half a step); o by those and one rounding to bf16; the log by the sum's and its own."""
    k, v, ks, vs = _host(cache)
    table, q, o, lse = table.cpu(), q.cpu(), o.double().cpu(), lse.double().cpu()
    d, group = cache.d, q.shape[1] // cache.H_kv
    for b in range(q.shape[0]):
        for g in range(cache.H_kv):
            pos = visible(b, g)
            kk, vv = (K.rows(x, s, table[b], g, pos) for x, s in ((k, ks), (v, vs)))
            hs = slice(g * group, (g + 1) * group)
            want, wl, size, mag = K.decode(q[b, hs], kk, vv, scale)
            if len(pos) == 0:
                assert not o[b, hs].any() and (lse[b, hs] == -math.inf).all(), (b, g)
                continue
            ds = (d + 8) * 2 * F32_HALF * size + 16 * F32_HALF
            bound = BF16_HALF * want.abs() + (BF16_HALF + 2 * ds + 2.0 ** -14) * mag + 1e-30
            assert ((o[b, hs] - want).abs() <= bound).all(), (b, g, ((o[b, hs] - want).abs() / bound).max())
            assert ((lse[b, hs] - wl).abs() <= ds + 2.0 ** -20 * (1 + wl.abs())).all(), (b, g)


# ---- append ----------------------------------------------------------------------------------
def _rope(n, rot, gen):
    angle = torch.rand(n, rot // 2, generator=gen, dtype=F64) * 50
    return torch.stack([angle.cos(), angle.sin()], 2).float()


APPEND = [
    # d, P, kv, H_kv, H_q, held, new, packed, rot, interleaved, summary
    (128, 64, "bf16", 2, 6, [0, 63, 64, 200], [1, 1, 1, 1], False, 128, False, False),
    (128, 16, "e4m3", 3, 3, [5, 0, 31], [1, 1, 1], True, 128, True, True),
    (64, 128, "bf16", 1, 5, [0, 127, 130], [300, 1, 0], True, 32, True, True),
    (64, 32, "e4m3", 4, 4, [31, 1], [33, 70], False, 64, False, True),
    (128, 128, "bf16", 2, 0, [7, 0, 3], [17, 129, 0], True, 96, False, True),
    (128, 16, "bf16", 8, 8, [3] * 5, [0, 1, 2, 16, 40], False, 0, False, True),
    (64, 64, "bf16", 3, 9, [100], [65], False, 16, True, False),
]


@pytest.mark.parametrize("d,P,kv,H,Hq,held,new,packed,rot,inter,summ", APPEND)
def test_append(B, d, P, kv, H, Hq, held, new, packed, rot, inter, summ):
    gen = torch.Generator().manual_seed(11)
    n_seq, T = len(held), max(new)
    cache, table, lens = _filled(B, held, H, P, d, kv, gen, joint=packed)
    need = [(a + b + P - 1) // P for a, b in zip(held, new)]
    # room for the new tokens: fresh pages behind the held ones
    grown, pages = _table(need, 0, gen)
    old_pages = cache.num_pages
    wide = torch.full((n_seq, max(max(need), 1)), -7, dtype=torch.int32)
    fresh = iter(range(old_pages, old_pages + pages))
    for b in range(n_seq):
        have = (held[b] + P - 1) // P
        wide[b, :have] = table[b, :have].cpu()
        for i in range(have, need[b]):
            wide[b, i] = next(fresh)
    dtype = cache.k.dtype
    joint = torch.full((old_pages + pages, 2, H, P, d), math.nan, device="cuda").to(dtype)
    joint.view(torch.uint8)[:old_pages, 0] = cache.k.contiguous().view(torch.uint8)
    joint.view(torch.uint8)[:old_pages, 1] = cache.v.contiguous().view(torch.uint8)
    more = {}
    if summ:
        more = {"summary": torch.full((old_pages + pages, H, 2, d), 99, dtype=torch.int8, device="cuda"),
                "summary_scale": torch.full((old_pages + pages, H), 7.0, device="cuda")}
    cache = B.KVCache(joint[:, 0], joint[:, 1], cache.k_scale, cache.v_scale, **more)
    before = joint.view(torch.uint8).clone()
    total, wide = sum(new), wide.cuda()
    rope = _rope(wide.shape[1] * P, rot, gen).cuda() if rot else None
    new_lens = torch.full_like(lens, -5)
    shape = (lambda h: (total + 3, h, d)) if packed else (lambda h: (n_seq, h, T, d))

    def strided(h, fill=None):  # a slice of a wider projection: token rows lie apart
        s = list(shape(h))
        s[-2 if packed else 1] += 2
        x = torch.randn(s, generator=gen) if fill is None else torch.full(s, fill)
        return x.to(torch.bfloat16).cuda()[:, 1:h + 1]

    k, v = strided(H), strided(H)
    k_out = strided(H, 5.0)
    more = {}
    if Hq:
        more = {"q": strided(Hq), "q_out": strided(Hq, 6.0)}
    if packed:
        more["cu_new"] = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda")
        more["max_new"] = T
    else:
        more["n_new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
    B.cm_kv_append(cache, wide, lens, k, v, k_out=k_out, rope=rope, interleaved=inter, new_lens=new_lens, **more)
    assert B.cm_kv_status(cache) == B.CM_OK
    assert new_lens.tolist() == [a + b for a, b in zip(held, new)] and lens.tolist() == held

    pool_k, pool_v, ks, vs = _host(cache)
    touched = torch.zeros(joint.shape[:4], dtype=torch.bool)
    outs = [(k.cpu(), k_out.cpu(), 5.0)] + ([(more["q"].cpu(), more["q_out"].cpu(), 6.0)] if Hq else [])
    written = [torch.zeros(x.shape, dtype=torch.bool) for _, x, _ in outs]
    v, host_table, host_rope = v.cpu(), wide.cpu(), None if rope is None else rope.cpu()
    base = 0
    for b in range(n_seq):
        for i in range(new[b]):
            p = held[b] + i
            at = (base + i,) if packed else (b, slice(None), i)
            for (src, dst, _), w in zip(outs, written):
                want, size = (K.rotate(src[at], host_rope[p, :, 0], host_rope[p, :, 1], inter) if rot
                              else (src[at].to(F64), src[at].to(F64).abs()))
                err = (dst[at].to(F64) - want).abs()
                assert (err <= BF16_HALF * want.abs() + 4 * F32_HALF * size).all(), (b, i)
                w[at] = True
            page, row = int(host_table[b, p // P]), p % P
            touched[page, :, :, row] = True
            for pool, s, val in ((pool_k, ks, k_out.cpu()[at]), (pool_v, vs, v[at])):
                got = pool[page, :, row].float()
                if s is None:
                    assert torch.equal(got, val.float()), (b, i)  # the cache holds what k_out says
                else:
                    x = (val.to(F64) / s.to(F64)[:, None]).clamp(-448, 448)
                    assert ((got.to(F64) - x).abs() <= E4M3_HALF * x.abs() * (1 + 2.0 ** -20) + 2.0 ** -10).all(), (b, i)
        base += new[b]
    # nothing else changed: outputs of no token, rows of no new token
    for (_, dst, fill), w in zip(outs, written):
        assert (dst[~w] == fill).all()
    after = joint.view(torch.uint8).cpu().view(*joint.shape[:4], -1)
    same = (after == before.cpu().view(*joint.shape[:4], -1)).all(-1)
    assert same[~touched].all()
    if summ:
        got, scale = cache.summary.cpu(), cache.summary_scale.cpu()
        fresh = torch.zeros(got.shape[0], dtype=torch.bool)
        for b in range(n_seq):
            for i in range(held[b] // P, need[b] if new[b] else 0):
                page, pos = int(host_table[b, i]), torch.arange(i * P, min((i + 1) * P, held[b] + new[b]))
                fresh[page] = True
                for h in range(H):
                    s, e = K.summary(K.rows(pool_k, ks, host_table[b], h, pos).float())
                    assert torch.equal(got[page, h], s) and scale[page, h] == e, (b, i, h)
        assert (got[~fresh] == 99).all() and (scale[~fresh] == 7.0).all()


def test_append_in_place_and_special_values(B):
    """q_out = q and k_out = k; NaN, infinities and values beyond the 8-bit range."""
    gen = torch.Generator().manual_seed(12)
    cache, table, lens = _filled(B, [10], 2, 16, 64, "e4m3", gen)
    cache = B.KVCache(cache.k, cache.v, cache.k_scale, cache.v_scale,
                      torch.zeros(cache.num_pages, 2, 2, 64, dtype=torch.int8, device="cuda"),
                      torch.zeros(cache.num_pages, 2, device="cuda"))
    k = torch.randn(1, 2, 1, 64, generator=gen).to(torch.bfloat16).cuda()
    k[0, 0, 0, :3] = torch.tensor([math.nan, math.inf, -1e30])
    v, q = k.clone(), k.repeat(1, 2, 1, 1)
    want_k, want_q = k.clone(), q.clone()
    B.cm_kv_append(cache, table, lens, k, v, q=q, q_out=q, k_out=k)
    page, row = int(table[0, 0]), 10
    got = cache.k[page, :, row].float().cpu()
    assert math.isnan(got[0, 0]) and got[0, 1] == 448 and got[0, 2] == -448
    assert torch.equal(torch.nan_to_num(k, 9.0), torch.nan_to_num(want_k, 9.0))
    assert torch.equal(torch.nan_to_num(q, 9.0), torch.nan_to_num(want_q, 9.0))
    pool, _, ks, _ = _host(cache)
    for h in range(2):
        s, e = K.summary(K.rows(pool, ks, table[0].cpu(), h, torch.arange(11)).float())
        assert torch.equal(cache.summary[page, h].cpu(), s) and cache.summary_scale[page, h].item() == e
    assert B.cm_kv_status(cache) == B.CM_OK


def test_append_token_by_token_gives_the_same_cache(B):
    """Prompt at once or one token a call: the same bits, summaries among them."""
    gen = torch.Generator().manual_seed(13)
    H, P, d, n = 2, 32, 128, 75
    k, v = (torch.randn(1, H, n, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    rope = _rope(n, d, gen).cuda()
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    caches = [B.KVCache.alloc(3, H, P, d, summaries=True) for _ in range(2)]
    for c in caches:
        c.k.zero_(), c.v.zero_()
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.cm_kv_append(caches[0], table, lens, k, v, rope=rope)
    for i in range(n):
        after = torch.empty_like(lens)
        B.cm_kv_append(caches[1], table, lens, k[:, :, i:i + 1], v[:, :, i:i + 1], rope=rope, new_lens=after)
        lens = after
    assert lens.item() == n
    for a, b in ((caches[0].k, caches[1].k), (caches[0].v, caches[1].v),
                 (caches[0].summary, caches[1].summary), (caches[0].summary_scale, caches[1].summary_scale)):
        assert torch.equal(a, b)


def test_append_reports_what_it_leaves_out(B):
    """A sequence out of range appends nothing, a page outside the pool is skipped, the others are whole."""
    H, P, d = 1, 16, 64
    cache = B.KVCache.alloc(4, H, P, d)
    cache.k.zero_(), cache.v.zero_()
    table = torch.tensor([[0, 1], [2, 77], [3, 3], [1, -1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([0, 15, 31, -1], dtype=torch.int32, device="cuda")  # the third has no room for 2
    k = torch.ones(4, H, 2, d, dtype=torch.bfloat16, device="cuda")
    new_lens, k_out = torch.empty_like(lens), torch.zeros_like(k)
    B.cm_kv_append(cache, table, lens, k, k, k_out=k_out, new_lens=new_lens)
    assert B.cm_kv_status(cache) == B.CM_ERR_DEVICE_CHECK and B.cm_kv_status(cache) == B.CM_OK
    assert new_lens.tolist() == [2, 17, 31, -1]
    rows = cache.k[..., 0].float().sum(1).cpu()
    want = torch.zeros(4, P)
    want[0, :2] = 1
    want[2, 15] = 1
    assert torch.equal(rows, want)
    assert k_out[..., 0].float().sum((1, 2)).tolist() == [2, 2, 0, 0]
    # token counts outside the tensors
    lens.zero_()
    for bad in ([0, 3, 3, 3, 3], [-1, 1, 2, 2, 2], [0, 1, 0, 1, 9]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        B.cm_kv_append(cache, torch.arange(4, dtype=torch.int32, device="cuda").view(4, 1), lens, k.view(8, H, d)[:4],
                       k.view(8, H, d)[:4], cu_new=cu, max_new=2)
        assert B.cm_kv_status(cache) == B.CM_ERR_DEVICE_CHECK, bad
    # a position behind the rotation's table
    rope = torch.zeros(1, d // 2, 2, device="cuda")
    B.cm_kv_append(cache, table, lens, k, k, rope=rope)
    assert B.cm_kv_status(cache) == B.CM_ERR_DEVICE_CHECK


def test_append_of_nothing(B):
    cache = B.KVCache.alloc(2, 1, 16, 64)
    table = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    new_lens = torch.empty_like(lens)
    none = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    B.cm_kv_append(cache, table, lens, none, none, cu_new=cu, max_new=0, new_lens=new_lens)
    assert new_lens.tolist() == [3, 0] and B.cm_kv_status(cache) == B.CM_OK


# ---- decode ----------------------------------------------------------------------------------
DECODE = [
    # d, P, kv, H_kv, group, lens
    (128, 64, "bf16", 2, 4, [1, 63, 64, 65, 0, 1000]),
    (128, 16, "bf16", 8, 1, [17, 16, 15, 1, 300]),
    (64, 16, "bf16", 3, 5, [0, 0, 33, 129]),
    (64, 128, "bf16", 1, 8, [127, 128, 129, 2500]),
    (128, 128, "bf16", 2, 16, [31, 32, 33, 700]),
    (128, 32, "bf16", 1, 24, [32, 511]),
    (128, 32, "e4m3", 2, 4, [1, 31, 32, 33, 0, 1025]),
    (64, 64, "e4m3", 4, 1, [100, 64, 7]),
    (128, 16, "e4m3", 1, 16, [400, 3]),
    (64, 16, "e4m3", 2, 9, [1, 200]),
    (128, 128, "e4m3", 1, 40, [513]),
    (128, 64, "bf16", 1, 7, [20000]),
    (64, 16, "e4m3", 1, 2, [9001, 1]),
    (128, 16, "bf16", 2, 3, [(7 * i) % 97 for i in range(150)]),
]


@pytest.mark.parametrize("d,P,kv,H,group,lens", DECODE)
def test_decode(B, d, P, kv, H, group, lens):
    gen = torch.Generator().manual_seed(21)
    cache, table, n = _filled(B, lens, H, P, d, kv, gen, joint=group % 2 == 0)
    wide = (torch.randn(len(lens), H * group + 2, d, generator=gen) * 2).to(torch.bfloat16).cuda()
    q = wide[:, 1:-1]
    o = torch.full((len(lens), H * group, 2 * d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(len(lens), H * group, device="cuda")
    work = torch.full((B.cm_attn_decode_workspace_size(len(lens), H * group, H, d),), 255, dtype=torch.uint8, device="cuda")
    B.cm_attn_decode(cache, table, n, q, o[..., :d], lse, work, scale=0.11)
    assert B.cm_kv_status(cache) == B.CM_OK
    assert (o[..., d:] == 3.0).all()
    _check_decode(cache, table, lens, q, o[..., :d], lse, 0.11, lambda b, g: torch.arange(lens[b]))
    # the same call gives the same bits, with no lse too
    o2 = torch.empty_like(o)
    B.cm_attn_decode(cache, table, n, q, o2[..., :d], None, work, scale=0.11)
    assert torch.equal(o2[..., :d], o[..., :d])


def test_decode_large_and_equal_scores(B):
    """Scores whose exponentials overflow without the running maximum, and rows of equal scores."""
    gen = torch.Generator().manual_seed(22)
    lens, H, P, d = [900, 900], 1, 32, 64
    cache, table, n = _filled(B, lens, H, P, d, "bf16", gen)
    q = torch.zeros(2, 8, d, dtype=torch.bfloat16, device="cuda")
    q[0] = (torch.randn(8, d, generator=gen) * 60).to(torch.bfloat16).cuda()
    o, lse = B.decode_attention(cache, table, n, q)
    _check_decode(cache, table, lens, q, o, lse, 1 / 8, lambda b, g: torch.arange(900))
    assert lse[1].sub(math.log(900)).abs().max() < 1e-5


MASKS = {
    "documents": "region all : j >= seg_start(i) && j <= i",
    "window": "region all : j > i - 70 && j <= i",
    "sinks": "region all : j < 5 || (j > i - 33 && j <= i) || j == 77",
    "far": "region all : j <= i - 600",  # rows below 600 see nothing
    "past": "region all : j <= i + 40",  # cut at the length
    "overlap": "region all : j < 200 || (j >= 100 && j < 250) || (j >= 240 && j <= i) || j == 130",
    "reversed": "region all : (j > i - 20 && j <= i) || (j >= 300 && j < 340) || (j >= 290 && j < 301) || j < 16",
}


@pytest.mark.parametrize("group", [1, 12])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_many_small_weights_beside_a_large_one(B, kv, group):
    """One key whose value is 0 and n - 1 of 2^-25.2 its weight whose values are 1: the small weights are
    all of the output, and 2^-25.2 is less than half of fp16's smallest number.  Bounds: a weight is off by half of that
    number (2^-25) times 2^-7 of the largest at most, o by n of those, the weights' 2^-14 and one rounding to bf16;
    the log by its own (2^-20) and the sum's: additions of up to n / (4 warps x 8 lanes) terms."""
    n, P, d = 1 << 19, 128, 64
    k, v = (torch.zeros(n // P, 1, P, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    v += 1
    k[0, 0, 5, 0] = 1
    v[0, 0, 5] = 0
    one = torch.ones(1, device="cuda")
    scales = {}
    if kv == "e4m3":
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
        scales = {"k_scale": one, "v_scale": one}
    cache = B.KVCache(k, v, **scales)
    table = torch.arange(n // P, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.zeros(1, group, d, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 1
    o, lse = B.decode_attention(cache, table, lens, q, scale=25.2 * math.log(2))
    assert B.cm_kv_status(cache) == B.CM_OK
    rest = (n - 1) * 2.0 ** -25.2
    want, wl = rest / (1 + rest), 25.2 * math.log(2) + math.log1p(rest)
    assert ((o.double() - want).abs() <= (BF16_HALF + 2.0 ** -14) * want + n * 2.0 ** -32).all(), (o, want)
    assert ((lse.double() - wl).abs() <= 2.0 ** -20 * (1 + wl) + n / 32 * 2 * F32_HALF * rest).all(), (lse, wl)


@pytest.mark.parametrize("name", MASKS)
@pytest.mark.parametrize("d,P,kv,H,group", [(128, 64, "bf16", 2, 4), (64, 16, "e4m3", 1, 9)])
def test_decode_masked(B, name, d, P, kv, H, group):
    gen = torch.Generator().manual_seed(23)
    lens, S = [1, 599, 601, 1024, 0, 777], 1024
    cache, table, n = _filled(B, lens, H, P, d, kv, gen)
    spec = B.cm_compile_spec(MASKS[name])
    desc = B.Descriptor(spec, spec, len(lens), S)
    seg = torch.tensor([[0, 100, 600, 640, S]] * len(lens), dtype=torch.int32, device="cuda")
    nseg = torch.full((len(lens),), 4, dtype=torch.int32, device="cuda")
    B.cm_build_descriptor(spec, spec, seg, nseg, desc)
    q = torch.randn(len(lens), H * group, d, generator=gen).to(torch.bfloat16).cuda()
    o, lse = B.decode_attention(cache, table, n, q, desc=desc)
    assert B.cm_kv_status(cache) == B.CM_OK

    def visible(b, g):
        if lens[b] == 0:
            return torch.arange(0)
        i, j = lens[b] - 1, np.arange(lens[b])
        start = max(x for x in (0, 100, 600, 640) if x <= i)
        see = {"documents": j >= start, "window": j > i - 70, "sinks": (j < 5) | (j > i - 33) | (j == 77),
               "far": j <= i - 600, "past": j >= 0,
               "overlap": (j < 200) | ((j >= 100) & (j < 250)) | (j >= 240) | (j == 130),
               "reversed": (j > i - 20) | ((j >= 290) & (j < 340)) | (j < 16)}[name]
        return torch.from_numpy(np.nonzero(see & (j <= i))[0])

    _check_decode(cache, table, lens, q, o, lse, 1 / math.sqrt(d), visible)


@pytest.mark.parametrize("d,P,kv,H,group", [(128, 64, "bf16", 2, 4), (64, 16, "e4m3", 3, 1), (128, 32, "e4m3", 1, 16)])
def test_decode_of_selected_pages(B, d, P, kv, H, group):
    gen = torch.Generator().manual_seed(24)
    lens = [P * 9 + 1, 3, 0, P * 40, P * 2]
    cache, table, n = _filled(B, lens, H, P, d, kv, gen)
    sel = torch.full((len(lens), H, 7), 123456, dtype=torch.int32)  # behind nsel: anything
    nsel = torch.zeros(len(lens), H, dtype=torch.int32)
    chosen = {}
    for b, m in enumerate(lens):
        pages = (m + P - 1) // P
        for h in range(H):
            pick = sorted(torch.randperm(pages, generator=gen)[:7 if h else 5].tolist())
            if b == 3 and h == 0:
                pick = []  # a row that keeps no page
            nsel[b, h] = len(pick)
            sel[b, h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
            chosen[b, h] = torch.tensor([p for x in pick for p in range(x * P, min(m, (x + 1) * P))], dtype=torch.long)
    q = torch.randn(len(lens), H * group, d, generator=gen).to(torch.bfloat16).cuda()
    o, lse = B.decode_attention(cache, table, n, q, sel=sel.cuda(), nsel=nsel.cuda())
    assert B.cm_kv_status(cache) == B.CM_OK
    _check_decode(cache, table, lens, q, o, lse, 1 / math.sqrt(d), lambda b, g: chosen[b, g])


def test_decode_reports_what_it_leaves_out(B):
    """Bad lengths give empty rows, bad pages and bad selections are skipped; the rest is right."""
    gen = torch.Generator().manual_seed(25)
    P, d = 16, 64
    lens = [40, 40, 40]
    cache, table, n = _filled(B, lens, 1, P, d, "bf16", gen)
    q = torch.randn(3, 2, d, generator=gen).to(torch.bfloat16).cuda()
    n = torch.tensor([40, -3, 49], dtype=torch.int32, device="cuda")
    o, lse = B.decode_attention(cache, table, n, q)
    assert B.cm_kv_status(cache) == B.CM_ERR_DEVICE_CHECK
    _check_decode(cache, table, lens, q, o, lse, 1 / 8, lambda b, g: torch.arange([40, 0, 0][b]))
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    bad = table.clone()
    bad[1, 1], bad[2, 0] = cache.num_pages, -1
    o, lse = B.decode_attention(cache, bad, n, q)
    assert B.cm_kv_status(cache) == B.CM_ERR_DEVICE_CHECK
    seen = [torch.arange(40), torch.tensor([*range(16), *range(32, 40)]), torch.arange(16, 40)]
    _check_decode(cache, table, lens, q, o, lse, 1 / 8, lambda b, g: seen[b])
    sel = torch.tensor([[[0, 0, 2]], [[2, 1, -1]], [[1, 3, 9]]], dtype=torch.int32, device="cuda")
    nsel = torch.tensor([[3], [3], [9]], dtype=torch.int32, device="cuda")
    o, lse = B.decode_attention(cache, table, n, q, sel=sel, nsel=nsel)
    assert B.cm_kv_status(cache) == B.CM_ERR_DEVICE_CHECK
    seen = [torch.tensor([*range(16), *range(32, 40)]), torch.arange(32, 40), torch.arange(16, 32)]
    _check_decode(cache, table, lens, q, o, lse, 1 / 8, lambda b, g: seen[b])
    spec = B.cm_compile_spec("region all : j <= i")
    desc = B.Descriptor(spec, spec, 3, 128)
    big, big_table, m = _filled(B, [129, 128, 5], 1, P, d, "bf16", gen)
    B.cm_build_descriptor(spec, spec, torch.tensor([[0, 128]] * 3, dtype=torch.int32, device="cuda"),
                          torch.ones(3, dtype=torch.int32, device="cuda"), desc)
    o, lse = B.decode_attention(big, big_table, m, q, desc=desc)
    assert B.cm_kv_status(big) == B.CM_ERR_DEVICE_CHECK
    _check_decode(big, big_table, [129, 128, 5], q, o, lse, 1 / 8, lambda b, g: torch.arange([0, 128, 5][b]))


# ---- selection -------------------------------------------------------------------------------
SELECT = [
    # d, P, kv, H_kv, group, lens, n, first, last
    (128, 16, "bf16", 2, 4, [1000, 16, 17, 1, 0], 8, 1, 2),
    (64, 16, "e4m3", 3, 1, [500, 129], 5, 0, 0),
    (128, 32, "bf16", 1, 17, [3000], 20, 20, 0),
    (64, 64, "bf16", 4, 8, [640, 641], 10, 0, 10),
    (128, 128, "e4m3", 1, 3, [900, 128, 129], 1, 0, 1),
    (64, 16, "bf16", 1, 5, [9000], 300, 2, 3),
    (128, 16, "e4m3", 1, 19, [9001, 7000], 100, 0, 1),  # several blocks a row, several rounds of heads
]


@pytest.mark.parametrize("d,P,kv,H,group,lens,n,first,last", SELECT)
@pytest.mark.parametrize("equal", [False, True])
def test_select_pages(B, d, P, kv, H, group, lens, n, first, last, equal):
    """equal: summaries of few values, so that many pages have the same score."""
    gen = torch.Generator().manual_seed(31)
    cache, table, m = _filled(B, lens, H, P, d, kv, gen)
    k = torch.zeros(cache.num_pages, H, 2, d, dtype=torch.int8)
    pages = cache.num_pages
    if equal:
        k[:, :, 0] = torch.randint(0, 2, (pages, H, 1), generator=gen, dtype=torch.int8)
        scale = torch.ones(pages, H)
    else:
        k = torch.randint(-127, 128, (pages, H, 2, d), generator=gen, dtype=torch.int8)
        scale = 2.0 ** torch.randint(-3, 2, (pages, H), generator=gen).float()
    cache = B.KVCache(cache.k, cache.v, cache.k_scale, cache.v_scale, k.cuda(), scale.cuda())
    q = torch.randn(len(lens), H * group, d, generator=gen).to(torch.bfloat16)
    sel, nsel = B.select_pages(cache, table, m, q.cuda(), n, first, last)
    assert B.cm_kv_status(cache) == B.CM_OK
    sel, nsel, table = sel.cpu(), nsel.cpu(), table.cpu()
    for b, t in enumerate(lens):
        at = table[b, :(t + P - 1) // P].long()
        for h in range(H):
            want = K.pick(K.scores(q[b, h * group:(h + 1) * group], k[at, h], scale[at, h]), n, first, last)
            assert sel[b, h].tolist() == want + [-1] * (n - len(want)) and nsel[b, h] == len(want), (b, h)


def test_select_reports_what_it_leaves_out(B):
    gen = torch.Generator().manual_seed(32)
    P, d = 16, 64
    cache, table, _ = _filled(B, [64, 64, 64], 1, P, d, "bf16", gen)
    s = torch.zeros(cache.num_pages, 1, 2, d, dtype=torch.int8, device="cuda")
    cache = B.KVCache(cache.k, cache.v, summary=s, summary_scale=torch.ones(cache.num_pages, 1, device="cuda"))
    q = torch.ones(3, 1, d, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([-1, 65, 64], dtype=torch.int32, device="cuda")
    table[2, 1] = -9
    sel, nsel = B.select_pages(cache, table, lens, q, 3)
    assert B.cm_kv_status(cache) == B.CM_ERR_DEVICE_CHECK
    assert sel.tolist() == [[[-1, -1, -1]], [[-1, -1, -1]], [[0, 2, 3]]] and nsel.tolist() == [[0], [0], [3]]


# ---- together --------------------------------------------------------------------------------
def test_prompt_then_tokens_under_one_mask(B):
    """A prompt through the attention forward and its keys into the cache, then one token after
    another by append and decode with the same descriptor: every token's output is the row that the
    forward gives for the whole sequence."""
    from masked_flashattention_gb300 import specs
    gen = torch.Generator().manual_seed(41)
    Bn, H, S, d, P = 2, 4, 512, 64, 32
    cuts = [[0, 20, 150, 300, S], [0, 40, 390, S, S]]
    seg = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    nseg = torch.tensor([4, 3], dtype=torch.int32, device="cuda")
    f, b = B.cm_compile_spec(specs.FWD[5]), B.cm_compile_spec(specs.BWD[5])
    desc = B.Descriptor(f, b, Bn, S)
    B.cm_build_descriptor(f, b, seg, nseg, desc)
    q, k, v = (torch.randn(Bn, H, S, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(3))
    rope = _rope(S, d, gen).cuda()
    prompt = [390, 410]
    cache = B.KVCache.alloc(Bn * (S // P), H, P, d)
    table = torch.randperm(Bn * (S // P), generator=gen).to(torch.int32).view(Bn, -1).cuda()
    lens = torch.zeros(Bn, dtype=torch.int32, device="cuda")
    qr, kr = q.clone(), k.clone()
    # rotate everything once for the whole-sequence forward (a scratch cache takes the keys)
    scratch = B.KVCache.alloc(Bn * (S // P), H, P, d)
    B.cm_kv_append(scratch, table, lens, k, v, q=q, q_out=qr, k_out=kr, rope=rope)
    full_o, full_lse = B.attention_forward(desc, qr, kr, v)
    after = torch.empty_like(lens)
    B.cm_kv_append(cache, table, lens, k, v, rope=rope, max_new=max(prompt), new_lens=after,
                   n_new=torch.tensor(prompt, dtype=torch.int32, device="cuda"))
    lens = after
    rows = torch.arange(Bn, device="cuda")
    for _ in range(101):
        at = lens.long()
        kt, vt, qt = (x[rows, :, at][:, :, None] for x in (k, v, q))
        one, after = torch.empty_like(qt), torch.empty_like(lens)
        B.cm_kv_append(cache, table, lens, kt, vt, q=qt, q_out=one, rope=rope, new_lens=after)
        o, lse = B.decode_attention(cache, table, after, one[:, :, 0], desc=desc)
        want, wl = full_o[rows, :, at].double(), full_lse[rows, :, at].double()
        # two bf16 roundings of the output and of the probabilities lie between them
        assert (o.double() - want).abs().max() <= 4 * BF16_HALF * 4.0
        assert (lse.double() - wl).abs().max() <= 1e-4
        lens = after
    assert B.cm_kv_status(cache) == B.CM_OK and B.cm_get_status(desc) == B.CM_OK


def test_sparse_step_in_a_graph(B):
    """Append, selection and decode captured once and replayed with new lengths, tokens and page tables, two
    graphs sharing the workspaces; replays equal eager calls."""
    gen = torch.Generator().manual_seed(42)
    Bn, H, group, P, d, cap, n = 3, 2, 4, 16, 128, 20, 6
    cache = B.KVCache.alloc(Bn * cap + 1, H, P, d, summaries=True)
    table = torch.randperm(Bn * cap, generator=gen).to(torch.int32).view(Bn, cap).cuda()
    rope = _rope(cap * P, d, gen).cuda()
    lens = torch.zeros(Bn, dtype=torch.int32, device="cuda")
    start = torch.tensor([200, 15, 0], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(Bn, H, 300, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    B.cm_kv_append(cache, table, lens, k, v, rope=rope, n_new=start, max_new=200, new_lens=lens.clone())
    work = torch.empty(B.cm_attn_decode_workspace_size(Bn, H * group, H, d), dtype=torch.uint8, device="cuda")
    swork = torch.empty(B.cm_select_pages_workspace_size(Bn, H, cap), dtype=torch.uint8, device="cuda")

    class Step:
        def __init__(self):
            self.lens, self.after = start.clone(), torch.zeros_like(start)
            self.q = torch.zeros(Bn, H * group, 1, d, dtype=torch.bfloat16, device="cuda")
            self.kt, self.vt = (torch.zeros(Bn, H, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.sel = torch.zeros(Bn, H, n, dtype=torch.int32, device="cuda")
            self.nsel = torch.zeros(Bn, H, dtype=torch.int32, device="cuda")
            self.o = torch.zeros(Bn, H * group, d, dtype=torch.bfloat16, device="cuda")
            self.dense = torch.zeros_like(self.o)
            self.lse = torch.zeros(Bn, H * group, device="cuda")

        def run(self):
            qr = self.q[:, :, 0]
            B.cm_kv_append(cache, table, self.lens, self.kt, self.vt, q=self.q, q_out=self.q, rope=rope, new_lens=self.after)
            B.cm_select_pages(cache, table, self.after, qr, self.sel, self.nsel, swork, 1, 1)
            B.cm_attn_decode(cache, table, self.after, qr, self.o, self.lse, work, sel=self.sel, nsel=self.nsel)
            B.cm_attn_decode(cache, table, self.after, qr, self.dense, None, work)

    steps, graphs = [Step(), Step(), Step()], []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        steps[0].run()
    torch.cuda.synchronize()
    for s in steps[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    eager = steps[2]
    for t in range(40):
        s, g = steps[t % 2], graphs[t % 2]
        q = torch.randn(Bn, H * group, 1, d, generator=gen).to(torch.bfloat16).cuda()
        for x in (s, eager):
            x.q.copy_(q), x.lens.copy_(start)
            x.kt.copy_(k[:, :, 250 + t % 40][:, :, None]), x.vt.copy_(v[:, :, 250 + t % 40][:, :, None])
        g.replay()
        eager.run()
        for name in ("q", "after", "sel", "nsel", "o", "lse", "dense"):
            assert torch.equal(getattr(s, name), getattr(eager, name)), (t, name)
        start = s.after.clone()
    assert B.cm_kv_status(cache) == B.CM_OK
    # dense attention over what the cache now holds
    final = start.tolist()
    o, lse = B.decode_attention(cache, table, start, q[:, :, 0])
    _check_decode(cache, table, final, q[:, :, 0], o, lse, 1 / math.sqrt(d), lambda b, g: torch.arange(final[b]))


def test_two_streams_with_workspaces_of_their_own(B):
    gen = torch.Generator().manual_seed(43)
    lens = [3000, 10, 700]
    cache, table, n = _filled(B, lens, 2, 64, 128, "bf16", gen)
    q = [torch.randn(3, 8, 128, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    want = [B.decode_attention(cache, table, n, x) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(B.decode_attention(cache, table, n, q[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_results_for_another_stream_keep_their_memory(B):
    """Memory that the current stream has given back but still writes to does not serve a call on another
    stream; nor does a later call there get memory whose contents the current stream still reads."""
    gen = torch.Generator().manual_seed(44)
    lens = [3000, 10, 700]
    cache, table, n = _filled(B, lens, 2, 64, 128, "bf16", gen)
    q = [torch.randn(3, 8, 128, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    want = [B.decode_attention(cache, table, n, x) for x in q]
    sizes = [B.cm_attn_decode_workspace_size(3, 8, 2, 128), 3 * 8 * 128 * 2, 3 * 8 * 4]
    torch.cuda.synchronize()
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    held = [torch.empty(b, dtype=torch.uint8, device="cuda") for b in sizes]
    torch.cuda._sleep(50_000_000)
    for t in held:
        t.fill_(255)
    del held, t
    o, lse = B.decode_attention(cache, table, n, q[0], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0][0]) and torch.equal(lse, want[0][1])
    o, lse = B.decode_attention(cache, table, n, q[0], stream=side)
    here.wait_stream(side)
    torch.cuda._sleep(50_000_000)
    kept = o.clone(), lse.clone()
    del o, lse
    for _ in range(4):
        B.decode_attention(cache, table, n, q[1], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(kept[0], want[0][0]) and torch.equal(kept[1], want[0][1])
    assert B.cm_kv_status(cache) == B.CM_OK


def test_many_sequences_sharing_pages(B):
    """More sequences than a block has threads, most of them short or empty, with a common prefix in
    shared pages; the same through selected pages, one row of pages a sequence and head."""
    gen = torch.Generator().manual_seed(51)
    Bn, H, group, P, d = 1300, 2, 2, 16, 64
    lens = [int(x) for x in torch.randint(0, 50, (Bn,), generator=gen)]
    for b in range(0, Bn, 3):
        lens[b] = 0
    cache, table, _ = _filled(B, [64] * 20, H, P, d, "bf16", gen)
    own = table.cpu()
    rows = torch.full((Bn, 4), -7, dtype=torch.int32)
    for b in range(Bn):
        rows[b] = own[b % 20]
        rows[b, 0] = own[0, 0]  # everybody's first page
    table, n = rows.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(Bn, H * group, d, generator=gen).to(torch.bfloat16).cuda()
    o, lse = B.decode_attention(cache, table, n, q)
    _check_decode(cache, table, lens, q, o, lse, 1 / 8, lambda b, g: torch.arange(lens[b]))
    pages = [(m + P - 1) // P for m in lens]
    nsel = torch.tensor([[p, max(p - 1, 0)] for p in pages], dtype=torch.int32)
    sel = torch.arange(4, dtype=torch.int32).repeat(Bn, H, 1)
    sel[:, 1] += 1  # the second head leaves the first page out
    o, lse = B.decode_attention(cache, table, n, q, sel=sel.cuda(), nsel=nsel.cuda())
    assert B.cm_kv_status(cache) == B.CM_OK
    _check_decode(cache, table, lens, q, o, lse, 1 / 8, lambda b, g: torch.arange(16 if g else 0, max(lens[b], 16 if g else 0)))
    # a table with room for long sequences takes the other way through the kernel
    wide = torch.full((Bn, 200), -7, dtype=torch.int32, device="cuda")
    wide[:, :4] = table
    o, lse = B.decode_attention(cache, wide, n, q)
    _check_decode(cache, wide, lens, q, o, lse, 1 / 8, lambda b, g: torch.arange(lens[b]))


def test_scales_of_either_sign_and_none(B):
    gen = torch.Generator().manual_seed(52)
    lens = [70, 33]
    for kv in ("bf16", "e4m3"):
        cache, table, n = _filled(B, lens, 1, 32, 128, kv, gen)
        q = torch.randn(2, 3, 128, generator=gen).to(torch.bfloat16).cuda()
        for scale in (0.0, -0.2):
            o, lse = B.decode_attention(cache, table, n, q, scale=scale)
            _check_decode(cache, table, lens, q, o, lse, scale, lambda b, g: torch.arange(lens[b]))


def test_values_of_one_head_do_not_reach_another(B):
    """A query of NaN, infinities or zeros spoils its own row alone; infinite keys give what the formula gives."""
    gen = torch.Generator().manual_seed(53)
    for kv in ("bf16", "e4m3"):
        cache, table, n = _filled(B, [50, 50], 2, 16, 64, kv, gen)
        q = torch.randn(2, 8, 64, generator=gen).to(torch.bfloat16).cuda()
        want, wl = B.decode_attention(cache, table, n, q)
        bad = q.clone()
        bad[0, 1], bad[1, 6, 3], bad[1, 2] = math.nan, math.inf, 0
        o, lse = B.decode_attention(cache, table, n, bad)
        assert o[0, 1].isnan().all() and lse[0, 1].isnan() and not o[1, 2].isnan().any()
        assert abs(lse[1, 2].item() - math.log(50)) < 1e-5
        keep = torch.ones(2, 8, dtype=torch.bool, device="cuda")
        keep[0, 1] = keep[1, 6] = keep[1, 2] = False
        assert torch.equal(o[keep], want[keep]) and torch.equal(lse[keep], wl[keep])


def test_many_key_value_heads(B):
    """12 key-value heads: more than the 8 warps of a block take at once."""
    gen = torch.Generator().manual_seed(54)
    H, P, d, lens = 12, 16, 64, [40, 7]
    cache = B.KVCache.alloc(8, H, P, d, summaries=True)
    table = torch.randperm(8, generator=gen).to(torch.int32).view(2, 4).cuda()
    k, v = (torch.randn(2, H, 40, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    zero, n = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    B.cm_kv_append(cache, table, zero, k, v, n_new=n)
    pool, _, _, _ = _host(cache)
    q = torch.randn(2, H, d, generator=gen).to(torch.bfloat16)
    sel, nsel = B.select_pages(cache, table, n, q.cuda(), 2)
    for b in range(2):
        at = table[b, :(lens[b] + P - 1) // P].cpu().long()
        for h in range(H):
            parts = [K.summary(K.rows(pool, None, table[b].cpu(), h, torch.arange(i * P, min(lens[b], i * P + P))).float())
                     for i in range(len(at))]
            for i, (s, e) in enumerate(parts):
                assert torch.equal(cache.summary[at[i], h].cpu(), s) and cache.summary_scale[at[i], h].item() == e
            want = K.pick(K.scores(q[b, h:h + 1], torch.stack([s for s, _ in parts]), [e for _, e in parts]), 2, 0, 0)
            assert sel[b, h, :len(want)].tolist() == want and nsel[b, h] == len(want)
    o, lse = B.decode_attention(cache, table, n, q.cuda(), sel=sel, nsel=nsel)
    chosen = {(b, h): torch.tensor([p for x in sel[b, h].tolist() if x >= 0 for p in range(x * P, min(lens[b], x * P + P))])
              for b in range(2) for h in range(H)}
    _check_decode(cache, table, lens, q, o, lse, 1 / 8, lambda b, g: chosen[b, g])
    assert B.cm_kv_status(cache) == B.CM_OK


@pytest.mark.parametrize("equal", [False, True])
def test_select_among_many_pages(B, equal):
    """9000 pages of one sequence: the wide form of the selection, and (equal scores) thousands of pages at the
    border; against a sort of the same scores."""
    gen = torch.Generator().manual_seed(55)
    pages, P, d, n = 9000, 16, 64, 1500
    s = torch.randint(-127, 128, (pages, 1, 2, d), generator=gen, dtype=torch.int8)
    if equal:
        s[:] = s[:1]
        s[::7] = 0
    cache = B.KVCache.alloc(pages, 1, P, d)
    cache = B.KVCache(cache.k, cache.v, summary=s.cuda(), summary_scale=torch.ones(pages, 1, device="cuda"))
    table = torch.randperm(pages, generator=gen).to(torch.int32).view(1, -1)
    lens = torch.tensor([pages * P - 3], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 2, d, generator=gen).to(torch.bfloat16)
    sel, nsel = B.select_pages(cache, table.cuda(), lens, q.cuda(), n, 2, 3)
    rows, best = s[table[0].long(), 0].to(F64), None
    for x in q[0].to(F64):
        f = K.exponent(x.abs().max().item())
        x = torch.round(x * 2.0 ** -f).clamp(-127, 127)
        score = (x.clamp(min=0) * rows[:, 0] + x.clamp(max=0) * rows[:, 1]).sum(1) * 2.0 ** f
        best = score if best is None else torch.maximum(best, score)
    best[:2] = best[-3:] = math.inf
    want = torch.sort(torch.sort(best, descending=True, stable=True)[1][:n])[0]
    assert nsel.item() == n and torch.equal(sel[0, 0].cpu().long(), want)
    assert B.cm_kv_status(cache) == B.CM_OK


def test_pool_beyond_32_bits(B):
    """Pages whose elements start beyond 2^32: 34,000 pages of 2^17 elements."""
    gen = torch.Generator().manual_seed(56)
    pages, H, P, d = 34000, 8, 128, 128
    k, v = (torch.empty(pages, H, P, d, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    scale = torch.full((H,), 0.02, device="cuda")
    s = torch.empty(pages, H, 2, d, dtype=torch.int8, device="cuda")
    cache = B.KVCache(k, v, scale, scale, s, torch.empty(pages, H, device="cuda"))
    table = torch.tensor([[33999, 5, 33000]], dtype=torch.int32, device="cuda")
    for i in table[0].tolist():
        k.view(torch.uint8)[i] = 127  # NaN
        v.view(torch.uint8)[i] = 127
    n = 300
    x, y = (torch.randn(1, H, n, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    B.cm_kv_append(cache, table, torch.zeros_like(lens), x, y)
    q = torch.randn(1, H * 2, d, generator=gen).to(torch.bfloat16).cuda()
    sel, nsel = B.select_pages(cache, table, lens, q, 2)
    o, lse = B.decode_attention(cache, table, lens, q)
    assert B.cm_kv_status(cache) == B.CM_OK
    at = table[0].long()
    small = B.KVCache(*(t.view(torch.uint8)[at].view(t.dtype) for t in (k, v)), scale, scale, s[at], cache.summary_scale[at])
    order = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    _check_decode(small, order, [n], q, o, lse, 1 / math.sqrt(d), lambda b, g: torch.arange(n))
    got, many = B.select_pages(small, order, lens, q, 2)
    assert torch.equal(got, sel) and torch.equal(many, nsel)


def test_expired_waits_are_reported_and_the_next_call_is_correct(B):
    """A wait limit of 1 ns makes ordinary waits of the attention kernel expire: CM_ERR_TIMEOUT, and with the
    default limit the same call succeeds (in both forms: rows kept whole, and rows split)."""
    gen = torch.Generator().manual_seed(57)
    for lens in ([100, 300], [5000, 9000]):
        cache, table, n = _filled(B, lens, 2, 64, 128, "bf16", gen)
        q = torch.randn(2, 4, 128, generator=gen).to(torch.bfloat16).cuda()
        B.cm_set_wait_limit_ns(1)
        try:
            B.decode_attention(cache, table, n, q)
            torch.cuda.synchronize()
        finally:
            B.cm_set_wait_limit_ns(0)
        assert B.cm_kv_status(cache) == B.CM_ERR_TIMEOUT
        o, lse = B.decode_attention(cache, table, n, q)
        assert B.cm_kv_status(cache) == B.CM_OK
        _check_decode(cache, table, lens, q, o, lse, 1 / math.sqrt(128), lambda b, g: torch.arange(lens[b]))


def test_binding_refusals(B):
    """What the binding turns down before the library is called."""
    cache = B.KVCache.alloc(4, 2, 16, 64)
    table, lens = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    work = torch.empty(B.cm_attn_decode_workspace_size(1, 4, 2, 64), dtype=torch.uint8, device="cuda")
    k = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    one = q[:, :2]
    decode = lambda **x: B.cm_attn_decode(*[x.get(n, y) for n, y in (("cache", cache), ("table", table), ("lens", lens),  # noqa: E731
                                            ("q", q), ("o", torch.empty_like(q)), ("lse", None), ("work", work))],
                                          **{n: x[n] for n in ("sel", "nsel") if n in x})
    sel = torch.zeros(1, 2, 3, dtype=torch.int32, device="cuda")
    for bad in ({"table": table.long()}, {"table": table[0]}, {"table": table.cpu()}, {"lens": lens.cpu()}, {"lens": lens[:0]},
                {"q": q.float()}, {"q": q[..., :32]}, {"q": q.transpose(1, 2)}, {"o": q[:, :2].clone()}, {"lse": torch.zeros(1, 4)},
                {"work": work.cpu()}, {"sel": sel}, {"nsel": sel[..., 0]}, {"sel": sel[:, :1], "nsel": sel[..., 0].contiguous()},
                {"lens": torch.ones(2, dtype=torch.int32, device="cuda")[::2].expand(1).repeat(2)}):
        with pytest.raises(ValueError):
            decode(**bad)
    for args, more in (((k, k[:, :1]), {}), ((k[:, :1], k[:, :1]), {}), ((k.float(), k), {}), ((k, k), {"q": k}),
                       ((k, k), {"k_out": k[:, :, :2]}), ((k, k), {"cu_new": cu}), ((one, one), {"cu_new": cu, "n_new": lens}),
                       ((k, k), {"n_new": cu}), ((k, k), {"rope": torch.zeros(9, 8, 3, device="cuda")}),
                       ((k, k), {"rope": torch.zeros(9, 8, 2)}), ((k, k), {"new_lens": lens.long()})):
        with pytest.raises(ValueError):
            B.cm_kv_append(cache, table, lens, *args, **more)
    with pytest.raises(B.CMError):
        B.cm_kv_append(cache, table, lens, k, k, new_lens=lens)  # lens is read while it would be written
    with pytest.raises(B.CMError):
        decode(work=work[:16])
    with pytest.raises(ValueError):
        B.select_pages(cache, table, lens, q, 2)  # no summaries
    e4m3 = torch.zeros(4, 2, 16, 64, device="cuda").to(torch.float8_e4m3fn)
    for args in ((e4m3, e4m3), (cache.k, e4m3), (cache.k, cache.v[:2]), (cache.k.transpose(1, 2), cache.v),
                 (cache.k, cache.v, lens.float(), lens.float()), (cache.k, cache.v, None, None, torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            B.KVCache(*args)


@pytest.mark.parametrize("summaries", [False, True])
def test_append_of_a_mixed_batch(B, summaries):
    """700 sequences, most with one new token, some with none, a few with long prompts, packed: the same cache as
    one sequence a call."""
    gen = torch.Generator().manual_seed(58)
    n, H, P, d, cap = 700, 9, 16, 64, 24
    held = torch.randint(0, 60, (n,), generator=gen)
    new = (torch.rand(n, generator=gen) < 0.9).long()
    for b, m in ((0, 250), (1, 0), (300, 97), (511, 16), (512, 300), (699, 33)):
        new[b] = m
    table = torch.randperm(n * cap, generator=gen).to(torch.int32).view(n, cap).cuda()
    lens, cu = held.to(torch.int32).cuda(), torch.cat([torch.zeros(1, dtype=torch.long), new.cumsum(0)]).to(torch.int32).cuda()
    total = int(new.sum())
    k, v = (torch.randn(total, H, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    rope = _rope(cap * P, 32, gen).cuda()
    first = torch.randn(n * cap, H, P, d, device="cuda").to(torch.bfloat16)
    caches = []
    for _ in range(2):
        more = {"summary": torch.zeros(n * cap, H, 2, d, dtype=torch.int8, device="cuda"),
                "summary_scale": torch.zeros(n * cap, H, device="cuda")} if summaries else {}
        caches.append(B.KVCache(first.clone(), first.clone(), **more))
    new_lens = torch.zeros_like(lens)
    B.cm_kv_append(caches[0], table, lens, k, v, rope=rope, cu_new=cu, max_new=300, new_lens=new_lens)
    assert torch.equal(new_lens.cpu().long(), held + new)
    at = cu.tolist()
    for b in range(n):
        t = slice(at[b], at[b + 1])
        if at[b] < at[b + 1]:
            B.cm_kv_append(caches[1], table[b:b + 1], lens[b:b + 1], k[t].transpose(0, 1)[None], v[t].transpose(0, 1)[None], rope=rope)
    assert B.cm_kv_status(caches[0]) == B.CM_OK and B.cm_kv_status(caches[1]) == B.CM_OK
    for name in ("k", "v") + (("summary", "summary_scale") if summaries else ()):
        assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), name
