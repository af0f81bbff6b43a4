"""Caches in 8 bits with a scale for each block of 16 tokens and head, on the GPU: append bit by bit against the
oracle's blocks, attention over them against the 64-bit form.

Cache memory that no token was written to holds NaN (e4m3) or 127 (int8), with NaN for scales, so that a key past a
length or behind a mask that reached an output would show."""
import math

import pytest
import torch

from oracle import kv_cache as K
from tests.test_kv_cache_gpu import BF16_HALF, F32_HALF, F64, _rope, _table
from tests.test_window_gpu import _forget, _visible

pytestmark = pytest.mark.gpu

DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


def _empty(B, pages, H, P, d, kind, summaries=False, joint=False):
    """A cache of memory that must not be used; joint: K and V halves of one tensor, so that pages lie apart."""
    both = torch.full((pages, 2, H, P, d), 0x7F, dtype=torch.uint8, device="cuda").view(DTYPE[kind])
    k, v = (both[:, i] if joint else both[:, i].view(torch.uint8).contiguous().view(DTYPE[kind]) for i in range(2))
    ks, vs = (torch.full((pages, H, P // 16), math.nan, device="cuda") for _ in range(2))
    more = {}
    if summaries:
        more = {"summary": torch.full((pages, H, 2, d), 99, dtype=torch.int8, device="cuda"),
                "summary_scale": torch.full((pages, H), 7.0, device="cuda")}
    return B.KVCache(k, v, ks, vs, **more)


def _filled(B, lens, H, P, d, kind, gen, joint=False, low=-3, high=3):
    """A cache whose sequences hold lens tokens of random numbers, blocks with scales of 2^low .. 2^high / 32."""
    need = [(n + P - 1) // P for n in lens]
    table, pages = _table(need, 2, gen)
    cache = _empty(B, pages, H, P, d, kind, joint=joint)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pos = torch.arange(n)
        at, row = table[b, pos // P].long().cuda(), (pos % P).cuda()
        for pool, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            x = torch.randn(n, H, d, generator=gen) * 32
            x = x.round().clamp(-128, 127).to(torch.int8) if kind == "int8" else x.to(torch.float8_e4m3fn)
            pool.view(torch.uint8)[at, :, row] = x.view(torch.uint8).cuda()
            first = pos[pos % 16 == 0]
            e = torch.randint(low, high + 1, (len(first), H), generator=gen) - 5
            scale[table[b, first // P].long().cuda(), :, (first % P // 16).cuda()] = (2.0 ** e.to(F64)).float().cuda()
    return cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def _check(cache, table, q, o, lse, scale, visible):
    """visible(b, h_kv) -> ascending positions.  A score is off by the fp32 sum of d exact products (one step a term, as the
    tensor core may cut) and its scaling, and in log2 units by one rounding beside the exponent of the value's scale (below
    64).  A weight is off by that and by its rounding to fp16; sums of n terms by a step each (a lane adds an eighth
    of them, the tensor core 16 at once); o by one rounding to bf16."""
    k, v, ks, vs, table, q = (x.cpu() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale, table, q))
    o, lse = o.double().cpu(), lse.double().cpu()
    d, group = cache.d, q.shape[1] // cache.H_kv
    for b in range(q.shape[0]):
        for g in range(cache.H_kv):
            pos = visible(b, g)
            hs = slice(g * group, (g + 1) * group)
            if len(pos) == 0:
                assert not o[b, hs].any() and (lse[b, hs] == -math.inf).all(), (b, g)
                continue
            kk, vv = K.block_rows(k, ks, table[b], g, pos), K.block_rows(v, vs, table[b], g, pos)
            want, wl, size, mag = K.decode(q[b, hs], kk, vv, scale)
            ds = (d + 8) * 2 * F32_HALF * size + 128 * F32_HALF
            sums = len(pos) / 8 * 2 * F32_HALF + 2.0 ** -18
            bound = BF16_HALF * want.abs() + (2.0 ** -11 + 2 * ds + sums) * mag + 1e-30
            assert ((o[b, hs] - want).abs() <= bound).all(), (b, g, ((o[b, hs] - want).abs() / bound).max())
            assert ((lse[b, hs] - wl).abs() <= ds + sums + 2.0 ** -20 * (1 + wl.abs())).all(), (b, g)


# ---- append ----------------------------------------------------------------------------------
APPEND = [
    # kind, d, P, H_kv, H_q, calls (new tokens of each sequence), packed, rot, interleaved, summary
    ("int8", 128, 64, 2, 6, [[1, 63, 64, 200], [1, 1, 1, 1], [15, 2, 17, 0], [1, 1, 1, 1]], False, 128, False, False),
    ("e4m3", 128, 16, 3, 3, [[5, 0, 31], [1, 1, 1], [1, 16, 1]], True, 128, True, True),
    ("int8", 64, 128, 1, 5, [[0, 127, 130], [300, 1, 0], [1, 1, 1]], True, 32, True, True),
    ("e4m3", 64, 32, 4, 4, [[31, 1], [33, 70], [1, 1]], False, 64, False, True),
    ("int8", 128, 128, 2, 0, [[7, 0, 3], [17, 129, 0], [1, 1, 1]], True, 96, False, True),
    ("e4m3", 128, 16, 8, 8, [[3] * 5, [0, 1, 2, 16, 40]], False, 0, False, False),
    ("int8", 64, 64, 3, 9, [[100], [65], [1], [1], [1]], False, 16, True, False),
    ("int8", 64, 16, 5, 1, [[1] * 40, [2000] + [1] * 39, [1] * 40], True, 64, False, False),
    ("e4m3", 64, 16, 9, 1, [[1] * 40, [2000] + [1] * 39, [1] * 40], True, 0, False, True),
]


@pytest.mark.parametrize("kind,d,P,H,Hq,calls,packed,rot,inter,summ", APPEND)
def test_append(B, kind, d, P, H, Hq, calls, packed, rot, inter, summ):
    """Calls one after another, larger and smaller than the ones before: every code, scale and summary, and nothing else."""
    gen = torch.Generator().manual_seed(71)
    n_seq = len(calls[0])
    total = [sum(c[b] for c in calls) for b in range(n_seq)]
    table, pages = _table([(t + P - 1) // P for t in total], 2, gen)
    cache = _empty(B, pages, H, P, d, kind, summaries=summ, joint=packed)
    wide = table.cuda()
    rope = _rope(wide.shape[1] * P, rot, gen) if rot else None
    rows = {x: [[K.BlockRow(kind) for _ in range(H)] for _ in range(n_seq)] for x in "kv"}
    held = [0] * n_seq
    for turn, new in enumerate(calls):
        size = [1.0, 9.0, 0.03, 700.0, 1.0][turn]
        lens = torch.tensor(held, dtype=torch.int32, device="cuda")
        new_lens = torch.full_like(lens, -5)
        T, n = max(new), sum(new)
        shape = (lambda h: (n + 3, h, d)) if packed else (lambda h: (n_seq, h, T, d))

        def strided(h, fill=None):  # a slice of a wider projection: token rows lie apart
            s = list(shape(h))
            s[-2 if packed else 1] += 2
            x = size * torch.randn(s, generator=gen) if fill is None else torch.full(s, fill)
            return x.to(torch.bfloat16).cuda()[:, 1:h + 1]

        k, v, k_out = strided(H), strided(H), strided(H, 5.0)
        more = {"q": strided(Hq), "q_out": strided(Hq, 6.0)} if Hq else {}
        if packed:
            more["cu_new"] = torch.tensor([0] + new, dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32)
            more["max_new"] = T
        else:
            more["n_new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        B.cm_kv_append(cache, wide, lens, k, v, k_out=k_out, rope=None if rope is None else rope.cuda(), interleaved=inter,
                       new_lens=new_lens, **more)
        assert B.cm_kv_status(cache) == B.CM_OK
        outs = [(k.cpu(), k_out.cpu(), 5.0)] + ([(more["q"].cpu(), more["q_out"].cpu(), 6.0)] if Hq else [])
        written = [torch.zeros(x.shape, dtype=torch.bool) for _, x, _ in outs]
        base, host_v = 0, v.cpu()
        for b in range(n_seq):
            for i in range(new[b]):
                at = (base + i,) if packed else (b, slice(None), i)
                for (src, dst, _), w in zip(outs, written):
                    w[at] = True
                    if i > 70:  # the rotation is tested elsewhere too
                        continue
                    p = held[b] + i
                    want, mag = (K.rotate(src[at], rope[p, :, 0], rope[p, :, 1], inter) if rot
                                 else (src[at].to(F64), src[at].to(F64).abs()))
                    assert ((dst[at].to(F64) - want).abs() <= BF16_HALF * want.abs() + 4 * F32_HALF * mag).all(), (b, i)
            for x, y in (("k", outs[0][1]), ("v", host_v)):
                part = y[base:base + new[b]].transpose(0, 1) if packed else y[b, :, :new[b]]
                for h in range(H):
                    if new[b]:
                        rows[x][b][h].append(part[h])
            base += new[b]
        for (_, dst, fill), w in zip(outs, written):
            assert (dst[~w] == fill).all()
        held = [a + c for a, c in zip(held, new)]
        assert new_lens.tolist() == held

        # the whole memory, as it ought to be
        for x, pool, scales in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
            want = torch.full((pages, H, P, d), 0x7F, dtype=torch.uint8)
            want_scale = torch.full((pages, H, P // 16), math.nan)
            for b in range(n_seq):
                for h in range(H):
                    r = rows[x][b][h]
                    if not r.codes:
                        continue
                    codes, pos = torch.stack(r.codes), torch.arange(held[b])
                    codes = codes.to(torch.int8) if kind == "int8" else codes.float().to(torch.float8_e4m3fn)
                    want[table[b, pos // P].long(), h, pos % P] = codes.view(torch.uint8)
                    first = torch.arange(0, held[b], 16)
                    want_scale[table[b, first // P].long(), h, first % P // 16] = torch.tensor([2.0 ** e for e in r.exps])
            assert torch.equal(scales.cpu().nan_to_num(-1.0), want_scale.nan_to_num(-1.0)), (turn, x)
            got = pool.cpu().view(torch.uint8)
            if kind == "e4m3":  # the two zeros are one
                got, want = (torch.where(y == 0x80, 0, y) for y in (got, want))
            assert torch.equal(got, want), (turn, x)
        if summ:
            got, scale = cache.summary.cpu(), cache.summary_scale.cpu()
            fresh = torch.zeros(pages, dtype=torch.bool)
            for b in range(n_seq):
                for i in range((held[b] + P - 1) // P):
                    page = int(table[b, i])
                    fresh[page] = True
                    for h in range(H):
                        part = rows["k"][b][h].values()[i * P:(i + 1) * P]
                        s, e = K.summary(part.float())
                        assert torch.equal(got[page, h], s) and scale[page, h] == e, (turn, b, i, h)
            assert (got[~fresh] == 99).all() and (scale[~fresh] == 7.0).all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_append_special_values(B, kind):
    """NaN, infinities, zeros, borders of the scales, halves, and a block whose first call is all zeros."""
    H, P, d = 2, 16, 64
    cache = _empty(B, 3, H, P, d, kind)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    rows = [[K.BlockRow(kind) for _ in range(H)] for _ in "kv"]
    top = 127.0 if kind == "int8" else 448.0
    calls = [
        [[0.0] * 8],
        [[math.nan, 1.0, 0.5, -0.5, 1.5, 2.5, -126.5, 126.5]],
        [[top, top, -top, 3.0, 1e-30, -1e-38, 0.25, 0.75], [math.nan] * 8],
        [[top * 1.0078125, 5.0, 5.0, -7.0, 9.0, 11.0, 13.0, 0.0]],
        [[math.inf, -math.inf, 1e30, -1e30, 1e38, 2.0 ** 30, math.nan, 1.0]],
        [[2.0 ** 39, -2.0 ** 20, 1.0, 0, 0, 0, 0, 0]] * 14,
    ]
    n = 0
    for call in calls:
        x = torch.zeros(1, H, len(call), d)
        for i, values in enumerate(call):
            x[0, 0, i, :8] = torch.tensor(values)
            x[0, 1, i, 8:16] = -2.0 * torch.tensor(values)
        x = x.to(torch.bfloat16)
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        B.cm_kv_append(cache, table, lens, x.cuda(), x.flip(1).cuda())
        for part, y in zip(rows, (x, x.flip(1))):
            for h in range(H):
                part[h].append(y[0, h])
        n += len(call)
        pos = torch.arange(n)
        at = table[0].cpu()[pos // P].long()
        for part, pool, scales in zip(rows, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
            for h in range(H):
                got = pool.cpu().view(torch.uint8)[at, h, pos % P].view(DTYPE[kind]).to(F64)
                assert torch.equal(got.nan_to_num(1e9), torch.stack(part[h].codes).nan_to_num(1e9)), n
                first = torch.arange(0, n, 16)
                assert scales.cpu()[at[first], h, 0].tolist() == [2.0 ** e for e in part[h].exps], n
    assert B.cm_kv_status(cache) == B.CM_OK


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_append_reports_what_it_leaves_out(B, kind):
    """As for the other caches: a sequence out of range appends nothing, a page outside the pool is skipped."""
    H, P, d = 1, 16, 64
    cache = _empty(B, 4, H, P, d, kind)
    cache.k.view(torch.uint8).zero_(), cache.v.view(torch.uint8).zero_(), cache.k_scale.fill_(1.0), cache.v_scale.fill_(1.0)
    table = torch.tensor([[0, 1], [2, 77], [3, 3], [1, -1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([0, 15, 31, -1], dtype=torch.int32, device="cuda")  # the third has no room for 2
    k = torch.ones(4, H, 2, d, dtype=torch.bfloat16, device="cuda")
    new_lens, k_out = torch.empty_like(lens), torch.zeros_like(k)
    B.cm_kv_append(cache, table, lens, k, k, k_out=k_out, new_lens=new_lens)
    assert B.cm_kv_status(cache) == B.CM_ERR_DEVICE_CHECK and B.cm_kv_status(cache) == B.CM_OK
    assert new_lens.tolist() == [2, 17, 31, -1]
    want = torch.zeros(4, P, dtype=torch.bool)
    want[0, :2] = want[2, 15] = True
    assert torch.equal(cache.k[:, 0, :, 0].cpu().float() != 0, want) and torch.equal(cache.v[:, 0, :, 0].cpu().float() != 0, want)
    assert k_out[..., 0].float().sum((1, 2)).tolist() == [2, 2, 0, 0]
    need = 2.0 ** -6 if kind == "int8" else 2.0 ** -8
    assert cache.k_scale[:, 0, 0].tolist() == [need, 1.0, 1.0, 1.0]
    none = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    B.cm_kv_append(cache, table, lens, none, none, cu_new=torch.zeros(5, dtype=torch.int32, device="cuda"), max_new=0, new_lens=new_lens)
    assert new_lens.tolist() == lens.tolist()


# ---- decode ----------------------------------------------------------------------------------
DECODE = [
    # kind, d, P, H_kv, group, lens
    ("int8", 128, 32, 2, 4, [1, 31, 32, 33, 0, 1025]),
    ("int8", 64, 64, 4, 1, [100, 64, 7, 16, 17]),
    ("int8", 128, 16, 1, 16, [400, 3]),
    ("int8", 64, 16, 2, 9, [1, 200]),
    ("int8", 128, 128, 1, 40, [513]),
    ("int8", 64, 16, 1, 2, [9001, 1]),
    ("e4m3", 128, 64, 2, 4, [1, 63, 64, 65, 0, 1000]),
    ("e4m3", 128, 16, 8, 1, [17, 16, 15, 1, 300]),
    ("e4m3", 64, 128, 1, 8, [127, 128, 129, 2500]),
    ("e4m3", 64, 32, 1, 24, [32, 511]),
    ("e4m3", 128, 128, 2, 16, [31, 32, 33, 700]),
    ("int8", 128, 64, 1, 7, [20000]),
    ("int8", 128, 16, 2, 3, [(7 * i) % 97 for i in range(150)]),
    ("int8", 64, 16, 8, 2, [33 + (11 * i) % 40 for i in range(400)]),  # several whole rows a warp
    ("e4m3", 64, 128, 16, 1, [97 + (11 * i) % 40 for i in range(200)]),
]


@pytest.mark.parametrize("kind,d,P,H,group,lens", DECODE)
def test_decode(B, kind, d, P, H, group, lens):
    gen = torch.Generator().manual_seed(72)
    cache, table, n = _filled(B, lens, H, P, d, kind, gen, joint=group % 2 == 0)
    wide = (torch.randn(len(lens), H * group + 2, d, generator=gen) * 0.5).to(torch.bfloat16).cuda()
    q = wide[:, 1:-1]
    o, lse = B.decode_attention(cache, table, n, q)
    assert B.cm_kv_status(cache) == B.CM_OK
    _check(cache, table, q, o, lse, 1 / math.sqrt(d), lambda b, g: torch.arange(lens[b]))
    again = B.decode_attention(cache, table, n, q)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_scales_far_apart(B, kind):
    """Values whose blocks' scales lie 2^24 apart, in rows where small ones carry the weight and where large ones do; keys
    whose scales lie as far apart.  A weight (with its value's scale) keeps its 11 bits down to 2^-21 of the row's
    largest (2^7 and more, against fp16's 2^-14) and is off by 2^-32 of that below."""
    gen = torch.Generator().manual_seed(73)
    H, P, d, lens = 2, 16, 64, [500, 40, 33]
    cache, table, n = _filled(B, lens, H, P, d, kind, gen)
    blocks = cache.v_scale.numel()
    for scales, times in ((cache.k_scale, 2.0 ** -7), (cache.v_scale, 1.0)):
        e = torch.randint(-12, 13, (blocks,), generator=gen).view(scales.shape).cuda()
        scales.copy_(torch.where(scales.isnan(), scales, times * 2.0 ** e.float()))
    q = (torch.randn(3, H * 3, d, generator=gen) * 2.0 ** -7).to(torch.bfloat16).cuda()
    o, lse = B.decode_attention(cache, table, n, q)
    assert B.cm_kv_status(cache) == B.CM_OK
    k, v, ks, vs, host = (x.cpu() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale, table))
    for b in range(3):
        for g in range(H):
            pos, hs = torch.arange(lens[b]), slice(3 * g, 3 * g + 3)
            kk, vv = K.block_rows(k, ks, host[b], g, pos), K.block_rows(v, vs, host[b], g, pos)
            want, wl, size, mag = K.decode(q[b, hs].cpu(), kk, vv, d ** -0.5)
            p = torch.exp(d ** -0.5 * q[b, hs].cpu().to(F64) @ kk.T - wl[:, None])
            scale = vs[host[b, pos // P].long(), g, pos % P // 16].to(F64)
            lost = 2.0 ** -32 * (p * scale).amax(1, keepdim=True) * (127 if kind == "int8" else 448) * lens[b]
            ds = (d + 8) * 2 * F32_HALF * size + 128 * F32_HALF
            bound = BF16_HALF * want.abs() + (2.0 ** -11 + 2 * ds + 2.0 ** -14) * mag + lost
            assert ((o[b, hs].double().cpu() - want).abs() <= bound).all(), (b, g)
            assert ((lse[b, hs].double().cpu() - wl).abs() <= ds + 2.0 ** -14 + 2.0 ** -20 * wl.abs()).all(), (b, g)


@pytest.mark.parametrize("kind,d,P,group", [("int8", 128, 16, 4), ("e4m3", 64, 64, 12), ("int8", 64, 32, 1)])
def test_window_mask_and_selection(B, kind, d, P, group):
    """The other ways to say what is visible, over a cache with block scales."""
    gen = torch.Generator().manual_seed(74)
    lens, H = [700, 130, 1, 257], 2
    cache, table, n = _filled(B, lens, H, P, d, kind, gen)
    q = (torch.randn(4, H * group, d, generator=gen) * 0.5).to(torch.bfloat16).cuda()
    scale = 1 / math.sqrt(d)
    o, lse = B.decode_attention(cache, _forget(table, lens, P, 65, 5), n, q, window=65, sinks=5)
    _check(cache, table, q, o, lse, scale, lambda b, g: _visible(lens[b], 65, 5))
    from masked_flashattention_gb300 import specs
    f, b = (B.cm_compile_spec(t) for t in specs.sliding_window(65, 5))
    desc = B.Descriptor(f, b, 4, 768)
    B.cm_build_descriptor(f, b, torch.tensor([[0, 768]] * 4, dtype=torch.int32, device="cuda"),
                          torch.ones(4, dtype=torch.int32, device="cuda"), desc)
    o, lse = B.decode_attention(cache, table, n, q, desc=desc)
    _check(cache, table, q, o, lse, scale, lambda b, g: _visible(lens[b], 65, 5))
    keep = 3
    sel = torch.full((4, H, keep), -1, dtype=torch.int32)
    nsel = torch.zeros(4, H, dtype=torch.int32)
    for b in range(4):
        for g in range(H):
            pages = torch.randperm((lens[b] + P - 1) // P, generator=gen)[:keep].sort()[0]
            sel[b, g, :len(pages)], nsel[b, g] = pages, len(pages)
    o, lse = B.decode_attention(cache, table, n, q, sel=sel.cuda(), nsel=nsel.cuda())
    assert B.cm_kv_status(cache) == B.CM_OK

    def chosen(b, g):
        pos = torch.arange(lens[b])
        return pos[torch.isin(pos // P, sel[b, g, :nsel[b, g]])]

    _check(cache, table, q, o, lse, scale, chosen)


def test_beside_a_cache_with_one_scale_a_head(B):
    """The same e4m3 bytes and the same power of two for every block: the attention of the cache with scales per head."""
    gen = torch.Generator().manual_seed(75)
    lens, H, P, d = [300, 77, 1], 2, 32, 128
    cache, table, n = _filled(B, lens, H, P, d, "e4m3", gen)
    one = torch.full((H,), 2.0 ** -5, device="cuda")
    cache.k_scale.fill_(2.0 ** -5), cache.v_scale.fill_(2.0 ** -5)
    plain = B.KVCache(cache.k, cache.v, one, one)
    q = torch.randn(3, 8, d, generator=gen).to(torch.bfloat16).cuda()
    o, lse = B.decode_attention(cache, table, n, q)
    o2, lse2 = B.decode_attention(plain, table, n, q)
    assert torch.equal(o, o2)
    assert ((lse - lse2).abs() <= 8 * F32_HALF * (8 + lse.abs())).all()  # sums with another reference: exponents only


def test_pages_without_numbers_and_bad_scales(B):
    """A page outside the pool is skipped and reported; a scale that is no power of two counts as its exponent says."""
    gen = torch.Generator().manual_seed(76)
    cache, table, n = _filled(B, [60, 60], 1, 16, 64, "int8", gen)
    q = torch.randn(2, 2, 64, generator=gen).to(torch.bfloat16).cuda()
    want = B.decode_attention(cache, table, n, q)
    cache.k_scale.mul_(1.75), cache.v_scale.mul_(1.25)
    got = B.decode_attention(cache, table, n, q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    cache.k_scale.div_(1.75), cache.v_scale.div_(1.25)
    bad = table.clone()
    bad[1, 1] = cache.num_pages
    o, lse = B.decode_attention(cache, bad, n, q)
    assert B.cm_kv_status(cache) == B.CM_ERR_DEVICE_CHECK
    gone = torch.cat([torch.arange(16), torch.arange(32, 60)])
    _check(cache, table, q, o, lse, 1 / 8, lambda b, g: gone if b else torch.arange(60))


def test_refusals_of_the_binding(B):
    k = torch.zeros(3, 2, 32, 64, dtype=torch.int8, device="cuda")
    s = torch.ones(3, 2, 2, device="cuda")
    B.KVCache(k, k.clone(), s, s.clone())
    for args in ((k, k), (k, k, s), (k, k, s, s[:, :, 0].contiguous()), (k, k, s[0, :, 0].contiguous(), s[0, :, 0].contiguous()),
                 (k, k, s.double(), s), (k, k.view(torch.float8_e4m3fn), s, s), (k.to(torch.bfloat16), k.to(torch.bfloat16), s, s),
                 (k.view(torch.float8_e4m3fn), k.view(torch.float8_e4m3fn), s, s[0, :, 0].contiguous())):
        with pytest.raises(ValueError):
            B.KVCache(*args)
    with pytest.raises(ValueError):
        B.KVCache.alloc(3, 2, 32, 64, dtype=torch.int8, k_scale=s, v_scale=s)
    for dtype in (torch.int8, torch.float8_e4m3fn):
        c = B.KVCache.alloc(3, 2, 32, 64, dtype=dtype, block_scales=True, summaries=True)
        assert c.k_scale.shape == (3, 2, 2) and c.summary.shape == (3, 2, 2, 64)


# ---- a loop of all of them -----------------------------------------------------------------------
@pytest.mark.parametrize("kind,d,P,window,sinks", [("int8", 64, 16, 40, 4), ("e4m3", 128, 32, 70, 33)])
def test_generation_without_end(B, kind, d, P, window, sinks):
    """Reserve, append, attend, release, over a pool that holds far fewer tokens than are generated, one captured
    step replayed: every output is that of the window and the sinks, and every page has one owner."""
    from oracle import kv_pages as Q
    gen = torch.Generator().manual_seed(77)
    H, group, n_seq, T = 2, 3, 3, 20
    most = 40 * P
    pool_pages = n_seq * (-(-(window + T) // P) + 1 + -(-sinks // P))
    pages = B.KVPages.alloc(pool_pages, n_seq, most // P, P, window=window, sinks=sinks)
    cache = B.KVCache.alloc(pool_pages, H, P, d, dtype=DTYPE[kind], block_scales=True)
    rope = _rope(most, d, gen).cuda()
    lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
    after, granted, n_new = torch.empty_like(lens), torch.empty_like(lens), torch.empty_like(lens)
    done = torch.zeros_like(lens)
    k, v = (torch.empty(n_seq, H, T, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.empty(n_seq, H * group, T, d, dtype=torch.bfloat16, device="cuda")
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    last = torch.empty(n_seq, H * group, d, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(last), torch.empty(n_seq, H * group, device="cuda")
    work = torch.empty(B.cm_attn_decode_workspace_size(n_seq, H * group, H, d), dtype=torch.uint8, device="cuda")
    slots = torch.empty(n_seq, T, dtype=torch.int64, device="cuda")

    def step():
        B.cm_kv_reserve(pages, pages.state, pages.spare, lens, T, n_new=n_new, granted=granted, slots=slots)
        B.cm_kv_append(cache, pages.page_table, lens, k, v, q=q, q_out=q_out, k_out=k_out, rope=rope, n_new=granted,
                       max_new=T, new_lens=after)
        at = (granted - 1).clamp(min=0).long()
        last.copy_(q_out.gather(2, at[:, None, None, None].expand(-1, H * group, 1, d))[:, :, 0])
        B.cm_attn_decode(cache, pages.page_table, after, last, o, lse, work, window=window, sinks=sinks)
        B.cm_kv_release(pages, pages.spare, pages.state, after, done)
        lens.copy_(after * (1 - done))

    n_new.zero_()
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rows = {x: [[K.BlockRow(kind) for _ in range(H)] for _ in range(n_seq)] for x in "kv"}
    held = [0] * n_seq
    for turn in range(60):
        counts = [T, 1, 7] if turn in (0, 30) else [1 + (turn * 3 + b) % 9 * (b == 1) for b in range(n_seq)]
        over = [0, int(turn == 29), 0]
        n_new.copy_(torch.tensor(counts))
        done.copy_(torch.tensor(over))
        for x in (k, v, q):
            x.copy_((torch.randn(x.shape, generator=gen) * (0.5 + turn % 4)).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert granted.tolist() == counts and B.cm_kv_pages_status(pages) == B.CM_OK and B.cm_kv_status(cache) == B.CM_OK
        host_k, host_v, hq, ho, hl = k_out.cpu(), v.cpu(), last.cpu(), o.double().cpu(), lse.double().cpu()
        for b in range(n_seq):
            for h in range(H):
                rows["k"][b][h].append(host_k[b, h, :counts[b]])
                rows["v"][b][h].append(host_v[b, h, :counts[b]])
            held[b] += counts[b]
            pos = _visible(held[b], window, sinks)
            for h in range(H):
                hs = slice(h * group, (h + 1) * group)
                kk, vv = rows["k"][b][h].values()[pos], rows["v"][b][h].values()[pos]
                want, wl, size, mag = K.decode(hq[b, hs], kk, vv, d ** -0.5)
                ds = (d + 8) * 2 * F32_HALF * size + 128 * F32_HALF
                # fp16 weights (times their value's scale) are off by half its smallest number, 2^-25, where they are small; the
                # row's largest is 2^7 at least, so each of n is off by 2^-32 of that, times a stored number of at most 127 or 448
                p = torch.exp(d ** -0.5 * hq[b, hs].to(F64) @ kk.T - wl[:, None])
                scale = torch.tensor([2.0 ** rows["v"][b][h].exps[i // 16] for i in pos.tolist()], dtype=F64)
                lost = 2.0 ** -32 * (p * scale).amax(1, keepdim=True) * (127 if kind == "int8" else 448) * len(pos)
                bound = BF16_HALF * want.abs() + (2.0 ** -11 + 2 * ds + 2.0 ** -16) * mag + lost
                assert ((ho[b, hs] - want).abs() <= bound).all(), (turn, b, h)
                assert ((hl[b, hs] - wl).abs() <= ds + 2.0 ** -16 + 2.0 ** -20 * wl.abs()).all(), (turn, b, h)
            if over[b]:
                held[b] = 0
                for x in "kv":
                    rows[x][b] = [K.BlockRow(kind) for _ in range(H)]
        assert lens.tolist() == held
        state, table = pages.state.tolist(), pages.page_table.tolist()
        own = [x for row in Q.owned(table, state[:-1], sinks, P) for x in row]
        assert sorted(own + pages.free_pages.tolist()[:state[-1][0]]) == list(range(pool_pages))
    assert sum(held) > pool_pages * P // 2
