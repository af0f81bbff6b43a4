"""Caches with block scales and pools of pages at the edge of what is allowed: queries of any size, values that are no
numbers, offsets beyond 32 bits, lengths that go back, calls that overlap."""
import math

import pytest
import torch

from oracle import kv_cache as K
from tests.test_block_cache_gpu import DTYPE, _check, _empty, _filled
from tests.test_kv_cache_gpu import _rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("power", [-120, -60, 60, 100])
def test_queries_of_any_size(B, kind, power):
    """Queries of 2^power with a scale that brings the scores back: the same bounds as for ordinary ones."""
    gen = torch.Generator().manual_seed(81)
    lens, H, P, d = [90, 33], 2, 32, 64
    cache, table, n = _filled(B, lens, H, P, d, kind, gen)
    q = (torch.randn(2, H * 3, d, generator=gen) * 0.5 * 2.0 ** power).to(torch.bfloat16).cuda()
    scale = 2.0 ** -power / math.sqrt(d)
    o, lse = B.decode_attention(cache, table, n, q, scale=scale)
    _check(cache, table, q, o, lse, scale, lambda b, g: torch.arange(lens[b]))
    q.zero_()  # every weight the same
    o, lse = B.decode_attention(cache, table, n, q)
    _check(cache, table, q, o, lse, 1.0, lambda b, g: torch.arange(lens[b]))


@pytest.mark.parametrize("kind,group", [("int8", 3), ("e4m3", 3), ("int8", 12)])
def test_numbers_that_are_none_stay_in_their_head(B, kind, group):
    """A NaN or an infinite query makes its own head's output NaN; a visible NaN value (e4m3) its channel."""
    gen = torch.Generator().manual_seed(82)
    lens, H, P, d = [100, 40], 2, 16, 64
    cache, table, n = _filled(B, lens, H, P, d, kind, gen)
    q = torch.randn(2, H * group, d, generator=gen).to(torch.bfloat16).cuda()
    want = B.decode_attention(cache, table, n, q)
    bad = q.clone()
    bad[0, 1, 5] = math.nan
    bad[1, group, 7] = math.inf
    o, lse = B.decode_attention(cache, table, n, bad)
    hit = torch.zeros(2, H * group, dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[1, group] = True
    assert o[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(o[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])
    if kind == "e4m3":
        v = cache.v.view(torch.uint8)
        v[int(table[0, 1]), 0, 3, 9] = 0x7F  # position 19 of the first sequence
        o, lse = B.decode_attention(cache, table, n, q)
        assert o[0, :group, 9].isnan().all() and torch.equal(lse, want[1])
        o[0, :group, 9] = want[0][0, :group, 9]
        assert torch.equal(o, want[0])


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_pool_beyond_32_bits(B, kind):
    """Pages that lie more than 2^32 elements into the pool hold and give what those of a small pool do."""
    gen = torch.Generator().manual_seed(83)
    H, P, d, pages, n = 16, 128, 128, 17000, 300
    big, small = (B.KVCache.alloc(m, H, P, d, dtype=DTYPE[kind], block_scales=True, summaries=True) for m in (pages, 3))
    assert big.k.numel() > 2**32
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    far = table + pages - 3
    rope = _rope(n + 1, d, gen).cuda()
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    for c, t in ((small, table), (big, far)):
        lens.zero_()
        g = torch.Generator().manual_seed(84)
        for count in (n - 1, 1):
            k, v = (torch.randn(1, H, count, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
            after = torch.empty_like(lens)
            B.cm_kv_append(c, t, lens, k, v, rope=rope, new_lens=after)
            lens = after
        assert B.cm_kv_status(c) == B.CM_OK
    for i in range(3):
        rows = min(P, n - 128 * [1, 2, 0][i])
        for x in ("k", "v"):
            a, b = (getattr(c, x)[at].view(torch.uint8)[:, :rows] for c, at in ((small, i), (big, pages - 3 + i)))
            assert torch.equal(a, b), (i, x)
            a, b = (getattr(c, x + "_scale")[at][:, :(rows + 15) // 16] for c, at in ((small, i), (big, pages - 3 + i)))
            assert torch.equal(a, b), (i, x)
        assert torch.equal(small.summary[i], big.summary[pages - 3 + i])
    q = torch.randn(1, 2 * H, d, generator=gen).to(torch.bfloat16).cuda()
    for more in ({}, {"window": 40, "sinks": 3}):
        a, b = B.decode_attention(small, table, lens, q, **more), B.decode_attention(big, far, lens, q, **more)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_slots_beyond_32_bits(B):
    P, pages = 128, 1 << 25
    free = torch.tensor([5, pages - 1, pages - 2], dtype=torch.int32, device="cuda")
    free = torch.cat([free, torch.zeros(pages - 3, dtype=torch.int32, device="cuda")])
    state = torch.tensor([[0, 0], [3, 0]], dtype=torch.int32, device="cuda")
    pool = B.KVPages(torch.full((1, 4), -1, dtype=torch.int32, device="cuda"), free, P, state=state)
    granted, slots = B.reserve_pages(pool, torch.zeros(1, dtype=torch.int32, device="cuda"), 200, slots=True)
    want = [(pages - 2) * P + i for i in range(P)] + [(pages - 1) * P + i for i in range(72)]
    assert granted.tolist() == [200] and slots[0].tolist() == want and want[0] > 2**31


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_lengths_that_go_back(B, kind):
    """Tokens that a program takes back (a length lowered) leave nothing but their blocks' scales: what is appended there
    next is stored with the larger of them, and nothing of the old rows reaches an output."""
    gen = torch.Generator().manual_seed(85)
    H, P, d = 2, 32, 64
    cache = _empty(B, 4, H, P, d, kind)
    table = torch.tensor([[3, 1]], dtype=torch.int32, device="cuda")
    rows = {x: [K.BlockRow(kind) for _ in range(H)] for x in "kv"}

    def append(at, x, y):
        B.cm_kv_append(cache, table, torch.tensor([at], dtype=torch.int32, device="cuda"), x.cuda(), y.cuda())
        for name, part in (("k", x), ("v", y)):
            for h in range(H):
                r = rows[name][h]
                del r.codes[at:]
                del r.exps[(at + 15) // 16:]
                r.append(part[0, h])

    def new(count, size):
        return [(torch.randn(1, H, count, d, generator=gen) * size).to(torch.bfloat16) for _ in range(2)]

    append(0, *new(20, 1.0))
    append(20, *new(15, 500.0))  # the second block's scale grows, a third begins
    append(22, *new(3, 0.01))    # back to 22: the second block keeps its scale
    append(16, *new(5, 0.01))    # back to the block's beginning: a scale of its own
    n = torch.tensor([21], dtype=torch.int32, device="cuda")
    for name, pool, scales in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
        for h in range(H):
            r = rows[name][h]
            pos = torch.arange(21)
            got = K.block_rows(pool.cpu(), scales.cpu(), table[0].cpu(), h, pos)
            assert torch.equal(got, r.values()), (name, h)
    q = torch.randn(1, H, d, generator=gen).to(torch.bfloat16).cuda()
    o, lse = B.decode_attention(cache, table, n, q)
    _check(cache, table, q, o, lse, 1 / 8, lambda b, g: torch.arange(21))


def test_calls_that_overlap(B):
    """Two streams with a workspace each, over one cache: the results of the calls alone."""
    gen = torch.Generator().manual_seed(86)
    lens, H, P, d = [4000, 700, 9000], 4, 64, 128
    cache, table, n = _filled(B, lens, H, P, d, "int8", gen)
    qs = [torch.randn(3, 16, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    want = [B.decode_attention(cache, table, n, q, **more) for q, more in zip(qs, ({}, {"window": 500, "sinks": 4}))]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [B.decode_attention(cache, table, n, q, stream=s, **more)
               for q, s, more in zip(qs, streams, ({}, {"window": 500, "sinks": 4}))]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind,d,rot,inter", [("int8", 64, 64, False), ("e4m3", 128, 32, True), ("int8", 128, 0, False)])
def test_append_in_place_and_without_queries(B, kind, d, rot, inter):
    """k_out = k and q_out = q; expanded values (strides of 0); the same cache without queries at all."""
    gen = torch.Generator().manual_seed(87)
    H, P, n = 3, 32, 83
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    rope = _rope(n, rot, gen).cuda() if rot else None
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, q = (torch.randn(1, H * m, n, d, generator=gen).to(torch.bfloat16).cuda() for m in (1, 2))
    v = torch.randn(1, H, 1, d, generator=gen).to(torch.bfloat16).cuda().expand(1, H, n, d)
    caches = [_empty(B, 3, H, P, d, kind) for _ in range(3)]
    k_out, q_out = torch.empty_like(k), torch.empty_like(q)
    B.cm_kv_append(caches[0], table, lens, k, v, q=q, q_out=q_out, k_out=k_out, rope=rope, interleaved=inter)
    B.cm_kv_append(caches[1], table, lens, k, v, rope=rope, interleaved=inter)
    k_in, q_in = k.clone(), q.clone()
    B.cm_kv_append(caches[2], table, lens, k_in, v, q=q_in, q_out=q_in, k_out=k_in, rope=rope, interleaved=inter)
    assert torch.equal(k_in, k_out) and torch.equal(q_in, q_out)
    for c in caches[1:]:
        for x in ("k", "v"):
            assert torch.equal(getattr(c, x).view(torch.uint8), getattr(caches[0], x).view(torch.uint8))
            a, b = (getattr(y, x + "_scale").nan_to_num(-1.0) for y in (c, caches[0]))
            assert torch.equal(a, b)


def test_the_second_loop_of_the_readme(B):
    """The README's loop without end as it stands there: prompts of different lengths, then tokens; one sequence ends."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(root, "README.md")).read(), re.S)
    code, = (x for x in blocks if "KVPages.alloc" in x)
    gen = torch.Generator().manual_seed(88)
    Bn, H, Hq, d, num_pages = 2, 2, 4, 64, 9
    counts, over = [[130, 70], [1, 1], [1, 2], [3, 1]], [[0, 0], [0, 1], [0, 0], [0, 0]]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def draw(h, t):
        return torch.randn(Bn, h, t, d, generator=gen).to(torch.bfloat16).cuda()

    steps = [(draw(H, max(c)), draw(H, max(c)), draw(Hq, max(c)), ints(c), ints(x)) for c, x in zip(counts, over)]
    keep = [(k.clone(), v.clone(), q.clone()) for k, v, q, _, _ in steps]
    rope = _rope(512, d, gen)
    names = {"torch": torch, "cm": B, "num_pages": num_pages, "max_pages": 8, "H_kv": H, "d": d, "B": Bn, "rope": rope.cuda(),
             "steps": steps, "lens": ints([0, 0]), "after": ints([0, 0])}
    exec(code, names)
    cache, pages = names["cache"], names["pages"]
    assert names["lens"].tolist() == [135, 3] and B.cm_kv_status(cache) == B.CM_OK and B.cm_kv_pages_status(pages) == B.CM_OK
    assert pages.state.tolist() == [[0, 3], [0, 1], [num_pages - 4, 0]]
    # the values as the oracle's blocks hold them (the second sequence since its end), and the last step's attention
    values = [[K.BlockRow("int8") for _ in range(H)] for _ in range(Bn)]
    for (_, v, _), c, x in zip(keep, counts, over):
        for b in range(Bn):
            for h in range(H):
                values[b][h].append(v[b, h, :c[b]].cpu())
                if x[b]:
                    values[b][h] = K.BlockRow("int8")
    table = pages.page_table.cpu()
    for b, n in ((0, 135), (1, 3)):
        for h in range(H):
            assert torch.equal(K.block_rows(cache.v.cpu(), cache.v_scale.cpu(), table[b], h, torch.arange(n)), values[b][h].values())
    q = torch.stack([K.rotate(keep[-1][2][b, :, counts[-1][b] - 1].cpu(), rope[n - 1, :, 0], rope[n - 1, :, 1], False)[0]
                     for b, n in ((0, 135), (1, 3))]).to(torch.bfloat16)
    _check(cache, pages.page_table, q, names["o"], names["lse"], 1 / math.sqrt(d), lambda b, g: torch.arange([135, 3][b]))
