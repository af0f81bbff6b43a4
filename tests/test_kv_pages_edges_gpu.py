"""Pools of pages where they are used with what comes next, and at their ends."""
import pytest
import torch

from tests.test_kv_cache_gpu import _rope
from tests.test_kv_pages_gpu import Both, _ints

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "int8_block", "e4m3_block"]


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


# ---- appends of packed tokens that were not all granted -------------------------------------------
def _cache(B, kind, pages, H, P, d):
    """A cache with summaries whose memory is all zeros (scales: 1)."""
    dtype = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8_block": torch.int8, "e4m3_block": torch.float8_e4m3fn}[kind]
    k, v = (torch.zeros(pages, H, P, d, dtype=torch.uint8, device="cuda").view(dtype) if kind != "bf16" else
            torch.zeros(pages, H, P, d, dtype=dtype, device="cuda") for _ in range(2))
    scales = {}
    if kind != "bf16":
        shape = (H,) if kind == "e4m3" else (pages, H, P // 16)
        scales = {x: torch.ones(shape, device="cuda") for x in ("k_scale", "v_scale")}
    return B.KVCache(k, v, summary=torch.zeros(pages, H, 2, d, dtype=torch.int8, device="cuda"),
                     summary_scale=torch.ones(pages, H, device="cuda"), **scales)


def _memory(cache):
    return [x.view(torch.uint8).clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.summary, cache.summary_scale)
            if x is not None]


def _copy(B, kind, cache):
    other = _cache(B, kind, cache.num_pages, cache.H_kv, cache.page_size, cache.d)
    for x in ("k", "v", "k_scale", "v_scale", "summary", "summary_scale"):
        if getattr(cache, x) is not None:
            getattr(other, x).view(torch.uint8).copy_(getattr(cache, x).view(torch.uint8))
    return other


def _packed(counts, granted, H, Hq, d, gen):
    """Packed tokens, and the same where each sequence has only what it was granted, padded."""
    n, top = sum(counts), max(max(granted), 1)
    k, v, q = (torch.randn(n, h, d, generator=gen).to(torch.bfloat16).cuda() for h in (H, H, Hq))
    padded, at = [torch.zeros(len(counts), h, top, d, dtype=torch.bfloat16, device="cuda") for h in (H, H, Hq)], 0
    mine = torch.zeros(n, dtype=torch.bool, device="cuda")
    for b, (c, g) in enumerate(zip(counts, granted)):
        for x, y in zip((k, v, q), padded):
            y[b, :, :g] = x[at:at + g].transpose(0, 1)
        mine[at:at + g] = True
        at += c
    return (k, v, q), padded, mine


def _append_both(B, kind, cache, table, lens, counts, granted, gen, rope):
    """The packed call with `granted` beside the padded one of those tokens alone: all memory, outputs and lengths."""
    other, H, d, Hq = _copy(B, kind, cache), cache.H_kv, cache.d, 2 * cache.H_kv
    (k, v, q), (pk, pv, pq), mine = _packed(counts, granted, H, Hq, d, gen)
    cu = _ints([0] + counts).cumsum(0).to(torch.int32)
    q_out, k_out, after = torch.full_like(q, 5.0), torch.full_like(k, 6.0), torch.full_like(lens, -9)
    B.cm_kv_append(cache, table, lens, k, v, q=q, q_out=q_out, k_out=k_out, rope=rope, cu_new=cu, max_new=max(counts),
                   new_lens=after, granted=_ints(granted))
    assert B.cm_kv_status(cache) == B.CM_OK
    pq_out, pk_out, p_after = torch.empty_like(pq), torch.empty_like(pk), torch.empty_like(lens)
    B.cm_kv_append(other, table, lens, pk, pv, q=pq, q_out=pq_out, k_out=pk_out, rope=rope, n_new=_ints(granted), new_lens=p_after)
    assert after.tolist() == p_after.tolist() == [a + b for a, b in zip(lens.tolist(), granted)]
    for a, b in zip(_memory(cache), _memory(other)):
        assert torch.equal(a, b)
    assert (q_out[~mine] == 5.0).all() and (k_out[~mine] == 6.0).all()
    at = 0
    for b, (c, g) in enumerate(zip(counts, granted)):
        assert torch.equal(q_out[at:at + g].transpose(0, 1), pq_out[b, :, :g])
        assert torch.equal(k_out[at:at + g].transpose(0, 1), pk_out[b, :, :g])
        at += c
    return after


@pytest.mark.parametrize("kind", KINDS)
def test_a_packed_append_heeds_what_was_granted(B, kind):
    """The pool runs short in a step of packed tokens, and the row that gets nothing still names pages that are others' by now:
    these hold what their owners wrote, and nothing else."""
    gen = torch.Generator().manual_seed(95)
    H, P, d = 2, 16, 64
    x, cache, rope = Both(B, 6, 4, 8, P), _cache(B, kind, 6, 2, P, d), _rope(8 * P, d, gen).cuda()
    lens = _ints([0] * 4)
    first = x.reserve([0] * 4, [16, 16, 0, 40], packed=True)
    assert first == [16, 16, 0, 40]
    lens = _append_both(B, kind, cache, x.gpu.page_table, lens, [16, 16, 0, 40], first, gen, rope)
    x.release(lens.tolist(), [0, 0, 0, 1])
    lens[3] = 0
    counts = [33, 1, 20, 40]
    granted = x.reserve(lens.tolist(), counts, packed=True)
    assert granted == [33, 1, 0, 0]
    stale, owned = set(x.table[3][:3]), set(x.table[0][:4] + x.table[1][:2])
    assert stale <= owned  # what an append without `granted` would overwrite
    lens = _append_both(B, kind, cache, x.gpu.page_table, lens, counts, granted, gen, rope)
    assert lens.tolist() == [49, 17, 0, 0]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seqs,long", [(5, 100), (101, 2000), (40, 700)])
def test_granted_in_part(B, kind, seqs, long):
    """Any part of a sequence's tokens, in batches small and large enough for each way of finding them; none at all."""
    gen = torch.Generator().manual_seed(96)
    H, P, d, wide = 1, 16, 64, 200
    counts = [long] + torch.randint(0, 4, (seqs - 1,), generator=gen).tolist()
    held = torch.randint(0, 40, (seqs,), generator=gen).tolist()
    table = torch.randperm(seqs * wide, generator=gen).view(seqs, wide).to(torch.int32).cuda()
    cache = _cache(B, kind, seqs * wide, H, P, d)
    rope = _rope(wide * P, 32, gen).cuda()
    for part in (0.0, 0.5, 1.0):
        granted = [int(part * c + 0.5) for c in counts]
        lens = _append_both(B, kind, cache, table, _ints(held), counts, granted, gen, rope)
        held = lens.tolist() if part == 0.5 else held


def test_granted_out_of_range(B):
    """More than a sequence's tokens, or fewer than none: it appends nothing and is reported; the others are whole."""
    gen = torch.Generator().manual_seed(97)
    cache = _cache(B, "bf16", 8, 1, 16, 64)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    k = torch.randn(8, 1, 64, generator=gen).to(torch.bfloat16).cuda()
    lens, after = _ints([0] * 4), _ints([0] * 4)
    B.cm_kv_append(cache, table, lens, k, k, cu_new=_ints([0, 2, 4, 6, 8]), max_new=2, new_lens=after, granted=_ints([3, -1, 1, 2]))
    assert B.cm_kv_status(cache) == B.CM_ERR_DEVICE_CHECK and after.tolist() == [0, 0, 1, 2]
    assert (cache.v[:, 0, :, 0] != 0).sum((1,)).tolist() == [0, 0, 0, 0, 1, 0, 2, 0]
    pad = torch.zeros(4, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    for bad in ({"granted": lens}, {"cu_new": _ints([0, 2, 4, 6, 8]), "granted": lens[:3]}):
        with pytest.raises(ValueError):
            B.cm_kv_append(cache, table, lens, *((k, k) if "cu_new" in bad else (pad, pad)), **bad)
def test_more_pages_come_back_than_there_are(B):
    """Sequences whose states claim more pages than the pool has, from a list that is empty, partly full and full: what has
    no room is dropped and reported, and the list never names more than there are."""
    for left in (0, 2, 5):
        x = Both(B, 5, 3, 8, 16)
        x.table = [[0, 1, 2, 3, 4, 0, 1, 2], [3, 4, 0, 1, 2, 3, 4, 0], [1, 2, 3, 4, 0, 1, 2, 3]]
        x.state = [[0, 8], [0, 8], [0, 8], [left, 0]]
        x.gpu.page_table.copy_(_ints(x.table))
        x.gpu.state.copy_(_ints(x.state))
        x.release([0, 0, 0], [1, 0, 1], bad=True)
        assert x.state[3] == [5, 0]
