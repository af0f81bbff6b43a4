"""Single-token attention under a sliding window with sinks against the 64-bit form, over every kind of cache.

All cache memory that no token was written to holds NaN, and page table entries behind the window name no page."""
import math

import pytest
import torch

from tests.test_kv_cache_gpu import _check_decode, _filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


def _visible(n, window, sinks):
    pos = torch.arange(n)
    return pos[(pos < sinks) | (pos > n - 1 - window)]


def _forget(table, lens, P, window, sinks):
    """Entries of the pages that hold no visible key name no page."""
    t = table.cpu()
    for b, n in enumerate(lens):
        seen = set((_visible(n, window, sinks) // P).tolist())
        for i in range(t.shape[1]):
            if i not in seen:
                t[b, i] = -9
    return t.cuda()


WINDOW = [
    # d, P, kv, H_kv, group, lens, window, sinks
    (128, 64, "bf16", 2, 4, [0, 1, 63, 64, 65, 1000], 1, 0),
    (128, 64, "bf16", 2, 4, [0, 1, 100, 101, 102, 1000], 96, 5),
    (64, 16, "bf16", 3, 5, [1, 15, 16, 17, 300, 401, 402, 417], 17, 1),
    (64, 16, "bf16", 1, 2, [31, 32, 33, 48, 63, 64, 65, 500], 31, 16),
    (128, 16, "e4m3", 2, 3, [1, 40, 77, 200, 1025], 64, 20),
    (64, 32, "e4m3", 1, 16, [64, 65, 700], 33, 31),
    (128, 128, "bf16", 1, 16, [129, 2500], 200, 130),
    (128, 32, "bf16", 1, 24, [511, 97], 64, 0),
    (128, 64, "bf16", 1, 4, [700, 30], 100000, 2),
    (128, 64, "bf16", 1, 4, [700, 30], 3, 100000),
    (128, 64, "bf16", 1, 7, [20000], 9001, 4),
    (64, 128, "e4m3", 2, 1, [20001, 5], 4096, 1),
    (128, 16, "bf16", 2, 3, [(7 * i) % 97 for i in range(150)], 20, 3),
]


@pytest.mark.parametrize("d,P,kv,H,group,lens,window,sinks", WINDOW)
def test_window(B, d, P, kv, H, group, lens, window, sinks):
    gen = torch.Generator().manual_seed(51)
    cache, table, n = _filled(B, lens, H, P, d, kv, gen, joint=group % 2 == 0)
    q = (torch.randn(len(lens), H * group, d, generator=gen) * 2).to(torch.bfloat16).cuda()
    o, lse = B.decode_attention(cache, _forget(table, lens, P, window, sinks), n, q, window=window, sinks=sinks)
    assert B.cm_kv_status(cache) == B.CM_OK
    _check_decode(cache, table, n, q, o, lse, 1 / math.sqrt(d), lambda b, g: _visible(lens[b], window, sinks))


def test_a_window_of_everything_is_the_call_without(B):
    gen = torch.Generator().manual_seed(52)
    lens = [700, 1, 64, 0]
    cache, table, n = _filled(B, lens, 2, 32, 64, "bf16", gen)
    q = torch.randn(4, 6, 64, generator=gen).to(torch.bfloat16).cuda()
    want = B.decode_attention(cache, table, n, q)
    for window, sinks in ((700, 0), (2**31 - 1, 2**31 - 1), (1, 699), (350, 350)):
        got = B.decode_attention(cache, table, n, q, window=window, sinks=sinks)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (window, sinks)


def test_bad_pages_and_lengths(B):
    """A visible page outside the pool is skipped, a length out of range sees nothing; both are reported."""
    gen = torch.Generator().manual_seed(53)
    lens = [200, 200, 200]
    cache, table, n = _filled(B, lens, 1, 16, 64, "bf16", gen)
    q = torch.randn(3, 2, 64, generator=gen).to(torch.bfloat16).cuda()
    bad = table.clone()
    bad[0, 12] = cache.num_pages  # positions 192 to 199
    n[2] = 10000
    o, lse = B.decode_attention(cache, bad, n, q, window=20, sinks=3)
    assert B.cm_kv_status(cache) == B.CM_ERR_DEVICE_CHECK and B.cm_kv_status(cache) == B.CM_OK
    seen = [_visible(200, 20, 3), _visible(200, 20, 3), torch.arange(0)]
    seen[0] = seen[0][seen[0] < 192]
    _check_decode(cache, table, n, q, o, lse, 1 / 8, lambda b, g: seen[b])


def test_graph_follows_the_lengths(B):
    gen = torch.Generator().manual_seed(54)
    lens = [500, 333]
    cache, table, n = _filled(B, lens, 2, 32, 128, "bf16", gen)
    q = torch.randn(2, 8, 128, generator=gen).to(torch.bfloat16).cuda()
    o, lse = torch.empty_like(q), torch.empty(2, 8, device="cuda")
    work = torch.empty(B.cm_attn_decode_workspace_size(2, 8, 2, 128), dtype=torch.uint8, device="cuda")

    def call():
        B.cm_attn_decode(cache, table, n, q, o, lse, work, window=64, sinks=4)

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for now in ([500, 333], [90, 12], [68, 69]):
        n.copy_(torch.tensor(now))
        g.replay()
        torch.cuda.synchronize()
        _check_decode(cache, table, n, q, o, lse, 128 ** -0.5, lambda b, h: _visible(now[b], 64, 4))


def test_refusals_of_the_binding(B):
    gen = torch.Generator().manual_seed(55)
    cache, table, n = _filled(B, [40], 1, 16, 64, "bf16", gen)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    sel = torch.zeros(1, 1, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        B.decode_attention(cache, table, n, q, sinks=2)
    with pytest.raises(ValueError):
        B.decode_attention(cache, table, n, q, window=4, sel=sel, nsel=sel[..., 0].contiguous())
    for bad in ({"window": 2**32 + 4}, {"window": 4, "sinks": 2**31}):
        with pytest.raises(ValueError):
            B.decode_attention(cache, table, n, q, **bad)
    for bad in ({"window": 0}, {"window": -3}, {"window": 4, "sinks": -1}):
        with pytest.raises(B.CMError):
            B.decode_attention(cache, table, n, q, **bad)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (100, 4), (200, 150), (5000, 3)])
def test_mask_spec_is_the_same_mask(B, window, sinks):
    """The descriptor of specs.sliding_window, forward and backward, is what the token sees."""
    from masked_flashattention_gb300 import specs
    S = 512
    f, b = (B.cm_compile_spec(t) for t in specs.sliding_window(window, sinks))
    desc = B.Descriptor(f, b, 1, S)
    B.cm_build_descriptor(f, b, torch.tensor([[0, S]], dtype=torch.int32, device="cuda"),
                          torch.ones(1, dtype=torch.int32, device="cuda"), desc)
    assert B.cm_get_status(desc) == B.CM_OK
    want = torch.zeros(S, S, dtype=torch.bool)
    for i in range(S):
        want[i, _visible(i + 1, window, sinks)] = True
    for table, mask in ((desc.interval_table_fwd(), want), (desc.interval_table_bwd(), want.T)):
        got = torch.zeros(S, S, dtype=torch.bool)
        for i in range(S):
            for s, e in table[0, :, i]:
                got[i, s:e] = True
        assert torch.equal(got, mask)
