"""Windows where a call's numbers are at their ends."""
import math

import pytest
import torch

from tests.test_kv_cache_gpu import _check_decode, _filled
from tests.test_window_gpu import _visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


def test_numbers_beyond_32_bits_are_refused(B):
    """None is taken modulo 2^32: -(2^32) + 4 is no window of 4."""
    gen = torch.Generator().manual_seed(56)
    cache, table, n = _filled(B, [40], 1, 16, 64, "bf16", gen)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    for bad in ({"window": -2**32 + 4}, {"window": -2**31 - 1}, {"window": 2**31}, {"window": 4, "sinks": -2**32},
                {"window": 4, "sinks": -2**32 + 3}, {"window": 4, "sinks": 2**32}):
        with pytest.raises(ValueError):
            B.decode_attention(cache, table, n, q, **bad)
    t = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    for bad in (2**32 + 16, -2**32 + 16):
        with pytest.raises(ValueError):
            B.KVPages(t, t[0], bad)


@pytest.mark.parametrize("window,sinks", [(None, 0), (0, 0), (0, 5), (40, 0), (40, 5)])
def test_attention_takes_the_window_of_a_pool(B, window, sinks):
    """A loop hands its pool's window and sinks on, whether the pool has a window or none."""
    gen = torch.Generator().manual_seed(57)
    lens = [200, 1, 77]
    cache, table, n = _filled(B, lens, 1, 16, 64, "bf16", gen)
    pages = B.KVPages(table, torch.arange(8, dtype=torch.int32, device="cuda"), 16, window=window, sinks=sinks)
    q = torch.randn(3, 2, 64, generator=gen).to(torch.bfloat16).cuda()
    o, lse = B.decode_attention(cache, table, n, q, window=pages.window, sinks=pages.sinks)
    _check_decode(cache, table, n, q, o, lse, 1 / 8, lambda b, g: _visible(lens[b], window or 10**9, sinks))


def test_the_work_of_a_call_goes_by_its_window(B):
    """64 sequences of 8 heads with tables for 2^27 tokens each, 2^22 tiles, are more than a call takes; under a window it is
    what the window can cover that counts, to the tile: 512 rows * (tiles + 1 + 2) below 2^31 - 320."""
    gen = torch.Generator().manual_seed(58)
    lens = [0] * 64
    lens[0], lens[7], lens[63] = 300, 1, 129
    P, H, d = 128, 8, 64
    cache, narrow, n = _filled(B, lens, H, P, d, "bf16", gen)
    table = torch.full((64, (1 << 27) // P), -7, dtype=torch.int32, device="cuda")
    table[:, :narrow.shape[1]] = narrow
    q = torch.randn(64, H, d, generator=gen).to(torch.bfloat16).cuda()
    most = 32 * (2**22 - 4)
    for more in ({}, {"window": most + 1}, {"window": most - 32, "sinks": 33}, {"window": 2**31 - 1}):
        with pytest.raises(B.CMError) as e:
            B.decode_attention(cache, table, n, q, **more)
        assert e.value.code == B.CM_ERR_UNSUPPORTED
    for more in ({"window": most}, {"window": most - 32, "sinks": 32}, {"window": 100, "sinks": 3}):
        o, lse = B.decode_attention(cache, table, n, q, **more)
        assert B.cm_kv_status(cache) == B.CM_OK
        _check_decode(cache, table, n, q, o, lse, 1 / 8, lambda b, g: _visible(lens[b], more["window"], more.get("sinks", 0)))
