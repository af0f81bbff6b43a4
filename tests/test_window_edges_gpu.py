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
