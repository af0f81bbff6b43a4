"""Sliding window with sinks without a GPU: what the C ABI refuses, and the MaskSpec of the same mask."""
import ctypes
import math

import pytest

from tests.test_kv_cache_cpu import A16, BAD_CACHE, BAD_SEQS, _cache, _seqs


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import build as bld
    bld.build()
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


def _call(B, cache=None, seqs=None, window=8, sinks=2, q=A16, qs=(512, 128), o=A16, os=(512, 128), lse=A16, H_q=4,
          scale=0.1, work=A16, size=1 << 40):
    return B.lib().cm_attn_decode_window(cache or _cache(B), seqs or _seqs(B), window, sinks, q,
                                         (ctypes.c_int64 * 2)(*qs) if qs else None, o,
                                         (ctypes.c_int64 * 2)(*os) if os else None, lse, H_q, scale, work, size, None)


def test_refusals(B):
    for bad, rc in BAD_CACHE:
        assert _call(B, cache=_cache(B, **bad)) == rc, bad
    for bad, rc in BAD_SEQS:
        assert _call(B, seqs=_seqs(B, **bad)) == rc, bad
    size = B.cm_attn_decode_workspace_size(2, 4, 2, 128)
    for bad in ({"window": 0}, {"window": -1}, {"sinks": -1}, {"q": None}, {"q": A16 + 8}, {"qs": None}, {"qs": (512, 4)},
                {"o": None}, {"os": None}, {"os": (512, 8)}, {"lse": 2}, {"H_q": 3}, {"scale": math.nan},
                {"work": None}, {"size": size - 1}):
        assert _call(B, **bad) == B.CM_ERR_INVALID_ARG, bad
    assert _call(B, H_q=1 << 15) == B.CM_ERR_UNSUPPORTED
    # the work of a call: what the window can cover, where that is less than the table
    big = dict(cache=_cache(B, page_size=128, H_kv=64, k_page_stride=1 << 20, v_page_stride=1 << 20),
               seqs=_seqs(B, B=32767, max_pages=8192), H_q=64)
    assert _call(B, **big, window=2**31 - 1, sinks=2**31 - 1) == B.CM_ERR_UNSUPPORTED
    assert _call(B, **big, window=40000, sinks=0) == B.CM_ERR_UNSUPPORTED


def test_binding_takes_one_mask(B):
    from masked_flashattention_gb300 import specs
    with pytest.raises(ValueError):
        specs.sliding_window(0)
    with pytest.raises(ValueError):
        specs.sliding_window(4, -1)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 4), (1000, 5)])
def test_mask_spec_compiles(B, window, sinks):
    from masked_flashattention_gb300 import specs
    f, b = specs.sliding_window(window, sinks)
    assert B.cm_spec_num_intervals(B.cm_compile_spec(f)) == (2 if sinks else 1)
    assert B.cm_spec_num_intervals(B.cm_compile_spec(b)) == 1
