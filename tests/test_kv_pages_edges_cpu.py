"""What the C ABI and the binding refuse of pools of pages and of the appends that go with them, without a GPU (made-up
pointers: every case must return before anything is queued)."""
import pytest

from tests.test_kv_cache_cpu import A16, _cache, _new, _seqs
from tests.test_kv_pages_cpu import _pages


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import build as bld
    bld.build()
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


def test_what_was_granted_is_for_packed_tokens(B):
    for bad in ({"granted": A16}, {"granted": A16, "n_new": 2 * A16}, {"granted": A16 + 2, "cu_new": 2 * A16},
                {"granted": 3 * A16, "cu_new": 2 * A16, "new_lens": 3 * A16}):
        assert B.lib().cm_kv_append(_cache(B), _seqs(B), _new(B, **bad), None) == B.CM_ERR_INVALID_ARG, bad


def test_results_that_lie_in_what_is_read(B):
    """Three sequences: 12 bytes of a number each, 16 of packed bounds, 32 of state."""
    L, state, new, lens, cu, n_new, granted = B.lib(), *(i * A16 for i in range(2, 8))

    def reserve(**k):  # more tokens than a call takes: refused as unsupported where nothing else is wrong
        a = dict(state=state, new=new, lens=lens, cu=None, n=n_new, granted=granted)
        a.update(k)
        n = 2**31 - 1 if a["cu"] else 1 << 30
        return L.cm_kv_reserve(_pages(B), a["state"], a["new"], a["lens"], a["cu"], a["n"], n, n, a["granted"], None, None)

    packed = {"cu": cu, "n": None}
    for good in ({}, packed, {"new": state + 32}, {"new": state - 32}, {"granted": lens + 12}, {"granted": n_new - 12},
                 {**packed, "granted": cu + 16}, {"granted": state + 32}, {"granted": None}):
        assert reserve(**good) == B.CM_ERR_UNSUPPORTED, good
    for bad in ({"new": state + 8}, {"new": state - 24}, {"new": lens - 24}, {"new": lens + 8}, {"new": n_new},
                {**packed, "new": cu - 24}, {"granted": lens + 8}, {"granted": lens - 8}, {"granted": n_new + 4},
                {**packed, "granted": cu}, {**packed, "granted": cu + 12}, {"granted": state + 28}, {"granted": new - 8},
                {"granted": new + 28}):
        assert reserve(**bad) == B.CM_ERR_INVALID_ARG, bad
    for a, b, done in ((state, state - 24, None), (state, lens - 24, None), (state, n_new + 8, n_new), (state, n_new - 24, n_new)):
        assert L.cm_kv_release(_pages(B), a, b, lens, done, None) == B.CM_ERR_INVALID_ARG, (a, b, done)


def test_new_lengths_that_lie_in_what_an_append_reads(B):
    """Two sequences: lens at A16 + 4 (8 bytes)."""
    def append(**k):  # more tokens than a call takes: refused as unsupported where nothing else is wrong
        n = 2**31 - 1 if "cu_new" in k else 1 << 30
        return B.lib().cm_kv_append(_cache(B), _seqs(B), _new(B, n_tokens=n, max_new=n, **k), None)

    far = 8 * A16
    for good in ({}, {"new_lens": A16 + 12}, {"new_lens": A16 - 4}, {"new_lens": far, "n_new": far + 8},
                 {"new_lens": far, "cu_new": far - 12}, {"new_lens": far, "cu_new": far + 8, "granted": far - 8}):
        assert append(**good) == B.CM_ERR_UNSUPPORTED, good
    for bad in ({"new_lens": A16 + 4}, {"new_lens": A16 + 8}, {"new_lens": A16}, {"new_lens": far, "n_new": far},
                {"new_lens": far, "n_new": far + 4}, {"new_lens": far, "cu_new": far}, {"new_lens": far, "cu_new": far - 8},
                {"new_lens": far, "cu_new": 9 * A16, "granted": far + 4}):
        assert append(**bad) == B.CM_ERR_INVALID_ARG, bad
