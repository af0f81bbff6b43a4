"""What the C ABI and the binding refuse of pools of pages and of the appends that go with them, without a GPU (made-up
pointers: every case must return before anything is queued)."""
import pytest

from tests.test_kv_cache_cpu import A16, _cache, _new, _seqs


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
