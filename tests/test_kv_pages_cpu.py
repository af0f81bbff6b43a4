"""Pool of pages without a GPU: the oracle's pins, and what the C ABI refuses on the host."""
import pytest
import torch

from oracle import kv_pages as K

A16 = 0x1000


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import build as bld
    bld.build()
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


# ---- oracle ----------------------------------------------------------------------------------
def test_reserve_by_hand():
    """Three sequences, pages of 16, five free pages: 20 tokens behind 0 need two pages, 1 behind 15 fits the page
    it has, 60 behind 32 need four, of which three are left."""
    table = [[-1] * 8, [7] + [-1] * 7, [8, 9] + [-1] * 6]
    free, slots = [0, 1, 2, 3, 4, -1, -1, -1, -1, -1], [-2] * 81
    granted, state, bad = K.reserve(table, free, [[0, 0], [0, 1], [0, 2], [5, 0]], [0, 15, 32], [0, 20, 21], [20, 1, 60],
                                    slots, 16, 10, 60, 81)
    assert granted == [20, 1, 0] and state == [[0, 2], [0, 1], [0, 2], [3, 0]] and not bad
    assert table[0][:3] == [4, 3, -1] and table[2][2] == -1
    assert slots[:20] == [64 + i for i in range(16)] + [48 + i for i in range(4)]
    assert slots[20] == 7 * 16 + 15 and slots[21:] == [-1] * 60


def test_release_by_hand():
    """Pages of 16, a window of 20 behind one sink page: at 100 tokens the positions before 80 are out of sight."""
    table = [[5, 6, 7, 8, 9, 10, 11], [0, 1, 2, -1, -1, -1, -1]]
    free = [3, 4] + [-1] * 10
    state, bad = K.release(table, free, [[2, 7], [0, 3], [2, 0]], [100, 40], [0, 1], 20, 4, 16, 12)
    assert state == [[5, 7], [0, 0], [8, 0]] and free[:8] == [3, 4, 7, 8, 9, 0, 1, 2] and not bad
    assert K.owned(table, state, 4, 16) == [[5, 10, 11], []]


# ---- refusals (made-up pointers: every case must return before anything is queued) ---------------
def _pages(B, /, **k):
    g = B.cm_kv_pages(100, 16, 3, 8, 0, 0, A16, A16 + 4, A16 + 8)
    for n, v in k.items():
        setattr(g, n, v)
    return g


BAD_PAGES = [({"num_pages": 0}, -2), ({"B": 0}, -2), ({"max_pages": 0}, -2), ({"window": -1}, -2), ({"sinks": -1}, -2),
             ({"page_size": 8}, -3), ({"page_size": 0}, -3), ({"page_size": 256}, -3), ({"B": 32768}, -3),
             ({"max_pages": 1 << 24}, -3), ({"page_table": None}, -2), ({"page_table": A16 + 2}, -2),
             ({"free_pages": None}, -2), ({"status": None}, -2), ({"status": A16 + 1}, -2)]


def test_reserve_refusals(B):
    def call(pages=None, state=A16, new_state=2 * A16, lens=A16 + 4, cu=None, n_new=A16, n_tokens=5, max_new=5, granted=3 * A16,
             slots=4 * A16):
        return B.lib().cm_kv_reserve(pages if pages is not None else _pages(B), state, new_state, lens, cu, n_new, n_tokens,
                                     max_new, granted, slots, None)

    for bad, rc in BAD_PAGES:
        assert call(pages=_pages(B, **bad)) == rc, bad
    assert B.lib().cm_kv_reserve(None, A16, 2 * A16, A16, None, A16, 5, 5, None, None, None) == B.CM_ERR_INVALID_ARG
    for bad in ({"state": None}, {"state": A16 + 4}, {"new_state": None}, {"new_state": A16}, {"new_state": 2 * A16 + 4},
                {"lens": None}, {"lens": A16 + 2}, {"cu": A16}, {"cu": A16 + 2, "n_new": None}, {"n_new": A16 + 2},
                {"n_tokens": -1, "max_new": -1}, {"max_new": 6}, {"max_new": -1}, {"n_new": None, "max_new": 4},
                {"granted": 2}, {"slots": A16 + 4}, {"granted": A16 + 4}, {"granted": A16}):
        assert call(**bad) == B.CM_ERR_INVALID_ARG, bad
    for bad in ({"n_tokens": 1 << 30, "max_new": 1 << 30},
                {"cu": A16, "n_new": None, "n_tokens": 2**31 - 1}):
        assert call(**bad) == B.CM_ERR_UNSUPPORTED, bad


def test_release_refusals(B):
    def call(pages=None, state=A16, new_state=2 * A16, lens=A16, done=None):
        return B.lib().cm_kv_release(pages if pages is not None else _pages(B), state, new_state, lens, done, None)

    for bad, rc in BAD_PAGES:
        assert call(pages=_pages(B, **bad)) == rc, bad
    for bad in ({"state": None}, {"new_state": None}, {"new_state": A16}, {"lens": None}, {"lens": 2}, {"done": 2}):
        assert call(**bad) == B.CM_ERR_INVALID_ARG, bad
    assert B.lib().cm_kv_pages_status(None, None) == B.CM_ERR_INVALID_ARG
    assert B.lib().cm_kv_pages_status(_pages(B, status=2), None) == B.CM_ERR_INVALID_ARG


def test_binding_refuses_tensors_that_are_not_on_a_gpu(B):
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.KVPages(t, t[0], 16)
