"""Pool of pages on the GPU: reserve and release against plain loops (oracle/kv_pages.py), bit by bit."""
import random

import pytest
import torch

from oracle import kv_pages as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """A pool on the GPU beside the oracle's."""

    def __init__(self, B, num_pages, seqs, max_pages, P, window=0, sinks=0, seed=0):
        self.B, self.P, self.window, self.sinks, self.num_pages = B, P, window, sinks, num_pages
        self.free = list(range(num_pages))
        random.Random(seed).shuffle(self.free)
        self.table = [[-1] * max_pages for _ in range(seqs)]
        self.state = [[0, 0] for _ in range(seqs)] + [[num_pages, 0]]
        self.gpu = B.KVPages(_ints(self.table), _ints(self.free), P, window, sinks, _ints(self.state))

    def check(self, bad=False):
        assert self.gpu.page_table.tolist() == self.table
        assert self.gpu.state.tolist() == self.state
        left = self.state[-1][0]
        assert self.gpu.free_pages.tolist()[:left] == self.free[:left]
        assert self.B.cm_kv_pages_status(self.gpu) == (self.B.CM_ERR_DEVICE_CHECK if bad else self.B.CM_OK)

    def reserve(self, lens, counts, packed=False, room=None, gap=0, bad=False):
        n = len(lens)
        most = max(max(counts), 0)
        if packed:
            cu = [gap]
            for c in counts:
                cu.append(cu[-1] + c)
            total = max(cu) + 2
            bases, size = cu[:-1], total
            more = {"cu_new": _ints(cu), "max_new": most}
        else:
            total = room or most
            bases, size = None, n * total
            more = {"n_new": _ints(counts), "max_new": most}
        slots = [-7] * size
        got_slots = torch.full((size,), -7, dtype=torch.int64, device="cuda")
        got_slots = got_slots if packed else got_slots.view(n, total)
        granted = torch.full((n,), -7, dtype=torch.int32, device="cuda")
        self.B.cm_kv_reserve(self.gpu, self.gpu.state, self.gpu.spare, _ints(lens), total, granted=granted, slots=got_slots, **more)
        self.gpu.state, self.gpu.spare = self.gpu.spare, self.gpu.state
        want, self.state, was_bad = K.reserve(self.table, self.free, self.state, lens, bases, counts, slots, self.P,
                                              self.num_pages, most, total)
        assert was_bad == bad
        assert granted.tolist() == want and got_slots.flatten().tolist() == slots
        self.check(bad)
        return want

    def release(self, lens, done, bad=False):
        self.B.release_pages(self.gpu, _ints(lens), None if done is None else _ints(done))
        self.state, was_bad = K.release(self.table, self.free, self.state, lens, done or [0] * len(lens), self.window,
                                        self.sinks, self.P, self.num_pages)
        assert was_bad == bad
        self.check(bad)

    def whole(self):
        """Every page has one owner."""
        held = [x for row in K.owned(self.table, self.state[:-1], self.sinks, self.P) for x in row]
        assert sorted(held + self.free[:self.state[-1][0]]) == list(range(self.num_pages))


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("packed", [False, True])
def test_reserve(B, P, packed):
    x = Both(B, 60, 7, 30, P)
    lens = [0] * 7
    for counts in ([1, P, P - 1, 0, P + 1, 3 * P + 5, 2], [P - 1, 0, 1, 5, P - 1, 1, P], [4 * P + 1] * 7, [1] * 7):
        granted = x.reserve(lens, counts, packed, gap=3)
        lens = [a + b for a, b in zip(lens, granted)]
        x.whole()
    x.release(lens, [0, 1, 0, 0, 1, 0, 1])
    lens = [n * (b not in (1, 4, 6)) for b, n in enumerate(lens)]
    x.whole()
    x.reserve(lens, [P] * 7, packed)
    x.whole()


def test_too_few_pages(B):
    """Sequences are served in order; from the first that does not fit on, only those that need no page go on."""
    x = Both(B, 6, 5, 10, 16)
    assert x.reserve([0] * 5, [40, 16, 40, 16, 0]) == [40, 16, 0, 0, 0]
    assert x.reserve([40, 16, 0, 0, 0], [8, 1, 17, 16, 0]) == [8, 1, 0, 0, 0]
    assert x.reserve([48, 17, 0, 0, 0], [17, 15, 0, 16, 0]) == [0, 15, 0, 0, 0]
    x.release([48, 32, 0, 0, 0], [1, 0, 0, 0, 0])
    assert x.reserve([0, 32, 0, 0, 0], [17, 0, 33, 1, 0]) == [17, 0, 0, 0, 0]
    x.whole()


@pytest.mark.parametrize("seqs", [1, 31, 512, 513, 3000, 32767])
def test_many_sequences(B, seqs):
    r = random.Random(seqs)
    P = 16
    x = Both(B, 3 * seqs, seqs, 8, P, window=20, sinks=3)
    lens = [0] * seqs
    for step in range(3):
        counts = [r.randint(0, 25) for _ in range(seqs)]
        granted = x.reserve(lens, counts, packed=step == 1)
        lens = [a + b for a, b in zip(lens, granted)]
        done = [int(r.random() < 0.1) for _ in range(seqs)]
        x.release(lens, done if step else None)
        if step:
            lens = [n * (1 - d) for n, d in zip(lens, done)]
        x.whole()


def test_long_rows(B):
    """More new tokens and pages of a sequence than one warp's share."""
    x = Both(B, 30000, 3, 20000, 16)
    assert x.reserve([0, 0, 0], [1, 300001, 5000], packed=True) == [1, 300001, 5000]
    assert x.reserve([1, 300001, 5000], [2049, 1, 1023]) == [2049, 1, 1023]
    x.release([2050, 300002, 6023], [0, 1, 1])
    x.whole()


@pytest.mark.parametrize("P,window,sinks", [(16, 20, 0), (16, 16, 1), (32, 1, 33), (64, 200, 4), (16, 100, 500)])
def test_a_loop_under_a_window(B, P, window, sinks):
    """Steps of one and several tokens: pages behind the window come back, those of sinks stay."""
    r = random.Random(window)
    x = Both(B, 60, 4, 64, P, window, sinks)
    lens = [0] * 4
    for step in range(60):
        counts = [r.choice([0, 1, 1, 1, P // 2, 2 * P]) for _ in lens]
        counts = [min(c, 64 * P - n) for c, n in zip(counts, lens)]
        granted = x.reserve(lens, counts, packed=step % 2 == 1)
        lens = [a + b for a, b in zip(lens, granted)]
        done = [int(r.random() < 0.03) for _ in lens]
        x.release(lens, done)
        lens = [0 if d else n for n, d in zip(lens, done)]
        x.whole()
        for (lo, hi), n in zip(x.state, lens):  # what the next token sees is owned
            first = K.first_pages(sinks, P)
            for pos in range(n):
                if pos < sinks or pos > n - window:
                    assert pos // P < hi and (pos // P < first or pos // P >= lo)


def test_what_is_out_of_range(B):
    """A sequence out of range gets nothing and keeps its state; the others are whole."""
    x = Both(B, 40, 6, 8, 16)
    x.reserve([0] * 6, [16, 16, 16, 16, 16, 16])
    x.state[1] = [0, 9]    # more pages than its row
    x.state[2] = [2, 1]    # begins behind its end
    x.state[3] = [0, 0]    # holds tokens without pages
    x.gpu.state.copy_(_ints(x.state))
    x.reserve([16, 16, 16, 16, -1, 16], [20, 1, 1, 1, 1, 113], bad=True)  # negative length; beyond the row
    x.release([36, 16, 16, 16, 0, 16], [1, 1, 1, 1, 0, 0], bad=True)
    # token counts outside the tensors
    y = Both(B, 40, 4, 8, 16)
    for cu in ([0, 3, 3, 3, 3], [-1, 1, 2, 2, 2], [0, 1, 0, 1, 9]):
        bases, counts = cu[:-1], [b - a for a, b in zip(cu, cu[1:])]
        slots = torch.full((4,), -7, dtype=torch.int64, device="cuda")
        want = [-7] * 4
        granted = torch.empty(4, dtype=torch.int32, device="cuda")
        B.cm_kv_reserve(y.gpu, y.gpu.state, y.gpu.spare, _ints([0] * 4), 4, 2, cu_new=_ints(cu), granted=granted, slots=slots)
        y.gpu.state, y.gpu.spare = y.gpu.spare, y.gpu.state
        got, y.state, bad = K.reserve(y.table, y.free, y.state, [0] * 4, bases, counts, want, 16, 40, 2, 4)
        assert bad and granted.tolist() == got and slots.tolist() == want, cu
        y.check(bad=True)


def test_lengths_out_of_range_under_a_window(B):
    """A length that the pages do not cover gives nothing back, whatever a window would make of it; an ended one needs none."""
    x = Both(B, 40, 5, 16, 16, window=5, sinks=1)
    x.reserve([0] * 5, [100] * 5)
    x.release([100, -2**31, 113, 2**31 - 1, -1], [0, 0, 0, 1, 0], bad=True)
    assert x.state[:5] == [[5, 7], [0, 7], [0, 7], [0, 0], [0, 7]]
    x.whole()


def test_bounds_that_fall_past_32_bits(B):
    """cu_new falls by more than 2^31: nothing behind is granted."""
    x = Both(B, 40, 3, 8, 16)
    cu = [0, 5, -2**31, 3]
    slots = torch.full((5,), -7, dtype=torch.int64, device="cuda")
    granted = torch.empty(3, dtype=torch.int32, device="cuda")
    B.cm_kv_reserve(x.gpu, x.gpu.state, x.gpu.spare, _ints([0] * 3), 5, cu_new=_ints(cu), granted=granted, slots=slots)
    assert granted.tolist() == [5, 0, 0] and B.cm_kv_pages_status(x.gpu) == B.CM_ERR_DEVICE_CHECK
    assert slots.tolist() == [x.free[39] * 16 + i for i in range(5)]
    assert x.gpu.spare.tolist() == [[0, 1], [0, 0], [0, 0], [39, 0]]


def test_numbers_that_name_no_page(B):
    x = Both(B, 8, 2, 8, 16)
    x.free[6], x.free[3] = 99, -4
    x.gpu.free_pages.copy_(_ints(x.free))
    x.reserve([0, 0], [40, 0], bad=True)   # the second page is none
    x.reserve([40, 0], [0, 16])
    x.reserve([40, 16], [0, 16], bad=True)
    x.table[1][0] = 8
    x.gpu.page_table.copy_(_ints(x.table))
    x.release([40, 32], [0, 1], bad=True)  # goes into the list as it is


def test_lists_that_are_too_long(B):
    x = Both(B, 4, 2, 8, 16)
    x.reserve([0, 0], [64, 0])
    x.state[2] = [3, 0]
    x.gpu.state.copy_(_ints(x.state))
    x.release([64, 0], [1, 0], bad=True)   # three of the four have no room
    x.state[2] = [9, 0]
    x.gpu.state.copy_(_ints(x.state))
    x.reserve([0, 0], [16, 0], bad=True)
    x.state[2] = [-1, 0]
    x.gpu.state.copy_(_ints(x.state))
    x.reserve([16, 0], [1, 1], bad=True)


def test_nothing_to_do(B):
    x = Both(B, 4, 2, 8, 16)
    x.reserve([0, 0], [0, 0], packed=True)
    x.reserve([0, 0], [0, 0], room=3)
    x.release([0, 0], None)
    B.cm_kv_reserve(x.gpu, x.gpu.state, x.gpu.spare, _ints([0, 0]), 0)  # no tokens at all
    assert x.gpu.spare.tolist() == x.state and B.cm_kv_pages_status(x.gpu) == B.CM_OK
    B.cm_kv_reserve(x.gpu, x.gpu.state, x.gpu.spare, _ints([0, 0]), 3)  # all of three, no outputs
    assert x.gpu.spare.tolist() == [[0, 1], [0, 1], [2, 0]] and B.cm_kv_pages_status(x.gpu) == B.CM_OK


def test_a_captured_step(B):
    """Reserve and release in one graph: every replay goes on where the one before ended, with lengths from the device."""
    x = Both(B, 40, 3, 16, 16, window=24, sinks=2)
    lens, counts, done = _ints([0, 0, 0]), _ints([0, 0, 0]), _ints([0, 0, 0])
    side = torch.cuda.Stream()
    granted = torch.empty_like(lens)
    after = torch.empty_like(lens)

    def step():
        B.cm_kv_reserve(x.gpu, x.gpu.state, x.gpu.spare, lens, 40, n_new=counts, granted=granted)
        torch.add(lens, granted, out=after)
        B.cm_kv_release(x.gpu, x.gpu.spare, x.gpu.state, after, done)
        lens.copy_(after * (1 - done))

    with torch.cuda.stream(side):
        step()  # no tokens: nothing changes
    torch.cuda.synchronize()
    x.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    host = [0, 0, 0]
    for now, over in (([5, 40, 1], [0, 0, 0]), ([1, 40, 30], [0, 0, 1]), ([17, 1, 16], [0, 1, 0]), ([0, 40, 40], [0, 0, 0])):
        counts.copy_(torch.tensor(now))
        done.copy_(torch.tensor(over))
        g.replay()
        torch.cuda.synchronize()
        got, x.state, bad = K.reserve(x.table, x.free, x.state, host, None, now, [0] * 120, 16, 40, 40, 40)
        assert not bad
        host = [a + b for a, b in zip(host, got)]
        x.state, bad = K.release(x.table, x.free, x.state, host, over, 24, 2, 16, 40)
        assert not bad
        host = [0 if d else n for n, d in zip(host, over)]
        assert lens.tolist() == host
        x.check()
        x.whole()


def test_on_another_stream(B):
    x = Both(B, 40, 3, 16, 16)
    side = torch.cuda.Stream()
    lens = _ints([0, 0, 0])
    side.wait_stream(torch.cuda.current_stream())
    granted, slots = B.reserve_pages(x.gpu, lens, 20, slots=True, stream=side)
    B.release_pages(x.gpu, lens, _ints([0, 1, 0]), stream=side.cuda_stream)
    side.synchronize()
    assert granted.tolist() == [20] * 3 and x.gpu.state.tolist() == [[0, 2], [0, 0], [0, 2], [36, 0]]
    want = [-1] * 60
    K.reserve(x.table, x.free, x.state, [0] * 3, None, [20] * 3, want, 16, 40, 20, 20)
    assert slots.flatten().tolist() == want


def test_refusals_of_the_binding(B):
    x = Both(B, 40, 3, 16, 16)
    lens = _ints([0, 0, 0])
    s, n = x.gpu.state, x.gpu.spare
    for call in (lambda: B.cm_kv_reserve(x.gpu, s[:3], n, lens, 1), lambda: B.cm_kv_reserve(x.gpu, s, n.long(), lens, 1),
                 lambda: B.cm_kv_reserve(x.gpu, s, n, lens[:2], 1), lambda: B.cm_kv_reserve(x.gpu, s, n, lens.cpu(), 1),
                 lambda: B.cm_kv_reserve(x.gpu, s, n, lens, 1, slots=torch.zeros(3, 2, dtype=torch.int64, device="cuda")),
                 lambda: B.cm_kv_reserve(x.gpu, s, n, lens, 1, slots=torch.zeros(3, 1, dtype=torch.int32, device="cuda")),
                 lambda: B.cm_kv_reserve(x.gpu, s, n, lens, 1 << 32), lambda: B.cm_kv_reserve(x.gpu, s, n, lens, 4, cu_new=lens),
                 lambda: B.cm_kv_release(x.gpu, s, n, lens, done=lens[:2]),
                 lambda: B.KVPages(x.gpu.page_table[:, ::2], x.gpu.free_pages, 16),
                 lambda: B.KVPages(x.gpu.page_table, x.gpu.free_pages.long(), 16),
                 lambda: B.KVPages(x.gpu.page_table, x.gpu.free_pages, 16, window=-1),
                 lambda: B.reserve_pages(B.KVPages(x.gpu.page_table, x.gpu.free_pages, 16), lens, 1)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: B.cm_kv_reserve(x.gpu, s, s, lens, 1), lambda: B.cm_kv_reserve(x.gpu, s, n, lens, 1, 2),
                 lambda: B.cm_kv_reserve(x.gpu, s, n, lens, 1, granted=lens),
                 lambda: B.cm_kv_release(B.KVPages(x.gpu.page_table, x.gpu.free_pages, 24), s, n, lens)):
        with pytest.raises(B.CMError):
            call()
    pool = B.KVPages.alloc(5, 2, 4, 32)
    assert pool.state.tolist() == [[0, 0], [0, 0], [5, 0]] and pool.free_pages.tolist() == [0, 1, 2, 3, 4]
