"""Plain form of the pool of pages (test infrastructure; shares no code with the library): a list of free
pages and, for every sequence, its row of the page table, as loops over the definitions in include/cm.h.
Everything is Python lists on the host."""
from __future__ import annotations


def first_pages(sinks, P):
    return -(-sinks // P)


def good_state(lo, hi, held, P, max_pages):
    return 0 <= lo <= hi <= max_pages and lo * P <= held <= hi * P


def reserve(table, free, state, lens, bases, counts, slots, P, num_pages, max_new, n_tokens):
    """Changes table (rows) and slots (one list; token i of sequence b at bases[b] + i) in place; returns granted, new
    state and whether anything was out of range.  bases: None for padded tokens, [B][n_tokens]."""
    B, max_pages = len(lens), len(table[0])
    left = min(max(state[B][0], 0), num_pages)
    bad = left != state[B][0]
    granted, after, short = [0] * B, [list(x) for x in state], False
    for b in range(B):
        (lo, hi), held, n = state[b], lens[b], counts[b]
        base = b * n_tokens if bases is None else bases[b]
        ok = (held >= 0 and 0 <= n <= max_new and good_state(lo, hi, held, P, max_pages)
              and held + n <= max_pages * P)
        if bases is None:
            ok = ok and n <= n_tokens
        else:  # nothing behind a sequence at which the packed tokens' bounds fall
            ok = ok and base >= 0 and base + n <= n_tokens and min(counts[:b + 1]) >= 0
        if not ok:
            bad = True
            continue
        need = max(-(-(held + n) // P), hi) if n else hi
        if need > hi and (short or need - hi > left):
            short = True
            for i in range(n):
                slots[base + i] = -1
            continue
        for i in range(hi, need):
            left -= 1
            ok = 0 <= free[left] < num_pages
            bad = bad or not ok
            table[b][i] = free[left] if ok else -1
        after[b] = [lo, need]
        granted[b] = n
        for i in range(n):
            page = table[b][(held + i) // P]
            ok = 0 <= page < num_pages
            bad = bad or not ok
            slots[base + i] = page * P + (held + i) % P if ok else -1
    after[B] = [left, 0]
    return granted, after, bad


def release(table, free, state, lens, done, window, sinks, P, num_pages):
    """Changes free in place; returns the new state and whether anything was out of range."""
    B, first = len(lens), first_pages(sinks, P)
    left = min(max(state[B][0], 0), num_pages)
    bad = left != state[B][0]
    after = [list(x) for x in state]
    for b in range(B):
        lo, hi = state[b]
        if not 0 <= lo <= hi <= len(table[b]):
            bad = True
            continue
        if window and not done[b] and not 0 <= lens[b] <= hi * P:
            bad = True
            continue
        at = max(lo, first)
        if done[b]:
            places = list(range(min(first, hi))) + list(range(at, hi))
            after[b] = [0, 0]
        else:
            to = min(hi, max(0, lens[b] - window) // P) if window else 0
            places = list(range(at, to))
            if to > at:
                after[b] = [to, hi]
        for i in places:
            bad = bad or not 0 <= table[b][i] < num_pages
            if left < num_pages:
                free[left] = table[b][i]
                left += 1
            else:
                bad = True
    after[B] = [left, 0]
    return after, bad


def owned(table, state, sinks, P):
    """The pages that each sequence owns."""
    first = first_pages(sinks, P)
    return [[row[i] for i in range(hi) if i < first or i >= lo] for row, (lo, hi) in zip(table, state)]
