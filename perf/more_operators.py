"""Further serving operators of the library over its paged key-value cache: what is measured, and their plain forms.

A loop that generates without end keeps a few first tokens and a window of the last ones, in 8 bits, in pages that
come out of a pool on the GPU and go back to it:

  append   new tokens go into a cache held in 8 bits with one scale for each block of 16 tokens and head
  decode   attention of one new token per sequence over such a cache
  window   the same under a sliding window with a few first tokens that stay visible
  reserve  pages for the tokens to come, out of the pool's free list: page tables and the slot of every token
  release  pages of sequences that end, and pages that lie behind the window, back into the free list

The cache is ``k, v [pages, kv_heads, page, d]`` of int8 or e4m3 codes with ``k_scale, v_scale
[pages, kv_heads, page / 16]``: value = code * scale.  Scales are powers of two.  With a the largest |x| of a call's
new tokens in a block, 2^e is the smallest power of two with a <= top * 2^e, e within -32..32 (top = 127 for int8, 448
for e4m3).  A block without earlier tokens takes it; one that holds some takes the larger of it and its own, and where that
is a new one its earlier codes become round(code * old / new).  Codes are round(x / scale), halves to even, held to +-top.
So the codes are the same in any order and precision of the sums.

A page's summary is made of the keys that the page then stands for: per head and channel the largest (rounded up) and
the smallest (rounded down) in units of the smallest 2^e with max(|largest|, |smallest|) <= 127 * 2^e, e within -50..50.

Under a window w with s sinks the token at position p sees the positions j < s and p - w < j <= p.

The pool: ``free`` holds the numbers of the free pages, its first ``state[seqs, 0]`` entries; ``state[b] = (lo, hi)`` says that
sequence b owns the entries [0, f) and [max(lo, f), hi) of its table's row below hi, f = ceil(sinks / page).  Reserve takes pages
from the end of the list, sequence after sequence, in the order of the table; from the first sequence on that the
list has too few for, only those that need none go on (``granted`` says how many tokens may be appended).  Release puts pages back
behind the list's end in the same order.

Every length of a case follows from the case; the values follow from the seed.
"""
import math
import random

import torch

own = False

BLOCK = 16


# ---- cases -------------------------------------------------------------------------------------

def listed():
    base = {"d": 128, "heads": 32, "kv_heads": 8, "page": 64, "kv": "int8", "pick": 1}
    pool = {"page": 64, "packed": True, "spare": 1.5, "pick": 1}
    return [
        # a full serving batch's step, summaries kept for page selection
        {**base, "name": "append_256seqs_e4m3", "op": "append", "seqs": 256, "held": 200, "new": 1, "page": 32, "kv": "e4m3", "rot": 128, "interleaved": False, "summary": True},
        # prompts of different lengths, packed, written behind what the cache holds; a partial rotation
        {**base, "name": "append_prompts_int8", "op": "append", "seqs": 9, "held": 700, "new": 16384, "page": 128, "rot": 64, "interleaved": True, "summary": False},
        # a short chat with one user, every query head with its own key-value head
        {**base, "name": "decode_1seq_517_int8", "op": "decode", "seqs": 1, "longest": 517, "spread": "same", "d": 64, "heads": 16, "kv_heads": 16, "page": 16},
        # one long document: the work of one sequence spread over the whole GPU
        {**base, "name": "decode_1seq_131071_e4m3", "op": "decode", "seqs": 1, "longest": 131071, "spread": "same", "kv": "e4m3"},
        # an ordinary serving batch: lengths anywhere up to 16384
        {**base, "name": "decode_64seqs_16384_int8", "op": "decode", "seqs": 64, "longest": 16384, "spread": "even"},
        # 16 query heads to a key-value head
        {**base, "name": "decode_40seqs_int8", "op": "decode", "seqs": 40, "longest": 32768, "spread": "even", "kv_heads": 2, "page": 32},
        # one user far into a document, of which the model sees the last 4096 tokens and the first 4
        {**base, "name": "window_1seq_100003_bf16", "op": "window", "seqs": 1, "longest": 100003, "spread": "same", "kv": "bf16", "window": 4096, "sinks": 4},
        # a full batch under a short window, some sequences still inside it
        {**base, "name": "window_256seqs_int8", "op": "window", "seqs": 256, "longest": 8192, "spread": "log", "page": 32, "window": 1024, "sinks": 16},
        # a full batch's step: one token each, a page now and then
        {**pool, "name": "reserve_256seqs_step", "op": "reserve", "seqs": 256, "held": 4000, "new": 1, "packed": False},
        # new requests' prompts, packed, beside sequences that go on
        {**pool, "name": "reserve_prompts", "op": "reserve", "seqs": 500, "held": 300, "new": 8192, "page": 16},
        # a step in which a few sequences end and some have a page fall behind the window
        {**pool, "name": "release_256seqs_step", "op": "release", "seqs": 256, "longest": 8192, "ends": 0.02, "window": 1024, "sinks": 4, "behind": 1},
        # a whole batch of long requests is over
        {**pool, "name": "release_2000seqs_over", "op": "release", "seqs": 2000, "longest": 20000, "ends": 1.0, "window": 0, "sinks": 0, "behind": 0, "page": 16},
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    c = {"op": rng.choice(["append", "decode", "decode", "window", "window", "reserve", "release"]),
         "page": rng.choice([16, 32, 64, 128]), "pick": rng.randrange(1 << 20)}
    if c["op"] == "reserve":
        c.update(seqs=log(1, 4000), held=log(1, 20000), packed=rng.choice([False, True]), spare=rng.choice([1.5, 1.0, 0.6]))
        c["new"] = rng.choice([1, log(1, max(2, 2000000 // c["seqs"]))])
        return c
    if c["op"] == "release":
        c.update(seqs=log(1, 4000), longest=log(1, 20000), ends=rng.choice([0.0, 0.1, 1.0]), window=rng.choice([0, log(1, 4000)]),
                 sinks=rng.choice([0, 4, 100]), behind=rng.randint(0, 5), spare=1.5)
        return c
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 16])
    c.update(d=rng.choice([64, 128]), kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), kv=rng.choice(["int8", "int8", "e4m3"]))
    if c["op"] == "append":
        c.update(new=rng.choice([1, log(1, 9000)]), held=log(1, 1000), rot=rng.choice([0, 32, 64, c["d"]]),
                 interleaved=rng.choice([False, True]), summary=rng.choice([False, True]))
        c["seqs"] = log(1, 300) if c["new"] == 1 else log(1, max(2, min(40, 40000 // c["new"])))
        return c
    c.update(longest=log(1, 100000), spread=rng.choice(["same", "log", "even"]))
    token = 2 * c["kv_heads"] * c["d"]
    c["seqs"] = log(1, max(2, min(256, int(0.5e9) // (token * c["longest"]))))
    if c["op"] == "window":
        c.update(kv=rng.choice(["bf16", "int8", "e4m3"]), window=log(1, 8000), sinks=rng.choice([0, 1, 4, log(1, 300)]))
    return c


def _lengths(case):
    """Tokens of each sequence: before the call (append, reserve) or with the new token (the others)."""
    r, top = random.Random(case["pick"]), case["held"] if "held" in case else case["longest"]
    if "held" in case:
        return [r.randint(0, top) for _ in range(case["seqs"])]
    if case.get("spread", "even") == "same":
        return [top] * case["seqs"]
    if case.get("spread", "even") == "even":
        return [top] + [r.randint(1, top) for _ in range(case["seqs"] - 1)]
    return [top] + [int(round(math.exp(r.uniform(0, math.log(top))))) for _ in range(case["seqs"] - 1)]


def _new(case):
    r = random.Random(case["pick"] + 1)
    return [case["new"]] + [int(round(math.exp(r.uniform(0, math.log(case["new"]))))) for _ in range(case["seqs"] - 1)]


def _owned(case):
    """Before a release: (lo, hi) of each sequence, and which sequences end."""
    r, page, first = random.Random(case["pick"] + 2), case["page"], -(-case["sinks"] // case["page"])
    out = []
    for n in _lengths(case):
        hi, lo = -(-n // page), 0
        if case["window"]:  # `behind` pages more than the last release left
            lo = max(0, (n - case["window"]) // page - r.randint(0, case["behind"]))
            lo = lo if lo > first else 0
        out.append((lo, hi, r.random() < case["ends"]))
    return out


def _given_back(case):
    """Places of the table's rows that a release gives back, and the new (lo, hi)."""
    page, first = case["page"], -(-case["sinks"] // case["page"])
    places, after = [], []
    for n, (lo, hi, over) in zip(_lengths(case), _owned(case)):
        at = max(lo, first)
        if over:
            places.append(list(range(min(first, hi))) + list(range(at, hi)))
            after.append((0, 0))
            continue
        to = min(hi, max(0, n - case["window"]) // page) if case["window"] else 0
        places.append(list(range(at, to)))
        after.append((to, hi) if to > at else (lo, hi))
    return places, after


# ---- inputs ------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = _prepare_pool(case, gen) if case["op"] in ("reserve", "release") else _prepare_cache(case, gen)
    s["case"] = dict(case)
    if own:
        _handles(case, s)
    return s


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(need, wide, gen, spare, empty):
    """A table [seqs, wide] whose rows hold need[b] pages in random order, and the numbers of the free pages."""
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    count = torch.tensor(need, device="cuda")
    first = torch.cumsum(count, 0) - count
    at = torch.arange(wide, device="cuda")[None, :]
    table = torch.where(at < count[:, None], order[(first[:, None] + at).clamp(max=pages - 1)], empty)
    return table.to(torch.int32).contiguous(), order[sum(need):]


def _prepare_pool(case, gen):
    lens, page, seqs = _lengths(case), case["page"], case["seqs"]
    s = {"lens": _ints(lens)}
    if case["op"] == "reserve":
        new = _new(case)
        own_pages = [(0, -(-n // page)) for n in lens]
        more = sum(-(-(a + b) // page) - hi for a, b, (_, hi) in zip(lens, new, own_pages))
        wide = max(-(-(a + b) // page) for a, b in zip(lens, new))
        s["table"], free = _table([hi for _, hi in own_pages], max(wide, 1), gen, max(1, int(case["spare"] * more)), -1)
        s["n_new"] = _ints(new)
        s["cu"] = _ints([0] + new).cumsum(0).to(torch.int32) if case["packed"] else None
        s["tokens"], s["most"] = (sum(new) if case["packed"] else max(new)), max(new)
        s["granted"] = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        s["slots"] = torch.full((sum(new),) if case["packed"] else (seqs, max(new)), -2, dtype=torch.int64, device="cuda")
        s["wide_window"], s["sinks"] = 0, 0
    else:
        owned = _owned(case)
        own_pages = [(lo, hi) for lo, hi, _ in owned]
        s["done"] = _ints([int(x) for _, _, x in owned])
        s["table"], free = _table([hi for _, hi in own_pages], max(1, max(hi for _, hi in own_pages)), gen, 64, -1)
        s["wide_window"], s["sinks"] = case["window"], case["sinks"]
    pages = sum(hi for _, hi in own_pages) + len(free)
    s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    s["free"][:len(free)] = free
    s["state"] = _ints([list(x) for x in own_pages] + [[len(free), 0]])
    s["state_out"] = torch.zeros_like(s["state"])
    return s


def _prepare_cache(case, gen):
    dev, d, page, hk, hq, seqs = "cuda", case["d"], case["page"], case["kv_heads"], case["heads"], case["seqs"]
    lens, s = _lengths(case), {}
    new = _new(case) if case["op"] == "append" else [0] * seqs
    need = [(a + b + page - 1) // page for a, b in zip(lens, new)]
    s["table"], _ = _table(need, max(need), gen, 3, 0)
    pages = sum(need) + 3
    s["lens"] = _ints(lens)
    # keys: some channels are larger than others, as after a projection; values: plain
    spread = 0.7 * torch.exp(0.5 * torch.randn(hk, 1, d, generator=gen, device=dev))
    s["k"], s["k_scale"] = _random_pool(case, pages, spread, gen)
    s["v"], s["v_scale"] = _random_pool(case, pages, 1.0, gen)
    if case.get("summary"):
        s["summary"] = torch.zeros(pages, hk, 2, d, dtype=torch.int8, device=dev)
        s["summary_scale"] = torch.zeros(pages, hk, device=dev)
    if case["op"] == "append":
        total = sum(new)
        wide_row = (hq + 2 * hk) * d  # one projection gives all three
        qkv = torch.randn(total, wide_row, generator=gen, device=dev)
        qkv = (qkv * torch.exp(0.3 * torch.randn(total, 1, generator=gen, device=dev))).to(torch.bfloat16)
        q, k, v = qkv.split([hq * d, hk * d, hk * d], 1)
        s["q"], s["knew"], s["vnew"] = q.unflatten(1, (hq, d)), k.unflatten(1, (hk, d)), v.unflatten(1, (hk, d))
        s["cu"] = _ints([0] + new).cumsum(0).to(torch.int32)
        s["most"] = max(new)
        if case["rot"]:
            half = case["rot"] // 2
            freq = torch.tensor([10000.0 ** (-i / half) for i in range(half)], dtype=torch.float64, device=dev)
            angle = torch.arange(max(need) * page, dtype=torch.float64, device=dev)[:, None] * freq
            s["rope"] = torch.stack([angle.cos(), angle.sin()], 2).float().contiguous()
        s["q_out"] = torch.empty(total, hq, d, dtype=torch.bfloat16, device=dev)
        s["lens_out"] = torch.empty_like(s["lens"])
    else:
        s["q"] = torch.randn(seqs, hq, d, generator=gen, device=dev).to(torch.bfloat16)
        s["o"] = torch.empty(seqs, hq, d, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(seqs, hq, device=dev)
    return s


def _random_pool(case, pages, times, gen):
    """Codes [pages, kv_heads, page, d] of normal values, and their blocks' scales; bf16 values without."""
    hk, page, d, kind = case["kv_heads"], case["page"], case["d"], case["kv"]
    dtype = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[kind]
    out = torch.empty(pages, hk, page, d, dtype=dtype, device="cuda")
    scale = None if kind == "bf16" else torch.empty(pages, hk, page // BLOCK, device="cuda")
    step = max(1, (1 << 27) // (hk * page * d))
    for i in range(0, pages, step):
        x = torch.randn(out[i:i + step].shape, generator=gen, device="cuda", dtype=torch.float32) * times
        if kind == "bf16":
            out[i:i + step] = x.to(dtype)
            continue
        x = x.unflatten(2, (page // BLOCK, BLOCK))
        e = _exponent(x.abs().amax((3, 4)), kind)
        scale[i:i + step] = _power(e)
        out.view(torch.uint8)[i:i + step] = _codes(x / _power(e)[..., None, None], kind).flatten(2, 3).view(torch.uint8)
    return out, scale


def _handles(case, s):
    """The handles and the workspace that a program keeps from call to call."""
    from masked_flashattention_gb300 import binding as cm
    if case["op"] in ("reserve", "release"):
        s["pages"] = cm.KVPages(s["table"], s["free"], case["page"], window=s["wide_window"], sinks=s["sinks"])
        return
    s["cache"] = cm.KVCache(s["k"], s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                            summary=s.get("summary"), summary_scale=s.get("summary_scale"))
    if case["op"] != "append":
        size = cm.cm_attn_decode_workspace_size(case["seqs"], case["heads"], case["kv_heads"], case["d"])
        s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda")


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from masked_flashattention_gb300 import binding as cm
        if op == "append":
            cm.cm_kv_append(s["cache"], s["table"], s["lens"], s["knew"], s["vnew"], q=s["q"], q_out=s["q_out"], rope=s.get("rope"),
                            interleaved=case["interleaved"], cu_new=s["cu"], max_new=s["most"], new_lens=s["lens_out"])
        elif op == "decode":
            cm.cm_attn_decode(s["cache"], s["table"], s["lens"], s["q"], s["o"], s["lse"], s["work"])
        elif op == "window":
            cm.cm_attn_decode(s["cache"], s["table"], s["lens"], s["q"], s["o"], s["lse"], s["work"], window=case["window"], sinks=case["sinks"])
        elif op == "reserve":
            which = {"cu_new": s["cu"]} if case["packed"] else {"n_new": s["n_new"]}
            cm.cm_kv_reserve(s["pages"], s["state"], s["state_out"], s["lens"], s["tokens"], max_new=s["most"],
                             granted=s["granted"], slots=s["slots"], **which)
        else:
            cm.cm_kv_release(s["pages"], s["state"], s["state_out"], s["lens"], done=s["done"])
    else:
        {"append": _append, "decode": _decode, "window": _window, "reserve": _reserve, "release": _release}[op](s)
    if op == "append":
        out = {"q": s["q_out"], "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "lens": s["lens_out"]}
        if case["summary"]:
            out.update(summary=s["summary"], summary_scale=s["summary_scale"])
        return out
    if op == "reserve":
        return {"table": s["table"], "state": s["state_out"], "granted": s["granted"], "slots": s["slots"]}
    if op == "release":
        return {"free": s["free"], "state": s["state_out"]}
    return {"o": s["o"], "lse": s["lse"]}


def _exponent(a, kind):
    """e of the smallest 2^e with a <= top * 2^e: 127 = 127/128 * 2^7, 448 = 7/8 * 2^9."""
    m, e = torch.frexp(a)
    e = e - 7 + (m > 127 / 128).to(e.dtype) if kind == "int8" else e - 9 + (m > 7 / 8).to(e.dtype)
    return torch.where(a > 0, e, -32).clamp(-32, 32)


def _power(e):
    """2^e in fp32, by its bits: a power function may be a step off."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(x, kind):
    """fp32 values in units of the scale as the cache holds them."""
    return x.round().clamp(-127, 127).to(torch.int8) if kind == "int8" else x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _take(pool, *at):
    """pool[at], by its bytes where it holds 8 bits."""
    return pool.view(torch.uint8)[at].view(pool.dtype) if pool.element_size() == 1 else pool[at]


def _rotated(x, rope, rot, interleaved):
    """x [tokens, heads, d], rope [tokens, rot / 2, 2] (cos, sin): pairs (2i, 2i + 1) or (i, i + rot / 2)."""
    x, cos, sin = x.float(), rope[:, None, :, 0], rope[:, None, :, 1]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _append(s):
    case, page = s["case"], s["case"]["page"]
    lens, cu = s["lens"].long(), s["cu"].long()
    n = s["knew"].shape[0]
    token = torch.arange(n, device="cuda")
    seq = torch.searchsorted(cu, token, right=True) - 1
    pos = lens[seq] + token - cu[seq]
    q, k = s["q"].float(), s["knew"].float()
    if case["rot"]:
        rope = s["rope"][pos]
        q, k = (_rotated(x, rope, case["rot"], case["interleaved"]) for x in (q, k))
    k = k.to(torch.bfloat16).float()  # the rotated key is a bf16 tensor, whatever the cache holds
    s["q_out"].copy_(q.to(torch.bfloat16))
    s["lens_out"].copy_(s["lens"] + s["cu"][1:] - s["cu"][:-1])
    # the blocks that the call touches: [n] of them, their page, place in it and sequence
    end = s["lens_out"].long()
    block = lens[:, None] // BLOCK + torch.arange((s["most"] + BLOCK - 2) // BLOCK + 1, device="cuda")[None, :]
    seq, col = ((block * BLOCK < end[:, None]) & (end > lens)[:, None]).nonzero(as_tuple=True)
    first = block[seq, col] * BLOCK
    to, place = s["table"].long()[seq, first // page], first % page // BLOCK
    pos = first[:, None] + torch.arange(BLOCK, device="cuda")  # [n, 16]
    fresh = (pos >= lens[seq][:, None]) & (pos < end[seq][:, None])
    src = torch.where(fresh, cu[seq][:, None] + pos - lens[seq][:, None], 0)
    for name, x in (("k", k), ("v", s["vnew"].float())):
        _put_blocks(s, name, x, to, place, src, fresh, first < lens[seq], pos < end[seq][:, None])
    if case["summary"]:
        local = lens[:, None] // page + torch.arange((s["most"] + page - 2) // page + 1, device="cuda")[None, :]
        seq, col = ((local * page < end[:, None]) & (end > lens)[:, None]).nonzero(as_tuple=True)
        at = local[seq, col]
        _summarise(s, s["table"].long()[seq, at], (end[seq] - at * page).clamp(max=page))


def _put_blocks(s, name, x, to, place, src, fresh, carried, inside):
    """x [tokens, heads, d] into the blocks (to, place): rows `fresh` take x[src], the others keep what they hold."""
    kind, pool, scales = s["case"]["kv"], s[name], s[name + "_scale"]
    row = place[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    new = x[src]  # [n, 16, heads, d]
    held = _take(pool, to[:, None], slice(None), row).float()
    here = fresh[:, :, None, None]
    need = _power(_exponent(torch.where(here, new.abs(), 0.0).amax((1, 3)), kind))  # [n, heads]
    old = scales[to, :, place]
    scale = torch.where(carried[:, None], torch.maximum(old, need), need)
    held = held * (old / scale)[:, None, :, None]
    codes = _codes(torch.where(here, new / scale[:, None, :, None], held), kind).view(torch.uint8)
    b, r = inside.nonzero(as_tuple=True)
    pool.view(torch.uint8)[to[b], :, row[b, r]] = codes[b, r]
    scales[to, :, place] = scale


def _values(codes, scale):
    """codes [n, heads, page, d], scale [n, heads, page / 16] -> fp32 values."""
    return codes.float() if scale is None else codes.float() * scale.repeat_interleave(BLOCK, -1)[..., None]


def _summarise(s, pages, held):
    """Summaries of the pages from their first `held` tokens."""
    k = _values(_take(s["k"], pages), s["k_scale"][pages])
    here = (torch.arange(k.shape[2], device="cuda")[None, :] < held[:, None])[:, None, :, None]
    high, low = torch.where(here, k, -math.inf).amax(2), torch.where(here, k, math.inf).amin(2)
    a = torch.maximum(high.abs(), low.abs()).amax(2)
    m, e = torch.frexp(a)
    scale = _power(torch.where(a > 0, e - 7 + (m > 127 / 128).to(e.dtype), -50).clamp(-50, 50))[..., None]
    s["summary"][pages] = torch.stack([(high / scale).ceil(), (low / scale).floor()], 2).clamp(-127, 127).to(torch.int8)
    s["summary_scale"][pages] = scale[..., 0]


def _attend(q, k, v, seen, s):
    """q [b, hk, g, d]; k, v [b, hk, n, d]; seen [b, n] -> o and lse."""
    x = torch.matmul(q.float(), k.transpose(-1, -2)) * (1 / math.sqrt(q.shape[-1]))
    x = torch.where(seen[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    s["o"].copy_(o.reshape(s["o"].shape).to(torch.bfloat16))
    s["lse"].copy_((top + torch.log(total)).reshape(s["lse"].shape))


def _decode(s):
    b, hk, d = s["q"].shape[0], s["case"]["kv_heads"], s["case"]["d"]
    table = s["table"].long()
    k, v = (_values(_take(s[x], table).flatten(0, 1), s[x + "_scale"][table].flatten(0, 1)).unflatten(0, table.shape)
            .permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d) for x in "kv")
    seen = torch.arange(k.shape[2], device="cuda")[None, :] < s["lens"].long()[:, None]
    _attend(s["q"].reshape(b, hk, -1, d), k, v, seen, s)


def _window(s):
    """Only the positions that some sequence may see are gathered: the sinks, then the window."""
    case, b, hk, d, page = s["case"], s["q"].shape[0], s["case"]["kv_heads"], s["case"]["d"], s["case"]["page"]
    n = s["lens"].long()[:, None]
    sinks, window = min(case["sinks"], case["longest"]), min(case["window"], case["longest"])
    early = torch.arange(sinks, device="cuda")[None, :].expand(b, -1)
    late = n - window + torch.arange(window, device="cuda")[None, :]
    pos = torch.cat([early, late], 1)
    seen = torch.cat([(early < n), late >= sinks], 1)
    pos = torch.where(seen, pos, 0)
    at, row = s["table"].long().gather(1, pos // page), pos % page
    out = []
    for x in "kv":
        y = _take(s[x], at, slice(None), row).float()  # [b, n, hk, d]
        if case["kv"] != "bf16":
            y = y * s[x + "_scale"][at, :, row // BLOCK][..., None]
        out.append(y.transpose(1, 2))
    _attend(s["q"].reshape(b, hk, -1, d), *out, seen, s)


def _reserve(s):
    case, page, seqs = s["case"], s["case"]["page"], s["lens"].shape[0]
    lens, hi, left = s["lens"].long(), s["state"][:seqs, 1].long(), s["state"][seqs, 0].long()
    new = (s["cu"][1:] - s["cu"][:-1] if case["packed"] else s["n_new"]).long()
    need = (lens + new + page - 1) // page
    take = (need - hi).clamp(min=0)
    behind = torch.cumsum(take, 0)
    good = (take == 0) | (behind <= left)
    taken = torch.where(good, take, 0)
    place = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    mine = (place >= hi[:, None]) & (place < (hi + taken)[:, None])
    at = left - 1 - ((behind - take)[:, None] + place - hi[:, None])
    s["table"].copy_(torch.where(mine, s["free"][torch.where(mine, at, 0)], s["table"]))
    s["granted"].copy_(torch.where(good, new, 0))
    s["state_out"][:seqs, 0] = s["state"][:seqs, 0]
    s["state_out"][:seqs, 1] = (hi + taken).to(torch.int32)
    s["state_out"][seqs, 0] = (left - taken.sum()).to(torch.int32)
    if case["packed"]:
        cu = s["cu"].long()
        token = torch.arange(s["slots"].shape[0], device="cuda")
        seq = torch.searchsorted(cu, token, right=True) - 1
        pos = lens[seq] + token - cu[seq]
        page_of = s["table"][seq, torch.where(good[seq], pos // page, 0)].long()
        s["slots"].copy_(torch.where(good[seq], page_of * page + pos % page, -1))
    else:
        i = torch.arange(s["slots"].shape[1], device="cuda")[None, :]
        pos = lens[:, None] + i
        ok = good[:, None] & (i < new[:, None])
        page_of = s["table"].gather(1, torch.where(ok, pos // page, 0)).long()
        slot = torch.where(good[:, None], page_of * page + pos % page, -1)
        s["slots"].copy_(torch.where(i < new[:, None], slot, s["slots"]))


def _release(s):
    case, page, seqs = s["case"], s["case"]["page"], s["lens"].shape[0]
    first = -(-case["sinks"] // page)
    lo, hi, left = s["state"][:seqs, 0].long(), s["state"][:seqs, 1].long(), s["state"][seqs, 0].long()
    over = s["done"] != 0
    at = lo.clamp(min=first)
    to = torch.minimum(hi, (s["lens"].long() - case["window"]).clamp(min=0) // page) if case["window"] else torch.zeros_like(hi)
    place = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    ends = ((place < first) | (place >= at[:, None])) & (place < hi[:, None])
    back = torch.where(over[:, None], ends, (place >= at[:, None]) & (place < to[:, None]))
    pages = s["table"][back]  # sequence after sequence, in the table's order
    s["free"][left + torch.arange(pages.shape[0], device="cuda")] = pages
    s["state_out"][:seqs, 0] = torch.where(over, 0, torch.where(to > at, to, lo)).to(torch.int32)
    s["state_out"][:seqs, 1] = torch.where(over, 0, hi).to(torch.int32)
    s["state_out"][seqs, 0] = (left + pages.shape[0]).to(torch.int32)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    page, seqs, lens = case["page"], case["seqs"], _lengths(case)
    if case["op"] == "reserve":
        new = _new(case)
        touched = sum(-(-(a + b) // page) - a // page for a, b in zip(lens, new))  # pages that slots lie in
        fresh = sum(-(-(a + b) // page) + -a // page for a, b in zip(lens, new))
        # lengths, counts, (lo, hi) in and out, granted; the pages' numbers read and written; the slots
        return {"bytes": seqs * (4 + 4 + 8 + 8 + 4) + 4 * touched + 4 * fresh + 8 * sum(new), "flops": 2 * sum(new) + seqs}
    if case["op"] == "release":
        back = sum(map(len, _given_back(case)[0]))
        return {"bytes": seqs * (4 + 4 + 8 + 8) + 8 * back, "flops": back + seqs}
    d, hk, hq = case["d"], case["kv_heads"], case["heads"]
    item = 2 if case["kv"] == "bf16" else 1
    if case["op"] == "append":
        new = _new(case)
        n = sum(new)
        size = n * d * (2 * (2 * hq + 2 * hk) + 2 * hk * item) + 4 * case["rot"] * n + 12 * seqs
        blocks = sum((a + b + BLOCK - 1) // BLOCK - a // BLOCK for a, b in zip(lens, new))
        size += 2 * hk * 4 * (blocks + sum(a % BLOCK > 0 for a in lens))
        flops = 3 * n * case["rot"] * (hq + hk) + 4 * n * d * hk
        if case["summary"]:  # the earlier tokens of the pages that are carried on, and the summaries
            size += sum(a % page for a in lens) * hk * d * item
            size += sum((a + b + page - 1) // page - a // page for a, b in zip(lens, new)) * hk * (2 * d + 4)
            flops += 2 * n * hk * d
        return {"bytes": size, "flops": flops}
    if case["op"] == "window":
        lens = [min(n, case["sinks"] + case["window"]) for n in lens]
    size = seqs * hq * (4 * d + 4) + 4 * seqs + sum(lens) * hk * d * 2 * item + 4 * sum((n + page - 1) // page for n in lens)
    if item == 1:
        size += 2 * hk * 4 * sum((n + BLOCK - 1) // BLOCK for n in lens)
    return {"bytes": size, "flops": 4 * sum(lens) * hq * d}


# ---- from the definitions, in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "reserve":
        return _exact_reserve(case, s)
    if case["op"] == "release":
        return _exact_release(case, s)
    return _exact_attention(case, s)


def _exact_append(case, s):
    """Rotated queries.  Values are not rotated: their codes follow from the definition, sequence by sequence, block by
    block.  Keys' codes depend on the rounding of the rotated key, so they have no 64-bit value."""
    lens, new, page, rot = _lengths(case), _new(case), case["page"], case["rot"]
    q_out = s["q"].double().clone()
    v_codes, v_scale = s["v"].float().double(), s["v_scale"].double()
    top = 127.0 if case["kv"] == "int8" else 448.0
    i = 0
    for b, (held, count) in enumerate(zip(lens, new)):
        t, pos = slice(i, i + count), torch.arange(held, held + count, device="cuda")
        if rot:
            angle = s["rope"].double()[pos]
            turn = torch.complex(angle[..., 0], angle[..., 1])[:, None]
            part = q_out[t, :, :rot]
            pair = part.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
            turned = torch.view_as_real(torch.complex(pair[..., 0], pair[..., 1]) * turn)
            q_out[t, :, :rot] = (turned if case["interleaved"] else turned.transpose(-1, -2)).flatten(-2)
        v_new, row = s["vnew"][t].double(), s["table"][b].tolist()
        for start in range(held // BLOCK * BLOCK, held + count, BLOCK):
            at, place = row[start // page], start % page // BLOCK
            lo, hi = max(start, held), min(start + BLOCK, held + count)
            x = v_new[lo - held:hi - held].transpose(0, 1)  # [heads, rows, d]
            a = x.abs().amax((1, 2))
            e = torch.ceil(torch.log2(a / top) - 1e-9).clamp(-32, 32)
            need = torch.pow(torch.tensor(2.0, dtype=torch.float64), e.cpu()).to(a.device)
            rows = slice(place * BLOCK + lo - start, place * BLOCK + hi - start)
            if lo > start:
                was = v_scale[at, :, place].clone()
                need = torch.maximum(was, need)
                before = slice(place * BLOCK, place * BLOCK + lo - start)
                v_codes[at, :, before] = _exact_codes(v_codes[at, :, before] * (was / need)[:, None, None], top)
            v_codes[at, :, rows] = _exact_codes(x / need[:, None, None], top)
            v_scale[at, :, place] = need
        i += count
    out = {"q": q_out, "k": None, "v": v_codes, "k_scale": None, "v_scale": v_scale, "lens": None}
    if case["summary"]:
        out.update(summary=None, summary_scale=None)
    return out


def _exact_codes(x, top):
    return torch.round(x).clamp(-127, 127) if top == 127 else x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()


def _exact_attention(case, s):
    lens, page, hk = _lengths(case), case["page"], case["kv_heads"]
    group = case["heads"] // hk
    o, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        if case["op"] == "window":
            pos = pos[(pos < case["sinks"]) | (pos > n - 1 - case["window"])]
        at, row = s["table"][b].long()[pos // page], pos % page
        for h in range(hk):
            k, v = (_take(s[x], at, h, row).double() for x in "kv")
            if case["kv"] != "bf16":
                k, v = (y * s[x][at, h, row // BLOCK].double()[:, None] for y, x in ((k, "k_scale"), (v, "v_scale")))
            heads = slice(h * group, (h + 1) * group)
            x = s["q"][b, heads].double() @ k.T / math.sqrt(case["d"])
            lse[b, heads] = torch.logsumexp(x, 1)
            o[b, heads] = torch.softmax(x, 1) @ v
    return {"o": o, "lse": lse}


def _exact_reserve(case, s):
    """Sequence after sequence, as a program on the host would deal the pages out."""
    lens, new, page, seqs = _lengths(case), _new(case), case["page"], case["seqs"]
    table, state, free = (s[x].cpu().clone() for x in ("table", "state", "free"))
    slots, granted = s["slots"].cpu().clone(), torch.zeros(seqs, dtype=torch.int32)
    left, short, i = int(state[seqs, 0]), False, 0
    for b, (held, count) in enumerate(zip(lens, new)):
        hi, need = int(state[b, 1]), -(-(held + count) // page)
        short = short or (need > hi and need - hi > left)
        good = need <= hi or not short
        if good and need > hi:
            table[b, hi:need] = free[left - (need - hi):left].flip(0)
            left -= need - hi
            state[b, 1] = need
        granted[b] = count if good else 0
        pos = torch.arange(held, held + count)
        mine = table[b, pos // page].long() * page + pos % page if good else torch.full((count,), -1)
        if case["packed"]:
            slots[i:i + count] = mine
        else:
            slots[b, :count] = mine
        i += count
    state[seqs] = torch.tensor([left, 0])
    return {"table": table.cuda(), "state": state.cuda(), "granted": granted.cuda(), "slots": slots.cuda()}


def _exact_release(case, s):
    places, after = _given_back(case)
    free, table = s["free"].cpu().tolist(), s["table"].cpu()
    left = int(s["state"][case["seqs"], 0])
    for b, at in enumerate(places):
        free[left:left + len(at)] = table[b, at].tolist()
        left += len(at)
    return {"free": _ints(free), "state": _ints([list(x) for x in after] + [[left, 0]])}
