"""Serving operators of the library over a paged key-value cache: what is measured, and their plain forms.

Three operators, as a serving loop uses them:

  append   the new tokens' keys and values go into the cache's pages, with the position rotation
           applied to the queries and keys on the way, and the summaries of the pages they touch
  decode   attention of one new token per sequence over its pages, all of them or the intervals
           that the sequence's mask leaves visible
  sparse   the summaries score every page against the query, the best pages of each sequence and
           key-value head are taken, and the new token attends to them alone

The cache is ``k, v [pages, kv_heads, page, d]`` (bf16, or e4m3 with one fp32 scale per head), a
page table ``[seqs, max_pages]`` of page numbers, and ``lens``.  A page's summary is, per head and
channel, the largest and the smallest key of its tokens in 8 bits with a scale that is a power of two:
with kmax, kmin over the tokens and a = max(|kmax|, |kmin|) over the channels, 2^e is the smallest
power of two with a <= 127 * 2^e (e within -50..50), and the summary is ceil(kmax / 2^e),
floor(kmin / 2^e).  Queries are rounded to 8 bits the same way, x = rint(q / 2^f).  The score of a page
is the largest, over the query heads that share the key-value head, of
2^(e + f) * sum_c (x_c > 0 ? x_c * smax_c : x_c * smin_c): whole numbers and powers of two, so it is the
same in any order and precision.  The best pages are the highest scores, the lowest page first among equals.

Every length of a case follows from the case; the values follow from the seed.
"""
import math
import random

import torch

own = False

_specs = {}  # compiled mask rules, kept as a program keeps them


# ---- cases -------------------------------------------------------------------------------------

def listed():
    base = {"d": 128, "heads": 32, "kv_heads": 8, "page": 64, "kv": "bf16", "pick": 1}
    return [
        # one user's next token: the latency of a call
        {**base, "name": "append_1seq", "op": "append", "seqs": 1, "held": 4000, "new": 1, "rot": 128, "interleaved": False, "summary": False},
        # a full serving batch's step, 8-bit cache with summaries
        {**base, "name": "append_256seqs_e4m3", "op": "append", "seqs": 256, "held": 200, "new": 1, "page": 32, "kv": "e4m3", "rot": 128, "interleaved": False, "summary": True},
        # prompts of different lengths, packed, written behind what the cache holds; a partial rotation
        {**base, "name": "append_prompts", "op": "append", "seqs": 9, "held": 700, "new": 16384, "page": 128, "rot": 64, "interleaved": True, "summary": True},
        # a short chat with one user, every query head with its own key-value head
        {**base, "name": "decode_1seq_517", "op": "decode", "seqs": 1, "longest": 517, "spread": "same", "mask": False, "d": 64, "heads": 16, "kv_heads": 16, "page": 16},
        # one long document: the work of one sequence spread over the whole GPU
        {**base, "name": "decode_1seq_131071", "op": "decode", "seqs": 1, "longest": 131071, "spread": "same", "mask": False},
        # many short conversations
        {**base, "name": "decode_200seqs_short", "op": "decode", "seqs": 200, "longest": 333, "spread": "log", "mask": False, "page": 16},
        # an ordinary serving batch: lengths anywhere up to 16384
        {**base, "name": "decode_64seqs_16384", "op": "decode", "seqs": 64, "longest": 16384, "spread": "even", "mask": False},
        # 16 query heads to a key-value head, 8-bit cache
        {**base, "name": "decode_40seqs_e4m3", "op": "decode", "seqs": 40, "longest": 32768, "spread": "even", "mask": False, "kv_heads": 2, "page": 32, "kv": "e4m3"},
        # the three-interval packing mask of the prompts, carried on into the generated tokens
        {**base, "name": "decode_8seqs_masked", "op": "decode", "seqs": 8, "longest": 32768, "spread": "even", "mask": True, "page": 128},
        # one long document, 64 of its 2048 pages
        {**base, "name": "sparse_1seq_131072", "op": "sparse", "seqs": 1, "longest": 131072, "spread": "same", "keep": 64, "first": 1, "last": 2},
        # a batch of long documents, 8-bit cache, small pages
        {**base, "name": "sparse_32seqs_e4m3", "op": "sparse", "seqs": 32, "longest": 32768, "spread": "even", "page": 32, "kv": "e4m3", "keep": 96, "first": 1, "last": 4},
        # lengths on both sides of what is kept
        {**base, "name": "sparse_5seqs_short", "op": "sparse", "seqs": 5, "longest": 1500, "spread": "log", "d": 64, "heads": 12, "kv_heads": 4, "page": 16, "keep": 32, "first": 0, "last": 1},
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 16])
    c = {"op": rng.choice(["append", "decode", "decode", "sparse"]), "d": rng.choice([64, 128]), "kv_heads": kv_heads,
         "heads": kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), "page": rng.choice([16, 32, 64, 128]),
         "kv": rng.choice(["bf16", "bf16", "e4m3"]), "pick": rng.randrange(1 << 20)}
    if c["op"] == "append":
        c.update(new=rng.choice([1, log(1, 9000)]), held=log(1, 1000), rot=rng.choice([32, 64, c["d"]]),
                 interleaved=rng.choice([False, True]), summary=rng.choice([False, True]))
        c["seqs"] = log(1, 300) if c["new"] == 1 else log(1, max(2, min(40, 40000 // c["new"])))
        return c
    c.update(longest=log(1, 100000), spread=rng.choice(["same", "log", "even"]))
    token = 2 * c["kv_heads"] * c["d"] * (1 if c["kv"] == "e4m3" else 2)
    c["seqs"] = log(1, max(2, min(256, int(1.0e9) // (token * c["longest"]))))
    if c["op"] == "decode":
        c["mask"] = c["longest"] >= 256 and c["seqs"] * c["longest"] <= 2000000 and rng.random() < 0.3
    else:
        c["last"] = rng.randint(0, 3)
        c["first"] = rng.randint(0, 2)
        c["keep"] = log(max(2, c["first"] + c["last"]), 128)
    return c


def _lengths(case):
    """Tokens of each sequence: before the call (append) or with the new token (decode, sparse)."""
    r, top = random.Random(case["pick"]), case["held"] if case["op"] == "append" else case["longest"]
    if case["op"] == "append":
        return [r.randint(0, top) for _ in range(case["seqs"])]
    if case["spread"] == "same":
        return [top] * case["seqs"]
    if case["spread"] == "even":
        return [top] + [r.randint(1, top) for _ in range(case["seqs"] - 1)]
    return [top] + [int(round(math.exp(r.uniform(0, math.log(top))))) for _ in range(case["seqs"] - 1)]


def _new(case):
    r = random.Random(case["pick"] + 1)
    return [case["new"]] + [int(round(math.exp(r.uniform(0, math.log(case["new"]))))) for _ in range(case["seqs"] - 1)]


def _documents(case):
    """Segments of the three-interval mask: a prefix, then documents up to the capacity of the mask's
    table; the new token is in the document that holds it."""
    r, size = random.Random(case["pick"] + 2), _mask_rows(case)
    rows = []
    for _ in range(case["seqs"]):
        cuts = [0, max(1, size // 64)]
        while cuts[-1] < size:
            cuts.append(min(size, cuts[-1] + r.randint(max(1, size // 32), max(2, 3 * size // 16))))
        rows.append(cuts)
    return rows


def _mask_rows(case):
    return (case["longest"] + 127) // 128 * 128


def _visible(cuts, n):
    """Visible keys of the row n - 1: the prefix, the first 64 tokens of the previous document, and its
    own document up to itself."""
    k = max(i for i in range(len(cuts) - 1) if cuts[i] <= n - 1)
    if k == 0:
        return [(0, n)]
    spans = [(0, cuts[1]), (cuts[k], n)]
    if k >= 2:
        spans.append((cuts[k - 1], min(cuts[k - 1] + 64, cuts[k])))
    return spans


# ---- inputs ------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev, d, page, hk, hq, seqs = "cuda", case["d"], case["page"], case["kv_heads"], case["heads"], case["seqs"]
    lens, s = _lengths(case), {"case": dict(case)}
    new = _new(case) if case["op"] == "append" else [0] * seqs
    need = [(a + b + page - 1) // page for a, b in zip(lens, new)]
    pages, wide = sum(need) + 3, max(need)
    order = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int64).to(torch.int32)
    count = torch.tensor(need, device=dev)
    first = torch.cumsum(count, 0) - count
    at = torch.arange(wide, device=dev)[None, :]
    s["table"] = torch.where(at < count[:, None], order[(first[:, None] + at).clamp(max=pages - 1)], 0).to(torch.int32).contiguous()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    # keys: some channels are larger than others, as after a projection; values: plain
    spread = torch.exp(0.5 * torch.randn(hk, 1, d, generator=gen, device=dev))

    def pool(times):
        out = torch.empty(pages, hk, page, d, dtype=torch.bfloat16 if case["kv"] == "bf16" else torch.float8_e4m3fn, device=dev)
        step = max(1, (1 << 27) // (hk * page * d))
        for i in range(0, pages, step):
            part = torch.randn(out[i:i + step].shape, generator=gen, device=dev, dtype=torch.float32) * times
            out[i:i + step] = part.clamp(-448, 448).to(out.dtype)
        return out

    if case["kv"] == "e4m3":
        s["k_scale"] = 0.01 + 0.03 * torch.rand(hk, generator=gen, device=dev)
        s["v_scale"] = 0.01 + 0.03 * torch.rand(hk, generator=gen, device=dev)
        s["k"], s["v"] = (pool(1 / x[:, None, None] * y).clone() for x, y in ((s["k_scale"], 0.7 * spread.clamp(max=3)), (s["v_scale"], 0.7)))
    else:
        s["k_scale"] = s["v_scale"] = None
        s["k"], s["v"] = pool(0.7 * spread), pool(1.0)
    if case.get("summary") or case["op"] == "sparse":
        s["summary"] = torch.zeros(pages, hk, 2, d, dtype=torch.int8, device=dev)
        s["summary_scale"] = torch.zeros(pages, hk, device=dev)
    if case["op"] == "append":
        total = sum(new)
        wide_row = (hq + 2 * hk) * d  # one projection gives all three
        qkv = torch.randn(total, wide_row, generator=gen, device=dev).to(torch.bfloat16)
        q, k, v = qkv.split([hq * d, hk * d, hk * d], 1)
        s["q"], s["knew"], s["vnew"] = q.unflatten(1, (hq, d)), k.unflatten(1, (hk, d)), v.unflatten(1, (hk, d))
        s["cu"] = torch.tensor([0] + new, dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
        s["most"] = max(new)
        if case["rot"]:
            half = case["rot"] // 2
            freq = torch.tensor([10000.0 ** (-i / half) for i in range(half)], dtype=torch.float64, device=dev)
            angle = torch.arange(wide * page, dtype=torch.float64, device=dev)[:, None] * freq
            s["rope"] = torch.stack([angle.cos(), angle.sin()], 2).float().contiguous()
        s["q_out"] = torch.empty(total, hq, d, dtype=torch.bfloat16, device=dev)
        s["lens_out"] = torch.empty_like(s["lens"])
    else:
        s["q"] = torch.randn(seqs, hq, d, generator=gen, device=dev).to(torch.bfloat16)
        s["o"] = torch.empty(seqs, hq, d, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(seqs, hq, device=dev)
    if case["op"] == "sparse":
        every = torch.arange(pages, device=dev)
        held = torch.full((pages,), page, device=dev)
        ends = torch.arange(seqs, device=dev)
        held[s["table"][ends, count - 1].long()] = s["lens"].long() - (count - 1) * page
        step = max(1, (1 << 26) // (hk * page * d))
        for i in range(0, pages, step):
            _summarise(s, every[i:i + step], held[i:i + step])
        s["sel"] = torch.empty(seqs, hk, case["keep"], dtype=torch.int32, device=dev)
        s["nsel"] = torch.empty(seqs, hk, dtype=torch.int32, device=dev)
    if case.get("mask"):
        rows = _documents(case)
        most = max(map(len, rows))
        s["seg"] = torch.tensor([r + [r[-1]] * (most - len(r)) for r in rows], dtype=torch.int32, device=dev)
        s["nseg"] = torch.tensor([len(r) - 1 for r in rows], dtype=torch.int32, device=dev)
    if own:
        _handles(case, s)
    return s


def _handles(case, s):
    """The cache's handle, the workspace and the mask's descriptor that a program keeps from call to call."""
    from masked_flashattention_gb300 import binding as cm
    from masked_flashattention_gb300 import specs
    s["cache"] = cm.KVCache(s["k"], s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                            summary=s.get("summary"), summary_scale=s.get("summary_scale"))
    s["desc"] = None
    if case["op"] != "append":
        size = cm.cm_attn_decode_workspace_size(case["seqs"], case["heads"], case["kv_heads"], case["d"])
        s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if case["op"] == "sparse":
        size = cm.cm_select_pages_workspace_size(case["seqs"], case["kv_heads"], s["table"].shape[1])
        s["select_work"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if case.get("mask"):
        if not _specs:
            _specs.update(f=cm.cm_compile_spec(specs.FWD[5]), b=cm.cm_compile_spec(specs.BWD[5]))
        s["desc"] = cm.Descriptor(_specs["f"], _specs["b"], case["seqs"], _mask_rows(case))
        cm.cm_build_descriptor(_specs["f"], _specs["b"], s["seg"], s["nseg"], s["desc"])


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        from masked_flashattention_gb300 import binding as cm
        if op == "append":
            cm.cm_kv_append(s["cache"], s["table"], s["lens"], s["knew"], s["vnew"], q=s["q"], q_out=s["q_out"], rope=s.get("rope"),
                            interleaved=s["case"]["interleaved"], cu_new=s["cu"], max_new=s["most"], new_lens=s["lens_out"])
        elif op == "decode":
            cm.cm_attn_decode(s["cache"], s["table"], s["lens"], s["q"], s["o"], s["lse"], s["work"], desc=s["desc"])
        else:
            cm.cm_select_pages(s["cache"], s["table"], s["lens"], s["q"], s["sel"], s["nsel"], s["select_work"],
                               keep_first=s["case"]["first"], keep_last=s["case"]["last"])
            cm.cm_attn_decode(s["cache"], s["table"], s["lens"], s["q"], s["o"], s["lse"], s["work"], sel=s["sel"], nsel=s["nsel"])
    else:
        {"append": _append, "decode": _decode, "sparse": _sparse}[op](s)
    if op == "append":
        out = {"q": s["q_out"], "k": s["k"], "v": s["v"], "lens": s["lens_out"]}
        if s["case"]["summary"]:
            out.update(summary=s["summary"], summary_scale=s["summary_scale"])
        return out
    out = {"o": s["o"], "lse": s["lse"]}
    if op == "sparse":
        out.update(sel=s["sel"], nsel=s["nsel"])
    return out


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


def _put(pool, to, row, x, scale):
    """fp32 values [tokens, heads, d] into the pool's rows, as it holds them."""
    if scale is None:
        pool[to, :, row] = x.to(pool.dtype)
    else:
        pool.view(torch.uint8)[to, :, row] = (x / scale[:, None]).clamp(-448, 448).to(pool.dtype).view(torch.uint8)


def _take(pool, *at):
    """pool[at], by its bytes where it holds 8 bits."""
    return pool.view(torch.uint8)[at].view(pool.dtype) if pool.element_size() == 1 else pool[at]


def _append(s):
    case, page = s["case"], s["case"]["page"]
    n = s["knew"].shape[0]
    token = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["cu"], token, right=True) - 1
    pos = s["lens"].long()[seq] + token - s["cu"].long()[seq]
    to = s["table"].long()[seq, pos // page]
    q, k = s["q"].float(), s["knew"].float()
    if case["rot"]:
        rope = s["rope"][pos]
        q, k = (_rotated(x, rope, case["rot"], case["interleaved"]) for x in (q, k))
    k = k.to(torch.bfloat16).float()  # the rotated key is a bf16 tensor, whatever the cache holds
    s["q_out"].copy_(q.to(torch.bfloat16))
    _put(s["k"], to, pos % page, k, s["k_scale"])
    _put(s["v"], to, pos % page, s["vnew"].float(), s["v_scale"])
    s["lens_out"].copy_(s["lens"] + s["cu"][1:] - s["cu"][:-1])
    if case["summary"]:
        end = s["lens_out"].long()[:, None]
        local = s["lens"].long()[:, None] // page + torch.arange((s["most"] + page - 2) // page + 1, device="cuda")[None, :]
        seq, col = (local * page < end).nonzero(as_tuple=True)
        at = local[seq, col]
        _summarise(s, s["table"].long()[seq, at], (end[seq, 0] - at * page).clamp(max=page))


def _exponent(a):
    """e of the smallest 2^e with a <= 127 * 2^e, within -50..50."""
    m, e = torch.frexp(a)
    return torch.where(a > 0, e - 7 + (m > 127 / 128).to(e.dtype), -50).clamp(-50, 50)


def _power(e):
    """2^e in fp32, by its bits: a power function may be a step off."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _summarise(s, pages, held):
    """Summaries of the pages from their first `held` tokens."""
    k = _take(s["k"], pages).float()
    if s["k_scale"] is not None:
        k = k * s["k_scale"][:, None, None]
    here = (torch.arange(k.shape[2], device="cuda")[None, :] < held[:, None])[:, None, :, None]
    high, low = torch.where(here, k, -math.inf).amax(2), torch.where(here, k, math.inf).amin(2)
    e = _exponent(torch.maximum(high.abs(), low.abs()).amax(2))
    scale = _power(e)[..., None]
    s["summary"][pages] = torch.stack([(high / scale).ceil(), (low / scale).floor()], 2).clamp(-127, 127).to(torch.int8)
    s["summary_scale"][pages] = scale[..., 0]


def _attend(q, k, v, seen, s):
    """q [b, hk, g, d]; k, v [b, hk, n, d]; seen, broadcast to [b, hk, n] -> o and lse."""
    d = q.shape[-1]
    x = torch.matmul(q.float(), k.transpose(-1, -2)) * (1 / math.sqrt(d))
    x = torch.where(seen[:, :, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    s["o"].copy_(o.reshape(s["o"].shape).to(torch.bfloat16))
    s["lse"].copy_((top + torch.log(total)).reshape(s["lse"].shape))


def _decode(s):
    case, b, hk, d = s["case"], s["q"].shape[0], s["case"]["kv_heads"], s["case"]["d"]
    table = s["table"].long()
    k, v = (_take(s[x], table).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d).float() for x in "kv")
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    pos, n = torch.arange(k.shape[2], device="cuda")[None, :], s["lens"].long()[:, None]
    seen = pos < n
    if case["mask"]:
        seg, last = s["seg"].long(), s["nseg"].long()[:, None] - 1
        at = torch.minimum(torch.searchsorted(seg, n - 1, right=True) - 1, last)
        start, end = seg.gather(1, at), seg.gather(1, at + 1)
        before = seg.gather(1, (at - 1).clamp(min=0))
        prefix = (pos < seg[:, 1:2]) | (at == 0)
        previous = (at >= 2) & (pos >= before) & (pos < torch.minimum(before + 64, start))
        seen = seen & (prefix | previous | ((pos >= start) & (pos < end)))
    _attend(s["q"].reshape(b, hk, -1, d), k, v, seen[:, None], s)


def _sparse(s):
    case, b, hk, d, page = s["case"], s["q"].shape[0], s["case"]["kv_heads"], s["case"]["d"], s["case"]["page"]
    table, n = s["table"].long(), s["lens"].long()
    q = s["q"].reshape(b, hk, -1, d).float()
    e = _exponent(q.abs().amax(-1))
    scale = _power(e)
    x = (q / scale[..., None]).round().clamp(-127, 127)
    x = torch.cat([x.clamp(min=0), x.clamp(max=0)], -1)  # [b, hk, g, 2d]
    summary = s["summary"][table].permute(0, 2, 1, 3, 4).flatten(3).float()  # [b, hk, pages, 2d]
    score = torch.matmul(x, summary.transpose(-1, -2)) * scale[..., None]
    score = (score * s["summary_scale"][table].permute(0, 2, 1)[:, :, None]).amax(2)
    many = ((n + page - 1) // page)[:, None, None]
    at = torch.arange(table.shape[1], device="cuda")
    score = torch.where((at < case["first"]) | (at >= many - case["last"]), math.inf, score)
    score = torch.where(at < many, score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :case["keep"]]
    rank = torch.arange(best.shape[-1], device="cuda")
    best = torch.sort(torch.where(rank < many, best, 1 << 30), dim=-1)[0]
    good = best < (1 << 30)
    s["sel"].fill_(-1)
    s["sel"][..., :best.shape[-1]] = torch.where(good, best, -1).to(torch.int32)
    s["nsel"].copy_(good.sum(-1))
    best = torch.where(good, best, 0)
    where = table[:, None].expand(-1, hk, -1).gather(2, best)
    head = torch.arange(hk, device="cuda")[None, :, None]
    k, v = (_take(s[y], where, head).flatten(2, 3).float() for y in "kv")  # [b, hk, keep * page, d]
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    pos = best[..., None] * page + torch.arange(page, device="cuda")
    seen = (good[..., None] & (pos < n[:, None, None, None])).flatten(2)
    _attend(q, k, v, seen, s)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    d, hk, hq, page, seqs = case["d"], case["kv_heads"], case["heads"], case["page"], case["seqs"]
    item = 1 if case["kv"] == "e4m3" else 2
    lens = _lengths(case)
    if case["op"] == "append":
        new = _new(case)
        n = sum(new)
        size = n * d * (2 * (2 * hq + 2 * hk) + 2 * hk * item) + 4 * case["rot"] * n + 12 * seqs
        flops = 3 * n * case["rot"] * (hq + hk)
        if case["summary"]:  # the earlier tokens of the pages that are carried on, and the summaries
            size += sum(a % page for a in lens) * hk * d * item
            size += sum((a + b + page - 1) // page - a // page for a, b in zip(lens, new)) * hk * (2 * d + 4)
            flops += 2 * n * hk * d
        return {"bytes": size, "flops": flops}
    size = seqs * hq * (4 * d + 4) + 4 * seqs
    if case["op"] == "decode":
        keys = sum(lens)
        if case["mask"]:
            keys = sum(len(set().union(*(range(a, min(b, n)) for a, b in _visible(c, n)))) for c, n in zip(_documents(case), lens))
        size += keys * hk * d * 2 * item + 4 * sum((n + page - 1) // page for n in lens)
        return {"bytes": size, "flops": 4 * keys * hq * d}
    pages = sum((n + page - 1) // page for n in lens)
    keys = sum(min(n, case["keep"] * page) for n in lens)
    size += pages * hk * (2 * d + 4) + 4 * pages + keys * hk * d * 2 * item + 4 * seqs * hk * (case["keep"] + 1)
    return {"bytes": size, "flops": 4 * pages * hq * d + 4 * keys * hq * d}


# ---- from the definitions, in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attention(case, s)


def _exact_append(case, s):
    lens, new, page, rot = _lengths(case), _new(case), case["page"], case["rot"]
    q_out = s["q"].double().clone()
    k_new, v_new = s["knew"].double().clone(), s["vnew"].double().clone()
    pools = {"k": s["k"].double().clone(), "v": s["v"].double().clone()}
    i = 0
    for b, (held, count) in enumerate(zip(lens, new)):
        t, pos = slice(i, i + count), torch.arange(held, held + count, device="cuda")
        if rot:
            half = rot // 2
            angle = s["rope"].double()[pos]
            turn = torch.complex(angle[..., 0], angle[..., 1])[:, None]
            for x in (q_out, k_new):
                part = x[t, :, :rot]
                pair = part.unflatten(-1, (half, 2)) if case["interleaved"] else part.unflatten(-1, (2, half)).transpose(-1, -2)
                turned = torch.view_as_real(torch.complex(pair[..., 0], pair[..., 1]) * turn)
                x[t, :, :rot] = (turned if case["interleaved"] else turned.transpose(-1, -2)).flatten(-2)
        where, row = s["table"].long()[b, pos // page], pos % page
        for name, x in (("k", k_new[t]), ("v", v_new[t])):
            if case["kv"] == "e4m3":
                x = x.bfloat16().double() if name == "k" else x
                x = (x / s[name + "_scale"].double()[:, None]).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
            pools[name][where, :, row] = x
        i += count
    return {"q": q_out, "k": pools["k"], "v": pools["v"], "lens": None, "summary": None, "summary_scale": None}


def _exact_attention(case, s):
    lens, page, hk, d = _lengths(case), case["page"], case["kv_heads"], case["d"]
    group = case["heads"] // hk
    o, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    spans = [_visible(c, n) for c, n in zip(_documents(case), lens)] if case.get("mask") else None
    for b, n in enumerate(lens):
        row = s["table"][b, :(n + page - 1) // page].long()
        pos = torch.arange(n, device="cuda")
        if spans:
            keep = sum(((pos >= x) & (pos < y)).int() for x, y in spans[b]) > 0
        elif case["op"] == "sparse":
            keep = _exact_pages(case, s, b, row).repeat_interleave(page, 1)[:, :n]
        for h in range(hk):
            at = pos[keep[h] if case["op"] == "sparse" else keep] if spans or case["op"] == "sparse" else pos
            k, v = (_take(s[x], row[at // page], h, at % page).double() for x in "kv")
            if case["kv"] == "e4m3":
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            heads = slice(h * group, (h + 1) * group)
            x = s["q"][b, heads].double() @ k.T / math.sqrt(d)
            lse[b, heads] = torch.logsumexp(x, 1)
            o[b, heads] = torch.softmax(x, 1) @ v
    return {"o": o, "lse": lse, "sel": None, "nsel": None}


def _exact_pages(case, s, b, row):
    """Truth values [kv_heads, pages]: which pages of the sequence are taken."""
    hk, many = case["kv_heads"], len(row)
    if many <= case["keep"]:
        return torch.ones(hk, many, dtype=torch.bool, device="cuda")
    q = s["q"][b].double().unflatten(0, (hk, -1))
    top = q.abs().amax(-1, keepdim=True)
    f = torch.ceil(torch.log2(top / 127) - 1e-9).clamp(-50, 50)  # bf16 tops lie far from the borders
    f = ((f.long() + 1023) << 52).view(torch.float64)  # 2^f
    x = torch.round(q / f).clamp(-127, 127)
    high, low = s["summary"][row].double().unbind(2)  # [pages, hk, d]
    score = torch.einsum("hgc,phc->hgp", x.clamp(min=0), high) + torch.einsum("hgc,phc->hgp", x.clamp(max=0), low)
    score = (score * f * s["summary_scale"][row].double().T[:, None]).amax(1)
    score[:, :case["first"]] = math.inf
    score[:, many - case["last"]:] = math.inf
    order = torch.argsort(-score, dim=1, stable=True)[:, :case["keep"]]
    return torch.zeros(hk, many, dtype=torch.bool, device="cuda").scatter_(1, order, True)
