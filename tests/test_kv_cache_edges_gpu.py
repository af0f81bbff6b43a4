"""Paged key-value cache on the GPU: values, calls and interleavings at the edge of what is allowed,
against the plain 64-bit forms (oracle/kv_cache.py)."""
import math

import pytest
import torch

from oracle import kv_cache as K
from tests.test_kv_cache_gpu import BF16_HALF, B, F64, _check_decode, _filled, _host  # noqa: F401 (B is a fixture)

pytestmark = pytest.mark.gpu


# ---- values ----------------------------------------------------------------------------------
@pytest.mark.parametrize("d,P,H,group,lens", [(64, 16, 2, 3, [1, 2, 33, 700]), (128, 64, 1, 12, [1, 64, 9000]),
                                              (128, 128, 1, 8, [40000])])
def test_infinite_values(B, d, P, H, group, lens):
    """A visible infinite value makes its channel infinite (both signs: NaN) and no other; scores are close
    enough that no weight is below fp32's smallest."""
    gen = torch.Generator().manual_seed(61)
    cache, table, n = _filled(B, lens, H, P, d, "bf16", gen)
    where = table.cpu()
    for b, m in enumerate(lens):
        def put(pos, channel, value):
            cache.v[int(where[b, pos // P]), :, pos % P, channel] = value
        put(0, 0, math.inf)
        put(m - 1, 1, -math.inf)
        put(m // 2, 2, math.inf)
        put(0, 3, math.inf)
        put(m - 1, 3, -math.inf)  # of one token, the same value
        for pos in range(0, m, 7):
            put(pos, d - 1, -math.inf)
    q = torch.randn(len(lens), H * group, d, generator=gen).to(torch.bfloat16).cuda()
    scale = 1 / math.sqrt(d)
    o, lse = B.decode_attention(cache, table, n, q)
    assert B.cm_kv_status(cache) == B.CM_OK
    k, v, _, _ = _host(cache)
    o, q = o.double().cpu(), q.cpu()
    for b, m in enumerate(lens):
        for g in range(H):
            hs, pos = slice(g * group, (g + 1) * group), torch.arange(m)
            kk, vv = K.rows(k, None, where[b], g, pos), K.rows(v, None, where[b], g, pos)
            up, down = (vv == math.inf).any(0), (vv == -math.inf).any(0)
            want, wl, size, mag = K.decode(q[b, hs], kk, torch.where(vv.isinf(), 0.0, vv), scale)
            got, finite = o[b, hs], ~(up | down)
            assert (got[:, up & ~down] == math.inf).all() and (got[:, down & ~up] == -math.inf).all(), (b, g)
            assert got[:, up & down].isnan().all(), (b, g)
            ds = (d + 8) * 2 * 2.0 ** -24 * size + 2.0 ** -20
            bound = BF16_HALF * want.abs() + (BF16_HALF + 2 * ds + 2.0 ** -14) * mag
            assert ((got - want).abs() <= bound)[:, finite].all(), (b, g)
            assert ((lse[b, hs].double().cpu() - wl).abs() <= ds + 2.0 ** -20 * (1 + wl.abs())).all(), (b, g)


@pytest.mark.parametrize("group", [1, 12])
def test_large_values(B, group):
    """Values of 2^118 whose scores come 2^7.9 above those before them: sums of weights of at most 1 stay within fp32
    (250 * 2^118 < 2^128), weights of 2^7.9 would not.  Weights are off by 2^-14 at most, o by one rounding more."""
    P, d = 32, 64
    lens = [256, 500]
    cache = B.KVCache.alloc(24, 1, P, d)  # a page is a tile of the kernel
    cache.k.zero_(), cache.v.zero_()
    cache.k[1::2, :, :, 0] = 1
    cache.v[1::2] = 2.0 ** 118
    table = torch.stack([torch.arange(0, 16), torch.arange(8, 24)]).to(torch.int32).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, group, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    o, lse = B.decode_attention(cache, table, n, q, scale=7.9 * math.log(2))
    assert B.cm_kv_status(cache) == B.CM_OK
    for b, m in enumerate(lens):
        high = sum(1 for i in range(m) if (i // P) % 2)
        weight = high * 2.0 ** 7.9
        total = weight + m - high
        assert ((o[b].double() * 2.0 ** -118 - weight / total).abs() <= (BF16_HALF + 2.0 ** -14) * weight / total).all(), b
        assert (lse[b].double() - math.log(total)).abs().max() <= 2.0 ** -20 * (1 + math.log(total)), b


def test_queries_of_any_size_beside_an_e4m3_cache(B):
    """Queries up to 2^120 (the keys' scale brings the scores back), and queries whose channels are 2^-20 of the
    head's largest while the keys are 0 in that one: scores as in the other tests."""
    gen = torch.Generator().manual_seed(63)
    lens, H, P, d = [50, 700], 2, 16, 64
    cache, table, n = _filled(B, lens, H, P, d, "e4m3", gen)
    v = cache.v
    k = (torch.randn(cache.num_pages, H, P, d, generator=gen) * 2.0 ** -4).to(v.dtype).cuda()
    tiny = torch.full((H,), 2.0 ** -106, device="cuda")
    big = B.KVCache(k, v, tiny, cache.v_scale)
    q = (torch.randn(2, H * 3, d, generator=gen) * 2.0 ** 118).to(torch.bfloat16).cuda()
    scale = 2.0 ** -10
    o, lse = B.decode_attention(big, table, n, q, scale=scale)
    assert o.isfinite().all() and B.cm_kv_status(big) == B.CM_OK
    _check_decode(big, table, lens, q, o, lse, scale, lambda b, g: torch.arange(lens[b]))
    k.view(torch.uint8)[..., 0] = 0
    one = torch.ones(H, device="cuda")
    small = B.KVCache(k, v, one, cache.v_scale)
    q = (torch.randn(2, H * 3, d, generator=gen) * 2.0 ** -20).to(torch.bfloat16).cuda()
    q[..., 0] = 1
    scale = 2.0 ** 21
    o, lse = B.decode_attention(small, table, n, q, scale=scale)
    _check_decode(small, table, lens, q, o, lse, scale, lambda b, g: torch.arange(lens[b]))


# ---- calls that overlap ------------------------------------------------------------------------
def test_selection_sees_the_summaries_of_the_append_before_it(B):
    """Appends and selections in turn, without a wait between them: each selection goes by what the append just
    before it wrote.  A step writes row 0 of one page anew, whose summary then is that token's."""
    gen = torch.Generator().manual_seed(64)
    Bn, H, P, d, per, n, steps = 40, 4, 16, 128, 8, 3, 80
    cache = B.KVCache.alloc(Bn * per, H, P, d, summaries=True)
    table = torch.randperm(Bn * per, generator=gen).to(torch.int32).view(Bn, per).cuda()
    full = torch.full((Bn,), per * P, dtype=torch.int32, device="cuda")
    zeros = torch.zeros(Bn, H, per * P, d, dtype=torch.bfloat16, device="cuda")
    B.cm_kv_append(cache, table, torch.zeros_like(full), zeros, zeros)
    place = torch.randint(0, per, (steps, Bn), generator=gen)
    power = torch.randint(-6, 7, (steps, Bn, H), generator=gen)  # scores are d times these powers of two
    tokens = torch.exp2(power.float()).to(torch.bfloat16).cuda()[..., None, None].expand(steps, Bn, H, 1, d).contiguous()
    lens = (place * P).to(torch.int32).cuda()
    q = torch.ones(Bn, H * 2, d, dtype=torch.bfloat16, device="cuda")
    work = torch.empty(B.cm_select_pages_workspace_size(Bn, H, per), dtype=torch.uint8, device="cuda")
    sel = torch.empty(steps, Bn, H, n, dtype=torch.int32, device="cuda")
    nsel = torch.empty(steps, Bn, H, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for t in range(steps):
        B.cm_kv_append(cache, table, lens[t], tokens[t], tokens[t])
        B.cm_select_pages(cache, table, full, q, sel[t], nsel[t], work)
    assert B.cm_kv_status(cache) == B.CM_OK
    assert (nsel == n).all()
    sel, value = sel.cpu(), torch.zeros(Bn, H, per, dtype=F64)
    for t in range(steps):
        value[torch.arange(Bn), :, place[t]] = torch.exp2(power[t].double())
        for b in range(Bn):
            for h in range(H):
                assert sel[t, b, h].tolist() == K.pick(value[b, h].tolist(), n, 0, 0), (t, b, h)


_FIRST_CALLS = """
import threading, torch
from masked_flashattention_gb300 import binding as B
P, d, n = 64, 128, 300
gen = torch.Generator().manual_seed(5)
sets = []
for _ in range(4):
    cache = B.KVCache.alloc(5, 2, P, d)
    cache.k.copy_(torch.randn(5, 2, P, d, generator=gen)), cache.v.copy_(torch.randn(5, 2, P, d, generator=gen))
    q = torch.randn(1, 8, d, generator=gen).to(torch.bfloat16).cuda()
    work = torch.empty(B.cm_attn_decode_workspace_size(1, 8, 2, d), dtype=torch.uint8, device="cuda")
    sets.append((cache, q, torch.zeros_like(q), work, torch.cuda.Stream()))
table = torch.arange(5, dtype=torch.int32, device="cuda")[None]
lens = torch.tensor([n], dtype=torch.int32, device="cuda")
B._serving()
torch.cuda.synchronize()
gate, errors = threading.Barrier(4), []
def first(cache, q, o, work, stream):
    try:
        torch.cuda.set_device(0)
        gate.wait()
        B.cm_attn_decode(cache, table, lens, q, o, None, work, stream=stream)
    except Exception as e:
        errors.append(repr(e))
threads = [threading.Thread(target=first, args=s) for s in sets]
[t.start() for t in threads], [t.join() for t in threads]
torch.cuda.synchronize()
assert not errors, errors
for cache, q, o, work, _ in sets:
    again = torch.zeros_like(o)
    B.cm_attn_decode(cache, table, lens, q, again, None, work)
    assert torch.equal(o, again) and o.any() and B.cm_kv_status(cache) == 0
print("first calls ok")
"""


def test_first_calls_of_several_threads():
    """The first calls of a process may come from several host threads at once."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", _FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and "first calls ok" in r.stdout, r.stderr


def test_handle_0_is_the_default_stream(B):
    """Memory for work on stream handle 0 is the default stream's, from whatever stream the call comes."""
    with torch.cuda.stream(torch.cuda.Stream()):
        def make():
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
            return (torch.empty(8, device="cuda"),)
        B._for_stream(0, make)
        B._for_stream(torch.cuda.default_stream(), make)


def test_results_for_handle_0_from_another_stream(B):
    """decode_attention and select_pages on stream handle 0, called where another stream is current and has
    memory of the same sizes that it still writes to."""
    gen = torch.Generator().manual_seed(66)
    lens, H, P, d, n = [3000, 10, 700], 2, 64, 128, 5
    cache, table, m = _filled(B, lens, H, P, d, "bf16", gen)
    s = torch.randint(-127, 128, (cache.num_pages, H, 2, d), generator=gen, dtype=torch.int8).cuda()
    cache = B.KVCache(cache.k, cache.v, summary=s, summary_scale=torch.ones(cache.num_pages, H, device="cuda"))
    q = torch.randn(3, 8, d, generator=gen).to(torch.bfloat16).cuda()
    want, chosen = B.decode_attention(cache, table, m, q), B.select_pages(cache, table, m, q, n)
    sizes = [B.cm_attn_decode_workspace_size(3, 8, H, d), B.cm_select_pages_workspace_size(3, H, table.shape[1]),
             3 * 8 * d * 2, 3 * 8 * 4, 3 * H * n * 4, 3 * H * 4]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        held = [torch.empty(b, dtype=torch.uint8, device="cuda") for b in sizes]
        torch.cuda._sleep(50_000_000)
        for t in held:
            t.fill_(255)
        del held, t
        got = B.decode_attention(cache, table, m, q, stream=0), B.select_pages(cache, table, m, q, n, stream=0)
        torch.cuda.synchronize()
    for a, b in zip((*got[0], *got[1]), (*want, *chosen)):
        assert torch.equal(a, b)
    assert B.cm_kv_status(cache) == B.CM_OK


def test_status_of_a_cache_on_another_device(B):
    """Like the other calls, cm_kv_status wants the cache's device to be the current one: another device's stream
    would not wait for the work that it asks about."""
    cache = B.KVCache.alloc(2, 1, 16, 64)
    assert B.cm_kv_status(cache) == B.CM_OK
    cache.index += 1
    with pytest.raises(ValueError):
        B.cm_kv_status(cache)


def test_the_loop_of_the_readme(B):
    """The README's generation loop as it stands there: prompt, then tokens, each one further."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(root, "README.md")).read(), re.S)
    code, = (x for x in blocks if "KVCache.alloc" in x)
    gen = torch.Generator().manual_seed(69)
    Bn, H, Hq, T, d, S, num_pages, steps = 2, 2, 4, 37, 64, 256, 8, 30
    draw = lambda h, t: torch.randn(Bn, h, t, d, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    prompt = [draw(H, T), draw(H, T), draw(Hq, T)]
    tokens = [(draw(H, 1), draw(H, 1), draw(Hq, 1)) for _ in range(steps)]
    angle = torch.rand(S, d // 2, generator=gen, dtype=F64) * 50
    spec = B.cm_compile_spec("region all : j <= i")
    desc = B.Descriptor(spec, spec, Bn, S)
    B.cm_build_descriptor(spec, spec, torch.tensor([[0, S]] * Bn, dtype=torch.int32, device="cuda"),
                          torch.ones(Bn, dtype=torch.int32, device="cuda"), desc)
    names = {"torch": torch, "cm": B, "num_pages": num_pages, "H_kv": H, "d": d, "B": Bn, "desc": desc,
             "page_table": torch.arange(num_pages, dtype=torch.int32, device="cuda").view(Bn, -1).contiguous(),
             "rope": torch.stack([angle.cos(), angle.sin()], 2).float().cuda(), "tokens": [tuple(x.clone() for x in t) for t in tokens],
             "k": prompt[0], "v": prompt[1], "q": prompt[2], "q_rot": torch.empty_like(prompt[2]), "k_rot": torch.empty_like(prompt[0])}
    names["lens"], names["after"] = (torch.zeros(Bn, dtype=torch.int32, device="cuda") for _ in range(2))
    exec(code, names)
    cache = names["cache"]
    assert names["after"].tolist() == [T + steps] * Bn and B.cm_kv_status(cache) == B.CM_OK
    rows = torch.arange(T + steps)
    k, v, _, _ = _host(cache)
    for b in range(Bn):
        for g in range(H):
            want = torch.cat([prompt[1][b, g], *(t[1][b, g] for t in tokens)]).cpu().to(F64)
            assert torch.equal(K.rows(v, None, names["page_table"][b].cpu(), g, rows), want)
    # the last step attends to all of it (64 pages are more than there are, so the selection is every page)
    last = tokens[-1][2].cpu()
    q = torch.stack([K.rotate(last[b, :, 0], names["rope"][T + steps - 1, :, 0].cpu(),
                              names["rope"][T + steps - 1, :, 1].cpu(), False)[0] for b in range(Bn)]).to(torch.bfloat16)
    _check_decode(cache, names["page_table"], [T + steps] * Bn, q, names["o"], names["lse"], 1 / math.sqrt(d), lambda b, g: rows)


# ---- how far outputs may be off ------------------------------------------------------------------
def _sharp_bound(kv, n, want, mag, size, d):
    """The scores' error and the output's rounding as in _check_decode, and in place of a rounding of every weight
    to bf16 what the kernel rounds: a weight beside bf16 values is two bf16 numbers, the first cut (the rest is below
    2^-7 of it), the second rounded (half a step: 2^-8 of that); beside e4m3 values it is one fp16 number (2^-11).  Two
    exp2 of 2^-22 each.  The second product adds 16 terms and the sum so far up to 4 times a tile of 32 keys, and may cut
    each term at 2^-23 of the largest."""
    ds = (d + 8) * 2 * 2.0 ** -24 * size + 2.0 ** -20
    weight = 2.0 ** -15 if kv == "bf16" else 2.0 ** -11
    return BF16_HALF * want.abs() + (1 + BF16_HALF) * (weight + 2 * ds + 2.0 ** -21 + 4 * ((n + 31) // 32) * 17 * 2.0 ** -23) * mag


def _close_scores(heads, d):
    """Two keys whose weights differ by up to 6 %, with values 1 and -1: what is left of the values is less than
    their weights' rounding to 8 bits."""
    k = torch.zeros(2, d)
    k[0, 0], k[1, 0] = 1, 0.9375
    v = torch.ones(2, d)
    v[1] = -1
    q = torch.zeros(heads, d)
    q[:, 0] = torch.arange(heads) / heads + 1 / 128
    return q.to(torch.bfloat16), k, v


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [8, 16])
def test_cancelling_values(B, kv, group):
    """Beside bf16 values, weights rounded to bf16 alone would be outside the bound (shown on the plain form first)."""
    d, P = 64, 16
    q, k, v = _close_scores(group, d)
    dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    pools = [torch.zeros(1, 1, P, d) for _ in range(2)]
    pools[0][0, 0, :2], pools[1][0, 0, :2] = k, v
    pools = [x.to(dtype).cuda() for x in pools]
    one = torch.ones(1, device="cuda")
    scales = {"k_scale": one, "v_scale": one} if kv == "e4m3" else {}
    cache = B.KVCache(*pools, **scales)
    want, wl, size, mag = K.decode(q, k.to(F64), v.to(F64), 1.0)
    bound = _sharp_bound(kv, 2, want, mag, size, d)
    s = q.to(F64) @ k.to(F64).T
    p = torch.exp(s - s.amax(1, keepdim=True))
    rounded = p.to(torch.bfloat16).to(F64) @ v.to(F64) / p.sum(1, keepdim=True)
    assert kv == "e4m3" or ((rounded - want).abs() > bound).any()
    table, n = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda")
    o, lse = B.decode_attention(cache, table, n, q.cuda()[None], scale=1.0)
    err = (o[0].double().cpu() - want).abs()
    assert (err <= bound).all(), (err / bound).max()
    assert ((lse[0].double().cpu() - wl).abs() <= 2.0 ** -19 * (1 + wl.abs())).all()


@pytest.mark.parametrize("d,P,kv,H,group", [(128, 64, "bf16", 2, 4), (64, 16, "bf16", 1, 16), (128, 16, "e4m3", 2, 3),
                                            (64, 32, "e4m3", 1, 12)])
def test_decode_is_off_by_its_own_rounding(B, d, P, kv, H, group):
    """Values of magnitude 1 and random signs, so that the outputs are small beside the weighted magnitudes."""
    gen = torch.Generator().manual_seed(70)
    lens = [3, 17, 33, 100, 300]
    cache, table, n = _filled(B, lens, H, P, d, kv, gen)
    sign = torch.randint(0, 2, cache.v.shape, generator=gen).float() * 2 - 1
    v = sign.to(cache.v.dtype).cuda()
    scales = {} if kv == "bf16" else {"k_scale": cache.k_scale, "v_scale": torch.ones(H, device="cuda")}
    cache = B.KVCache(cache.k, v, **scales)
    q = torch.randn(len(lens), H * group, d, generator=gen).to(torch.bfloat16).cuda()
    o, lse = B.decode_attention(cache, table, n, q)
    assert B.cm_kv_status(cache) == B.CM_OK
    k, v, ks, vs = _host(cache)
    where, worst = table.cpu(), 0.0
    for b, m in enumerate(lens):
        for g in range(H):
            kk, vv = (K.rows(x, s, where[b], g, torch.arange(m)) for x, s in ((k, ks), (v, vs)))
            hs = slice(g * group, (g + 1) * group)
            want, _, size, mag = K.decode(q[b, hs].cpu(), kk, vv, 1 / math.sqrt(d))
            err = (o[b, hs].double().cpu() - want).abs() / _sharp_bound(kv, m, want, mag, size, d)
            worst = max(worst, err.max().item())
    assert worst <= 1, worst


def test_tokens_after_a_prompt_are_off_by_their_own_rounding(B):
    """A prompt and the tokens after it under one mask, token by token, against the 64-bit form of the rows."""
    from masked_flashattention_gb300 import specs
    from oracle import masks as M
    gen = torch.Generator().manual_seed(71)
    H, S, d, P, T, wid = 2, 256, 64, 32, 150, 5
    cuts = [0, 20, 100, 190, S]
    f, b = B.cm_compile_spec(specs.FWD[wid]), B.cm_compile_spec(specs.BWD[wid])
    desc = B.Descriptor(f, b, 1, S)
    B.cm_build_descriptor(f, b, torch.tensor([cuts], dtype=torch.int32, device="cuda"),
                          torch.tensor([4], dtype=torch.int32, device="cuda"), desc)
    mask = torch.from_numpy(M.dense_mask(wid, torch.tensor(cuts).numpy(), 4, S))
    q, k, v = (torch.randn(1, H, S, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(3))
    cache = B.KVCache.alloc(S // P, H, P, d)
    table = torch.randperm(S // P, generator=gen).to(torch.int32).view(1, -1).cuda()
    lens, after = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    B.cm_kv_append(cache, table, lens, k[:, :, :T], v[:, :, :T], new_lens=after)
    for i in range(T, S):
        lens, after = after, lens
        B.cm_kv_append(cache, table, lens, k[:, :, i:i + 1], v[:, :, i:i + 1], new_lens=after)
        o, lse = B.decode_attention(cache, table, after, q[:, :, i], desc=desc)
        see = mask[i].nonzero()[:, 0]
        for h in range(H):
            want, wl, size, mag = K.decode(q[0, h, i:i + 1].cpu(), k[0, h].double().cpu()[see], v[0, h].double().cpu()[see],
                                           1 / math.sqrt(d))
            assert ((o[0, h:h + 1].double().cpu() - want).abs() <= _sharp_bound("bf16", i + 1, want, mag, size, d)).all(), (i, h)
            assert (lse[0, h].double().cpu() - wl).abs().item() <= (d + 8) * 2.0 ** -23 * size + 2.0 ** -18 * (1 + wl.abs().item())
    assert B.cm_kv_status(cache) == B.CM_OK and B.cm_get_status(desc) == B.CM_OK


@pytest.mark.parametrize("lens", [[300, 0, 77], [20000, 5, 0]])
def test_outputs_in_place_of_the_queries(B, lens):
    """o may be q: a row's queries have been read by all that need them before its output is written."""
    gen = torch.Generator().manual_seed(72)
    cache, table, n = _filled(B, lens, 2, 64, 128, "bf16", gen)
    q = torch.randn(3, 2 * 20, 128, generator=gen).to(torch.bfloat16).cuda()
    want, wl = B.decode_attention(cache, table, n, q)
    work = torch.empty(B.cm_attn_decode_workspace_size(3, 40, 2, 128), dtype=torch.uint8, device="cuda")
    lse = torch.empty_like(wl)
    B.cm_attn_decode(cache, table, n, q, q, lse, work)
    assert torch.equal(q, want) and torch.equal(lse, wl) and B.cm_kv_status(cache) == B.CM_OK


_FIRST_CAPTURE = """
import torch
from masked_flashattention_gb300 import binding as B
P, d, n = 64, 128, 300
gen = torch.Generator().manual_seed(6)
caches = [B.KVCache.alloc(6, 2, P, d, summaries=True) for _ in range(2)]
draw = lambda h, t: torch.randn(1, h, t, d, generator=gen).to(torch.bfloat16).cuda()
k, v, q = draw(2, n), draw(2, n), draw(8, 1)
table = torch.arange(6, dtype=torch.int32, device="cuda")[None]
lens, after = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
def step(cache):
    B.cm_kv_append(cache, table, lens, k, v, new_lens=after)
    sel, nsel = B.select_pages(cache, table, after, q[:, :, 0], 3, 1, 1)
    return [sel, *B.decode_attention(cache, table, after, q[:, :, 0], sel=sel, nsel=nsel),
            *B.decode_attention(cache, table, after, q[:, :, 0])]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step(caches[0])
graph.replay()
want = step(caches[1])
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[1].any()
assert B.cm_kv_status(caches[0]) == 0 and B.cm_kv_status(caches[1]) == 0
print("first capture ok")
"""


def test_first_calls_of_a_process_in_a_capture():
    """Nothing has to be called before a step is captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first capture ok" in r.stdout, r.stderr


@pytest.mark.parametrize("group", [2, 10])
def test_infinite_keys(B, group):
    """A key of -inf against a positive channel has no weight; against a negative one it makes that head NaN; where
    every key is such a key, the row is empty."""
    gen = torch.Generator().manual_seed(73)
    lens, P, d = [40, 40, 3], 16, 64
    cache, table, n = _filled(B, lens, 1, P, d, "bf16", gen)
    where = table.cpu()
    cache.k[int(where[0, 1]), 0, 5, 7] = -math.inf  # position 21 of sequence 0
    cache.k[int(where[2, 0]), 0, :3, 7] = -math.inf
    q = torch.randn(3, group, d, generator=gen).to(torch.bfloat16).cuda()
    q[..., 7] = 1
    q[0, 1, 7] = -1
    o, lse = B.decode_attention(cache, table, n, q)
    assert B.cm_kv_status(cache) == B.CM_OK
    assert o[0, 1].isnan().all() and lse[0, 1].isnan()
    assert not o[2].any() and (lse[2] == -math.inf).all()
    keep = [h for h in range(group) if h != 1]
    q0, o0, l0 = q[:, keep].contiguous(), o[:, keep].contiguous(), lse[:, keep].contiguous()
    seen = [torch.tensor([p for p in range(40) if p != 21]), torch.arange(40), torch.arange(0)]
    _check_decode(cache, table, lens, q0, o0, l0, 1 / 8, lambda b, g: seen[b])
