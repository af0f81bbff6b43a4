"""The sparse step over caches with block scales: appends that keep summaries, the selection of pages by them, and attention over
what was selected."""
import math

import pytest
import torch

from oracle import kv_cache as K
from tests.test_block_cache_gpu import _empty
from tests.test_block_scores_gpu import check_far
from tests.test_kv_cache_gpu import _rope, _table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


@pytest.mark.parametrize("kind,d,P,H,group,prompts,n,first,last", [
    ("int8", 128, 64, 2, 4, [900, 64, 65, 0], 4, 1, 2),
    ("int8", 64, 16, 3, 1, [500, 31], 9, 0, 0),
    ("e4m3", 128, 16, 1, 12, [1000, 1], 20, 2, 1),
    ("e4m3", 64, 128, 2, 8, [1500, 300, 127], 2, 0, 1),
    ("int8", 128, 32, 1, 16, [700], 5, 0, 1),
])
def test_append_select_attend(B, kind, d, P, H, group, prompts, n, first, last):
    """Prompts, then tokens one by one: what is selected is what the definition picks from the keys as the cache holds them, and
    attention goes over these pages alone."""
    gen = torch.Generator().manual_seed(61)
    steps, Bn = 3, len(prompts)
    table, pages = _table([(t + steps + P - 1) // P for t in prompts], 2, gen)
    cache = _empty(B, pages, H, P, d, kind, summaries=True)
    wide = table.cuda()
    rope = _rope(wide.shape[1] * P, d, gen).cuda()
    lens = torch.zeros(Bn, dtype=torch.int32, device="cuda")
    spread = torch.exp(torch.randn(H, 1, d, generator=gen))  # some channels are larger than others
    for step in range(steps + 1):
        counts = [1] * Bn if step else prompts
        T = max(counts)
        k, v = (torch.randn(Bn, H, T, d, generator=gen) * (spread if i else 1.0) for i in (1, 0))
        k, v = (x.to(torch.bfloat16).cuda() for x in (k * torch.exp(torch.randn(Bn, 1, T, 1, generator=gen)), v))
        q = torch.randn(Bn, H * group, T, d, generator=gen).to(torch.bfloat16).cuda()
        after = torch.empty_like(lens)
        B.cm_kv_append(cache, wide, lens, k, v, q=q, q_out=q, rope=rope, new_lens=after,
                       n_new=torch.tensor(counts, dtype=torch.int32, device="cuda"))
        lens = after
        if not step:
            continue
        held = [t + step for t in prompts]
        assert lens.tolist() == held
        one = q[:, :, 0].contiguous()
        sel, nsel = B.select_pages(cache, wide, lens, one, n, first, last)
        o, lse = B.decode_attention(cache, wide, lens, one, sel=sel, nsel=nsel)
        assert B.cm_kv_status(cache) == B.CM_OK
        sel, nsel, host_q, hk, hs = (x.cpu() for x in (sel, nsel, one, cache.k, cache.k_scale))
        for b in range(Bn):
            for h in range(H):
                parts = [K.summary(K.block_rows(hk, hs, table[b], h, torch.arange(f, min(f + P, held[b]))).float())
                         for f in range(0, held[b], P)]
                score = K.scores(host_q[b, h * group:(h + 1) * group], torch.stack([s for s, _ in parts]), [e for _, e in parts])
                want = K.pick(score, n, first, last)
                assert sel[b, h].tolist() == want + [-1] * (n - len(want)) and nsel[b, h] == len(want), (step, b, h)

        def chosen(b, g):
            pos = torch.arange(held[b])
            return pos[torch.isin(pos // P, sel[b, g, :nsel[b, g]])]

        check_far(kind, cache, wide, one, o, lse, 1 / math.sqrt(d), chosen)
