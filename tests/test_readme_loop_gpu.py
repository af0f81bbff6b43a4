"""The README's loop without end where a program leaves its first lines: its step captured into a graph, and a pool that is too
small for a while."""
import math
import os
import re
import textwrap

import pytest
import torch

from oracle import kv_cache as K
from tests.test_kv_cache_gpu import _rope

pytestmark = pytest.mark.gpu

B_, H, HQ, D = 2, 2, 4, 64


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


def _readme():
    """What comes before the loop, the loop's step, and the whole."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(root, "README.md")).read(), re.S)
    code, = (x for x in blocks if "KVPages.alloc" in x)
    before, step = re.split(r"^for .*? in steps:.*\n", code, flags=re.M)
    return before, textwrap.dedent(step), code


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _names(B, num_pages, rope, **more):
    return {"torch": torch, "cm": B, "num_pages": num_pages, "max_pages": 8, "H_kv": H, "d": D, "B": B_, "rope": rope.cuda(),
            "lens": _ints([0, 0]), "after": _ints([0, 0]), **more}


def test_its_step_as_a_graph(B):
    """Every replay goes on where the one before ended: lengths, pages and outputs are those of the loop as it stands."""
    gen = torch.Generator().manual_seed(98)
    before, step, code = _readme()
    T, rope = 70, _rope(512, D, gen)
    counts, over = [[70, 65], [1, 1], [30, 1], [1, 64], [2, 1]], [[0, 0], [0, 0], [0, 1], [0, 0], [0, 0]]
    tokens = [[torch.randn(B_, h, T, D, generator=gen).to(torch.bfloat16).cuda() for h in (H, H, HQ)] for _ in counts]
    eager = _names(B, 9, rope)
    seen = []

    def steps():
        for (k, v, q), n, x in zip(tokens, counts, over):
            yield k.clone(), v.clone(), q.clone(), _ints(n), _ints(x)
            seen.append([eager[y].clone() for y in ("o", "lse", "lens")] + [eager["pages"].state.clone()])

    eager["steps"] = steps()
    exec(code, eager)
    names = _names(B, 9, rope)
    names.update(zip("kvq", (torch.zeros_like(x) for x in tokens[0])), n_new=_ints([0, 0]), done=_ints([0, 0]))
    exec(before, names)
    run = compile(step, "README", "exec")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        exec(run, names)  # no tokens: nothing changes
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        exec(run, names)
    for (k, v, q), n, x, (o, lse, lens, state) in zip(tokens, counts, over, seen):
        for name, y in zip(("k", "v", "q", "n_new", "done"), (k, v, q, _ints(n), _ints(x))):
            names[name].copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert names["lens"].tolist() == lens.tolist() and names["pages"].state.tolist() == state.tolist()
        assert torch.equal(names["o"], o) and torch.equal(names["lse"], lse)
    assert B.cm_kv_status(names["cache"]) == B.CM_OK and B.cm_kv_pages_status(names["pages"]) == B.CM_OK


def test_a_pool_that_is_too_small_for_a_while(B):
    """Tokens that were not granted are brought again, as the README says: none is lost, and each is attended to once it is
    stored."""
    gen = torch.Generator().manual_seed(99)
    code, rope = _readme()[2], _rope(512, D, gen)
    # three pages of 64: the second sequence's 70 tokens wait until the first, which fills all three, has ended
    queue = [[([torch.randn(h, n, D, generator=gen).to(torch.bfloat16) for h in (H, H, HQ)], x) for n, x in want]
             for want in ([(130, 0), (1, 1)], [(70, 0), (1, 0), (2, 0)])]
    names = _names(B, 3, rope)
    stored, turns = [[], []], []

    def steps():
        while any(queue):
            now = [q[0] if q else None for q in queue]
            T = max(x[0][0].shape[1] for x in now if x)
            k, v, q = (torch.zeros(B_, h, T, D, dtype=torch.bfloat16) for h in (H, H, HQ))
            n = [0, 0]
            for b, x in enumerate(now):
                if x:
                    n[b] = x[0][0].shape[1]
                    for to, y in zip((k, v, q), x[0]):
                        to[b, :, :n[b]] = y
            # a sequence ends in the step that stores its last token
            yield k.cuda(), v.cuda(), q.cuda(), _ints(n), _ints([int(bool(x) and x[1]) for x in now])
            granted = names["granted"].tolist()
            turns.append(granted)
            for b, x in enumerate(now):
                if x and granted[b] == n[b]:
                    queue[b].pop(0)
                    stored[b] += [x[0]]

    names["steps"] = steps()
    exec(code, names)
    assert turns == [[130, 0], [1, 0], [0, 70], [0, 1], [0, 2]]
    cache, pages = names["cache"], names["pages"]
    assert names["lens"].tolist() == [0, 73] and B.cm_kv_status(cache) == B.CM_OK and B.cm_kv_pages_status(pages) == B.CM_OK
    assert pages.state.tolist() == [[0, 0], [0, 2], [1, 0]]
    table, pos = pages.page_table.cpu()[1], torch.arange(73)
    for h in range(H):
        row = K.BlockRow("int8")
        for _, v, _ in stored[1]:
            row.append(v[h])
        vv = K.block_rows(cache.v.cpu(), cache.v_scale.cpu(), table, h, pos)
        assert torch.equal(vv, row.values())
        kk = K.block_rows(cache.k.cpu(), cache.k_scale.cpu(), table, h, pos)
        q = K.rotate(stored[1][-1][2][2 * h:2 * h + 2, 1], rope[72, :, 0], rope[72, :, 1], False)[0].to(torch.bfloat16)
        want, _, _, mag = K.decode(q, kk, vv, 1 / math.sqrt(D))
        assert ((names["o"][1, 2 * h:2 * h + 2].double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * mag).all()
