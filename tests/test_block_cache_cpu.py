"""Caches with a scale for each block, without a GPU: the oracle's pins, and what the C ABI refuses on the host."""
import math

import pytest
import torch

from oracle import kv_cache as K
from tests.test_kv_cache_cpu import A16, BAD_NEW, _cache, _new, _seqs


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import build as bld
    bld.build()
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


@pytest.mark.parametrize("a,int8,e4m3", [(127.0, 0, -1), (127.5, 1, -1), (448.0, 2, 0), (450.0, 2, 1), (1.0, -6, -8),
                                         (0.0, -32, -32), (1e-30, -32, -32), (3e38, 32, 32), (math.inf, 32, 32)])
def test_exponents(a, int8, e4m3):
    assert K.block_exponent(a, "int8") == int8 and K.block_exponent(a, "e4m3") == e4m3


def test_blocks_by_hand():
    """Two calls into one block: 100 fits a scale of 1; 300 needs 4, and the first token's 100 and 3 become 25 and 1 (3 / 4 =
    0.75), its 2 becomes 0 (a half goes to even)."""
    r = K.BlockRow("int8")
    r.append(torch.tensor([[100.0, 3.0, 2.0, -6.0]]))
    assert r.exps == [0] and r.codes[0].tolist() == [100, 3, 2, -6]
    r.append(torch.tensor([[300.0, 0.0, 0.0, 10.0]]))
    assert r.exps == [2] and r.codes[0].tolist() == [25, 1, 0, -2] and r.codes[1].tolist() == [75, 0, 0, 2]
    r.append(torch.ones(15, 4))  # 14 of them in the first block, whose scale stays
    assert r.exps == [2, -6] and r.codes[15].tolist() == [0] * 4 and r.codes[16].tolist() == [64] * 4
    assert r.values()[0].tolist() == [100, 4, 0, -8]


def test_e4m3_blocks_lose_nothing_when_a_scale_grows():
    """A power of two moves an e4m3 number's exponent alone, down to the smallest numbers."""
    r = K.BlockRow("e4m3")
    x = torch.tensor([[1.0, 1.125, -3.25, 0.875]])
    r.append(x)
    r.append(torch.full((1, 4), 30.0))
    assert r.values()[0].tolist() == x[0].tolist()


@pytest.mark.parametrize("dtype", [2, 3])
def test_refusals(B, dtype):
    import ctypes
    good = {"dtype": dtype, "k_scale": A16, "v_scale": A16}
    call = lambda **k: B.lib().cm_kv_append(_cache(B, **{**good, **k}), _seqs(B), _new(B), None)  # noqa: E731
    for bad, rc in (({"dtype": 4}, -2), ({"dtype": -1}, -2), ({"k_scale": None}, -2), ({"v_scale": None}, -2), ({"v_scale": 2}, -2),
                    ({"k_page_stride": 2 * 64 * 128 + 8}, -2), ({"page_size": 8}, -3), ({"d": 96}, -3), ({"k": A16 + 8}, -2),
                    ({"summary": A16}, -2)):
        assert call(**bad) == rc, bad
    for bad in BAD_NEW:
        assert B.lib().cm_kv_append(_cache(B, **good), _seqs(B), _new(B, **bad), None) == B.CM_ERR_INVALID_ARG, bad
    # more blocks than a grid takes
    assert B.lib().cm_kv_append(_cache(B, **good, page_size=16, H_kv=1024, k_page_stride=1 << 21, v_page_stride=1 << 21),
                                _seqs(B, B=32767), _new(B, n_tokens=32000, max_new=32000), None) == B.CM_ERR_UNSUPPORTED
    n = ctypes.c_size_t()
    assert B.lib().cm_attn_decode_workspace_size(2, 4, 2, 128, n) == B.CM_OK
    stride = (ctypes.c_int64 * 2)(512, 128)
    assert B.lib().cm_attn_decode(_cache(B, **{**good, "v_scale": None}), _seqs(B), None, None, None, 0, A16, stride, A16, stride,
                                  None, 4, 0.1, A16, n.value, None) == B.CM_ERR_INVALID_ARG
