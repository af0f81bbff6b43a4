"""Paged key-value cache without a GPU: the oracle's pins, and what the C ABI refuses on the host."""
import ctypes
import math

import pytest
import torch

from oracle import attention as A
from oracle import kv_cache as K


@pytest.fixture(scope="module")
def B():
    from masked_flashattention_gb300 import build as bld
    bld.build()
    from masked_flashattention_gb300 import binding
    binding.lib()
    return binding


# ---- oracle ----------------------------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_complex_multiplication(interleaved):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 10, generator=g, dtype=torch.float64)
    a = torch.randn(3, generator=g, dtype=torch.float64)
    got, _ = K.rotate(x, a.cos(), a.sin(), interleaved)
    pairs = [(2 * i, 2 * i + 1) if interleaved else (i, i + 3) for i in range(3)]
    for i, (p, q) in enumerate(pairs):
        z = torch.complex(x[:, p], x[:, q]) * complex(math.cos(a[i]), math.sin(a[i]))
        assert torch.allclose(got[:, p], z.real) and torch.allclose(got[:, q], z.imag)
    assert torch.equal(got[:, 6:], x[:, 6:])


@pytest.mark.parametrize("a,e", [(127.0, 0), (127.5, 1), (1.0, -6), (0.992, -7), (0.0, -50), (3e38, 50),
                                 (math.inf, 50), (254.0, 1), (1e-30, -50)])
def test_exponent(a, e):
    assert K.exponent(a) == e


def test_summary_of_two_keys():
    s, scale = K.summary(torch.tensor([[100.0, -3.5, math.nan], [-20.0, 2.25, 1.0]]))
    assert scale == 1.0 and s.tolist() == [[100, 3, 1], [-20, -4, 1]]


def test_decode_is_the_last_row_of_attention():
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(9, 16, generator=g, dtype=torch.float64) for _ in range(3))
    vis = torch.rand(9, 9, generator=g) < 0.6
    o, lse = A.attention_forward(q, k, v, vis, 0.3)
    at = vis[8].nonzero()[:, 0]
    got_o, got_l, _, _ = K.decode(q[8:], k[at], v[at], 0.3)
    assert torch.allclose(got_o[0], o[8]) and torch.allclose(got_l[0], lse[8])
    zero, none, _, _ = K.decode(q[:2], k[:0], v[:0], 0.3)
    assert not zero.any() and (none == -math.inf).all()


def test_scores_bound_the_keys_and_pick_orders_them():
    g = torch.Generator().manual_seed(3)
    q = torch.randint(-127, 128, (2, 8), generator=g).float()  # whole numbers: no rounding
    q[:, 0] = 127
    keys = torch.randint(-127, 128, (5, 4, 8), generator=g).float()
    keys[..., 0] = 127
    parts = [K.summary(x) for x in keys]
    got = K.scores(q, torch.stack([s for s, _ in parts]), [e for _, e in parts])
    for n in range(5):
        assert got[n] >= (q @ keys[n].T).max().item()
        assert got[n] <= (q.abs() @ keys[n].abs().amax(0)[:, None]).max().item()
    assert K.pick([5.0, 7.0, 7.0, 1.0, 7.0], 2, 0, 0) == [1, 2]
    assert K.pick([5.0, 7.0, 7.0, 1.0, 9.0], 3, 1, 0) == [0, 1, 4]
    assert K.pick([5.0, 7.0, 7.0, 1.0, 2.0], 2, 0, 1) == [1, 4]
    assert K.pick([5.0], 4, 1, 1) == [0]


# ---- refusals (made-up pointers: every case must return before anything is queued) ---------------
A16 = 0x1000


def _cache(B, /, **k):
    c = B.cm_kv_cache(8, 64, 2, 128, B.CM_KV_BF16, 2 * 64 * 128, 2 * 64 * 128, A16, A16, None, None,
                      None, None, A16)
    for n, v in k.items():
        setattr(c, n, v)
    return c


def _seqs(B, /, **k):
    s = B.cm_kv_seqs(2, 4, A16, A16 + 4)
    for n, v in k.items():
        setattr(s, n, v)
    return s


E4 = {"dtype": 1, "k_scale": A16, "v_scale": A16}
BAD_CACHE = [({"num_pages": 0}, -2), ({"page_size": 48}, -3), ({"page_size": 256}, -3),
             ({"H_kv": 0}, -2), ({"H_kv": 2000}, -3), ({"d": 96}, -3), ({"dtype": 2}, -2),
             ({"k_page_stride": 64}, -2), ({"v_page_stride": 2 * 64 * 128 + 4}, -2),
             ({"k_page_stride": 1 << 38}, -3), ({"k": None}, -2), ({"v": A16 + 8}, -2),
             ({"status": None}, -2), ({"status": 2}, -2), ({"k_scale": A16}, -2), ({"dtype": 1}, -2),
             ({**E4, "v_scale": None}, -2), ({"summary": A16}, -2), ({"summary_scale": A16}, -2),
             ({"summary": A16 + 4, "summary_scale": A16}, -2),
             ({"num_pages": 2**31 - 1, "H_kv": 1024, "k_page_stride": 1 << 30, "v_page_stride": 1 << 30}, -3)]
BAD_SEQS = [({"B": 0}, -2), ({"B": 40000}, -3), ({"max_pages": 0}, -2), ({"max_pages": 1 << 22}, -3),
            ({"page_table": None}, -2), ({"lens": 2}, -2)]


def _new(B, /, **k):
    t = B.cm_kv_new()
    t.k = t.v = t.q = t.q_out = A16
    for n in ("k", "v", "q", "q_out", "k_out"):
        getattr(t, n + "_stride")[:] = (1024, 512, 128)
    t.n_tokens = t.max_new = 3
    t.H_q = 4
    t.rope, t.rope_len, t.rot_dim = A16, 100, 128
    for n, v in k.items():
        if n.endswith("stride"):
            getattr(t, n)[:] = v
        else:
            setattr(t, n, v)
    return t


BAD_NEW = [{"k": None}, {"v": A16 + 2}, {"q": None}, {"q_out": None}, {"q_out": A16 + 8}, {"H_q": 0},
           {"k_stride": (1024, 512, 4)}, {"v_stride": (-1024, 512, 128)}, {"q_out_stride": (0, 0, 1)},
           {"q_out_stride": (1024, 256, 128)},  # in place with other strides
           {"k_out": A16, "k_out_stride": (1024, 256, 128)}, {"k_out": A16 + 8},
           {"n_tokens": -1, "max_new": -1}, {"max_new": 4}, {"max_new": 2}, {"n_tokens": 4},
           {"cu_new": A16, "n_new": A16}, {"cu_new": 2}, {"n_new": 2}, {"rot_dim": 24},
           {"rot_dim": 144}, {"rot_dim": -16}, {"rot_dim": 0}, {"rope": None}, {"rope": A16 + 8},
           {"rope_len": 0}, {"new_lens": A16 + 4}, {"new_lens": 2}]


def test_append_refusals(B):
    call = lambda c, s, t: B.lib().cm_kv_append(c, s, t, None)  # noqa: E731
    for bad, rc in BAD_CACHE:
        assert call(_cache(B, **bad), _seqs(B), _new(B)) == rc, bad
    for bad, rc in BAD_SEQS:
        assert call(_cache(B), _seqs(B, **bad), _new(B)) == rc, bad
    for bad in BAD_NEW:
        assert call(_cache(B), _seqs(B), _new(B, **bad)) == B.CM_ERR_INVALID_ARG, bad
    assert call(_cache(B), _seqs(B), _new(B, H_q=1 << 20)) == B.CM_ERR_UNSUPPORTED
    assert call(_cache(B, page_size=16), _seqs(B), _new(B, n_tokens=1 << 30, max_new=1 << 30)) == B.CM_ERR_UNSUPPORTED
    assert call(_cache(B, page_size=16, summary=A16, summary_scale=A16, H_kv=1024, k_page_stride=1 << 21, v_page_stride=1 << 21),
                _seqs(B, B=32767), _new(B, n_tokens=32000, max_new=32000)) == B.CM_ERR_UNSUPPORTED
    for args in ((None, _seqs(B), _new(B)), (_cache(B), None, _new(B)), (_cache(B), _seqs(B), None)):
        assert call(*args) == B.CM_ERR_INVALID_ARG


def _decode(B, cache=None, seqs=None, desc=None, sel=None, nsel=None, sel_max=0, q=A16, qs=(512, 128), o=A16,
            os=(512, 128), lse=A16, H_q=4, scale=0.1, work=A16, size=1 << 40):
    return B.lib().cm_attn_decode(cache or _cache(B), seqs or _seqs(B), desc, sel, nsel, sel_max, q,
                                  (ctypes.c_int64 * 2)(*qs) if qs else None, o,
                                  (ctypes.c_int64 * 2)(*os) if os else None, lse, H_q, scale, work, size, None)


def _desc(B, /, **k):
    d = B.cm_descriptor(2, 256, 128, 1, 1, 0, A16, A16, A16, A16, A16, A16, A16)
    for n, v in k.items():
        setattr(d, n, v)
    return ctypes.byref(d)


def test_decode_refusals(B):
    for bad, rc in BAD_CACHE:
        assert _decode(B, cache=_cache(B, **bad)) == rc, bad
    for bad, rc in BAD_SEQS:
        assert _decode(B, seqs=_seqs(B, **bad)) == rc, bad
    size = B.cm_attn_decode_workspace_size(2, 4, 2, 128)
    for bad in ({"q": None}, {"q": A16 + 8}, {"qs": (512, 4)}, {"qs": (-8, 128)}, {"qs": None}, {"os": None},
                {"o": None}, {"o": A16 + 2}, {"os": (1, 128)}, {"lse": 2}, {"H_q": 3}, {"H_q": 0},
                {"scale": math.inf}, {"scale": math.nan}, {"work": None}, {"work": A16 + 8},
                {"size": size - 1}, {"sel": A16}, {"nsel": A16}, {"sel": A16, "nsel": A16},
                {"sel": 2, "nsel": A16, "sel_max": 4},
                {"sel": A16, "nsel": A16, "sel_max": 4, "desc": _desc(B)},
                {"desc": _desc(B, B=3)}, {"desc": _desc(B, S=0)}, {"desc": _desc(B, ni_f=0)},
                {"desc": _desc(B, ni_f=9)}, {"desc": _desc(B, itab_f=None)}, {"desc": _desc(B, itab_f=A16 + 8)}):
        assert _decode(B, **bad) == B.CM_ERR_INVALID_ARG, bad
    for bad in ({"H_q": 1 << 15}, {"sel": A16, "nsel": A16, "sel_max": 9000}, {"desc": _desc(B, form=1)},
                {"cache": _cache(B, page_size=128, H_kv=64, k_page_stride=1 << 20, v_page_stride=1 << 20),
                 "seqs": _seqs(B, B=32767, max_pages=8192), "H_q": 64}):
        assert _decode(B, **bad) == B.CM_ERR_UNSUPPORTED, bad


def test_select_refusals(B):
    full = {"summary": A16, "summary_scale": A16}

    def call(cache=None, seqs=None, q=A16, qs=(512, 128), H_q=4, first=1, last=1, sel=A16, nsel=A16, n=4,
             work=A16, size=1 << 40):
        return B.lib().cm_select_pages(cache or _cache(B, **full), seqs or _seqs(B), q, (ctypes.c_int64 * 2)(*qs),
                                       H_q, first, last, sel, nsel, n, work, size, None)

    for bad, rc in BAD_CACHE:
        whole = {} if "summary" in bad or "summary_scale" in bad else full
        assert call(cache=_cache(B, **{**whole, **bad})) == rc, bad
    for bad, rc in BAD_SEQS:
        assert call(seqs=_seqs(B, **bad)) == rc, bad
    size = B.cm_select_pages_workspace_size(2, 2, 4)
    for bad in ({"cache": _cache(B)}, {"q": None}, {"qs": (512, 1)}, {"H_q": 3}, {"first": -1}, {"last": -1},
                {"first": 3, "last": 2}, {"first": 5, "last": 0}, {"sel": None}, {"nsel": 2}, {"n": 0},
                {"work": None}, {"size": size - 1}):
        assert call(**bad) == B.CM_ERR_INVALID_ARG, bad
    for bad in ({"n": 9000}, {"seqs": _seqs(B, max_pages=40000)}):
        assert call(**bad) == B.CM_ERR_UNSUPPORTED, bad


def test_workspace_sizes_and_status_refusals(B):
    n = ctypes.c_size_t()
    L = B.lib()
    assert L.cm_attn_decode_workspace_size(2, 3, 2, 128, n) == B.CM_ERR_INVALID_ARG
    assert L.cm_attn_decode_workspace_size(2, 4, 2, 96, n) == B.CM_ERR_UNSUPPORTED
    assert L.cm_attn_decode_workspace_size(2, 4, 2, 64, None) == B.CM_ERR_INVALID_ARG
    assert L.cm_select_pages_workspace_size(0, 2, 4, n) == B.CM_ERR_INVALID_ARG
    assert L.cm_select_pages_workspace_size(2, 2, 1 << 20, n) == B.CM_ERR_UNSUPPORTED
    assert L.cm_kv_status(None, None) == B.CM_ERR_INVALID_ARG
    assert L.cm_kv_status(_cache(B, status=2), None) == B.CM_ERR_INVALID_ARG


def test_binding_refuses_tensors_that_are_not_on_a_gpu(B):
    t = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.KVCache(t, t)
