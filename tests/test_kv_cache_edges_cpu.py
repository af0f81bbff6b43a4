"""Paged key-value cache without a GPU: host code at the edge of what is allowed."""
import os
import subprocess

import pytest
import torch

from tests.test_kv_cache_cpu import A16, B, _cache, _decode, _new, _seqs  # noqa: F401 (B is a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_SLOW_LOOKUP = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include "tma_host.h"
// the runtime's lookup, taking its time
extern "C" cudaError_t CUDARTAPI cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                                                  cudaDriverEntryPointQueryResult* q) {
  std::this_thread::sleep_for(std::chrono::milliseconds(100));
  *p = reinterpret_cast<void*>(0x1000);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
int main() {
  bool found[4] = {};
  std::thread all[4];
  for (int i = 0; i < 4; ++i) all[i] = std::thread([&found, i] { found[i] = cm::encode_tiled_fn() != nullptr; });
  for (auto& t : all) t.join();
  std::printf("%d%d%d%d\n", found[0], found[1], found[2], found[3]);
}
"""


def test_the_encoder_is_found_by_every_thread(tmp_path):
    """Threads that ask for the tensor maps' encoder while the first still looks it up get it too."""
    src, exe = tmp_path / "lookup.cpp", tmp_path / "lookup"
    src.write_text(_SLOW_LOOKUP)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I/usr/local/cuda/include",
                        "-I" + os.path.join(ROOT, "masked_flashattention_gb300", "csrc"), str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([str(exe)], capture_output=True, text=True, timeout=60).stdout.strip() == "1111"


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are made up: nothing may be queued")
def test_limit_of_a_decode_call(B):  # noqa: F811
    """Rows of tiles are counted in 31 bits, with room for the rounding of their division among up to 320 blocks:
    331 x 151 rows of one head with 42,966 places each are 2^31 - 2, one too many by that; with 42,959 they fit."""
    def call(pages, group=1, **more):
        c = _cache(B, num_pages=16, page_size=32, H_kv=151, k_page_stride=151 * 32 * 128, v_page_stride=151 * 32 * 128)
        return _decode(B, cache=c, seqs=_seqs(B, B=331, max_pages=pages), H_q=151 * group, **more)
    assert call(42964) == B.CM_ERR_UNSUPPORTED
    assert call(42957) == B.CM_ERR_CUDA  # goes on to the launch
    assert call(42957, group=16) == B.CM_ERR_CUDA
    assert call(42957, group=17) == B.CM_ERR_UNSUPPORTED  # two rows of 16
    assert call(42964, sel=A16, nsel=A16, sel_max=8192) == B.CM_ERR_CUDA  # what is selected counts


def test_outputs_that_overlap_themselves(B):  # noqa: F811
    """Heads, tokens or sequences of an output in the same memory (an expanded tensor) are refused; inputs may be."""
    for name in ("q_out", "k_out"):
        for s in ((1024, 0, 128), (0, 512, 128), (1024, 512, 64), (1024, 8, 128)):
            t = _new(B, **{name: 2 * A16, name + "_stride": s})
            assert B.lib().cm_kv_append(_cache(B), _seqs(B), t, None) == B.CM_ERR_INVALID_ARG, (name, s)
    t = _new(B, cu_new=A16, q_out=2 * A16, q_out_stride=(0, 512, 0))
    assert B.lib().cm_kv_append(_cache(B), _seqs(B), t, None) == B.CM_ERR_INVALID_ARG
    for s in ((0, 128), (512, 0), (512, 64)):
        assert _decode(B, os=s) == B.CM_ERR_INVALID_ARG, s


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are made up: nothing may be queued")
def test_inputs_that_are_expanded_and_axes_of_one_entry(B):  # noqa: F811
    """What goes on to the launch: inputs with strides of 0, and outputs whose axis of one entry has any."""
    t = _new(B, k_stride=(0, 0, 0), v_stride=(0, 0, 0), q_stride=(0, 0, 0), q_out=2 * A16)
    assert B.lib().cm_kv_append(_cache(B), _seqs(B), t, None) == B.CM_ERR_CUDA
    t = _new(B, n_tokens=1, max_new=1, H_q=1, q_out=2 * A16, q_out_stride=(1024, 0, 0))
    assert B.lib().cm_kv_append(_cache(B), _seqs(B), t, None) == B.CM_ERR_CUDA
    t = _new(B, cu_new=A16, q_out=2 * A16, q_out_stride=(0, 512, 128))
    assert B.lib().cm_kv_append(_cache(B), _seqs(B), t, None) == B.CM_ERR_CUDA
    one = _cache(B, H_kv=1)
    assert _decode(B, cache=one, seqs=_seqs(B, B=1), H_q=1, qs=(0, 0), os=(0, 0)) == B.CM_ERR_CUDA
    assert _decode(B, qs=(0, 0)) == B.CM_ERR_CUDA
