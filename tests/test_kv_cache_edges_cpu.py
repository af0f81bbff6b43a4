"""Paged key-value cache without a GPU: host code at the edge of what is allowed."""
import os
import subprocess

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
