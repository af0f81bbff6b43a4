// Between the host side of cm_attn_decode (attn_decode.cu) and its kernels (attn_decode.cuh), which are compiled once for each
// type of cache.
#pragma once
#include <cuda.h>

#include "kv_cache.h"

namespace cm {

constexpr int kTileKeys = 32;
constexpr int kMaxCtas = 320;
constexpr int kRowCost = 2;
constexpr int kMaxDevices = 64;  // beyond them, a device's properties are asked for at every call

// Division of 0 <= n < 2^31 by a fixed d >= 1: with 2^s >= d > 2^(s-1) and mul = ceil(2^(31+s) / d), the
// product's error stays below 2^s / 2^(31+s) * n < 1 / d.
struct Divisor {
  uint32_t mul, shift;
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
  }
};
inline Divisor make_divisor(uint32_t d) {
  uint32_t s = 0;
  while ((1u << s) < d) ++s;
  return {static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d), 31 + s};
}

struct DecodeArgs {
  DecodeParams p;
  int chunks;   // rows of one key-value head: ceil(group / heads of a row)
  int group;
  int heads;    // of a row: 8 or 16
  int units;    // B, or B * H_kv where pages are selected
  int rows;     // of a unit
  int ctas;
  int min_run;  // least cost a CTA's run is given
  int most_tiles;  // a row can have
  int whole_rows;  // a CTA's run is cut at rows' ends only
  Divisor by_chunks, by_heads;  // H_kv
  uint64_t wait_ns;
};

// Launches the kernels for caches of type KIND (one translation unit each).
template <int KIND>
int launch_decode_kind(DecodeArgs& a, int dev, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream);

}  // namespace cm
