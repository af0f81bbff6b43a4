// Append of new tokens to a paged key-value cache, with the rotation of queries and keys and the
// page summaries (cm_kv_append): one kernel whose blocks have two roles.
//
// What bounds it: each new query, key and value is read once and written once, and a row of the
// rotation's table is read per token.  A thread owns 16 channels of a token in two 16-byte pieces, the
// partners of a rotation among them (pieces j and j + rot / 16 of the rotated channels), so
// nothing crosses lanes; its pieces of the next heads (or tokens) are on their way into shared memory
// that no other thread reads (cp.async), which keeps 160 KB an SM in flight without the registers.
//   tokens  A block takes 1 to 8 tokens with all their heads; a thread goes through the heads with
//           the token's cosines and sines in registers.  The first loads do not depend on where the
//           token goes, so they are in flight while its sequence, position and page are looked up.
//   pages   With summaries, the keys go by page instead: one warp a (page, head) that the call
//           touches stores the new keys and takes the largest and smallest over all that the page
//           then holds, so a summary never depends on how its tokens arrived and needs no atomics.
//           Where blocks of 16 tokens have scales, keys and values go by block in this role (store_blocks).
// Measured: 42,000 new tokens of 9 sequences, 32 query and 8 key-value heads of 128, with summaries, 156 us =
// 6.7 TB/s, 99 % of the copy bandwidth (428 us with one unit a warp of 16 rows in registers, 265 with
// the heads' loads in registers, which held a quarter of the warps, 183 with neighbouring pieces a lane); one token
// of 256 sequences, e4m3, 9.2 us.  int8 with block scales, no summaries: 164 us = 5.9 TB/s (the rows of keys and values alone
// 3.9 TB/s: they are gone through twice, and a rotation's row is read again by every head);
// one token of 256 sequences, e4m3 with block scales and summaries, 9.5 us.
//
// Numerics: the rotation is fp32 with every product and sum rounded once (no fused
// multiply-add), so that it equals the formula evaluated step by step; one rounding to bf16, and
// for an e4m3 cache one more after the division by the scale (the cache holds what k_out says).  Scales of blocks are powers of
// two, so that the division is exact and what is stored depends on that one rounding; a scale that grows rounds its block's earlier
// tokens once more (e4m3: only where they become subnormal).
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <type_traits>

#include "kv_cache.h"
#include "ptx.cuh"

namespace cm {
namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 5;  // heads of a thread whose pieces are on their way: 40 KB a CTA, 4 CTAs an SM

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_float2(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// 8 fp32 values as e4m3 of value / scale, held to +-448 (NaN stays NaN)
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale)), __NV_SATFINITE,
        __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// two e4m3 as fp16x2
__device__ __forceinline__ uint32_t widen2(uint32_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x), __NV_E4M3);
  return h.x | (static_cast<uint32_t>(h.y) << 16);
}
// larger and smaller of two pairs of fp16 (F16) or bf16; NaN loses to any number
template <bool F16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t c;
  if constexpr (F16) asm("max.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  else asm("max.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}
template <bool F16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t c;
  if constexpr (F16) asm("min.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  else asm("min.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}
// values that such a pair stands for
template <bool F16>
__device__ __forceinline__ float2 value2(uint32_t x, float scale) {
  if constexpr (F16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
    return make_float2(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
  } else {
    return bf16x2_to_float2(x);
  }
}

// What a sequence appends: false (and the status word) where it is out of range.
__device__ __forceinline__ bool new_tokens(const AppendParams& p, int b, int& start, int& count,
                                           int& base) {
  start = p.c.lens[b];
  base = 0;
  if (p.cu_new) {
    base = p.cu_new[b];
    count = p.cu_new[b + 1] - base;
  } else {
    count = p.n_new ? p.n_new[b] : p.n_tokens;
  }
  bool good = start >= 0 && base >= 0 && count >= 0 && count <= p.max_new &&
              static_cast<int64_t>(base) + count <= p.n_tokens;
  if (p.granted) {  // of its tokens, the first so many
    const int given = p.granted[b];
    good = good && given >= 0 && given <= count;
    count = given;
  }
  const int64_t end = static_cast<int64_t>(start) + count;
  return good && end <= (static_cast<int64_t>(p.c.max_pages) << p.c.log2_page) &&
         (p.rot_dim == 0 || count == 0 || end <= p.rope_len);
}

// Rotates two pieces of 8 channels: (lo[i], hi[i]) are pairs, or each piece holds 4 pairs of its own.
// cs: cosine and sine of the 8 pairs.
__device__ __forceinline__ void rotate16(float (&lo)[8], float (&hi)[8], const float2 (&cs)[8], bool interleaved) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& x = interleaved ? (i < 4 ? lo[2 * (i & 3)] : hi[2 * (i & 3)]) : lo[i];
    float& y = interleaved ? (i < 4 ? lo[2 * (i & 3) + 1] : hi[2 * (i & 3) + 1]) : hi[i];
    const float a = x, b = y;
    x = __fsub_rn(__fmul_rn(a, cs[i].x), __fmul_rn(b, cs[i].y));
    y = __fadd_rn(__fmul_rn(b, cs[i].x), __fmul_rn(a, cs[i].y));
  }
}

// Channels of a lane's two pieces of 8: partners of a rotation for the first `pairs` lanes of a row, then as far apart as the
// lanes are many, so that what the lanes read or write at once lies side by side (neighbouring pieces instead took 200 us for
// 42,000 tokens without rotation, int8, 158 as it is).
__device__ __forceinline__ int first_piece(int j, int pairs) { return 8 * (j < pairs ? j : j + pairs); }
template <int PER>
__device__ __forceinline__ int second_piece(int j, int pairs) { return 8 * (j < pairs ? j + pairs : j + PER); }

struct Token {
  int seq, place, pos;  // sequence (-1: none), number among its new tokens, position
  int page;             // -1: outside the pool
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory"); }

// Cosines and sines of a thread's 8 pairs from the table's row of a position.
template <bool INTER>
__device__ __forceinline__ void load_turn(const float* rope, int64_t at, int j, int pairs, float2 (&cs)[8]) {
  const float4* row = reinterpret_cast<const float4*>(rope + at);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const float4 f = __ldg(row + (INTER ? (x < 2 ? 2 * j + x : 2 * (j + pairs) + x - 2) : 4 * j + x));
    cs[2 * x] = make_float2(f.x, f.y);
    cs[2 * x + 1] = make_float2(f.z, f.w);
  }
}
template <bool INTER>
__device__ __forceinline__ void rotate_pieces(uint4& w0, uint4& w1, const float2 (&cs)[8]) {
  float lo[8], hi[8];
  unpack8(w0, lo);
  unpack8(w1, hi);
  rotate16(lo, hi, cs, INTER);
  w0 = pack8(lo);
  w1 = pack8(hi);
}

// Sequence and page (of those that it adds to; or, with 2^log2_unit the tokens of a block, block) number `item` of all
// that the call touches; false where there are fewer.  SCAN: items are dealt out without gaps, by a scan over the sequences, 256 at a time, in which
// the whole block takes part; else a sequence has `segs` of them, and those it does not need end at once.
template <bool SCAN>
__device__ __forceinline__ bool find_page(const AppendParams& p, int item, int segs, int log2_unit, int& b, int& seg) {
  if constexpr (!SCAN) {
    b = item / segs;
    seg = item - b * segs;
    return true;
  }
  __shared__ int sums[kThreads / 32], found[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  if (p.c.B <= 64) {  // two steps of a warp at most: every warp for itself, without the block's barriers
    for (int b0 = 0, before = 0; b0 < p.c.B; b0 += 32) {
      int start, count, base, pages = 0;
      if (b0 + lane < p.c.B && new_tokens(p, b0 + lane, start, count, base) && count > 0)
        pages = ((start + count - 1) >> log2_unit) - (start >> log2_unit) + 1;
      int sum = pages;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += x;
      }
      sum += before;
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, item >= sum - pages && item < sum);
      if (hit) {
        b = b0 + __ffs(hit) - 1;
        seg = item - __shfl_sync(0xFFFFFFFFu, sum - pages, __ffs(hit) - 1);
        return true;
      }
      before = __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    return false;
  }
  if (tid == 0) found[0] = -1;
  for (int b0 = 0, before = 0; b0 < p.c.B && before <= item; b0 += kThreads) {
    int start, count, base, pages = 0;
    if (b0 + tid < p.c.B && new_tokens(p, b0 + tid, start, count, base) && count > 0)
      pages = ((start + count - 1) >> log2_unit) - (start >> log2_unit) + 1;
    int sum = pages;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += x;
    }
    __syncthreads();  // the sums before have been read
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    sum += before;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) sum += sums[w];
      before += sums[w];
    }
    if (item >= sum - pages && item < sum) {
      found[0] = b0 + tid;
      found[1] = item - (sum - pages);
    }
  }
  __syncthreads();
  b = found[0];
  seg = found[1];
  return b >= 0;
}

// A page's summary from each lane's largest and smallest of its 16 channels, as stored (fp16 or bf16 pairs, times scale).
// Lanes that hold the same channels halve them among themselves at every step, so that in the end each has 4 (or 2) of
// the row's channels to itself, and the rest of the work is spread over the warp.
template <int D, bool F16>
__device__ __forceinline__ void write_summary(const AppendParams& p, int64_t at, uint32_t (&high)[8], uint32_t (&low)[8],
                                              float scale, int c0, int c1, int lane) {
  constexpr int kPer = D / 16;
  int first = 0;  // of the pairs that are the lane's
  int n = 8;
#pragma unroll
  for (int d = 16; d >= kPer; d >>= 1) {
    n >>= 1;
    const bool upper = lane & d;
    first += upper ? n : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= n) break;
      const uint32_t h = __shfl_xor_sync(0xFFFFFFFFu, upper ? high[i] : high[i + n], d);
      const uint32_t l = __shfl_xor_sync(0xFFFFFFFFu, upper ? low[i] : low[i + n], d);
      high[i] = max2<F16>(upper ? high[i + n] : high[i], h);
      low[i] = min2<F16>(upper ? low[i + n] : low[i], l);
    }
  }
  constexpr int kPairs = kPer / 4;  // 2 of d = 128, 1 of 64
  float a = 0.f;
  float2 most[kPairs], least[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    most[i] = value2<F16>(high[i], scale);
    least[i] = value2<F16>(low[i], scale);
    a = fmaxf(a, fmaxf(fmaxf(fabsf(most[i].x), fabsf(most[i].y)), fmaxf(fabsf(least[i].x), fabsf(least[i].y))));
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, d));
  const int e = scale_exponent(a);
  const float inv = pow2_bits(-e);
  uint32_t up = 0, down = 0;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const float m[2] = {most[i].x, most[i].y}, l[2] = {least[i].x, least[i].y};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int u = static_cast<int>(fminf(fmaxf(ceilf(m[x] * inv), -127.f), 127.f));
      const int v = static_cast<int>(fminf(fmaxf(floorf(l[x] * inv), -127.f), 127.f));
      up |= static_cast<uint32_t>(u & 0xFF) << (8 * (2 * i + x));
      down |= static_cast<uint32_t>(v & 0xFF) << (8 * (2 * i + x));
    }
  }
  int8_t* to = p.c.summary + at * 2 * D + (first < 4 ? c0 : c1) + 2 * (first & 3);
  if constexpr (kPairs == 2) {
    *reinterpret_cast<uint32_t*>(to) = up;
    *reinterpret_cast<uint32_t*>(to + D) = down;
  } else {
    *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(up);
    *reinterpret_cast<uint16_t*>(to + D) = static_cast<uint16_t>(down);
  }
  if (lane == 0) p.c.summary_scale[at] = pow2_bits(e);
}

// A block's share of the second role.
template <int D, bool E4M3, bool INTER, bool SCAN>
__device__ __forceinline__ void store_keys_by_page(const AppendParams& p, int segs, uint4* ring) {
  constexpr int kPer = D / 16;       // threads of a row
  constexpr int kRows = 32 / kPer;   // rows of a step
  constexpr int kItem = E4M3 ? 1 : 2;
  const int tid = threadIdx.x, lane = tid & 31, P = 1 << p.c.log2_page;
  const int head_blocks = (p.c.H_kv + kThreads / 32 - 1) / (kThreads / 32);
  const int item = blockIdx.x / head_blocks;
  const int h = (blockIdx.x - item * head_blocks) * (kThreads / 32) + tid / 32;
  int b, seg, start, count, base;
  if (!find_page<SCAN>(p, item, segs, p.c.log2_page, b, seg)) return;
  if (!new_tokens(p, b, start, count, base) || h >= p.c.H_kv) return;
  const int place = (start >> p.c.log2_page) + seg, first = place << p.c.log2_page;
  const int lo = max(start, first) - first, hi = min(start + count, first + P) - first;  // new rows of the page
  if (lo >= hi) return;
  const int page = p.c.table[static_cast<int64_t>(b) * p.c.max_pages + place];
  const bool paged = static_cast<unsigned>(page) < static_cast<unsigned>(p.c.num_pages);
  if (!paged && h == 0 && lane == 0) set_status(p.c.status, kDevBadMeta, b);
  const int j = lane % kPer, sub = lane / kPer, pairs = p.rot_dim >> 4;
  const bool turns = j < pairs;
  const int c0 = first_piece(j, pairs), c1 = second_piece<kPer>(j, pairs);
  const __nv_bfloat16* src = p.k + h * p.ks.head + (p.cu_new ? base * p.ks.token : b * p.ks.seq) +
                             (first - start) * p.ks.token;
  char* pool = p.c.k + (paged ? page : 0) * p.c.k_page_bytes + (static_cast<int64_t>(h) << p.c.log2_page) * (D * kItem);
  const float scale = E4M3 ? p.c.k_scale[h] : 1.f;
  const int r0 = paged ? 0 : lo;  // what the page held before counts in its summary
  const uint32_t slots = smem_u32(ring) + tid * 16;
  auto load = [&](int r, int slot) {
    if (r < hi) {
      const uint32_t to0 = slots + 2 * slot * kThreads * 16, to1 = to0 + kThreads * 16;
      if (r >= lo) {
        copy_async<16>(to0, src + r * p.ks.token + c0);
        copy_async<16>(to1, src + r * p.ks.token + c1);
      } else {
        copy_async<8 * kItem>(to0, pool + (r * D + c0) * kItem);
        copy_async<8 * kItem>(to1, pool + (r * D + c1) * kItem);
      }
    }
    copies_end();
  };
#pragma unroll
  for (int x = 0; x < kSlots; ++x) load(r0 + x * kRows + sub, x);
  // largest and smallest of channel pairs, as stored (bf16, or e4m3 widened to fp16 and not yet scaled: a
  // positive factor keeps the order)
  uint32_t high[8], low[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    high[i] = E4M3 ? 0xFC00FC00u : 0xFF80FF80u;  // -inf
    low[i] = E4M3 ? 0x7C007C00u : 0x7F807F80u;
  }
  int slot = 0;
#pragma unroll 1
  for (int r = r0 + sub; r - sub < hi; r += kRows) {
    copies_wait();
    uint4 w0 = ring[(2 * slot) * kThreads + tid], w1 = ring[(2 * slot + 1) * kThreads + tid];
    load(r + kSlots * kRows, slot);  // its pieces are in registers by now
    slot = slot + 1 == kSlots ? 0 : slot + 1;
    if (r >= hi) continue;
    if (r >= lo) {
      if (turns) {
        float2 cs[8];
        load_turn<INTER>(p.rope, static_cast<int64_t>(first + r) * p.rot_dim, j, pairs, cs);
        rotate_pieces<INTER>(w0, w1, cs);
      }
      if (p.k_out) {
        __nv_bfloat16* to = p.k_out + h * p.kos.head + (p.cu_new ? base * p.kos.token : b * p.kos.seq) +
                            (first + r - start) * p.kos.token;
        *reinterpret_cast<uint4*>(to + c0) = w0;
        *reinterpret_cast<uint4*>(to + c1) = w1;
      }
      if (!paged) continue;
      char* to = pool + r * (D * kItem);
      if constexpr (E4M3) {
        float x[8];
        unpack8(w0, x);
        const uint2 u0 = pack8_e4m3(x, scale);
        unpack8(w1, x);
        const uint2 u1 = pack8_e4m3(x, scale);
        *reinterpret_cast<uint2*>(to + c0) = u0;
        *reinterpret_cast<uint2*>(to + c1) = u1;
        w0.x = u0.x;
        w0.y = u0.y;
        w1.x = u1.x;
        w1.y = u1.y;
      } else {
        *reinterpret_cast<uint4*>(to + c0 * 2) = w0;
        *reinterpret_cast<uint4*>(to + c1 * 2) = w1;
      }
    }
    uint32_t x[8];
    if constexpr (E4M3) {
      const uint32_t u[4] = {w0.x, w0.y, w1.x, w1.y};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = widen2(u[i >> 1] >> (16 * (i & 1)));
    } else {
      x[0] = w0.x, x[1] = w0.y, x[2] = w0.z, x[3] = w0.w, x[4] = w1.x, x[5] = w1.y, x[6] = w1.z, x[7] = w1.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      high[i] = max2<E4M3>(high[i], x[i]);
      low[i] = min2<E4M3>(low[i], x[i]);
    }
  }
  if (paged) write_summary<D, E4M3>(p, static_cast<int64_t>(page) * p.c.H_kv + h, high, low, scale, c0, c1, lane);
}

// ---- blocks with a scale each ---------------------------------------------------------------------
// e of the smallest power of two with a <= 127 * 2^e (int8) or a <= 448 * 2^e = 1.75 * 2^(e + 8) (e4m3), held to +-32
template <bool INT8>
__device__ __forceinline__ int needed_exponent(float a) {
  const uint32_t u = __float_as_uint(a), m = u & 0x7FFFFFu;
  const int x = static_cast<int>(u >> 23) - 127, e = INT8 ? x - 6 + (m > 0x7E0000u) : x - 8 + (m > 0x600000u);
  return min(max(e, -kMaxBlockExp), kMaxBlockExp);
}
// 8 fp32 values times a power of two as the cache holds them.  PLAIN: int8, and none is NaN or beyond 127 then: added to
// 1.5 * 2^23, a value is rounded to a whole number, halves to even, whose 8 bits are the sum's last.
template <bool INT8, bool PLAIN>
__device__ __forceinline__ uint2 pack8_block(const float (&x)[8], float times) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (INT8) {
      uint32_t q[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)  // NaN becomes 0
        q[c] = PLAIN ? __float_as_uint(fmaf(x[4 * i + c], times, 12582912.f))
                     : static_cast<uint32_t>(min(max(__float2int_rn(x[4 * i + c] * times), -127), 127));
      w[i] = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
    } else {
      uint32_t q[2];
#pragma unroll
      for (int c = 0; c < 2; ++c)
        q[c] = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2 * c] * times, x[4 * i + 2 * c + 1] * times),
                                        __NV_SATFINITE, __NV_E4M3);
      w[i] = q[0] | (q[1] << 16);
    }
  }
  return make_uint2(w[0], w[1]);
}
template <bool INT8>
__device__ __forceinline__ void unpack8_block(uint2 w, float (&x)[8]) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (INT8) {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[4 * i + c] = static_cast<float>(static_cast<int8_t>(u[i] >> (8 * c)));
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t h = widen2(u[i] >> (16 * c));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        x[4 * i + 2 * c] = f.x;
        x[4 * i + 2 * c + 1] = f.y;
      }
    }
  }
}
// a lane's 16 channels of a token, as stored times the block's scale, into the page's largest and smallest: a stored
// number has at most 8 bits, so bf16 holds it exactly
template <bool INT8>
__device__ __forceinline__ void take_in(uint2 a, uint2 b, float scale, uint32_t (&high)[8], uint32_t (&low)[8]) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float x[8];
    unpack8_block<INT8>(half ? b : a, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t y = pack_bf16x2(x[2 * i] * scale, x[2 * i + 1] * scale);
      high[4 * half + i] = max2<false>(high[4 * half + i], y);
      low[4 * half + i] = min2<false>(low[4 * half + i], y);
    }
  }
}

// Larger magnitudes of two pairs; NaN where one is NaN.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("{\n\t.reg .b32 x;\n\tabs.bf16x2 x, %2;\n\tmax.NaN.bf16x2 %0, %1, x;\n\t}" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

// The second role where blocks have scales: one warp a head's keys or values of one to four blocks, or with summaries of
// all the blocks of a page that the call touches.  A lane's pieces of a block's new rows (16 channels of one of 4 or 8 rows a
// step) come into shared memory that no other thread reads.  They are gone through twice: rotated, with
// their largest magnitude, and once that has settled the scale, stored.  Earlier rows are read only where the scale
// grows (or for the summary).
template <int D, bool INT8, bool INTER, bool SCAN>
__device__ __forceinline__ void store_blocks(const AppendParams& p, int segs, int log2_unit, uint4* ring) {
  constexpr int kPer = D / 16, kRows = 32 / kPer, kSteps = kBlockTokens / kRows;
  static_assert(kSteps <= kSlots, "a block's pieces fit the ring");
  const int tid = threadIdx.x, lane = tid & 31, P = 1 << p.c.log2_page;
  const bool whole_pages = p.c.summary != nullptr;
  const int head_blocks = (2 * p.c.H_kv + kThreads / 32 - 1) / (kThreads / 32);
  const int item = blockIdx.x / head_blocks;
  const int hh = (blockIdx.x - item * head_blocks) * (kThreads / 32) + tid / 32;
  int b, seg, start, count, base;
  if (!find_page<SCAN>(p, item, segs, log2_unit, b, seg)) return;
  if (!new_tokens(p, b, start, count, base) || hh >= 2 * p.c.H_kv) return;
  const bool is_v = hh >= p.c.H_kv;
  const int h = is_v ? hh - p.c.H_kv : hh;
  const int first = ((start >> log2_unit) + seg) << log2_unit;  // positions from here on
  const int lo = max(start, first), hi = min(start + count, first + (1 << log2_unit));
  if (lo >= hi) return;
  const int j = lane % kPer, sub = lane / kPer, pairs = is_v ? 0 : p.rot_dim >> 4;
  const bool turns = j < pairs;
  const int c0 = first_piece(j, pairs), c1 = second_piece<kPer>(j, pairs);
  const Strides& st = is_v ? p.vs : p.ks;
  const __nv_bfloat16* src = (is_v ? p.v : p.k) + h * st.head + (p.cu_new ? base * st.token : b * st.seq);
  const uint32_t slots = smem_u32(ring) + tid * 16;
  auto load_new = [&](int pos, int s) {
    if (pos >= lo && pos < hi) {
      const __nv_bfloat16* x = src + static_cast<int64_t>(pos - start) * st.token;
      copy_async<16>(slots + (2 * s) * kThreads * 16, x + c0);
      copy_async<16>(slots + (2 * s + 1) * kThreads * 16, x + c1);
    }
  };
#pragma unroll
  for (int s = 0; s < kSteps; ++s) load_new((lo & ~15) + s * kRows + sub, s);  // while their page is looked up
  // a block's rows of the rotation's table, into the cache that the heads' warps share
  const int log2_lines = p.rot_dim > 64 ? 2 : p.rot_dim > 32 ? 1 : 0;  // of 128 bytes, of a row
  auto warm = [&](int f) {
#pragma unroll
    for (int x = lane; x < 64; x += 32) {
      const int pos = f + (x >> log2_lines), c = (x & ((1 << log2_lines) - 1)) * 32;
      if (!is_v && x >> log2_lines < kBlockTokens && pos >= lo && pos < hi && c < p.rot_dim)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.rope + static_cast<int64_t>(pos) * p.rot_dim + c));
    }
  };
  const bool many = hi - lo >= kBlockTokens;
  if (many) warm(lo & ~15);
  const int page = p.c.table[static_cast<int64_t>(b) * p.c.max_pages + (first >> p.c.log2_page)];
  const bool paged = static_cast<unsigned>(page) < static_cast<unsigned>(p.c.num_pages);
  if (!paged && hh == 0 && lane == 0) set_status(p.c.status, kDevBadMeta, b);
  const int64_t at = static_cast<int64_t>(paged ? page : 0) * p.c.H_kv + h;
  char* pool = (is_v ? p.c.v + (paged ? page : 0) * p.c.v_page_bytes : p.c.k + (paged ? page : 0) * p.c.k_page_bytes) +
               (static_cast<int64_t>(h) << p.c.log2_page) * D;
  float* scales = const_cast<float*>(is_v ? p.c.v_scale : p.c.k_scale) + (at << (p.c.log2_page - 4));
  const bool sums = whole_pages && !is_v && paged;
  uint32_t high[8], low[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    high[i] = 0xFF80FF80u;  // -inf
    low[i] = 0x7F807F80u;
  }
  if (sums)  // blocks that the call leaves as they are count in the summary
#pragma unroll 4
    for (int pos = first + sub; pos < (lo & ~15); pos += kRows) {
      const int row = pos & (P - 1);
      const char* from = pool + row * D;
      take_in<INT8>(*reinterpret_cast<const uint2*>(from + c0), *reinterpret_cast<const uint2*>(from + c1),
                    pow2_bits(block_exponent(__float_as_uint(scales[row >> 4]))), high, low);
    }
#pragma unroll 1
  for (int f = lo & ~15; f < hi; f += kBlockTokens) {
    const int row = f & (P - 1);
    char* to = pool + row * D;
    const bool carried = lo > f;  // holds earlier tokens
    const int e_old = carried && paged ? block_exponent(__float_as_uint(scales[row >> 4])) : -kMaxBlockExp;
    if (many) warm(f + kBlockTokens);
    asm volatile("cp.async.wait_all;" ::: "memory");
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int pos = f + s * kRows + sub;
      if (pos < lo || pos >= hi) continue;
      uint4 w0 = ring[(2 * s) * kThreads + tid], w1 = ring[(2 * s + 1) * kThreads + tid];
      if (turns) {
        float2 cs[8];
        load_turn<INTER>(p.rope, static_cast<int64_t>(pos) * p.rot_dim, j, pairs, cs);
        rotate_pieces<INTER>(w0, w1, cs);
        ring[(2 * s) * kThreads + tid] = w0;
        ring[(2 * s + 1) * kThreads + tid] = w1;
      }
      if (p.k_out && !is_v) {
        __nv_bfloat16* out = p.k_out + h * p.kos.head + (p.cu_new ? base * p.kos.token : b * p.kos.seq) +
                             static_cast<int64_t>(pos - start) * p.kos.token;
        *reinterpret_cast<uint4*>(out + c0) = w0;
        *reinterpret_cast<uint4*>(out + c1) = w1;
      }
      const uint32_t u[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max_abs_bf16x2(top, u[i]);
    }
    if (!paged) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) load_new(f + kBlockTokens + s * kRows + sub, s);
      continue;
    }
    top = max_abs_bf16x2(top, top >> 16);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) top = max_abs_bf16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    float a = __uint_as_float(top << 16);
    const bool plain = a <= (INT8 ? 127.f : 448.f) * 4294967296.f;
    if (!(a <= INFINITY)) {  // some are NaN: passed over
      top = 0;
#pragma unroll 1
      for (int s = 0; s < kSteps; ++s) {
        const int pos = f + s * kRows + sub;
        if (pos < lo || pos >= hi) continue;
        const uint4 w0 = ring[(2 * s) * kThreads + tid], w1 = ring[(2 * s + 1) * kThreads + tid];
        const uint32_t u[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max2<false>(top, u[i] & 0x7FFF7FFFu);
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) top = max2<false>(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      const float2 tops = bf16x2_to_float2(top);
      a = fmaxf(tops.x, tops.y);
    }
    const int e = max(e_old, needed_exponent<INT8>(a));
    const float scale = pow2_bits(e), inv = pow2_bits(-e), fade = pow2_bits(e_old - e);
    // new rows; the next block's pieces are asked for once these are in registers
    auto store_new = [&](int s, auto is_plain, auto in_sums) {
      const int pos = f + s * kRows + sub;
      if (pos >= lo && pos < hi) {
        uint2* out = reinterpret_cast<uint2*>(to + (s * kRows + sub) * D);
        float x[8];
        unpack8(ring[(2 * s) * kThreads + tid], x);
        const uint2 u0 = pack8_block<INT8, is_plain.value>(x, inv);
        unpack8(ring[(2 * s + 1) * kThreads + tid], x);
        const uint2 u1 = pack8_block<INT8, is_plain.value>(x, inv);
        out[c0 >> 3] = u0;
        out[c1 >> 3] = u1;
        if constexpr (in_sums.value) take_in<INT8>(u0, u1, scale, high, low);
      }
      load_new(pos + kBlockTokens, s);
    };
    if ((plain || !INT8) && !sums) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) store_new(s, std::true_type(), std::false_type());
    } else if (plain || !INT8) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) store_new(s, std::true_type(), std::true_type());
    } else {
#pragma unroll 1
      for (int s = 0; s < kSteps; ++s) store_new(s, std::false_type(), std::true_type());
    }
    if (carried && (e > e_old || sums)) {  // earlier rows
      uint2 u[kSteps][2];
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint2* from = reinterpret_cast<const uint2*>(to + (s * kRows + sub) * D);
        const bool in = f + s * kRows + sub < lo;
        u[s][0] = in ? from[c0 >> 3] : make_uint2(0, 0);
        u[s][1] = in ? from[c1 >> 3] : make_uint2(0, 0);
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (f + s * kRows + sub >= lo) continue;
        uint2* out = reinterpret_cast<uint2*>(to + (s * kRows + sub) * D);
        if (e > e_old) {
          float x[8];
          unpack8_block<INT8>(u[s][0], x);
          out[c0 >> 3] = u[s][0] = pack8_block<INT8, true>(x, fade);
          unpack8_block<INT8>(u[s][1], x);
          out[c1 >> 3] = u[s][1] = pack8_block<INT8, true>(x, fade);
        }
        if (sums) take_in<INT8>(u[s][0], u[s][1], scale, high, low);
      }
    }
    if (lane == 0) scales[row >> 4] = scale;
  }
  if (sums) write_summary<D, false>(p, at, high, low, 1.f, c0, c1, lane);
}

// Blocks 0 .. page_blocks-1 have the second role.
template <int D, int KIND, bool INTER, bool SCAN>
__global__ void __launch_bounds__(kThreads, 4)
    append_kernel(const AppendParams p, int log2_tokens, int page_blocks, int segs, int log2_unit) {
  constexpr bool E4M3 = KIND == kE4m3, BLOCKS = KIND >= kE4m3Block;
  constexpr int kPer = D / 16;  // threads of a token's head
  constexpr int kItem = KIND == kBf16 ? 2 : 1;
  __shared__ Token tokens[8];
  extern __shared__ __align__(16) uint4 ring[];  // [kSlots][2][kThreads]: a thread's own 16-byte pieces
  let_next_start();
  wait_for_previous();
  if (static_cast<int>(blockIdx.x) < page_blocks) {
    if constexpr (BLOCKS) store_blocks<D, KIND == kInt8Block, INTER, SCAN>(p, segs, log2_unit, ring);
    else store_keys_by_page<D, E4M3, INTER, SCAN>(p, segs, ring);
    return;
  }
  const int block = blockIdx.x - page_blocks;
  // heads in the order queries, keys (unless they go by page), values (unless blocks have scales)
  const int H_k = page_blocks ? 0 : p.c.H_kv, values = p.H_q + H_k;
  const int tid = threadIdx.x, P = 1 << p.c.log2_page, n = 1 << log2_tokens;
  const int j = tid % kPer, tt = (tid / kPer) & (n - 1), h0 = (tid / kPer) >> log2_tokens;
  const int step = kThreads / kPer >> log2_tokens;
  const bool packed = p.cu_new != nullptr;
  const int total = packed ? p.n_tokens : p.c.B * p.max_new;
  const int i0 = block << log2_tokens, i = i0 + tt;
  const int heads = BLOCKS ? p.H_q : values + p.c.H_kv;

  // channels of the thread: pieces of 8
  const int pairs = p.rot_dim >> 4;  // threads that rotate
  const bool turns = j < pairs;
  const int c0 = first_piece(j, pairs), c1 = second_piece<kPer>(j, pairs);

  const int row_seq = packed ? 0 : i / max(p.max_new, 1), row_tok = packed ? i : i - row_seq * p.max_new;
  auto source = [&](int h) -> const __nv_bfloat16* {
    const bool q = h < p.H_q, k = h < values;
    const Strides& s = q ? p.qs : k ? p.ks : p.vs;
    return (q ? p.q : k ? p.k : p.v) + (q ? h : k ? h - p.H_q : h - values) * s.head +
           (packed ? 0 : row_seq * s.seq) + row_tok * s.token;
  };
  const uint32_t slots = smem_u32(ring) + tid * 16;
  auto load = [&](int h, int slot) {
    if (h < heads && i < total) {
      const __nv_bfloat16* s = source(h);
      copy_async<16>(slots + (2 * slot) * kThreads * 16, s + c0);
      copy_async<16>(slots + (2 * slot + 1) * kThreads * 16, s + c1);
    }
    copies_end();
  };
#pragma unroll
  for (int x = 0; x < kSlots; ++x) load(h0 + x * step, x);

  // the tokens' sequences; the first block also writes the new lengths and reports bad sequences
  if (tid < n) tokens[tid].seq = -1;
  __syncthreads();
  const bool first = block == 0;
  if (packed || first) {
    for (int b = tid; b < p.c.B; b += kThreads) {
      int start, count, base;
      const bool good = new_tokens(p, b, start, count, base);
      if (first) {
        if (!good) set_status(p.c.status, kDevBadMeta, b);
        if (p.new_lens) p.new_lens[b] = good ? start + count : start;
      }
      if (packed && good)
        for (int x = max(base, i0); x < min(base + count, i0 + n); ++x) {
          tokens[x - i0].seq = b;
          tokens[x - i0].place = x - base;
          tokens[x - i0].pos = start + x - base;
        }
    }
  }
  if (packed) __syncthreads();
  if (tid < n) {
    Token& t = tokens[tid];
    if (!packed && i0 + tid < total) {
      const int b = (i0 + tid) / p.max_new, place = i0 + tid - b * p.max_new;
      int start, count, base;
      if (new_tokens(p, b, start, count, base) && place < count) {
        t.seq = b;
        t.place = place;
        t.pos = start + place;
      }
    }
    if (!BLOCKS && t.seq >= 0) {
      t.page = p.c.table[static_cast<int64_t>(t.seq) * p.c.max_pages + (t.pos >> p.c.log2_page)];
      if (static_cast<unsigned>(t.page) >= static_cast<unsigned>(p.c.num_pages)) {
        set_status(p.c.status, kDevBadMeta, t.seq);
        t.page = -1;
      }
    }
  }
  __syncthreads();
  const Token t = tokens[tt];
  if (t.seq < 0) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }

  float2 cs[8];
  if (turns) load_turn<INTER>(p.rope, static_cast<int64_t>(t.pos) * p.rot_dim, j, pairs, cs);
  int slot = 0;
#pragma unroll 1
  for (int head = h0; head < heads; head += step) {
    copies_wait();
    uint4 out0 = ring[(2 * slot) * kThreads + tid], out1 = ring[(2 * slot + 1) * kThreads + tid];
    load(head + kSlots * step, slot);  // its pieces are in registers by now
    slot = slot + 1 == kSlots ? 0 : slot + 1;
    const bool is_q = head < p.H_q, is_v = head >= values;
    const int hh = is_q ? head : is_v ? head - values : head - p.H_q;
    if (turns && !is_v) rotate_pieces<INTER>(out0, out1, cs);
    __nv_bfloat16* to = is_q ? p.q_out : is_v ? nullptr : p.k_out;
    if (to) {
      const Strides& s = is_q ? p.qos : p.kos;
      to += hh * s.head + (packed ? 0 : row_seq * s.seq) + row_tok * s.token;
      *reinterpret_cast<uint4*>(to + c0) = out0;
      *reinterpret_cast<uint4*>(to + c1) = out1;
    }
    if (BLOCKS || is_q || t.page < 0) continue;
    char* row = (is_v ? p.c.v + t.page * p.c.v_page_bytes : p.c.k + t.page * p.c.k_page_bytes) +
                ((static_cast<int64_t>(hh) << p.c.log2_page) + (t.pos & (P - 1))) * (D * kItem);
    if constexpr (E4M3) {
      const float scale = __ldg((is_v ? p.c.v_scale : p.c.k_scale) + hh);
      float x[8];
      unpack8(out0, x);
      *reinterpret_cast<uint2*>(row + c0) = pack8_e4m3(x, scale);
      unpack8(out1, x);
      *reinterpret_cast<uint2*>(row + c1) = pack8_e4m3(x, scale);
    } else {
      *reinterpret_cast<uint4*>(row + c0 * 2) = out0;
      *reinterpret_cast<uint4*>(row + c1 * 2) = out1;
    }
  }
}

// Whether blocks of the grid go by page (for the summaries) or by block of tokens, and how many tokens that is.
bool has_scaled_blocks(const AppendParams& p) { return p.c.kind >= kE4m3Block; }
bool goes_by_page(const AppendParams& p) { return p.max_new > 0 && (p.c.summary || has_scaled_blocks(p)); }
// Blocks with scales: four a warp, within a page, where every warp of the GPU then still has some (the next block's
// pieces are on their way while one is stored; 42,000 tokens took 197 us with one a warp, 186 with four, before the
// lanes' pieces lay as they do).
int log2_unit(const AppendParams& p) {
  if (p.c.summary) return p.c.log2_page;
  const int64_t tokens = p.cu_new ? p.n_tokens : static_cast<int64_t>(p.c.B) * p.max_new;
  return tokens * 2 * p.c.H_kv < 152 * 32 * 64 ? 4 : p.c.log2_page < 6 ? p.c.log2_page : 6;
}
int head_blocks(const AppendParams& p) {
  const int heads = has_scaled_blocks(p) ? 2 * p.c.H_kv : p.c.H_kv;
  return (heads + kThreads / 32 - 1) / (kThreads / 32);
}

// The most pages (or blocks) a run of max_new tokens can touch.
int append_segments(const AppendParams& p) {
  const int P = 1 << log2_unit(p);
  return (p.max_new + P - 2) / P + 1;
}
// Pages that blocks are launched for, and whether they are dealt out by a scan.  Packed tokens: every page but a
// sequence's first and last takes a page's worth of them, so a batch of a few long prompts among many
// single tokens has far fewer than `segs` for each sequence: 17.8 us instead of 53.6 for 255 single tokens
// and 2048 of one sequence (pages of 16).  A block that finds nothing to do takes about 1 us of one of 608
// places, the scan's barriers about 0.5 us of each block that has work: it pays from a few rounds of idle
// blocks on.
int64_t append_pages(const AppendParams& p, bool& scan) {
  const int64_t all = static_cast<int64_t>(append_segments(p)) * p.c.B;
  const int64_t most = (p.n_tokens >> log2_unit(p)) + 2 * static_cast<int64_t>(p.c.B);
  scan = p.cu_new != nullptr && (all - most) * head_blocks(p) > 4 * 608;
  return (scan ? most : all) * head_blocks(p);
}

template <int D, int KIND>
bool launch(const AppendParams& p, cudaStream_t stream) {
  const bool none = KIND >= kE4m3Block && p.H_q == 0;  // nothing goes by token
  const int total = none ? 0 : p.cu_new ? p.n_tokens : p.c.B * p.max_new;
  bool scan = false;
  const int segs = append_segments(p);
  const int pages = goes_by_page(p) ? static_cast<int>(append_pages(p, scan)) : 0;
  // tokens of a CTA: one while there are few (16 CTAs an SM at most), up to 8 that share the lookups
  int log2_tokens = 0;
  while (log2_tokens < 3 && total >> log2_tokens > 152 * 16) ++log2_tokens;
  const int blocks = total > 0 ? (total + (1 << log2_tokens) - 1) >> log2_tokens : 1;  // new_lens needs one
  auto* kernel = p.interleaved ? (scan ? append_kernel<D, KIND, true, true> : append_kernel<D, KIND, true, false>)
                               : (scan ? append_kernel<D, KIND, false, true> : append_kernel<D, KIND, false, false>);
  return launch_after(kernel, dim3(pages + blocks), kThreads, kSlots * 2 * kThreads * 16, stream, p, log2_tokens, pages,
                      segs, log2_unit(p));
}

}  // namespace

int64_t append_page_blocks(const AppendParams& p) {
  bool scan;
  return goes_by_page(p) ? append_pages(p, scan) : 0;
}

int launch_kv_append(const AppendParams& p, cudaStream_t stream) {
  bool ok = false;
  switch (p.c.kind) {
    case kBf16: ok = p.c.d == 128 ? launch<128, kBf16>(p, stream) : launch<64, kBf16>(p, stream); break;
    case kE4m3: ok = p.c.d == 128 ? launch<128, kE4m3>(p, stream) : launch<64, kE4m3>(p, stream); break;
    case kE4m3Block: ok = p.c.d == 128 ? launch<128, kE4m3Block>(p, stream) : launch<64, kE4m3Block>(p, stream); break;
    case kInt8Block: ok = p.c.d == 128 ? launch<128, kInt8Block>(p, stream) : launch<64, kInt8Block>(p, stream); break;
  }
  return ok ? 0 : -1;
}

}  // namespace cm
