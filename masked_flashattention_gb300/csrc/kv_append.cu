// Append of new tokens to a paged key-value cache, with the rotation of queries and keys and the
// page summaries (cm_kv_append): two kernels.
//
// append_kernel.  What bounds it: each new query, key and value is read once and written once, and
// a row of the rotation's table is read per token.  A CTA takes 1 to 8 tokens with all their heads;
// a thread owns 16 channels of a token in two 16-byte pieces, the partners of a rotation among
// them (pieces j and j + rot / 16 of the rotated channels), so nothing crosses lanes, and goes
// through the heads with the token's cosines and sines in registers.  The first heads' loads do not depend on
// where the token goes, so they are in flight while its sequence, position and page are looked up.
//
// summary_kernel.  One warp a (page, head) that the call touched: the largest and smallest of the
// page's stored keys, taken anew, so that a summary never depends on how its tokens arrived and
// needs no atomics.
//
// Numerics: the rotation is fp32 with every product and sum rounded once (no fused
// multiply-add), so that it equals the formula evaluated step by step; one rounding to bf16, and
// for an e4m3 cache one more after the division by the scale (the cache holds what k_out says).
#include <cuda_fp8.h>

#include "kv_cache.h"
#include "ptx.cuh"

namespace cm {
namespace {

constexpr int kThreads = 256;

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

__device__ __forceinline__ void unpack8_e4m3(const uint2& w, float scale, float (&x)[8]) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(u[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * i] = __fmul_rn(f.x, scale);
    x[2 * i + 1] = __fmul_rn(f.y, scale);
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
  const int64_t end = static_cast<int64_t>(start) + count;
  return start >= 0 && base >= 0 && count >= 0 && count <= p.max_new &&
         static_cast<int64_t>(base) + count <= p.n_tokens &&
         end <= (static_cast<int64_t>(p.c.max_pages) << p.c.log2_page) &&
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

struct Token {
  int seq, place, pos;  // sequence (-1: none), number among its new tokens, position
  int page;             // -1: outside the pool
};

template <int D, bool E4M3, bool INTER>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p, int log2_tokens) {
  constexpr int kPer = D / 16;  // threads of a token's head
  constexpr int kAtOnce = 4;    // heads whose loads are in flight
  constexpr int kItem = E4M3 ? 1 : 2;
  __shared__ Token tokens[8];
  let_next_start();
  wait_for_previous();
  const int tid = threadIdx.x, P = 1 << p.c.log2_page, n = 1 << log2_tokens;
  const int j = tid % kPer, tt = (tid / kPer) & (n - 1), h0 = (tid / kPer) >> log2_tokens;
  const int step = kThreads / kPer >> log2_tokens;
  const bool packed = p.cu_new != nullptr;
  const int total = packed ? p.n_tokens : p.c.B * p.max_new;
  const int i0 = blockIdx.x << log2_tokens, i = i0 + tt;
  const int heads = p.H_q + 2 * p.c.H_kv;

  // channels of the thread: pieces of 8
  const int pairs = p.rot_dim >> 4;  // threads that rotate
  const bool turns = j < pairs;
  const int c0 = 8 * (turns ? j : 2 * j), c1 = 8 * (turns ? j + pairs : 2 * j + 1);

  const int row_seq = packed ? 0 : i / max(p.max_new, 1), row_tok = packed ? i : i - row_seq * p.max_new;
  auto source = [&](int h) -> const __nv_bfloat16* {
    const bool q = h < p.H_q, k = h < p.H_q + p.c.H_kv;
    const Strides& s = q ? p.qs : k ? p.ks : p.vs;
    return (q ? p.q : k ? p.k : p.v) + (q ? h : k ? h - p.H_q : h - p.H_q - p.c.H_kv) * s.head +
           (packed ? 0 : row_seq * s.seq) + row_tok * s.token;
  };
  uint4 w[kAtOnce][2];
  auto load = [&](int h) {
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x)
      if (h + x * step < heads && i < total) {
        const __nv_bfloat16* s = source(h + x * step);
        w[x][0] = *reinterpret_cast<const uint4*>(s + c0);
        w[x][1] = *reinterpret_cast<const uint4*>(s + c1);
      }
  };
  load(h0);

  // the tokens' sequences; the first block also writes the new lengths and reports bad sequences
  if (tid < n) tokens[tid].seq = -1;
  __syncthreads();
  const bool first = blockIdx.x == 0;
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
    if (t.seq >= 0) {
      t.page = p.c.table[static_cast<int64_t>(t.seq) * p.c.max_pages + (t.pos >> p.c.log2_page)];
      if (static_cast<unsigned>(t.page) >= static_cast<unsigned>(p.c.num_pages)) {
        set_status(p.c.status, kDevBadMeta, t.seq);
        t.page = -1;
      }
    }
  }
  __syncthreads();
  const Token t = tokens[tt];
  if (t.seq < 0) return;

  float2 cs[8];
  if (turns) {
    const float4* row = reinterpret_cast<const float4*>(p.rope + static_cast<int64_t>(t.pos) * p.rot_dim);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float4 f = __ldg(row + (INTER ? (x < 2 ? 2 * j + x : 2 * (j + pairs) + x - 2) : 4 * j + x));
      cs[2 * x] = make_float2(f.x, f.y);
      cs[2 * x + 1] = make_float2(f.z, f.w);
    }
  }
  for (int h = h0; h < heads; h += kAtOnce * step) {
    if (h != h0) load(h);
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      const int head = h + x * step;
      if (head >= heads) break;
      const bool is_q = head < p.H_q, is_v = head >= p.H_q + p.c.H_kv;
      const int hh = is_q ? head : is_v ? head - p.H_q - p.c.H_kv : head - p.H_q;
      float lo[8], hi[8];
      unpack8(w[x][0], lo);
      unpack8(w[x][1], hi);
      uint4 out0 = w[x][0], out1 = w[x][1];
      if (turns && !is_v) {
        rotate16(lo, hi, cs, INTER);
        out0 = pack8(lo);
        out1 = pack8(hi);
      }
      __nv_bfloat16* to = is_q ? p.q_out : is_v ? nullptr : p.k_out;
      if (to) {
        const Strides& s = is_q ? p.qos : p.kos;
        to += hh * s.head + (packed ? 0 : row_seq * s.seq) + row_tok * s.token;
        *reinterpret_cast<uint4*>(to + c0) = out0;
        *reinterpret_cast<uint4*>(to + c1) = out1;
      }
      if (is_q || t.page < 0) continue;
      char* row = (is_v ? p.c.v + t.page * p.c.v_page_bytes : p.c.k + t.page * p.c.k_page_bytes) +
                  ((static_cast<int64_t>(hh) << p.c.log2_page) + (t.pos & (P - 1))) * (D * kItem);
      if constexpr (E4M3) {
        const float scale = __ldg((is_v ? p.c.v_scale : p.c.k_scale) + hh);
        unpack8(out0, lo);
        unpack8(out1, hi);
        *reinterpret_cast<uint2*>(row + c0) = pack8_e4m3(lo, scale);
        *reinterpret_cast<uint2*>(row + c1) = pack8_e4m3(hi, scale);
      } else {
        *reinterpret_cast<uint4*>(row + c0 * 2) = out0;
        *reinterpret_cast<uint4*>(row + c1 * 2) = out1;
      }
    }
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) summary_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8;       // lanes of a row
  constexpr int kRows = 32 / kLanes;  // rows of a load
  constexpr int kItem = E4M3 ? 1 : 2;
  let_next_start();
  wait_for_previous();
  const int b = blockIdx.z, P = 1 << p.c.log2_page, lane = lane_id();
  const int h = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  int start, count, base;
  if (!new_tokens(p, b, start, count, base) || count == 0 || h >= p.c.H_kv) return;
  const int place = (start >> p.c.log2_page) + blockIdx.y, first = place << p.c.log2_page;
  const int held = min(start + count - first, P);  // tokens of the page
  if (held <= 0) return;
  const int page = p.c.table[static_cast<int64_t>(b) * p.c.max_pages + place];
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.c.num_pages)) return;
  const int c = lane & (kLanes - 1), sub = lane / kLanes;
  const char* rows = p.c.k + page * p.c.k_page_bytes + ((static_cast<int64_t>(h) << p.c.log2_page) * D + c * 8) * kItem;
  const float scale = E4M3 ? p.c.k_scale[h] : 1.f;
  float high[8], low[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    high[i] = -INFINITY;
    low[i] = INFINITY;
  }
  for (int r0 = 0; r0 < held; r0 += 8 * kRows) {
    uint4 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = min(r0 + i * kRows + sub, held - 1);  // the last token again does no harm
      if constexpr (E4M3) {
        const uint2 u = *reinterpret_cast<const uint2*>(rows + r * D);
        w[i] = make_uint4(u.x, u.y, 0, 0);
      } else {
        w[i] = *reinterpret_cast<const uint4*>(rows + r * D * 2);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      if constexpr (E4M3) unpack8_e4m3(make_uint2(w[i].x, w[i].y), scale, x);
      else unpack8(w[i], x);
#pragma unroll
      for (int k = 0; k < 8; ++k) {  // NaN loses to any number
        high[k] = fmaxf(high[k], x[k]);
        low[k] = fminf(low[k], x[k]);
      }
    }
  }
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int d = kLanes; d < 32; d <<= 1) {
      high[i] = fmaxf(high[i], __shfl_xor_sync(0xFFFFFFFFu, high[i], d));
      low[i] = fminf(low[i], __shfl_xor_sync(0xFFFFFFFFu, low[i], d));
    }
    a = fmaxf(a, fmaxf(fabsf(high[i]), fabsf(low[i])));
  }
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, d));
  const int e = scale_exponent(a);
  const float inv = pow2_bits(-e);
  if (lane >= kLanes) return;
  uint32_t up[2] = {0, 0}, down[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int u = static_cast<int>(fminf(fmaxf(ceilf(high[i] * inv), -127.f), 127.f));
    const int l = static_cast<int>(fminf(fmaxf(floorf(low[i] * inv), -127.f), 127.f));
    up[i >> 2] |= static_cast<uint32_t>(u & 0xFF) << (8 * (i & 3));
    down[i >> 2] |= static_cast<uint32_t>(l & 0xFF) << (8 * (i & 3));
  }
  const int64_t at = static_cast<int64_t>(page) * p.c.H_kv + h;
  int8_t* s = p.c.summary + at * 2 * D + c * 8;
  *reinterpret_cast<uint2*>(s) = make_uint2(up[0], up[1]);
  *reinterpret_cast<uint2*>(s + D) = make_uint2(down[0], down[1]);
  if (lane == 0) p.c.summary_scale[at] = pow2_bits(e);
}

template <int D, bool E4M3>
bool launch(const AppendParams& p, cudaStream_t stream) {
  const int total = p.cu_new ? p.n_tokens : p.c.B * p.max_new;
  // tokens of a CTA: one while there are few (16 CTAs an SM at most), up to 8 that share the lookups
  int log2_tokens = 0;
  while (log2_tokens < 3 && total >> log2_tokens > 152 * 16) ++log2_tokens;
  const int blocks = total > 0 ? (total + (1 << log2_tokens) - 1) >> log2_tokens : 1;  // new_lens needs one
  if (!launch_after(p.interleaved ? append_kernel<D, E4M3, true> : append_kernel<D, E4M3, false>, dim3(blocks),
                    kThreads, 0, stream, p, log2_tokens))
    return false;
  if (!p.c.summary || p.max_new == 0) return true;
  const int P = 1 << p.c.log2_page, warps = p.c.H_kv < 8 ? p.c.H_kv : 8;
  // the most pages a run of max_new tokens can touch
  const dim3 grid((p.c.H_kv + warps - 1) / warps, (p.max_new + P - 2) / P + 1, p.c.B);
  return launch_after(summary_kernel<D, E4M3>, grid, 32 * warps, 0, stream, p);
}

}  // namespace

int launch_kv_append(const AppendParams& p, cudaStream_t stream) {
  const bool ok = p.c.d == 128 ? (p.c.e4m3 ? launch<128, true>(p, stream) : launch<128, false>(p, stream))
                               : (p.c.e4m3 ? launch<64, true>(p, stream) : launch<64, false>(p, stream));
  return ok ? 0 : -1;
}

}  // namespace cm
