// Append of new tokens to a paged key-value cache, with the rotation of queries and keys and the
// page summaries (cm_kv_append).
//
// A token at position p of its sequence goes to row p % P of page table[p / P].  A unit of work is
// one head's rows of one page: the tokens of a sequence that fall into the same page.  A warp holds
// 16 rows of a unit (P / 16 warps a unit, 8 warps a CTA), 8 channels a lane in one 16-byte load,
// all of its rows' loads in flight at once; the partner of a channel half the rotated width away
// comes from another lane by shuffle.  A unit owns its page's summary, so the largest and smallest
// keys need no atomics: they are taken over the page's rows in the warp's registers, then over the
// unit's warps through shared memory.
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

// Rotates the 8 channels [8c, 8c + 8) of a row held by this lane; `row` is the row's table
// entry [rot / 2][2].  Every lane of the warp takes part in the shuffles.
__device__ __forceinline__ void rotate8(float (&x)[8], const float* row, int c, int rot,
                                        bool interleaved, bool active) {
  if (interleaved) {
    if (active && 8 * c < rot) {
      const float4* t = reinterpret_cast<const float4*>(row) + 2 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 f = __ldg(t + i);  // cos, sin of two pairs
        const float a = x[4 * i], b = x[4 * i + 1], e = x[4 * i + 2], g = x[4 * i + 3];
        x[4 * i] = __fsub_rn(__fmul_rn(a, f.x), __fmul_rn(b, f.y));
        x[4 * i + 1] = __fadd_rn(__fmul_rn(b, f.x), __fmul_rn(a, f.y));
        x[4 * i + 2] = __fsub_rn(__fmul_rn(e, f.z), __fmul_rn(g, f.w));
        x[4 * i + 3] = __fadd_rn(__fmul_rn(g, f.z), __fmul_rn(e, f.w));
      }
    }
    return;
  }
  const int half = rot >> 4;  // lanes of one half of the rotated channels
  const bool low = c < half, in = c < 2 * half;
  const int lane = lane_id();
  const int partner = in ? (low ? lane + half : lane - half) : lane;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xFFFFFFFFu, x[i], partner);
  if (active && in) {
    const float4* t = reinterpret_cast<const float4*>(row) + 4 * (low ? c : c - half);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldg(t + i);
      const float p0 = __fmul_rn(x[2 * i], f.x), q0 = __fmul_rn(y[2 * i], f.y);
      const float p1 = __fmul_rn(x[2 * i + 1], f.z), q1 = __fmul_rn(y[2 * i + 1], f.w);
      x[2 * i] = low ? __fsub_rn(p0, q0) : __fadd_rn(p0, q0);
      x[2 * i + 1] = low ? __fsub_rn(p1, q1) : __fadd_rn(p1, q1);
    }
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

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8;       // lanes of a row
  constexpr int kRows = 32 / kLanes;  // rows a warp touches at once
  constexpr int kSteps = 16 / kRows;
  constexpr int kItem = E4M3 ? 1 : 2;
  __shared__ float red[kThreads / 32][2][D];

  let_next_start();
  wait_for_previous();
  const int b = blockIdx.z, P = 1 << p.c.log2_page;
  int start, count, base;
  const bool good = new_tokens(p, b, start, count, base);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    if (!good) set_status(p.c.status, kDevBadMeta, b);
    if (p.new_lens) p.new_lens[b] = good ? start + count : start;
  }
  if (!good) return;
  const int place = (start >> p.c.log2_page) + blockIdx.y;  // page of the sequence
  const int first = place << p.c.log2_page;
  const int lo = max(start, first), hi = min(start + count, first + P);
  if (lo >= hi) return;
  const int page = p.c.table[static_cast<size_t>(b) * p.c.max_pages + place];
  const bool paged = static_cast<unsigned>(page) < static_cast<unsigned>(p.c.num_pages);
  if (!paged && blockIdx.x == 0 && threadIdx.x == 0) set_status(p.c.status, kDevBadMeta, b);

  const int warps = P / 16;  // of a unit
  const int warp = threadIdx.x / 32, lane = lane_id();
  const int chunk = warp & (warps - 1);
  const int head = blockIdx.x * (8 / warps) + warp / warps;  // keys, values, then queries
  const int H_kv = p.c.H_kv;
  const bool is_k = head < H_kv, is_v = !is_k && head < 2 * H_kv;
  const bool is_q = head >= 2 * H_kv && head < 2 * H_kv + p.H_q;
  const int h = is_k ? head : is_v ? head - H_kv : head - 2 * H_kv;
  const int c = lane & (kLanes - 1), sub = lane / kLanes;
  const bool summed = is_k && p.c.summary != nullptr && paged;

  float high[8], low[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    high[i] = -INFINITY;
    low[i] = INFINITY;
  }
  if (is_k || is_v || is_q) {
    const __nv_bfloat16* src = is_k ? p.k : is_v ? p.v : p.q;
    const Strides& ss = is_k ? p.ks : is_v ? p.vs : p.qs;
    src += h * ss.head + (p.cu_new ? base * ss.token : b * ss.seq) + c * 8;
    char* pool = is_k ? p.c.k : p.c.v;
    char* rows = paged && !is_q
                     ? pool + page * (is_k ? p.c.k_page_bytes : p.c.v_page_bytes) +
                           ((static_cast<int64_t>(h) << p.c.log2_page) * D + c * 8) * kItem
                     : nullptr;
    const float scale = E4M3 && !is_q ? (is_k ? p.c.k_scale[h] : p.c.v_scale[h]) : 1.f;
    uint4 w[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int r = chunk * 16 + j * kRows + sub, pos = first + r;
      w[j] = make_uint4(0, 0, 0, 0);
      if (pos >= lo && pos < hi) {
        w[j] = *reinterpret_cast<const uint4*>(src + (pos - start) * ss.token);
      } else if (summed && pos < lo) {  // a token the page held before
        if (E4M3) {
          const uint2 u = *reinterpret_cast<const uint2*>(rows + r * D);
          w[j].x = u.x;
          w[j].y = u.y;
        } else {
          w[j] = *reinterpret_cast<const uint4*>(rows + r * D * 2);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int r = chunk * 16 + j * kRows + sub, pos = first + r;
      const bool active = pos >= lo && pos < hi, held = summed && pos < lo;
      float x[8];
      unpack8(w[j], x);
      if (!is_v && p.rot_dim)
        rotate8(x, p.rope + static_cast<int64_t>(active ? pos : 0) * p.rot_dim, c, p.rot_dim,
                p.interleaved != 0, active);
      if (active) {
        const uint4 out = pack8(x);
        __nv_bfloat16* to = is_q ? p.q_out : is_k ? p.k_out : nullptr;
        if (to) {
          const Strides& os = is_q ? p.qos : p.kos;
          to += h * os.head + (p.cu_new ? base * os.token : b * os.seq) + c * 8;
          *reinterpret_cast<uint4*>(to + (pos - start) * os.token) = out;
        }
        unpack8(out, x);
        if (rows) {
          if (E4M3) {
            const uint2 u = pack8_e4m3(x, scale);
            *reinterpret_cast<uint2*>(rows + r * D) = u;
            if (summed) unpack8_e4m3(u, scale, x);
          } else {
            *reinterpret_cast<uint4*>(rows + r * D * 2) = out;
          }
        }
      } else if (held) {
        if (E4M3) unpack8_e4m3(make_uint2(w[j].x, w[j].y), scale, x);
        else unpack8(w[j], x);
      }
      if (summed && (active || held)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          high[i] = fmaxf(high[i], x[i]);
          low[i] = fminf(low[i], x[i]);
        }
      }
    }
  }
  if (p.c.summary == nullptr) return;
  // rows of the warp, then warps of the unit
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int d = kLanes; d < 32; d <<= 1) {
      high[i] = fmaxf(high[i], __shfl_xor_sync(0xFFFFFFFFu, high[i], d));
      low[i] = fminf(low[i], __shfl_xor_sync(0xFFFFFFFFu, low[i], d));
    }
  if (summed && lane < kLanes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      red[warp][0][c * 8 + i] = high[i];
      red[warp][1][c * 8 + i] = low[i];
    }
  }
  __syncthreads();
  if (!summed || chunk != 0) return;
  for (int o = 1; o < warps; ++o)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      high[i] = fmaxf(high[i], red[warp + o][0][c * 8 + i]);
      low[i] = fminf(low[i], red[warp + o][1][c * 8 + i]);
    }
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fmaxf(fabsf(high[i]), fabsf(low[i])));
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, d));
  const int e = scale_exponent(a);
  const float inv = pow2_bits(-e);
  if (lane < kLanes) {
    uint32_t up[2] = {0, 0}, down[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = static_cast<int>(fminf(fmaxf(ceilf(high[i] * inv), -127.f), 127.f));
      const int l = static_cast<int>(fminf(fmaxf(floorf(low[i] * inv), -127.f), 127.f));
      up[i >> 2] |= static_cast<uint32_t>(u & 0xFF) << (8 * (i & 3));
      down[i >> 2] |= static_cast<uint32_t>(l & 0xFF) << (8 * (i & 3));
    }
    const int64_t at = static_cast<int64_t>(page) * H_kv + h;
    int8_t* s = p.c.summary + at * 2 * D + c * 8;
    *reinterpret_cast<uint2*>(s) = make_uint2(up[0], up[1]);
    *reinterpret_cast<uint2*>(s + D) = make_uint2(down[0], down[1]);
    if (lane == 0) p.c.summary_scale[at] = pow2_bits(e);
  }
}

}  // namespace

int launch_kv_append(const AppendParams& p, cudaStream_t stream) {
  const int P = 1 << p.c.log2_page;
  const int heads = 2 * p.c.H_kv + (p.q ? p.H_q : 0);
  const int units = 128 / P;  // a CTA
  // the most pages a run of max_new tokens can touch (no tokens still write new_lens)
  const int segs = p.max_new > 0 ? (p.max_new + P - 2) / P + 1 : 1;
  const dim3 grid((heads + units - 1) / units, segs, p.c.B);
  const bool ok = p.c.d == 128 ? (p.c.e4m3 ? launch_after(kv_append_kernel<128, true>, grid, kThreads, 0, stream, p)
                                           : launch_after(kv_append_kernel<128, false>, grid, kThreads, 0, stream, p))
                               : (p.c.e4m3 ? launch_after(kv_append_kernel<64, true>, grid, kThreads, 0, stream, p)
                                           : launch_after(kv_append_kernel<64, false>, grid, kThreads, 0, stream, p));
  return ok ? 0 : -1;
}

}  // namespace cm
