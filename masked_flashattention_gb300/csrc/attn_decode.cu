// Attention of one new token per sequence over a paged key-value cache (cm_attn_decode).
//
// First form: one CTA per (sequence, query head).  Each of its 4 warps takes every fourth key, with
// the row's channels spread over its lanes and a running maximum and sum (one pass over the keys);
// the warps are joined through shared memory.
#include <cuda_fp8.h>

#include "kv_cache.h"
#include "ptx.cuh"

namespace cm {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxIntervals = 8;

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps) decode_kernel(const DecodeParams p) {
  constexpr int N = D / 32;  // channels of a lane
  __shared__ float part[kWarps][D + 2];
  const int b = blockIdx.y, h = blockIdx.x, P = 1 << p.c.log2_page;
  const int g = h / (p.H_q / p.c.H_kv);
  const int warp = threadIdx.x / 32, lane = lane_id();
  int len = p.c.lens[b];
  bool good = len >= 0 && static_cast<int64_t>(len) <= (static_cast<int64_t>(p.c.max_pages) << p.c.log2_page);
  if (p.itab && len > p.S) good = false;
  if (!good) {
    if (threadIdx.x == 0) set_status(p.c.status, kDevBadMeta, b);
    len = 0;
  }
  int ni = 1, st[kMaxIntervals], en[kMaxIntervals];
  st[0] = 0;
  en[0] = len;
  if (p.itab && len > 0) {
    ni = p.NI;
#pragma unroll
    for (int n = 0; n < kMaxIntervals; ++n)
      if (n < ni) {
        const int2 iv = reinterpret_cast<const int2*>(p.itab)[(static_cast<int64_t>(b) * ni + n) * p.S + len - 1];
        st[n] = iv.x;
        en[n] = min(iv.y, len);
      }
  }
  float q[N], o[N], m = -INFINITY, l = 0.f;
  const __nv_bfloat16* qr = p.q + b * p.qs.seq + h * p.qs.head;
  const float ks = E4M3 ? p.c.k_scale[g] : 1.f, vs = E4M3 ? p.c.v_scale[g] : 1.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = __bfloat162float(qr[lane + 32 * i]) * (p.scale * ks);
    o[i] = 0.f;
  }
  const int pages = (len + P - 1) >> p.c.log2_page;
  const int64_t row = static_cast<int64_t>(b) * p.c.H_kv + g;
  const int entries = p.sel ? min(max(p.nsel[row], 0), p.sel_max) : pages;
  int before = -1;
  for (int e = 0; e < entries; ++e) {
    int place = e;
    if (p.sel) {
      place = p.sel[row * p.sel_max + e];
      if (place <= before || place >= pages) {
        if (threadIdx.x == 0) set_status(p.c.status, kDevBadMeta, b);
        continue;
      }
      before = place;
    }
    const int page = p.c.table[static_cast<int64_t>(b) * p.c.max_pages + place];
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.c.num_pages)) {
      if (threadIdx.x == 0) set_status(p.c.status, kDevBadMeta, b);
      continue;
    }
    const int64_t at = (static_cast<int64_t>(g) << p.c.log2_page) * D;
    for (int r = warp; r < P; r += kWarps) {
      const int pos = (place << p.c.log2_page) + r;
      bool seen = false;
#pragma unroll
      for (int n = 0; n < kMaxIntervals; ++n)
        if (n < ni) seen |= pos >= st[n] && pos < en[n];
      if (!seen) continue;
      float k[N], v[N], s = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t x = at + r * D + lane + 32 * i;
        if (E4M3) {
          k[i] = static_cast<float>(reinterpret_cast<const __nv_fp8_e4m3*>(p.c.k + page * p.c.k_page_bytes)[x]);
          v[i] = static_cast<float>(reinterpret_cast<const __nv_fp8_e4m3*>(p.c.v + page * p.c.v_page_bytes)[x]);
        } else {
          k[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.c.k + page * p.c.k_page_bytes)[x]);
          v[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.c.v + page * p.c.v_page_bytes)[x]);
        }
        s += q[i] * k[i];
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
      const float top = fmaxf(m, s), keep = top == -INFINITY ? 0.f : top;
      const float a = __expf(m - keep), w = __expf(s - keep);
      l = l * a + w;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = o[i] * a + w * v[i];
      m = top;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) part[warp][lane + 32 * i] = o[i];
  if (lane == 0) {
    part[warp][D] = m;
    part[warp][D + 1] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part[w][D]);
  const float keep = top == -INFINITY ? 0.f : top;
  for (int w = 0; w < kWarps; ++w) sum += part[w][D + 1] * __expf(part[w][D] - keep);
  for (int c = threadIdx.x; c < D; c += 32 * kWarps) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += part[w][c] * __expf(part[w][D] - keep);
    p.o[b * p.os.seq + h * p.os.head + c] = __float2bfloat16(sum > 0.f ? x * vs / sum : sum == 0.f ? 0.f : sum);
  }
  if (threadIdx.x == 0 && p.lse) p.lse[static_cast<int64_t>(b) * p.H_q + h] = sum == 0.f ? -INFINITY : keep + logf(sum);
}

}  // namespace

size_t decode_workspace_bytes(int, int, int, int) { return 16; }

int launch_attn_decode(const DecodeParams& p, cudaStream_t stream) {
  const dim3 grid(p.H_q, p.c.B);
  if (p.c.d == 128) {
    if (p.c.e4m3) decode_kernel<128, true><<<grid, 32 * kWarps, 0, stream>>>(p);
    else decode_kernel<128, false><<<grid, 32 * kWarps, 0, stream>>>(p);
  } else {
    if (p.c.e4m3) decode_kernel<64, true><<<grid, 32 * kWarps, 0, stream>>>(p);
    else decode_kernel<64, false><<<grid, 32 * kWarps, 0, stream>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace cm
