// Selection of the pages a new token attends to (cm_select_pages).
//
// First form: one thread scores one page of a (sequence, key-value head) by integer dot products;
// a second kernel ranks every page by counting the pages that come before it.
#include "kv_cache.h"
#include "ptx.cuh"

namespace cm {
namespace {

constexpr int kThreads = 256;

// 8-bit queries of one key-value head's group in shared memory, and the powers of two of their
// scales: x = rint(q / 2^f).
template <int D>
__device__ __forceinline__ void load_queries(const SelectParams& p, int b, int g, int group,
                                             int first, int n, int8_t* x, float* power) {
  const int warp = threadIdx.x / 32, lane = lane_id();
  for (int i = warp; i < n; i += kThreads / 32) {
    const __nv_bfloat16* q = p.q + b * p.qs.seq + (static_cast<int64_t>(g) * group + first + i) * p.qs.head;
    float v[D / 32], a = 0.f;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      v[j] = __bfloat162float(q[lane + 32 * j]);
      a = fmaxf(a, fabsf(v[j]));
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, d));
    const int f = scale_exponent(a);
    const float inv = pow2_bits(-f);
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
      x[i * D + lane + 32 * j] = static_cast<int8_t>(fminf(fmaxf(rintf(v[j] * inv), -127.f), 127.f));
    if (lane == 0) power[i] = pow2_bits(f);
  }
}

__device__ __forceinline__ int pages_of(const SelectParams& p, int b) {
  const int len = p.c.lens[b];
  if (len < 0 || static_cast<int64_t>(len) > (static_cast<int64_t>(p.c.max_pages) << p.c.log2_page)) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(p.c.status, kDevBadMeta, b);
    return 0;
  }
  return (len + (1 << p.c.log2_page) - 1) >> p.c.log2_page;
}

template <int D>
__global__ void __launch_bounds__(kThreads) score_kernel(const SelectParams p) {
  __shared__ int8_t x[16 * D];
  __shared__ float power[16];
  const int b = blockIdx.z, g = blockIdx.y, group = p.H_q / p.c.H_kv;
  const int pages = pages_of(p, b);
  const int n = blockIdx.x * kThreads + threadIdx.x;
  float best = -INFINITY;
  int page = -1;
  if (n < pages) {
    page = p.c.table[static_cast<int64_t>(b) * p.c.max_pages + n];
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.c.num_pages)) {
      set_status(p.c.status, kDevBadMeta, b);
      page = -1;
    }
  }
  const int64_t at = static_cast<int64_t>(page < 0 ? 0 : page) * p.c.H_kv + g;
  for (int first = 0; first < group; first += 16) {
    const int m = min(16, group - first);
    __syncthreads();
    load_queries<D>(p, b, g, group, first, m, x, power);
    __syncthreads();
    if (page < 0) continue;
    const int8_t* s = p.c.summary + at * 2 * D;
    for (int i = 0; i < m; ++i) {
      int sum = 0;
      for (int c = 0; c < D; ++c) {
        const int q = x[i * D + c];
        sum += q * (q > 0 ? s[c] : s[D + c]);
      }
      best = fmaxf(best, static_cast<float>(sum) * power[i] * p.c.summary_scale[at]);
    }
  }
  if (n < pages) {
    if (n < p.keep_first || n >= pages - p.keep_last) best = INFINITY;
    p.scores[(static_cast<int64_t>(b) * p.c.H_kv + g) * p.c.max_pages + n] = best;
  }
}

__global__ void __launch_bounds__(kThreads) pick_kernel(const SelectParams p) {
  const int b = blockIdx.y, g = blockIdx.x;
  const int pages = pages_of(p, b);
  const int64_t row = static_cast<int64_t>(b) * p.c.H_kv + g;
  const float* s = p.scores + row * p.c.max_pages;
  __shared__ int taken;
  int32_t* sel = p.sel + row * p.sel_max;
  if (threadIdx.x == 0) taken = 0;
  __syncthreads();
  for (int n0 = 0; n0 < pages; n0 += kThreads) {
    const int n = n0 + threadIdx.x;
    bool in = false;
    if (n < pages) {
      int ahead = 0;
      for (int m = 0; m < pages; ++m) ahead += s[m] > s[n] || (s[m] == s[n] && m < n);
      in = ahead < p.sel_max;
    }
    // ascending order: one thread after another
    for (int w = 0; w < kThreads / 32; ++w) {
      if (static_cast<int>(threadIdx.x) / 32 == w) {
        const uint32_t all = __ballot_sync(0xFFFFFFFFu, in);
        if (in) sel[taken + __popc(all & ((1u << lane_id()) - 1))] = n;
        __syncwarp();
        if (lane_id() == 0) taken += __popc(all);
      }
      __syncthreads();
    }
  }
  for (int i = taken + threadIdx.x; i < p.sel_max; i += kThreads) sel[i] = -1;
  if (threadIdx.x == 0) p.nsel[row] = taken;
}

}  // namespace

int launch_select_pages(const SelectParams& p, cudaStream_t stream) {
  const dim3 grid((p.c.max_pages + kThreads - 1) / kThreads, p.c.H_kv, p.c.B);
  if (p.c.d == 128) score_kernel<128><<<grid, kThreads, 0, stream>>>(p);
  else score_kernel<64><<<grid, kThreads, 0, stream>>>(p);
  pick_kernel<<<dim3(p.c.H_kv, p.c.B), kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace cm
