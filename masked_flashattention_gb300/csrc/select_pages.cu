// Selection of the pages a new token attends to (cm_select_pages): two kernels.
//
// score_kernel.  What bounds it: the summaries, 2 d + 4 bytes a page and key-value head, each read
// once.  A warp takes one key-value head and up to 128 pages of a sequence, 16 at a time: the
// summaries go from memory straight into the A operand of an integer tensor-core product
// (m16n8k32, 16 pages x 8 query heads), 16 bytes a lane; since a dot product takes its channels in any order, the
// lanes' own 16 bytes serve as the k index and nothing is rearranged.  With x split into its positive
// and negative part, the score is one dot product over 2 d channels:
//   sum_c (x_c > 0 ? x_c largest_c : x_c smallest_c) = x+ . largest + x- . smallest.
// Sums are 32-bit integers (at most 2 * 128 * 127^2 < 2^23), and fp32 holds them and their
// scaling by powers of two exactly, so no order of summation shows in the selection.
//
// pick_kernel.  One block a row.  Every thread holds consecutive pages in registers.  A histogram of
// 1024 equal ranges of the row's scores finds the range that the last page taken falls into; only
// the few pages in that range are ranked against each other (a bisection over the score's bits where they
// are many, as with equal scores), and two scans over the block write the pages in order.
#include "kv_cache.h"
#include "ptx.cuh"

namespace cm {
namespace {

constexpr int kScoreWarps = 8;
constexpr int kMaxSteps = 8;   // of 16 pages a warp
constexpr int kBins = 1024;
constexpr int kListed = 1024;  // pages of a range that are ranked by comparing all pairs

__device__ __forceinline__ void mma16832_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int pages_of(const SelectParams& p, int b, bool report) {
  const int len = p.c.lens[b];
  if (len < 0 || static_cast<int64_t>(len) > (static_cast<int64_t>(p.c.max_pages) << p.c.log2_page)) {
    if (report) set_status(p.c.status, kDevBadMeta, b);
    return 0;
  }
  return (len + (1 << p.c.log2_page) - 1) >> p.c.log2_page;
}

// 8-bit queries of up to 8 heads, x+ then x-, into the warp's shared memory; returns the power of two of head
// lane / 4 (each head's 4 lanes hold D / 4 channels each).
template <int D, int PITCH>
__device__ __forceinline__ float quantise(const __nv_bfloat16* q, int64_t head_stride, int heads, int8_t* to,
                                          int lane) {
  const int h = lane >> 2, c0 = (lane & 3) * (D / 4);
  uint4 w[D / 32];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    w[i] = h < heads ? *reinterpret_cast<const uint4*>(q + h * head_stride + c0 + 8 * i) : make_uint4(0, 0, 0, 0);
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xFFFF0000u))));
  }
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  const int f = scale_exponent(top);
  const float inv = pow2_bits(-f);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    uint32_t pos[2] = {0, 0}, neg[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = __uint_as_float(j & 1 ? u[j >> 1] & 0xFFFF0000u : u[j >> 1] << 16);
      const int x = static_cast<int>(fminf(fmaxf(rintf(v * inv), -127.f), 127.f));
      pos[j >> 2] |= static_cast<uint32_t>(max(x, 0)) << (8 * (j & 3));
      neg[j >> 2] |= static_cast<uint32_t>(min(x, 0) & 0xFF) << (8 * (j & 3));
    }
    *reinterpret_cast<uint2*>(to + h * PITCH + c0 + 8 * i) = make_uint2(pos[0], pos[1]);
    *reinterpret_cast<uint2*>(to + h * PITCH + D + c0 + 8 * i) = make_uint2(neg[0], neg[1]);
  }
  return pow2_bits(f);
}

template <int D>
__global__ void __launch_bounds__(32 * kScoreWarps) score_kernel(const SelectParams p, int steps) {
  constexpr int kPitch = 2 * D + 64;  // keeps the fragments' reads free of bank conflicts
  constexpr int kLoads = 2 * D / 64;  // 16-byte loads of a lane for one row
  __shared__ __align__(16) int8_t queries[kScoreWarps][8 * kPitch];
  let_next_start();
  wait_for_previous();
  const int warp = threadIdx.x / 32, lane = lane_id(), t = lane & 3, r = lane >> 2;
  const int b = blockIdx.z, g = blockIdx.y * (blockDim.x / 32) + warp, first = blockIdx.x * 16 * steps;
  if (g >= p.c.H_kv) return;
  const int pages = pages_of(p, b, blockIdx.x == 0 && threadIdx.x == 0);
  if (first >= pages) return;
  const int group = p.H_q / p.c.H_kv, n = min(16 * steps, pages - first);
  // page numbers: page 32 i + lane of the warp's
  int number[kMaxSteps / 2];
#pragma unroll
  for (int i = 0; i < kMaxSteps / 2; ++i) {
    number[i] = -1;
    if (32 * i + lane < n) {
      number[i] = p.c.table[static_cast<int64_t>(b) * p.c.max_pages + first + 32 * i + lane];
      if (static_cast<unsigned>(number[i]) >= static_cast<unsigned>(p.c.num_pages)) {
        set_status(p.c.status, kDevBadMeta, b);
        number[i] = -1;
      }
    }
  }
  float best[kMaxSteps][2];
#pragma unroll
  for (int s = 0; s < kMaxSteps; ++s) best[s][0] = best[s][1] = -INFINITY;
  for (int h0 = 0; h0 < group; h0 += 8) {
    const int heads = min(8, group - h0);
    const __nv_bfloat16* q = p.q + b * p.qs.seq + static_cast<int64_t>(g * group + h0) * p.qs.head;
    __syncwarp();
    const float power = quantise<D, kPitch>(q, p.qs.head, heads, queries[warp], lane);
    __syncwarp();
    uint4 x[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      x[j] = *reinterpret_cast<const uint4*>(&queries[warp][r * kPitch + j * 64 + t * 16]);
    const float power0 = __shfl_sync(0xFFFFFFFFu, power, t * 8), power1 = __shfl_sync(0xFFFFFFFFu, power, t * 8 + 4);
#pragma unroll
    for (int s = 0; s < kMaxSteps; ++s) {
      if (16 * s >= n) break;
      int64_t at[2];
      uint4 y[2][kLoads];
      float scale[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int page = __shfl_sync(0xFFFFFFFFu, number[s / 2], (s & 1) * 16 + i * 8 + r);
        at[i] = page < 0 ? -1 : static_cast<int64_t>(page) * p.c.H_kv + g;
        scale[i] = page < 0 ? 0.f : __ldg(p.c.summary_scale + at[i]);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
          y[i][j] = page < 0 ? make_uint4(0, 0, 0, 0)
                             : __ldg(reinterpret_cast<const uint4*>(p.c.summary + at[i] * 2 * D + j * 64 + t * 16));
      }
      int c[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        mma16832_s8(c, y[0][j].x, y[1][j].x, y[0][j].y, y[1][j].y, x[j].x, x[j].y);
        mma16832_s8(c, y[0][j].z, y[1][j].z, y[0][j].w, y[1][j].w, x[j].z, x[j].w);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (at[i] < 0) continue;
        if (2 * t < heads) best[s][i] = fmaxf(best[s][i], static_cast<float>(c[2 * i]) * power0 * scale[i]);
        if (2 * t + 1 < heads) best[s][i] = fmaxf(best[s][i], static_cast<float>(c[2 * i + 1]) * power1 * scale[i]);
      }
    }
  }
  float* out = p.scores + (static_cast<int64_t>(b) * p.c.H_kv + g) * score_pitch(p.c.max_pages);
#pragma unroll
  for (int s = 0; s < kMaxSteps; ++s)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float v = best[s][i];
      v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
      v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
      const int m = 16 * s + 8 * i + r;
      if (t == 0 && m < n) out[first + m] = v;
    }
}

// Exclusive scan of one number a thread over the block; `total` is the sum.  `sums` [32].
__device__ __forceinline__ int block_scan(int x, int* sums, int& total) {
  const int lane = lane_id(), warp = threadIdx.x / 32, warps = blockDim.x / 32;
  int s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, s, d);
    if (lane >= d) s += y;
  }
  __syncthreads();  // sums of an earlier scan have been read
  if (lane == 31) sums[warp] = s;
  __syncthreads();
  int w = lane < warps ? sums[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, w, d);
    if (lane >= d) w += y;
  }
  total = __shfl_sync(0xFFFFFFFFu, w, 31);
  const int before = __shfl_sync(0xFFFFFFFFu, w, max(warp - 1, 0));
  return s - x + (warp ? before : 0);
}

// Bits of a score in an order-keeping unsigned form.
__device__ __forceinline__ uint32_t key_of(float s) {
  const uint32_t u = __float_as_uint(s);
  return u ^ (u & 0x80000000u ? 0xFFFFFFFFu : 0x80000000u);
}

template <int E>  // pages of a thread
__global__ void __launch_bounds__(1024) pick_kernel(const SelectParams p) {
  __shared__ int bins[kBins + kBins / 32];  // one spare word a 32, for the scan's reads
  __shared__ uint32_t listed[kListed];
  __shared__ int sums[32];
  __shared__ float range[2][32];
  __shared__ int found[4];                  // range, pages needed of it, pages in it
  __shared__ uint32_t limit[2];             // score of the last page taken, pages of that score taken
  let_next_start();
  wait_for_previous();
  const int b = blockIdx.y, tid = threadIdx.x, lane = lane_id(), warp = tid / 32, warps = blockDim.x / 32;
  const int64_t row = static_cast<int64_t>(b) * p.c.H_kv + blockIdx.x;
  const int pages = pages_of(p, b, false), take = min(pages, p.sel_max);
  int32_t* sel = p.sel + row * p.sel_max;
  if (tid == 0) p.nsel[row] = take;
  for (int i = take + tid; i < p.sel_max; i += blockDim.x) sel[i] = -1;
  if (take == pages) {
    for (int i = tid; i < pages; i += blockDim.x) sel[i] = i;
    return;
  }
  const float* from = p.scores + row * score_pitch(p.c.max_pages) + tid * E;
  const int base = tid * E, last = pages - p.keep_last;
  float s[E];
  float low = INFINITY, high = -INFINITY;
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (base + e < pages) v = *reinterpret_cast<const float4*>(from + e);
    s[e] = v.x;
    s[e + 1] = v.y;
    s[e + 2] = v.z;
    s[e + 3] = v.w;
  }
  // pages in the running: neither kept anyway nor behind the end
  auto runs = [&](int e) { return base + e >= p.keep_first && base + e < last; };
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (runs(e) && s[e] > -INFINITY) {
      low = fminf(low, s[e]);
      high = fmaxf(high, s[e]);
    }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, d));
    high = fmaxf(high, __shfl_xor_sync(0xFFFFFFFFu, high, d));
  }
  if (lane == 0) {
    range[0][warp] = low;
    range[1][warp] = high;
  }
  for (int i = tid; i < kBins + kBins / 32; i += blockDim.x) bins[i] = 0;
  __syncthreads();
  low = lane < warps ? range[0][lane] : INFINITY;
  high = lane < warps ? range[1][lane] : -INFINITY;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, d));
    high = fmaxf(high, __shfl_xor_sync(0xFFFFFFFFu, high, d));
  }
  // the map to ranges never falls where the score rises, whatever it rounds to
  const float per = high > low ? (kBins - 1) / (high - low) : 0.f;
  auto bin_of = [&](float x) {
    const float f = (x - low) * per;
    return f > 0.f ? static_cast<int>(fminf(f, kBins - 1)) : 0;  // -inf and 0 * inf too
  };
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (runs(e)) {
      const int i = bin_of(s[e]);
      atomicAdd(&bins[i + (i >> 5)], 1);
    }
  __syncthreads();
  const int need = take - min(p.keep_first, pages) - p.keep_last;  // of those in the running; may be 0
  if (warp == 0) {  // lane 0 has the highest 32 ranges
    int mine = 0;
    for (int i = 0; i < 32; ++i) mine += bins[(31 - lane) * 33 + i];
    int above = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, above, d);
      if (lane >= d) above += y;
    }
    above -= mine;
    if (above < need && above + mine >= need) {
      int i = 31;
      for (; above + bins[(31 - lane) * 33 + i] < need; --i) above += bins[(31 - lane) * 33 + i];
      found[0] = (31 - lane) * 32 + i;
      found[1] = need - above;
      found[2] = bins[(31 - lane) * 33 + i];
    }
  }
  if (tid == 0) {
    found[3] = 0;
    limit[0] = limit[1] = 0;
  }
  __syncthreads();
  const int bin = need > 0 ? found[0] : kBins, want = found[1], many = found[2];
  if (need > 0 && many <= kListed) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (runs(e) && bin_of(s[e]) == bin) listed[atomicAdd(&found[3], 1)] = key_of(s[e]);
    __syncthreads();
    for (int i = tid; i < many; i += blockDim.x) {
      const uint32_t k = listed[i];
      int above = 0, equal = 0;
      for (int j = 0; j < many; ++j) {
        above += listed[j] > k;
        equal += listed[j] == k;
      }
      if (above < want && above + equal >= want) {  // the same numbers from every page of this score
        limit[0] = k;
        limit[1] = want - above;
      }
    }
    __syncthreads();
  } else if (need > 0) {  // the largest key that `want` pages of the range reach
    uint32_t k = 0;
    int above = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t trial = k | (1u << bit);
      int n = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) n += runs(e) && bin_of(s[e]) == bin && key_of(s[e]) >= trial;
      int total;
      block_scan(n, sums, total);
      if (total >= want) k = trial;
    }
    int n = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) n += runs(e) && bin_of(s[e]) == bin && key_of(s[e]) > k;
    block_scan(n, sums, above);
    if (tid == 0) {
      limit[0] = k;
      limit[1] = want - above;
    }
    __syncthreads();
  }
  const uint32_t border = limit[0];
  const int ties = static_cast<int>(limit[1]);
  // in order: the pages of the border's score, then all pages taken
  uint32_t taken = 0, equal = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (base + e >= pages) continue;
    if (!runs(e)) {
      taken |= 1u << e;
      continue;
    }
    const int i = bin_of(s[e]);
    const uint32_t k = key_of(s[e]);
    if (i > bin || (i == bin && k > border)) taken |= 1u << e;
    if (i == bin && k == border) equal |= 1u << e;
  }
  int total;
  int rank = block_scan(__popc(equal), sums, total);
#pragma unroll
  for (int e = 0; e < E; ++e)
    if ((equal >> e) & 1u) {
      if (rank < ties) taken |= 1u << e;
      ++rank;
    }
  int at = block_scan(__popc(taken), sums, total);
#pragma unroll
  for (int e = 0; e < E; ++e)
    if ((taken >> e) & 1u) sel[at++] = base + e;
}

}  // namespace

int launch_select_pages(const SelectParams& p, cudaStream_t stream) {
  const int warps = p.c.H_kv < kScoreWarps ? p.c.H_kv : kScoreWarps;
  // pages of a warp: enough warps to fill the GPU first (152 SMs x 16), then fewer queries to round
  int steps = 1;
  while (steps < kMaxSteps &&
         static_cast<int64_t>(p.c.B) * p.c.H_kv * ((p.c.max_pages + 32 * steps - 1) / (32 * steps)) >= 152 * 16)
    steps *= 2;
  const dim3 grid((p.c.max_pages + 16 * steps - 1) / (16 * steps), (p.c.H_kv + warps - 1) / warps, p.c.B);
  const bool scored = p.c.d == 128 ? launch_after(score_kernel<128>, grid, 32 * warps, 0, stream, p, steps)
                                   : launch_after(score_kernel<64>, grid, 32 * warps, 0, stream, p, steps);
  if (!scored) return -1;
  const dim3 rows(p.c.H_kv, p.c.B);
  const int e = p.c.max_pages <= 8192 ? 8 : 32;
  const int threads = ((p.c.max_pages + e - 1) / e + 31) / 32 * 32;
  return (e == 8 ? launch_after(pick_kernel<8>, rows, threads, 0, stream, p)
                 : launch_after(pick_kernel<32>, rows, threads, 0, stream, p))
             ? 0
             : -1;
}

}  // namespace cm
