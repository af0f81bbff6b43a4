// Selection of the pages a new token attends to (cm_select_pages): one kernel, one cluster of blocks a row (a
// sequence's key-value head).
//
// Scores.  What bounds them: the summaries, 2 d + 4 bytes a page and key-value head, each read once.  A
// warp takes 32 pages at a time: the summaries go from memory straight into the A operand of a tensor-core
// product (m16n8k16, 16 pages x 8 query heads), 16 bytes a lane; since a dot product takes its channels
// in any order, the lanes' own 16 bytes serve as the k index and nothing is rearranged.  With x split
// into its positive and negative part, the score is one dot product over 2 d channels:
//   sum_c (x_c > 0 ? x_c largest_c : x_c smallest_c) = x+ . largest + x- . smallest.
// An 8-bit integer product would be its natural form, but this GPU takes 65 cycles for an m16n8k32 of
// that type (8 for an m16n8k16 of fp16, measured), which bound the kernel.  A byte y + 128 behind a
// zero byte is the fp16 number (y + 128) * 2^-24, so one permutation a channel pair makes
// the operand, and 128 * sum x is taken off at the end.  Every partial sum is a whole number below 2^23 (2 * 128 *
// 127 * 255) times 2^-24: fp32 holds it, and the scaling by powers of two, exactly, so no order of summation
// shows in the selection.  A row's blocks take every cs-th 32 pages, so that any length is dealt out
// evenly; one block a row where there are rows enough for the GPU, up to 8 where there are few.
//
// Choice, by a row's first block: every thread holds consecutive pages in registers.  A histogram of 1024
// equal ranges of the row's scores finds the range that the last page taken falls into; only the few
// pages in that range are ranked against each other (a bisection over the score's bits where they are
// many, as with equal scores), and scans over the block write the pages in order.
//
// Measured (d = 128, 8 key-value heads, groups of 4): one sequence of 2048 pages, 8.1 us; 32 of up to 1024, 18 us, of
// which the scores are half (34 MB: 5 us at the copy bandwidth; rows of unequal length, one a block), the
// choice 4.  As two kernels, scores by a warp a head with 16 to 64 pages, then the choice, they took
// 8.7 and 19.7: rounding the queries for so few pages took more instructions than the products.
#include <cuda_fp16.h>
#include <type_traits>

#include "kv_cache.h"
#include "ptx.cuh"

namespace cm {
namespace {

constexpr int kBins = 1024;
constexpr int kListed = 1024;  // pages of a range that are ranked by comparing all pairs

__device__ __forceinline__ void mma16816_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int pages_of(const SelectParams& p, int b, int len, bool report) {
  if (len < 0 || static_cast<int64_t>(len) > (static_cast<int64_t>(p.c.max_pages) << p.c.log2_page)) {
    if (report) set_status(p.c.status, kDevBadMeta, b);
    return 0;
  }
  return (len + (1 << p.c.log2_page) - 1) >> p.c.log2_page;
}

// 8-bit queries of up to 8 heads as fp16, x+ then x-, in shared memory; the powers of two of their scales, and
// 128 * sum x: a warp a head, D / 32 channels a lane.
template <int D, int T>
__device__ __forceinline__ void quantise(const SelectParams& p, const __nv_bfloat16* q, int heads, __half* to,
                                         int pitch, float* power, float* excess) {
  constexpr int kWords = D / 64;  // of two channels
  const int lane = lane_id();
  for (int h = threadIdx.x / 32; h < 8; h += T / 32) {
    uint32_t w[kWords];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      w[i] = h < heads ? *reinterpret_cast<const uint32_t*>(q + h * p.qs.head + lane * 2 * kWords + 2 * i) : 0u;
      top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const int f = scale_exponent(top);
    const float inv = pow2_bits(-f);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const float a = fminf(fmaxf(rintf(__uint_as_float(w[i] << 16) * inv), -127.f), 127.f);
      const float b = fminf(fmaxf(rintf(__uint_as_float(w[i] & 0xFFFF0000u) * inv), -127.f), 127.f);
      __half2* row = reinterpret_cast<__half2*>(to + h * pitch + lane * 2 * kWords) + i;
      row[0] = __floats2half2_rn(fmaxf(a, 0.f), fmaxf(b, 0.f));
      row[D / 2] = __floats2half2_rn(fminf(a, 0.f), fminf(b, 0.f));
      sum += a + b;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if (lane == 0) {
      power[h] = pow2_bits(f);
      excess[h] = 128.f * sum;
    }
  }
}

// Summaries of 16 pages as a lane holds them: 16-byte pieces of pages lane / 4 and 8 further.  Loaded from L2 (ld.cg)
// rather than as read-only data: the append before may still be writing them when this kernel's blocks start.
template <int D>
struct Summaries {
  static constexpr int kLoads = 2 * D / 64;
  uint4 y[2][kLoads];
  float scale[2];  // -1: no such page
  __device__ __forceinline__ void load(const SelectParams& p, int g, int number, int half, int lane) {
    const int t = lane & 3, r = lane >> 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int page = __shfl_sync(0xFFFFFFFFu, number, half * 16 + i * 8 + r);
      const int64_t at = static_cast<int64_t>(page) * p.c.H_kv + g;
      scale[i] = page < 0 ? -1.f : __ldcg(p.c.summary_scale + at);
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        y[i][j] = page < 0 ? make_uint4(0, 0, 0, 0)
                           : __ldcg(reinterpret_cast<const uint4*>(p.c.summary + at * 2 * D + j * 64 + t * 16));
    }
  }
};

// The block's share of a row's scores: 32 pages a warp, every cs-th such piece.
template <int D, int T>
__device__ __forceinline__ void score_pages(const SelectParams& p, int b, int g, int pages, int rank, int cs, int number,
                                            float* out, __half* queries, float* power, float* excess) {
  constexpr int kPitch = 2 * D + 32;  // 64 spare bytes keep the fragments' reads free of bank conflicts
  constexpr int kLoads = Summaries<D>::kLoads;
  const int warp = threadIdx.x / 32, lane = lane_id(), t = lane & 3, r = lane >> 2;
  const int group = p.H_q / p.c.H_kv;
  const int32_t* table = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
  const int piece0 = warp * cs + rank;
#pragma unroll 1
  for (int h0 = 0; h0 < group; h0 += 8) {
    const int heads = min(8, group - h0);
    if (h0 > 0) __syncthreads();
    quantise<D, T>(p, p.q + b * p.qs.seq + static_cast<int64_t>(g * group + h0) * p.qs.head, heads, queries, kPitch, power, excess);
    __syncthreads();
    uint4 x[kLoads][2];  // channels of the lane's 16 bytes
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        x[j][i] = *reinterpret_cast<const uint4*>(queries + r * kPitch + j * 64 + t * 16 + i * 8);
    const float excess0 = excess[2 * t], excess1 = excess[2 * t + 1];
    const float power0 = power[2 * t], power1 = power[2 * t + 1];
    const bool in0 = 2 * t < heads, in1 = 2 * t + 1 < heads;
    const int stride = 32 * (T / 32) * cs;  // pages from a warp's piece to its next
    int next = number;
#pragma unroll 1
    for (int m0 = 32 * piece0; m0 < pages; m0 += stride) {
      int page = m0 + lane < pages ? next : -1;
      if (m0 + lane < pages && static_cast<unsigned>(page) >= static_cast<unsigned>(p.c.num_pages)) {
        set_status(p.c.status, kDevBadMeta, b);
        page = -1;
      }
      Summaries<D> now[2];
      now[0].load(p, g, page, 0, lane);
      now[1].load(p, g, page, 1, lane);
      const int ahead = m0 + stride + lane;
      next = ahead < pages ? table[ahead] : -1;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        auto product = [&](uint32_t y0, uint32_t y1, uint32_t b0, uint32_t b1) {  // 4 channels a lane
          y0 ^= 0x80808080u;
          y1 ^= 0x80808080u;
          mma16816_f16(c, __byte_perm(y0, 0, 0x4140), __byte_perm(y1, 0, 0x4140), __byte_perm(y0, 0, 0x4342),
                       __byte_perm(y1, 0, 0x4342), b0, b1);
        };
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const uint4 y0 = now[half].y[0][j], y1 = now[half].y[1][j];
          product(y0.x, y1.x, x[j][0].x, x[j][0].y);
          product(y0.y, y1.y, x[j][0].z, x[j][0].w);
          product(y0.z, y1.z, x[j][1].x, x[j][1].y);
          product(y0.w, y1.w, x[j][1].z, x[j][1].w);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float scale = now[half].scale[i];
          float v = -INFINITY;
          if (scale >= 0.f) {
            if (in0) v = __fmaf_rn(c[2 * i], 16777216.f, -excess0) * power0 * scale;
            if (in1) v = fmaxf(v, __fmaf_rn(c[2 * i + 1], 16777216.f, -excess1) * power1 * scale);
          }
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
          const int at = m0 + 16 * half + 8 * i + r;
          if (t == 0 && at < pages) {
            if (h0 > 0) v = fmaxf(v, __ldcg(out + at));  // of the group's heads before
            out[at] = v;
          }
        }
      }
    }
  }
}

// Exclusive scan of one number a thread over the block; `total` is the sum.  `sums` [32].
template <int T>
__device__ __forceinline__ int block_scan(int x, int* sums, int& total) {
  const int lane = lane_id(), warp = threadIdx.x / 32;
  constexpr int warps = T / 32;
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

template <int D, int T, int E>  // T threads, E pages of a thread
__global__ void __launch_bounds__(T, 512 / T) select_kernel(const SelectParams p, int cs) {
  __shared__ __align__(16) __half queries[8 * (2 * D + 32)];
  __shared__ float power[8], excess[8];
  __shared__ int bins[kBins + kBins / 32];  // one spare word a 32, for the scan's reads
  __shared__ uint32_t listed[kListed];
  __shared__ int sums[32];
  __shared__ float range[2][32];
  __shared__ int found[4];                  // range, pages needed of it, pages in it
  __shared__ uint32_t limit[3];             // score of the last page taken; pages of it taken, and in all
  let_next_start();
  wait_for_previous();
  const int g = blockIdx.x / cs, rank = blockIdx.x - g * cs, b = blockIdx.y;
  const int tid = threadIdx.x, lane = lane_id(), warp = tid / 32;
  constexpr int warps = T / 32;
  const int64_t row = static_cast<int64_t>(b) * p.c.H_kv + g;
  // the first page numbers are read beside the length, before it is known how many of them count
  const int first = 32 * (warp * cs + rank) + lane;
  const int number = first < p.c.max_pages ? p.c.table[static_cast<int64_t>(b) * p.c.max_pages + first] : -1;
  const int len = p.c.lens[b];
  const int pages = pages_of(p, b, len, g == 0 && rank == 0 && tid == 0);
  const int take = min(pages, p.sel_max), last = pages - p.keep_last;
  int32_t* sel = p.sel + row * p.sel_max;
  if (rank == 0) {
    if (tid == 0) p.nsel[row] = take;
    for (int i = take + tid; i < p.sel_max; i += T) sel[i] = -1;
  }
  if (take == pages) {  // all of them: the same answer in every block of the row
    if (rank == 0)
      for (int i = tid; i < pages; i += T) sel[i] = i;
    return;
  }
  float* scores = p.scores + row * score_pitch(p.c.max_pages);
  score_pages<D, T>(p, b, g, pages, rank, cs, number, scores, queries, power, excess);
  if (cs > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank != 0) return;
  } else {
    __syncthreads();
  }
  const int base = tid * E;
  float s[E];
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (base + e < pages) v = __ldcg(reinterpret_cast<const float4*>(scores + base + e));
    s[e] = v.x;
    s[e + 1] = v.y;
    s[e + 2] = v.z;
    s[e + 3] = v.w;
  }
  float low = INFINITY, high = -INFINITY;
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
  for (int i = tid; i < kBins + kBins / 32; i += T) bins[i] = 0;
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
#pragma unroll
    for (int i = 0; i < 32; ++i) mine += bins[(31 - lane) * 33 + i];
    auto scan = [&](int x) {  // of the lanes up to this one
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
        if (lane >= d) x += y;
      }
      return x;
    };
    const int sum = scan(mine), part = __ffs(__ballot_sync(0xFFFFFFFFu, sum >= need)) - 1;
    const int above = __shfl_sync(0xFFFFFFFFu, sum - mine, max(part, 0));
    const int count = bins[(31 - max(part, 0)) * 33 + 31 - lane];  // lane 0 has the highest range of the 32
    const int upto = above + scan(count), one = __ffs(__ballot_sync(0xFFFFFFFFu, upto >= need)) - 1;
    if (lane == one && part >= 0) {
      found[0] = (31 - part) * 32 + 31 - lane;
      found[1] = need - (upto - count);
      found[2] = count;
    }
  }
  if (tid == 0) {
    found[3] = 0;
    limit[0] = limit[1] = limit[2] = 0;
  }
  __syncthreads();
  const int bin = need > 0 ? found[0] : kBins, want = found[1], many = found[2];
  if (need > 0 && many <= kListed) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (runs(e) && bin_of(s[e]) == bin) listed[atomicAdd(&found[3], 1)] = key_of(s[e]);
    __syncthreads();
    for (int i = tid; i < many; i += T) {
      const uint32_t k = listed[i];
      int above = 0, equal = 0;
      for (int j = 0; j < many; ++j) {
        above += listed[j] > k;
        equal += listed[j] == k;
      }
      if (above < want && above + equal >= want) {  // the same numbers from every page of this score
        limit[0] = k;
        limit[1] = want - above;
        limit[2] = equal;
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
      block_scan<T>(n, sums, total);
      if (total >= want) k = trial;
    }
    int n = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) n += runs(e) && bin_of(s[e]) == bin && key_of(s[e]) > k;
    block_scan<T>(n, sums, above);
    if (tid == 0) {
      limit[0] = k;
      limit[1] = want - above;
      limit[2] = many;  // not counted: at least limit[1]
    }
    __syncthreads();
  }
  const uint32_t border = limit[0];
  const int ties = static_cast<int>(limit[1]);
  // in order: the pages of the border's score, then all pages taken
  using Mask = std::conditional_t<(E > 32), uint64_t, uint32_t>;
  Mask taken = 0, equal = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (base + e >= pages) continue;
    if (!runs(e)) {
      taken |= Mask(1) << e;
      continue;
    }
    const int i = bin_of(s[e]);
    const uint32_t k = key_of(s[e]);
    if (i > bin || (i == bin && k > border)) taken |= Mask(1) << e;
    if (i == bin && k == border) equal |= Mask(1) << e;
  }
  int total;
  if (limit[2] == limit[1]) {
    taken |= equal;
  } else {  // the first of equals
    int rank = block_scan<T>(__popcll(equal), sums, total);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if ((equal >> e) & 1u) {
        if (rank < ties) taken |= Mask(1) << e;
        ++rank;
      }
  }
  int at = block_scan<T>(__popcll(taken), sums, total);
#pragma unroll
  for (int e = 0; e < E; ++e)
    if ((taken >> e) & 1u) sel[at++] = base + e;
}

template <int D, int T, int E>
bool launch(const SelectParams& p, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.c.B) * p.c.H_kv;
  // blocks of a row: as many as leave every block of all rows resident (512 threads an SM), and 32 pages for
  // each of their warps
  int cs = 1;
  while (cs < 8 && rows * 2 * cs <= 152 * (512 / T) && p.c.max_pages > T * cs) cs *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cs;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.c.H_kv * cs, p.c.B);
  cfg.blockDim = dim3(T);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_kernel<D, T, E>, p, cs) == cudaSuccess;
}

template <int D>
bool launch(const SelectParams& p, cudaStream_t stream) {
  if (p.c.max_pages <= 2048) return launch<D, 256, 8>(p, stream);
  if (p.c.max_pages <= 8192) return launch<D, 512, 16>(p, stream);
  return launch<D, 512, 64>(p, stream);  // its scores spill: 9000 pages 27 us, 8192 by the form above 14
}

}  // namespace

int launch_select_pages(const SelectParams& p, cudaStream_t stream) {
  return (p.c.d == 128 ? launch<128>(p, stream) : launch<64>(p, stream)) ? 0 : -1;
}

}  // namespace cm
