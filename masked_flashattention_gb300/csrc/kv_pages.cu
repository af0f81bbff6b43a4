// Pages of a paged key-value cache dealt out on the GPU: page tables and slot maps from request lengths
// (cm_kv_reserve), and pages given back to the pool (cm_kv_release).
//
// What bounds it: a few bytes a sequence, a page and a token, so the time is that of the launch and of a chain of three
// loads (lengths and state, then page numbers out of the list or the table, then the stores).  So it is one launch:
// every block adds up the pages of all sequences for itself (16 bytes a sequence, from L2 for all blocks but the
// first), which gives each sequence its place in the free list without a second kernel and without blocks that wait
// for one another, and then takes its share of the page numbers and slots, a warp a piece of a sequence.  Input and
// output state are separate memory, so no block's reading meets another's writing.  Prefix sums make
// the result the same as that of a loop over the sequences; there are no atomics but the status word's.
#include <cstdint>

#include "kv_cache.h"
#include "ptx.cuh"

namespace cm {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxBlocks = 304;     // two an SM
constexpr int kTokens = 1024;       // slots of a warp's piece (256 bytes a step)
constexpr int kEntries = 256;       // page numbers of a warp's piece (at most 64 pieces a sequence)
constexpr int kShort = -1, kBad = -2;  // instead of a place in the list: too few pages, out of range

__device__ __forceinline__ int first_pages(const PagesParams& p) {  // that hold the sinks
  return static_cast<int>((static_cast<int64_t>(p.sinks) + (1 << p.log2_page) - 1) >> p.log2_page);
}

// What a sequence appends, and the pages it needs for that; false where it is out of range.
struct Request {
  int held, count, base, lo, hi, need;
};
__device__ __forceinline__ bool request(const PagesParams& p, int b, Request& r) {
  const int2 own = p.state[b];
  r.lo = own.x;
  r.hi = own.y;
  r.held = p.lens[b];
  r.base = 0;
  if (p.cu_new) {
    r.base = p.cu_new[b];
    r.count = p.cu_new[b + 1] - r.base;
  } else {
    r.count = p.n_new ? p.n_new[b] : p.n_tokens;
  }
  const int64_t end = static_cast<int64_t>(r.held) + r.count, P = 1LL << p.log2_page;
  const bool good = r.held >= 0 && r.base >= 0 && r.count >= 0 && r.count <= p.max_new &&
                    static_cast<int64_t>(r.base) + r.count <= p.n_tokens && end <= p.max_pages * P && r.lo >= 0 &&
                    r.lo <= r.hi && r.hi <= p.max_pages && r.hi * P >= r.held && r.lo * P <= r.held;
  r.need = good && r.count > 0 ? max(static_cast<int>((end + P - 1) >> p.log2_page), r.hi) : r.hi;
  return good;
}

// What a sequence gives back: the entries [0, early) and [at, to) of its row, and what it owns afterwards.
struct Return {
  int early, at, to;
  int2 left;
};
__device__ __forceinline__ bool give_back(const PagesParams& p, int b, Return& r) {
  const int2 own = p.state[b];
  const int first = first_pages(p), held = p.lens[b], over = p.done ? p.done[b] : 0;
  r.early = 0;
  r.at = r.to = 0;
  r.left = own;
  if (own.x < 0 || own.x > own.y || own.y > p.max_pages) return false;
  r.at = max(own.x, first);
  if (over) {
    r.early = min(first, own.y);
    r.to = own.y;
    r.left = make_int2(0, 0);
  } else if (p.window) {
    r.to = min(own.y, max(held - p.window, 0) >> p.log2_page);
    if (r.to > r.at) r.left.x = r.to;
  }
  r.to = max(r.to, r.at);
  return true;
}

// Dynamic shared memory: places[B], first the pages of each sequence, then its place in the list.
template <bool RELEASE>
__global__ void __launch_bounds__(kThreads) pages_kernel(const PagesParams p, int pieces) {
  extern __shared__ int places[];
  __shared__ int64_t warp_sum[kWarps];
  __shared__ int used;  // pages taken, or given back
  __shared__ int fall;  // first sequence behind which cu_new falls
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, P = 1 << p.log2_page;
  let_next_start();
  wait_for_previous();
  if (tid == 0) {
    used = 0;
    fall = p.B;
  }
  __syncthreads();
  const int listed = p.state[p.B].x, free = min(max(listed, 0), p.num_pages);
  if (blockIdx.x == 0 && tid == 0 && listed != free) set_status(p.status, kDevBadMeta, 0xFFFF);
#pragma unroll 4
  for (int b = tid; b < p.B; b += kThreads) {
    int n;
    bool good;
    if constexpr (RELEASE) {
      Return r;
      good = give_back(p, b, r);
      n = r.early + r.to - r.at;
    } else {
      Request r;
      good = request(p, b, r);
      n = r.need - r.hi;
      if (p.cu_new && r.count < 0) atomicMin(&fall, b);
    }
    if (!good && blockIdx.x == 0) set_status(p.status, kDevBadMeta, b);
    places[b] = good ? n : kBad;
  }
  __syncthreads();
  // prefix sums: a run of sequences a thread, then over the threads
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += b > fall ? 0 : max(places[b], 0);
  int64_t sum = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, sum, d);
    if (lane >= d) sum += x;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) sum += warp_sum[w];
  int64_t at = sum - mine;
  int most = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = places[b];
    if (n < 0) continue;
    if (!RELEASE && b > fall) {  // its tokens may be another's too
      places[b] = kBad;
      continue;
    }
    if constexpr (RELEASE) {
      places[b] = static_cast<int>(min(at, static_cast<int64_t>(p.num_pages)));
      at += n;
      most = static_cast<int>(min(at, static_cast<int64_t>(p.num_pages)));
    } else {  // sums only grow, so from the first that does not fit on none does
      const bool fits = n == 0 || at + n <= free;
      places[b] = n == 0 ? 0 : fits ? static_cast<int>(at) : kShort;
      at += n;
      if (fits && n > 0) most = static_cast<int>(at);
    }
  }
  if (most > 0) atomicMax(&used, most);
  __syncthreads();

  // state after the call
  for (int b = blockIdx.x * kThreads + tid; b < p.B; b += gridDim.x * kThreads) {
    if constexpr (RELEASE) {
      Return r;
      give_back(p, b, r);
      p.new_state[b] = r.left;
    } else {
      Request r;
      request(p, b, r);
      const bool good = places[b] >= 0;
      p.new_state[b] = make_int2(r.lo, good ? r.need : r.hi);
      if (p.granted) p.granted[b] = good ? r.count : 0;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (RELEASE && used > p.num_pages - free) set_status(p.status, kDevBadMeta, 0xFFFF);  // more pages than there are
    p.new_state[p.B] = make_int2(RELEASE ? min(free + used, p.num_pages) : free - used, 0);
  }

  const int64_t items = static_cast<int64_t>(p.B) * pieces;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp; item < items; item += gridDim.x * kWarps) {
    const int b = static_cast<int>(item / pieces), piece = static_cast<int>(item - static_cast<int64_t>(b) * pieces);
    const int place = places[b];
    if (place == kBad) continue;
    int32_t* row = p.page_table + static_cast<int64_t>(b) * p.max_pages;
    if constexpr (RELEASE) {
      Return r;
      give_back(p, b, r);
      const int n = r.early + r.to - r.at;
#pragma unroll 4
      for (int i = piece * 32 + lane; i < n; i += pieces * 32) {
        const int page = row[i < r.early ? i : r.at + i - r.early];
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) set_status(p.status, kDevBadMeta, b);
        const int64_t to = static_cast<int64_t>(free) + place + i;
        if (to < p.num_pages) p.free_pages[to] = page;
      }
    } else {
      Request r;
      request(p, b, r);
      // k-th new page of the sequence, and whether it is one
      auto fresh = [&](int k) {
        const int page = p.free_pages[free - 1 - place - k];
        return static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages) ? page : -1;
      };
      if (place >= 0) {
#pragma unroll 4
        for (int k = piece * 32 + lane; k < r.need - r.hi; k += pieces * 32) {
          const int page = fresh(k);
          if (page < 0) set_status(p.status, kDevBadMeta, b);
          row[r.hi + k] = page;
        }
      }
      if (p.slots == nullptr) continue;
      int64_t* slots = p.slots + (p.cu_new ? r.base : static_cast<int64_t>(b) * p.n_tokens);
      const int end = min(r.count, (piece + 1) * kTokens);
#pragma unroll 4
      for (int i = piece * kTokens + lane; i < end; i += 32) {
        int64_t slot = -1;
        if (place >= 0) {
          const int pos = r.held + i, k = pos >> p.log2_page;
          const int page = k < r.hi ? row[k] : fresh(k - r.hi);
          if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages))
            slot = (static_cast<int64_t>(page) << p.log2_page) + (pos & (P - 1));
          else
            set_status(p.status, kDevBadMeta, b);
        }
        slots[i] = slot;
      }
    }
  }
}

template <bool RELEASE>
int launch(const PagesParams& p, int pieces, cudaStream_t stream) {
  const int64_t blocks = (static_cast<int64_t>(p.B) * pieces + kWarps - 1) / kWarps;
  const size_t smem = static_cast<size_t>(p.B) * 4;
  if (smem > (47 << 10) && cudaFuncSetAttribute(pages_kernel<RELEASE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                32768 * 4) != cudaSuccess)
    return -1;
  return launch_after(pages_kernel<RELEASE>, dim3(static_cast<unsigned>(blocks < kMaxBlocks ? blocks : kMaxBlocks)),
                      kThreads, smem, stream, p, pieces)
             ? 0
             : -1;
}

}  // namespace

int launch_kv_reserve(const PagesParams& p, cudaStream_t stream) {
  return launch<false>(p, p.max_new > kTokens ? (p.max_new + kTokens - 1) / kTokens : 1, stream);
}

int launch_kv_release(const PagesParams& p, cudaStream_t stream) {
  const int pieces = (p.max_pages + kEntries - 1) / kEntries;
  return launch<true>(p, pieces < 64 ? pieces : 64, stream);
}

}  // namespace cm
