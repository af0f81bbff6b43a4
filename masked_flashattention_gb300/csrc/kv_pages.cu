// Pages of a paged key-value cache dealt out on the GPU: page tables and slot maps from request lengths
// (cm_kv_reserve), and pages given back to the pool (cm_kv_release).
//
// What bounds it: a few bytes a sequence, a page and a token, so the time is that of the launch and of a chain of three
// loads (lengths and state, then page numbers out of the list or the table, then the stores).  So it is one launch:
// every block adds up the pages of all sequences for itself (16 bytes a sequence, from L2 for all blocks but the
// first), which gives each sequence its place in the free list without a second kernel and without blocks that wait
// for one another, and then takes its share of the page numbers and slots, a warp a piece of a sequence.  Input and
// output state are separate memory, so no block's reading meets another's writing.  Prefix sums make
// the result the same as that of a loop over the sequences; there are no atomics but the status word's and the block's own.
// Measured: a step of 256 sequences 2.8 us (reserve) and 3.2 (release), of which a launch is 2.2; 500 prompts, 483,000
// slots, 9.2 us (9.7 and 14.3 with pieces of 512 and 2048 slots); 2000 sequences that end with 1.28 million pages
// 6.8 us.  With blocks of 512 threads and 64-bit sums: 3.5, 3.4, 12.4 and 10.1 us.
#include <cstdint>

#include "kv_cache.h"
#include "ptx.cuh"

namespace cm {
namespace {

constexpr int kSms = 152;           // blocks of 1024 threads, or as many threads in smaller ones
constexpr int kTokens = 1024;       // slots of a warp's piece, one a lane and step; eight steps' page numbers are on their way at once
constexpr int kEntries = 256;       // page numbers of a warp's piece (at most 64 pieces a sequence), the same
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

// The same where it has been found in range: no more than the table's room, so 32 bits hold everything.
__device__ __forceinline__ Request known_request(const PagesParams& p, int b) {
  Request r;
  const int2 own = p.state[b];
  r.lo = own.x;
  r.hi = own.y;
  r.held = p.lens[b];
  r.base = p.cu_new ? p.cu_new[b] : 0;
  r.count = p.cu_new ? p.cu_new[b + 1] - r.base : p.n_new ? p.n_new[b] : p.n_tokens;
  r.need = r.count > 0 ? max((r.held + r.count - 1 + (1 << p.log2_page)) >> p.log2_page, r.hi) : r.hi;
  return r;
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
    if (held < 0 || held > static_cast<int64_t>(own.y) << p.log2_page) return false;
    r.to = min(own.y, max(held - p.window, 0) >> p.log2_page);
    if (r.to > r.at) r.left.x = r.to;
  }
  r.to = max(r.to, r.at);
  return true;
}

// Dynamic shared memory: places[B], first the pages of each sequence, then its place in the list.  Sum: 64 bits where 32
// may not hold the pages of all sequences.
template <bool RELEASE, class Sum, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) pages_kernel(const PagesParams p, int pieces) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ int places[];
  __shared__ Sum warp_sum[kWarps];
  __shared__ int used;  // pages taken, or given back
  __shared__ int fall;  // first sequence behind which cu_new falls
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, P = 1 << p.log2_page;
  let_next_start();
  if (tid == 0) {
    used = 0;
    fall = p.B;
  }
  __syncthreads();
  wait_for_previous();
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
      if (p.cu_new && p.cu_new[b + 1] < r.base) atomicMin(&fall, b);
    }
    if (!good && blockIdx.x == 0) set_status(p.status, kDevBadMeta, b);
    places[b] = good ? n : kBad;
  }
  __syncthreads();
  // prefix sums: a run of sequences a thread, then over the threads
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  Sum mine = 0;
  for (int b = b0; b < b1; ++b) mine += b > fall ? 0 : max(places[b], 0);
  Sum sum = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sum x = __shfl_up_sync(0xFFFFFFFFu, sum, d);
    if (lane >= d) sum += x;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  if (warp > 0) {
    Sum before = lane < warp ? warp_sum[lane] : 0;
#pragma unroll
    for (int d = 1; d < kWarps; d <<= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, d);
    sum += __shfl_sync(0xFFFFFFFFu, before, 0);
  }
  Sum at = sum - mine;
  int most = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = places[b];
    if (n < 0) continue;
    if (!RELEASE && b > fall) {  // its tokens may be another's too
      places[b] = kBad;
      continue;
    }
    if constexpr (RELEASE) {
      places[b] = static_cast<int>(min(at, static_cast<Sum>(p.num_pages)));
      at += n;
      most = static_cast<int>(min(at, static_cast<Sum>(p.num_pages)));
      if (blockIdx.x == 0 && at > p.num_pages - free) set_status(p.status, kDevBadMeta, 0xFFFF);  // more pages than there are
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
      const bool good = places[b] >= 0;
      const Request r = known_request(p, b);
      p.new_state[b] = make_int2(r.lo, good ? r.need : r.hi);
      if (p.granted) p.granted[b] = good ? r.count : 0;
    }
  }
  if (blockIdx.x == 0 && tid == 0)
    p.new_state[p.B] = make_int2(!RELEASE ? free - used : used > p.num_pages - free ? p.num_pages : free + used, 0);

  // pieces of sequences, one a warp, in turn
  const int step = gridDim.x * kWarps, step_b = step / pieces, step_piece = step - step_b * pieces;
  int b = (blockIdx.x * kWarps + warp) / pieces, piece = blockIdx.x * kWarps + warp - b * pieces;
  for (; b < p.B; b += step_b, piece += step_piece) {
    if (piece >= pieces) {
      piece -= pieces;
      if (++b >= p.B) break;
    }
    const int place = places[b];
    if (place == kBad) continue;
    int32_t* row = p.page_table + static_cast<int64_t>(b) * p.max_pages;
    if constexpr (RELEASE) {
      Return r;
      give_back(p, b, r);
      const int n = r.early + r.to - r.at;
      constexpr int kSteps = kEntries / 32;
      for (int i0 = piece * kEntries + lane; i0 < n; i0 += pieces * kEntries) {
        int page[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int i = i0 + s * 32;
          page[s] = i < n ? row[i < r.early ? i : r.at + i - r.early] : 0;
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int i = i0 + s * 32;
          if (static_cast<unsigned>(page[s]) >= static_cast<unsigned>(p.num_pages)) set_status(p.status, kDevBadMeta, b);
          const int64_t to = static_cast<int64_t>(free) + place + i;
          if (i < n && to < p.num_pages) p.free_pages[to] = page[s];
        }
      }
    } else {
      const Request r = known_request(p, b);
      // k-th new page of the sequence, and whether it is one
      auto fresh = [&](int k) {
        const int page = p.free_pages[free - 1 - place - k];
        return static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages) ? page : -1;
      };
      if (p.slots == nullptr) {
        if (place >= 0) {
#pragma unroll 4
          for (int k = piece * 32 + lane; k < r.need - r.hi; k += pieces * 32) {
            const int page = fresh(k);
            if (page < 0) set_status(p.status, kDevBadMeta, b);
            row[r.hi + k] = page;
          }
        }
        continue;
      }
      if (r.count == 0) continue;
      // with slots, a new page's first token is one of these: its lane writes the table's entry too
      int64_t* slots = p.slots + (p.cu_new ? r.base : static_cast<int64_t>(b) * p.n_tokens);
      constexpr int kSteps = 8;
      const int end = min(r.count, (piece + 1) * kTokens);
#pragma unroll 1
      for (int first = piece * kTokens + lane; first < end; first += kSteps * 32) {
        int page[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int i = first + s * 32, k = (r.held + i) >> p.log2_page;
          page[s] = place >= 0 && i < end ? (k < r.hi ? row[k] : fresh(k - r.hi)) : -1;
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int i = first + s * 32, pos = r.held + i, k = pos >> p.log2_page;
          if (i >= end) break;
          const bool good = static_cast<unsigned>(page[s]) < static_cast<unsigned>(p.num_pages);
          if (place >= 0) {
            if (k >= r.hi && (pos & (P - 1)) == 0) row[k] = page[s];
            if (!good) set_status(p.status, kDevBadMeta, b);
          }
          slots[i] = good ? (static_cast<int64_t>(page[s]) << p.log2_page) + (pos & (P - 1)) : -1;
        }
      }
    }
  }
}

template <bool RELEASE, class Sum, int kThreads>
int launch(const PagesParams& p, int pieces, cudaStream_t stream) {
  constexpr int kWarps = kThreads / 32, kMaxBlocks = kSms * (1024 / kThreads);
  const int64_t blocks = (static_cast<int64_t>(p.B) * pieces + kWarps - 1) / kWarps;
  const size_t smem = static_cast<size_t>(p.B) * 4;
  auto* kernel = pages_kernel<RELEASE, Sum, kThreads>;
  if (smem > (47 << 10) &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 32768 * 4) != cudaSuccess)
    return -1;
  return launch_after(kernel, dim3(static_cast<unsigned>(blocks < kMaxBlocks ? blocks : kMaxBlocks)), kThreads, smem,
                      stream, p, pieces)
             ? 0
             : -1;
}

// Every block adds up all sequences, so blocks are as large as they can be where there is work for all SMs (2000 sequences
// of 20000 tokens that end, pages of 16: 6.8 us, 12.7 with 256 threads); where a step has few pieces, barriers of
// small blocks cost less (256 sequences, one token each, before table and slots were written in one pass: 3.1 us, 3.9 with 1024
// threads).
template <bool RELEASE>
int launch(const PagesParams& p, int pieces, cudaStream_t stream) {
  if (static_cast<int64_t>(p.B) * p.max_pages >= (1LL << 31)) return launch<RELEASE, int64_t, 1024>(p, pieces, stream);
  if (p.B <= 1024 && static_cast<int64_t>(p.B) * pieces <= kSms * 16) return launch<RELEASE, int, 256>(p, pieces, stream);
  return launch<RELEASE, int, 1024>(p, pieces, stream);
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
