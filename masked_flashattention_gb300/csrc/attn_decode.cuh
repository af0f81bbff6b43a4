// Attention of one new token per sequence over a paged key-value cache (cm_attn_decode).
//
// What bounds it: every visible key and value is read once for 4 * (query heads a key-value head)
// flops an element pair, so up to 16 heads a group (128 flops every 4 bytes of a bf16 cache, every 2
// of an e4m3 one) the bytes bound it, far below the tensor cores' rate.
//
// Work.  A row is one key-value head of one sequence with up to 8 * NB of its query heads; its keys
// are cut into tiles of 32.  All rows' tiles, one after another, are dealt out in equal runs: one
// run a CTA (one CTA an SM), and within it one run a warp, so a batch of any lengths keeps every SM
// equally busy and a single long sequence is split over all of them.  Where a run ends inside a row, the row's
// parts are joined: within a CTA through shared memory, between CTAs by a second small kernel that
// is already resident when the first ends.  The dealing goes by the lengths on the device, which
// every CTA adds up for itself (a scan over the batch).
//
// A warp pair works alone: one warp fetches tiles by TMA into a ring of its own (page numbers are
// read 32 tiles ahead), the other computes; no barrier of the CTA until the run's end.  The
// tensor-core shape is turned around so that few query heads waste little of it:
//   S^T [32 keys x 8 heads] = K Q^T          A = K rows as they lie in shared memory (ldmatrix)
//   O^T [d x 8 heads]      += V^T P^T        A = V transposed on the way (ldmatrix.trans)
// (tcgen05 is the wrong tool for this one: its products start at 64 rows and take B from shared memory alone, so P would
// go there and back for a pipe that is busy 13 % of the time.)
// There is a running maximum and sum per head (one pass).  The reference that weights are taken by is
// renewed only when a score passes it, and then put 2^8 above that maximum (all in log2 units), which
// bounds p by 1 and spares the cross-lane maximum on most tiles; beside an e4m3 cache p is fp16 and taken
// 2^15 larger (kLift).  P is rounded to the values' 16-bit type for the second product; sums, maxima and O are fp32.
// An 8-bit cache is widened to fp16 (exactly) between shared memory and the product; queries become
// fp16 scaled by a power of two per head so that none overflows (scale_q).
// With a scale for each block of 16 keys, half a tile, the fetching warp hands the four exponents of a tile's blocks
// along with it.  The keys' is a factor of the scores.  The values' is added to the scores in log2 units, so that a weight is
// that of the stored numbers and the running maximum bounds it however far scales lie apart; the sum of the weights
// takes it off again.  Neither is an instruction more a score than one scale a head takes.
// Under a sliding window a row's tiles are those of the first keys and of the last (WINDOW, kernels of their own: as a
// further case of the mask's intervals the case below took 46.9 us where it then took 45.6, and the calls without one slowed by 1 to 3 %).
//
// Measured (8 key-value heads of 128, 4 query heads each, bf16): 64 sequences of up to 16384 keys, 332 us =
// 6.9 TB/s, 102 % of the copy bandwidth; one of 131071, 85 us = 6.3 TB/s; 200 of up to 333, 17.6 us.  What
// stands above the bytes is the start, 4 us from the launch to the first tile on its way (length, place, page
// number: one load behind another) and up to 4 more until the memory's address translations are warm, and the end,
// 4 to 5 us where rows are split (join, launch, join).  One CTA a head took 52 ms for the one of 131071.
// With block scales: the 64 sequences, int8, 180 us = 6.4 TB/s, 94 %; the one of 131071, e4m3, 50 us; 40 of up to 32768
// with 16 heads a group, int8, 70 us (67 with one scale a head, e4m3: the widening of the bytes holds both).  Windows: 256 sequences
// under 1024 keys and 16 sinks, int8, 44.5 us = 4.3 TB/s (start, row ends and join); one of 100,003 under 4096, bf16, 9.1 us.
#pragma once
#include <cuda_fp16.h>
#include <atomic>

#include "attn_decode.h"
#include "ptx.cuh"

namespace cm {
namespace {

constexpr int kMaxIntervals = 8;
constexpr float kRenew = 8.f;       // log2 units a score may pass the maximum by that the reference was set from
// Log2 units that the reference of the weights lies below that maximum.  bf16 weights have fp32's range: 8 above
// it, no weight is beyond 1, and O stays within fp32 where the sum of |v| does (with weights up to 2^8,
// values of 2^118 overflowed).  fp16 weights reach up to 2^(8 + 7), and what fp16 cannot hold is below 2^-32 of the
// largest: with 2^8, a million keys of 2^-25 each beside one large one lost 3 % of the sum.
template <int KIND>
constexpr float kLift = KIND != kBf16 ? 7.f : -kRenew;
// What the reference starts from.  With block scales a score is taken over it in the same step that scales it, so it is a
// number: a score of -inf over a reference of -inf would be NaN, and not the 0 that its weight is.
template <int KIND>
constexpr float kLowest = KIND >= kE4m3Block ? -3.402823466e38f : -INFINITY;
constexpr size_t kSmemMax = 232448;

// flags of a tile
constexpr int kFirst = 1;   // first tile of the warp's part of the row
constexpr int kLast = 2;    // last tile of that part
constexpr int kStarts = 4;  // the part begins where the row begins
constexpr int kEnds = 8;    // the part ends where the row ends
constexpr int kFlagBits = 4;  // above them: the CTAs that hold parts of the row

// Shared memory: 32 keys of 128 bf16 channels, K and V, are 16 KB, and 4 pairs with 3 such stages are what fits.
// The smaller rows take more instructions a byte, so 8 pairs share the ring's memory (one computing warp
// a scheduler left an e4m3 cache at 47 % of the bandwidth).  Their 16 warps start with 128 registers a thread and
// trade: 184 for a computing warp, 72 for a fetching one.
template <int D, int KIND, int NB>
struct Cfg {
  static constexpr int kItem = KIND == kBf16 ? 2 : 1;
  static constexpr int kRowBytes = D * kItem;
  static constexpr int kPairs = kRowBytes == 256 ? 4 : 8;  // warp pairs of a CTA
  static constexpr int kThreads = 64 * kPairs;
  static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;  // inner width of a TMA box
  static constexpr int kBoxes = kRowBytes / kBoxBytes;
  static constexpr int kMatrix = kTileKeys * kRowBytes;
  static constexpr int kStage = 2 * kMatrix;  // K, then V
  static constexpr int kHeads = 8 * NB;
  // floats of a head in a part: 4 spare keep a warp's fragment stores free of conflicts, where there is room
  static constexpr int kHeadPitch = NB == 1 ? D + 4 : D;
  static constexpr int kPiece = kHeads * kHeadPitch * 4 + 2 * kHeads * 4;  // O, m, l
  static constexpr int kFit = (static_cast<int>(kSmemMax) - 1024 - kPairs * kPiece) / (kPairs * kStage);
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  // Stages in flight where rows are long: 128 KB an SM.  With all that fits, some SMs get their data a third
  // faster than others (one sequence of 131071: blocks were done after 60 to 87 us), and the slowest decide.
  // Short rows are better off with every stage: the next rows' tiles are on their way during the ends of these.
  static constexpr int kSteady = (128 << 10) / (kPairs * kStage) < kStages ? (128 << 10) / (kPairs * kStage) : kStages;
  static constexpr int kRing = kPairs * kStages * kStage;
  static constexpr int kOffPiece = kRing;
  static constexpr int kOffMeta = kOffPiece + kPairs * kPiece;
  static constexpr int kOffBars = kOffMeta + kPairs * kStages * 16;
  static constexpr int kOffHead = kOffBars + kPairs * kStages * 16;   // int4 per piece
  static constexpr int kOffMisc = kOffHead + 2 * kPairs * 16;         // starts, counts, abort flag
  static constexpr int kOffExps = kOffMisc + 64;                      // a word a stage: exponents of its blocks' scales
  static constexpr int kSmem = kOffMisc + 256;
  static_assert(KIND < kE4m3Block || kPairs * kStages * 4 <= 256 - 64, "the exponents lie behind the abort flag");
  static_assert(kStages >= 2 && kSmem <= static_cast<int>(kSmemMax), "shared memory");
  static_assert(kOffPiece % 16 == 0 && kPiece % 16 == 0 && kOffMeta % 16 == 0, "alignment");
  static_assert(kPairs * kPiece >= (3 * kThreads + kThreads / 32) * 4, "the search borrows the pieces' memory");
  static_assert(kStages * kStage >= kPiece, "the last piece of a warp borrows its ring");
};

// Workspace: per CTA a header (int4, .x = parts of the row whose start its second part holds, .y = that
// row) and two parts, the first of a row begun earlier, the second of a row carried on.
struct Part {
  float* o;  // [heads][D]
  float* m;  // [heads], log2 units
  float* l;
};
template <int D>
__device__ __forceinline__ Part part_at(void* workspace, int heads, int cta, int slot) {
  float* f = reinterpret_cast<float*>(static_cast<char*>(workspace) + kMaxCtas * 16) +
             static_cast<size_t>(cta * 2 + slot) * heads * (D + 2);
  return {f, f + heads * D, f + heads * (D + 1)};
}

// Sequence, key-value head and place among its rows of a row.
struct RowIndex {
  int b, h, chunk;
};
__device__ __forceinline__ RowIndex row_index(const DecodeArgs& a, int row) {
  const int bh = a.by_chunks(row), b = a.by_heads(bh);
  return {b, bh - b * a.p.c.H_kv, row - bh * a.chunks};
}

// ---- instructions -----------------------------------------------------------------------------
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movm_trans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two of the four 8-bit numbers of x as fp16x2, exact: bytes 0 and 1, or 2 and 3; ODD: bytes 0 and 2, or 1 and 3.
// A whole number n is the fp16 1024 + (n + 128), whose bits are 0x6400 + (n + 128), less 1152.  (Keys as the bits n + 128 alone,
// which as fp16 are (n + 128) * 2^-24, with the sum's excess taken off in fp32, were 0.4 to 1.2 % faster; but a score was then off
// by the rounding of 128 * sum |q|, whatever the keys were.)
template <int KIND, bool ODD = false>
__device__ __forceinline__ void widen(uint32_t x, uint32_t& lo, uint32_t& hi) {
  if constexpr (KIND == kInt8Block) {
    x ^= 0x80808080u;
    const uint32_t top = 0x64646464u;
    lo = __byte_perm(x, top, ODD ? 0x4240 : 0x4140);
    hi = __byte_perm(x, top, ODD ? 0x4341 : 0x4342);
    const __half2 less = __half2half2(__ushort_as_half(0x6480));
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&lo), less), z = __hsub2(*reinterpret_cast<const __half2*>(&hi), less);
    lo = *reinterpret_cast<const uint32_t*>(&y);
    hi = *reinterpret_cast<const uint32_t*>(&z);
  } else {
    if constexpr (ODD) x = __byte_perm(x, 0, 0x3120);
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
  }
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int32_t x, int32_t y,
                                            int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// ---- the plan of a unit: which tiles it has ------------------------------------------------------
// A unit is a sequence (all its key-value heads see the same keys), or with selected pages one
// key-value head of a sequence.  Intervals [st, en) of keys become tile ranges; a tile that several touch
// belongs to the first in the order of the ranges' starts, so with `before` that order, interval i
// owns the tiles [max(a_i, max of b_j before i), b_i).
__device__ __forceinline__ int checked_length(const DecodeArgs& a, int b, int len, bool report) {
  const DecodeParams& p = a.p;
  const bool good = len >= 0 &&
                    static_cast<int64_t>(len) <= (static_cast<int64_t>(p.c.max_pages) << p.c.log2_page) &&
                    (p.itab == nullptr || len <= p.S);
  if (!good && report) set_status(p.c.status, kDevBadMeta, b);
  return good ? len : 0;
}
// Under a window: the keys [0, early) and [start, len) are visible; one interval where the sinks reach the window, so
// that its tiles count as full.
struct Window {
  int early, start;
  __device__ __forceinline__ Window(const DecodeParams& p, int len) : early(0), start(max(len - p.window, 0)) {
    if (p.sinks >= start) start = 0;
    else early = p.sinks;
  }
  __device__ __forceinline__ int early_tiles() const { return (early + kTileKeys - 1) / kTileKeys; }
  // the first tile of the second interval that the first has not
  __device__ __forceinline__ int from() const { return max(start / kTileKeys, early_tiles()); }
  __device__ __forceinline__ bool sees(int key, int len) const { return key < early || (key >= start && key < len); }
};
__device__ __forceinline__ int2 unit_interval(const DecodeArgs& a, int b, int n, int len) {
  if (a.p.itab == nullptr) return make_int2(0, n == 0 ? len : 0);
  if (n >= a.p.NI || len == 0) return make_int2(0, 0);
  const int2 iv = reinterpret_cast<const int2*>(
      a.p.itab)[(static_cast<int64_t>(b) * a.p.NI + n) * a.p.S + (len - 1)];
  const int s = max(iv.x, 0), e = min(iv.y, len);
  return e > s ? make_int2(s, e) : make_int2(0, 0);
}
// Tiles of a unit's rows, and its sequence's length (0 where that is out of range).
template <bool WINDOW>
__device__ __forceinline__ int unit_tiles(const DecodeArgs& a, int u, bool report, int& len) {
  if constexpr (WINDOW) {
    len = checked_length(a, u, a.p.c.lens[u], report);
    const Window w(a.p, len);
    return w.early_tiles() + max((len + kTileKeys - 1) / kTileKeys - w.from(), 0);
  }
  const int b = a.p.sel ? a.by_heads(u) : u;
  const int held = a.p.c.lens[b], chosen = a.p.sel ? a.p.nsel[u] : 0;  // both on their way at once
  len = checked_length(a, b, held, report);
  if (a.p.sel) {
    const int n = len ? min(max(chosen, 0), a.p.sel_max) : 0;
    return a.p.c.log2_page == 4 ? (n + 1) / 2 : n << (a.p.c.log2_page - 5);
  }
  if (a.p.itab == nullptr) return (len + kTileKeys - 1) / kTileKeys;
  int lo[kMaxIntervals], hi[kMaxIntervals], total = 0;
#pragma unroll
  for (int n = 0; n < kMaxIntervals; ++n) {
    const int2 iv = unit_interval(a, b, n, len);
    lo[n] = iv.x / kTileKeys;
    hi[n] = (iv.y + kTileKeys - 1) / kTileKeys;
  }
  // one interval after another comes to the front (small code: instructions fetched for the first time
  // cost more than these)
#pragma unroll 1
  for (int i = 0; i < a.p.NI; ++i) {
    int from = lo[0];
#pragma unroll
    for (int k = 1; k < kMaxIntervals; ++k)
      if (lo[k] < lo[0] || (lo[k] == lo[0] && i + k >= kMaxIntervals)) from = max(from, hi[k]);
    total += max(hi[0] - from, 0);
    const int l = lo[0], h = hi[0];
#pragma unroll
    for (int k = 1; k < kMaxIntervals; ++k) {
      lo[k - 1] = lo[k];
      hi[k - 1] = hi[k];
    }
    lo[kMaxIntervals - 1] = l;
    hi[kMaxIntervals - 1] = h;
  }
  return total;
}
// What a row costs: its tiles, and about two more for its queries, its end and its output (of 0 to 3, the best for
// batches of short rows: 128 sequences of up to 1024 keys 53.3 us, 55.2 with one more).
__device__ __forceinline__ int row_cost(int tiles) { return tiles ? tiles + kRowCost : 0; }

// The same by a warp: lane n < 8 holds interval n.
struct Plan {
  int b, len, tiles;
  int st, en;         // keys of the lane's interval
  int from, cnt, off; // its own tiles, and their place in the unit's order
};
template <bool WINDOW>
__device__ __forceinline__ Plan make_plan(const DecodeArgs& a, int u, int len, int tiles, int lane) {
  Plan w;
  w.b = !WINDOW && a.p.sel ? a.by_heads(u) : u;
  w.len = len;
  w.tiles = tiles;
  w.st = w.en = w.from = w.cnt = w.off = 0;
  if (WINDOW || a.p.itab == nullptr) return w;  // its tiles in order, every key below the length (or of the window)
  const int2 iv = lane < kMaxIntervals ? unit_interval(a, w.b, lane, w.len) : make_int2(0, 0);
  w.st = iv.x;
  w.en = iv.y;
  const int lo = iv.x / kTileKeys, hi = (iv.y + kTileKeys - 1) / kTileKeys;
  w.from = lo;
#pragma unroll 1
  for (int j = 0; j < a.p.NI; ++j) {
    const int lj = __shfl_sync(0xFFFFFFFFu, lo, j), hj = __shfl_sync(0xFFFFFFFFu, hi, j);
    if (j != lane && (lj < lo || (lj == lo && j < lane))) w.from = max(w.from, hj);
  }
  w.cnt = lane < kMaxIntervals ? max(hi - w.from, 0) : 0;
#pragma unroll 1
  for (int j = 0; j < a.p.NI; ++j) {
    const int lj = __shfl_sync(0xFFFFFFFFu, lo, j), cj = __shfl_sync(0xFFFFFFFFu, w.cnt, j);
    if (lj < lo || (lj == lo && j < lane)) w.off += cj;
  }
  return w;
}

struct Place {
  int u, m, c;     // unit, row of the unit, tile of the row
  int len, tiles;  // of the unit
};

// Up to 32 consecutive tiles of a row, one per lane.
struct Chunk {
  int row, n, c0;        // row, tiles, place of the first in the row
  int h;                 // key-value head
  int page0, page1;      // pages of the tile (page1: second half of a tile of two 16-key pages); -1: none
  int key0, key1;        // first keys of these
  uint32_t k0, k1, v0, v1;  // scales of their two blocks of 16 keys, as they lie in memory
  bool full;             // every key of the tile is visible
  bool whole;            // the chunk is a whole row
};

// Positions count costs: a row's tiles, then kRowCost places without a tile.
struct Walk {
  int u, m, c;   // unit, row of the unit, tile of the row: what comes next
  int pos, end;  // of the warp's run
  Plan plan;
};

// Scales of the chunk's tiles, for its key-value head: asked for once the page numbers are there, and not looked at
// before the chunk is fetched.
__device__ __forceinline__ void load_scales(const DecodeParams& p, Chunk& k) {
  const int log2_page = p.c.log2_page, per = log2_page - 4, block = (k.key0 & ((1 << log2_page) - 1)) >> 4;
  const bool two = log2_page == 4;
  const int64_t at0 = ((static_cast<int64_t>(k.page0) * p.c.H_kv + k.h) << per) + block;
  const int64_t at1 = two ? static_cast<int64_t>(k.page1) * p.c.H_kv + k.h : at0 + 1;
  const bool in0 = k.page0 >= 0, in1 = two ? k.page1 >= 0 : in0;
  k.k0 = in0 ? __float_as_uint(p.c.k_scale[at0]) : 0u;
  k.v0 = in0 ? __float_as_uint(p.c.v_scale[at0]) : 0u;
  k.k1 = in1 ? __float_as_uint(p.c.k_scale[at1]) : 0u;
  k.v1 = in1 ? __float_as_uint(p.c.v_scale[at1]) : 0u;
}

template <int D, int KIND, bool WINDOW>
__device__ __forceinline__ void next_chunk(const DecodeArgs& a, Walk& w, Chunk& k, int lane) {
  if (w.c >= w.plan.tiles) {  // next row
    w.pos += kRowCost - (w.c - w.plan.tiles);
    w.c = 0;
    if (w.m + 1 < a.rows) {
      ++w.m;
      if (k.whole && w.end - w.pos >= w.plan.tiles) {  // the last chunk was all of a row with the same tiles
        ++k.row;
        k.h = row_index(a, k.row).h;
        k.n = w.c = w.plan.tiles;
        w.pos += k.n;
        if constexpr (KIND >= kE4m3Block) load_scales(a.p, k);
        return;
      }
    } else if (w.pos < w.end) {  // next unit that has tiles: there is one, or the run would have ended
      w.m = 0;
      do {
        if (w.u + 1 >= a.units) {
          k.n = 0;
          return;
        }
        int len;
        const int tiles = unit_tiles<WINDOW>(a, ++w.u, false, len);
        w.plan = make_plan<WINDOW>(a, w.u, len, tiles, lane);
      } while (w.plan.tiles == 0);
    }
  }
  k.n = max(min(min(32, w.plan.tiles - w.c), w.end - w.pos), 0);
  if (k.n == 0) return;
  const DecodeParams& p = a.p;
  const int log2_page = p.c.log2_page, P = 1 << log2_page;
  k.row = w.u * a.rows + w.m;
  k.h = row_index(a, k.row).h;
  const int bh = w.plan.b * p.c.H_kv + k.h;
  k.c0 = w.c;
  k.whole = k.n == w.plan.tiles;
  const int c = w.c + lane;
  const bool in = lane < k.n;
  const int pages = (w.plan.len + P - 1) >> log2_page;
  int place0 = -1, place1 = -1;
  k.key0 = k.key1 = 0;
  k.full = false;
  if (!WINDOW && p.sel) {
    const int32_t* sel = p.sel + static_cast<int64_t>(bh) * p.sel_max;
    const int entries = log2_page == 4 ? min(p.nsel[bh], p.sel_max) : 0;  // there may be one page too few for the last tile
    const int e0 = log2_page == 4 ? 2 * c : c >> (log2_page - 5);
    if (in) {
      place0 = sel[e0];
      const int before = e0 > 0 ? sel[e0 - 1] : -1;
      int place = place0;
      if (log2_page == 4 && e0 + 1 < entries) {
        place1 = sel[e0 + 1];
        if (place1 <= place0 || place1 >= pages) {
          set_status(p.c.status, kDevBadMeta, w.plan.b);
          place1 = -1;
        }
      }
      if (place <= before || place >= pages) {
        set_status(p.c.status, kDevBadMeta, w.plan.b);
        place0 = -1;
      }
      k.key0 = (place0 << log2_page) + (log2_page == 4 ? 0 : (c & ((P >> 5) - 1)) * kTileKeys);
      k.key1 = place1 << 4;
    }
  } else {
    int tile = c;
    const Window win(p, w.plan.len);
    if constexpr (WINDOW) {
      tile = c < win.early_tiles() ? c : win.from() + c - win.early_tiles();
    } else if (p.itab) {
#pragma unroll 1
      for (int j = 0; j < p.NI; ++j) {
        const int from = __shfl_sync(0xFFFFFFFFu, w.plan.from, j);
        const int off = __shfl_sync(0xFFFFFFFFu, w.plan.off, j);
        const int cnt = __shfl_sync(0xFFFFFFFFu, w.plan.cnt, j);
        if (c >= off && c < off + cnt) tile = from + c - off;
      }
    }
    if (in) {
      k.key0 = tile * kTileKeys;
      k.key1 = k.key0 + 16;
      place0 = k.key0 >> log2_page;
      if (log2_page == 4 && place0 + 1 < pages) place1 = place0 + 1;
      if (WINDOW && log2_page == 4) {  // a page that lies behind the window is no longer the sequence's
        if (k.key0 >= win.early && k.key1 <= win.start) place0 = -1;
        if (k.key1 >= win.early && k.key1 + 16 <= win.start) place1 = -1;
      }
    }
  }
  // visible keys are [st, en) of the intervals; without intervals, [0, len)
  const bool two = log2_page == 4;
  const int end0 = k.key0 + (two ? 16 : kTileKeys);
  if constexpr (WINDOW) {
    const Window win(p, w.plan.len);
    k.full = in && (k.key0 + kTileKeys <= win.early || (k.key0 >= win.start && k.key0 + kTileKeys <= w.plan.len));
  } else if (p.itab) {
#pragma unroll 1
    for (int j = 0; j < p.NI; ++j) {
      const int st = __shfl_sync(0xFFFFFFFFu, w.plan.st, j), en = __shfl_sync(0xFFFFFFFFu, w.plan.en, j);
      k.full |= st <= k.key0 && k.key0 + kTileKeys <= en;
    }
    k.full = k.full && in;
  } else {
    k.full = in && place0 >= 0 && end0 <= w.plan.len && (!two || (place1 >= 0 && k.key1 + 16 <= w.plan.len));
  }
  const int32_t* table = p.c.table + static_cast<int64_t>(w.plan.b) * p.c.max_pages;
  k.page0 = place0 >= 0 ? table[place0] : -1;
  k.page1 = place1 >= 0 ? table[place1] : -1;
  if ((place0 >= 0 && static_cast<unsigned>(k.page0) >= static_cast<unsigned>(p.c.num_pages)) ||
      (place1 >= 0 && static_cast<unsigned>(k.page1) >= static_cast<unsigned>(p.c.num_pages))) {
    set_status(p.c.status, kDevBadMeta, w.plan.b);
    if (static_cast<unsigned>(k.page0) >= static_cast<unsigned>(p.c.num_pages)) k.page0 = -1;
    if (static_cast<unsigned>(k.page1) >= static_cast<unsigned>(p.c.num_pages)) k.page1 = -1;
    k.full = false;
  }
  if constexpr (KIND >= kE4m3Block) load_scales(p, k);
  w.c += k.n;
  w.pos += k.n;
}

// A warp's wait: whole or not at all, so that its lanes go on together.  Bounded as WaitCtl's are.  The
// waits here are a microsecond or two, and a try may sleep longer than that by itself: under a
// short limit (cm_set_wait_limit_ns) the phase is only looked at.
__device__ __forceinline__ bool warp_wait(const WaitCtl& w, uint32_t bar, uint32_t parity, int where) {
  if (w.limit_ns >= 20000) return __all_sync(0xFFFFFFFFu, w(bar, parity, where));
  const uint64_t t0 = globaltimer_ns();
  bool got = false;
  while (!got && !*w.abort) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    got = ok != 0;
    if (!got && globaltimer_ns() - t0 > w.limit_ns) {
      *w.abort = 1;
      set_status(w.status, kDevTimeout, where);
    }
  }
  return __all_sync(0xFFFFFFFFu, got);
}

// Two fp32 operations an instruction, each rounded as by itself.
struct F2 {
  float x, y;
};
__device__ __forceinline__ uint64_t as_pair(F2 a) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a.x), "f"(a.y));
  return p;
}
__device__ __forceinline__ F2 from_pair(uint64_t p) {
  F2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(p));
  return a;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  uint64_t c;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(c) : "l"(as_pair(a)), "l"(as_pair(b)));
  return from_pair(c);
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as_pair(a)), "l"(as_pair(b)), "l"(as_pair(c)));
  return from_pair(d);
}

// Exponents of a tile's block scales (keys' two, then values' two), a byte each.
__device__ __forceinline__ uint32_t pack_exponents(uint32_t k0, uint32_t k1, uint32_t v0, uint32_t v1) {
  const uint32_t a = __byte_perm(block_exponent(k0), block_exponent(k1), 0x0040);
  const uint32_t b = __byte_perm(block_exponent(v0), block_exponent(v1), 0x0040);
  return __byte_perm(a, b, 0x5410);
}
__device__ __forceinline__ int exponent_at(uint32_t word, int i) { return static_cast<int8_t>(word >> (8 * i)); }

// ---- fetching warp ------------------------------------------------------------------------------
// Returns the tiles fetched; `rest` is the first of them whose copy the computing warp need not have
// waited for, were it to give up.
template <int D, int KIND, int NB, bool WINDOW>
__device__ __forceinline__ int fetch(const DecodeArgs& a, const CUtensorMap* kmap,
                                     const CUtensorMap* vmap, Walk w, uint32_t ring,
                                     uint32_t meta, uint32_t bars, uint32_t exps, int run, const WaitCtl& wait,
                                     int lane, int& rest) {
  using C = Cfg<D, KIND, NB>;
  const DecodeParams& p = a.p;
  const int log2_page = p.c.log2_page, P = 1 << log2_page;
  const int depth = a.whole_rows ? C::kStages : C::kSteady;
  int issued = 0;
  const int begin = w.pos, end = w.end;
  Chunk next;
  next.whole = false;
  next_chunk<D, KIND, WINDOW>(a, w, next, lane);
  bool ok = true;
  while (next.n > 0 && ok) {
    const Chunk cur = next;
    const Plan plan = w.plan;  // of cur's unit
    const int at = w.pos - cur.n, row_begin = at - cur.c0;
    // parts of the row, one a CTA's run; asked for where the row is not all this warp's
    const int parts = row_begin < begin || row_begin + plan.tiles > end
                          ? (row_begin + plan.tiles - 1) / run - row_begin / run + 1
                          : 1;
    next_chunk<D, KIND, WINDOW>(a, w, next, lane);  // its loads are on their way while cur is fetched
    for (int j = 0; j < cur.n; ++j) {
      const int stage = issued % C::kStages;
      const uint32_t full = bars + stage * 16;
      const int before = issued - depth;  // that tile has to be done with
      if (before >= 0 && !warp_wait(wait, bars + before % C::kStages * 16 + 8, (before / C::kStages) & 1, 1)) {
        ok = false;
        break;
      }
      const int page0 = __shfl_sync(0xFFFFFFFFu, cur.page0, j), page1 = __shfl_sync(0xFFFFFFFFu, cur.page1, j);
      const int key0 = __shfl_sync(0xFFFFFFFFu, cur.key0, j), key1 = __shfl_sync(0xFFFFFFFFu, cur.key1, j);
      uint32_t seen = 0xFFFFFFFFu;
      if (!__shfl_sync(0xFFFFFFFFu, static_cast<int>(cur.full), j)) {  // one lane a key
        const bool second = log2_page == 4 && lane >= 16;
        const int key = second ? key1 + lane - 16 : key0 + lane;
        bool in = key < plan.len;
        if constexpr (WINDOW) {
          in = Window(p, plan.len).sees(key, plan.len);
        } else if (p.itab) {
          in = false;
#pragma unroll 1
          for (int n = 0; n < p.NI; ++n) {
            const int st = __shfl_sync(0xFFFFFFFFu, plan.st, n), en = __shfl_sync(0xFFFFFFFFu, plan.en, n);
            in |= key >= st && key < en;
          }
        }
        seen = __ballot_sync(0xFFFFFFFFu, in && (second ? page1 : page0) >= 0);
      }
      uint32_t scales = 0;
      if constexpr (KIND >= kE4m3Block) {
        const uint32_t mine = pack_exponents(cur.k0, cur.k1, cur.v0, cur.v1);
        scales = __shfl_sync(0xFFFFFFFFu, mine, j);
      }
      if (lane == 0) {
        const int c = cur.c0 + j;
        if constexpr (KIND >= kE4m3Block) asm volatile("st.shared.b32 [%0], %1;" ::"r"(exps + stage * 4), "r"(scales) : "memory");
        int flags = 0;
        if (c == 0) flags |= kFirst | kStarts;
        if (at + j == begin) flags |= kFirst;
        if (c == plan.tiles - 1) flags |= kLast | kEnds;
        if (at + j == end - 1) flags |= kLast;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(meta + stage * 16), "r"(cur.row),
                     "r"(seen), "r"(flags | (parts << kFlagBits)), "r"(next.n > 0 ? next.row : -1)
                     : "memory");
        const uint32_t k_at = ring + stage * C::kStage, v_at = k_at + C::kMatrix;
        const int half = log2_page == 4 ? 2 : 1;  // boxes of 16 or 32 keys
        const bool get0 = page0 >= 0, get1 = half == 2 && page1 >= 0;
        mbar_arrive_expect_tx(full, C::kStage / half * (static_cast<int>(get0) + static_cast<int>(get1)));
        if (get0) {
          const int y = (cur.h << log2_page) + (key0 & (P - 1));
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x) {
            tma_load_3d(k_at + x * kTileKeys * C::kBoxBytes, kmap, x * C::kBoxBytes / C::kItem, y, page0, full);
            tma_load_3d(v_at + x * kTileKeys * C::kBoxBytes, vmap, x * C::kBoxBytes / C::kItem, y, page0, full);
          }
        }
        if (get1) {
          const int y = cur.h << log2_page;
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x) {
            const uint32_t to = (x * kTileKeys + 16) * C::kBoxBytes;
            tma_load_3d(k_at + to, kmap, x * C::kBoxBytes / C::kItem, y, page1, full);
            tma_load_3d(v_at + to, vmap, x * C::kBoxBytes / C::kItem, y, page1, full);
          }
        }
      }
      __syncwarp();
      ++issued;
    }
  }
  rest = max(issued - C::kStages, 0);
  if (ok) {  // tell the computing warp that there is no more
    const int stage = issued % C::kStages;
    const uint32_t full = bars + stage * 16, empty = full + 8;
    if (issued < C::kStages || warp_wait(wait, empty, ((issued / C::kStages) & 1) ^ 1, 2)) {
      rest = max(issued + 1 - C::kStages, 0);
      if (lane == 0) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(meta + stage * 16), "r"(-1) : "memory");
        mbar_arrive(full);
      }
    }
  }
  return issued;
}

// ---- computing warp -------------------------------------------------------------------------------
// Query fragments of a row: B operand [16 channels x 8 heads] of each step, thread (head lane / 4,
// channels by lane % 4).  bf16 steps take channels 2t, 2t+1 and 2t+8, 2t+9; e4m3 steps take
// 4t .. 4t+3, the order in which a lane gets the keys' bytes.
template <int D, int KIND>
__device__ __forceinline__ void read_q(const DecodeArgs& a, int row, int n, int lane, uint32_t (&q)[D / 16][2]) {
  const DecodeParams& p = a.p;
  const auto [b, h, chunk] = row_index(a, row);
  const int i = chunk * a.heads + n * 8 + lane / 4;
  const bool in = i < a.group;
  const __nv_bfloat16* src = p.q + b * p.qs.seq + static_cast<int64_t>(h * a.group + (in ? i : 0)) * p.qs.head;
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    if constexpr (KIND != kBf16) {
      const uint2 w = in ? *reinterpret_cast<const uint2*>(src + s * 16 + (lane & 3) * 4) : make_uint2(0, 0);
      q[s][0] = w.x;
      q[s][1] = w.y;
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x)
        q[s][x] = in ? *reinterpret_cast<const uint32_t*>(src + s * 16 + x * 8 + (lane & 3) * 2) : 0u;
    }
  }
}

// Factor of the scores (log2 units) of the lane's two columns; for an e4m3 cache the fragments become
// fp16, scaled by a power of two per head to a largest value in [2^14, 2^15): no more (65504) fits, and
// what is smaller loses no bits down to 2^-31 of it.  (Powers of two are held to fp32's normal numbers: a head
// whose largest value is below 2^-112 stays below 2^14.)
template <int D, int KIND, int NB>
__device__ __forceinline__ void scale_q(const DecodeArgs& a, int row, int lane, uint32_t (&q)[NB][D / 16][2],
                                        float (&scale)[NB][2]) {
  const float base = a.p.scale * 1.4426950408889634f * (KIND == kE4m3 ? a.p.c.k_scale[row_index(a, row).h] : 1.f);
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    if constexpr (KIND == kBf16) {
      scale[n][0] = scale[n][1] = base;
    } else {
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          top = fmaxf(top, fabsf(__uint_as_float(q[n][s][x] << 16)));
          top = fmaxf(top, fabsf(__uint_as_float(q[n][s][x] & 0xFFFF0000u)));
        }
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const int e = max(min(static_cast<int>(__float_as_uint(top) >> 23) - 127, 127) - 14, -126);
      const float inv = pow2_bits(-e);
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const __half2 f = __floats2half2_rn(__uint_as_float(q[n][s][x] << 16) * inv,
                                              __uint_as_float(q[n][s][x] & 0xFFFF0000u) * inv);
          q[n][s][x] = *reinterpret_cast<const uint32_t*>(&f);
        }
      float mine = base * pow2_bits(e);
      // times a block's scale of at most 2^32 it stays finite, so that a key of zeros scores 0 beside any query
      if constexpr (KIND >= kE4m3Block) mine = fminf(fmaxf(mine, -0x1p95f), 0x1p95f);
      scale[n][0] = __shfl_sync(0xFFFFFFFFu, mine, (lane & 3) * 8);  // heads of the lane's columns
      scale[n][1] = __shfl_sync(0xFFFFFFFFu, mine, (lane & 3) * 8 + 4);
    }
  }
}

// Address of the 16-byte piece `c` of key `r` in a matrix of the ring (TMA's swizzle).
template <int D, int KIND>
__device__ __forceinline__ uint32_t piece_at(uint32_t matrix, int r, int c) {
  if constexpr (KIND != kBf16 && D == 64) {  // 64-byte rows
    return matrix + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  } else {
    return matrix + (c >> 3) * (kTileKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  }
}

template <int D, int KIND, int NB>
struct State {
  uint32_t q[NB][D / 16][2];
  float scale[NB][2];
  float m[NB][2], l[NB][2];
  float o[NB][D / 16][4];
};

// What is left of a weight p beside its first 8 bits: never negative, and of a weight that is not 0 never 0, as
// an infinite value would make NaN of either (inf - inf, 0 * inf) where p * inf is infinite.  The floor, fp32's
// smallest normal number, is far below p's own last bit unless p is as small.
__device__ __forceinline__ float left_over(float p, float cut) { return fmaxf(p - cut, fminf(p, 1.17549435e-38f)); }

template <int D, int KIND, int NB>
__device__ __forceinline__ void compute_tile(State<D, KIND, NB>& t, uint32_t k_at, uint32_t v_at,
                                             uint32_t seen, uint32_t exps, int lane) {
  constexpr bool k8 = KIND != kBf16, kBlocks = KIND >= kE4m3Block;
  // One or two warps a scheduler: latencies are hidden within the warp, by loading ahead of the
  // products and by two sets of sums each.
  float s[2][NB][4], s2[2][NB][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[i][n][x] = s2[i][n][x] = 0.f;
  // S^T = K Q^T: matrices of ldmatrix are (keys 0-7, 8-15) x (pieces 2j, 2j+1)
  constexpr int kSteps = D * (k8 ? 1 : 2) / 32, kGroup = kSteps < 4 ? kSteps : 4;
  const int row = lane & 15, col = lane >> 4;
#pragma unroll
  for (int j0 = 0; j0 < kSteps; j0 += kGroup) {
    uint32_t w[kGroup][2][4];
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) ldsm4(w[j][i], piece_at<D, KIND>(k_at, i * 16 + row, 2 * (j0 + j) + col));
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (!k8) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
            mma16816<false>(j & 1 ? s2[i][n] : s[i][n], w[j][i], t.q[n][j0 + j][0], t.q[n][j0 + j][1]);
        } else {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t f[4];
            widen<KIND>(w[j][i][2 * x], f[0], f[2]);
            widen<KIND>(w[j][i][2 * x + 1], f[1], f[3]);
#pragma unroll
            for (int n = 0; n < NB; ++n)
              mma16816<true>(x ? s2[i][n] : s[i][n], f, t.q[n][2 * (j0 + j) + x][0], t.q[n][2 * (j0 + j) + x][1]);
          }
        }
      }
  }
  // values of the first 16 keys, for the second product
  constexpr int kValues = k8 ? D / 32 : D / 16;
  const int key = k8 ? row : (lane & 7) + ((lane >> 4) << 3), piece = k8 ? col : (lane >> 3) & 1;
  uint32_t v[kValues][4];
#pragma unroll
  for (int j = 0; j < kValues; ++j) ldsm4t(v[j], piece_at<D, KIND>(v_at, key, 2 * j + piece));
  const bool whole = seen == 0xFFFFFFFFu;
  auto hide = [&] {  // keys of the lane: lane / 4 and 8 further, of both halves
    const uint32_t bits = seen >> (lane >> 2);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          s[i][n][x] = (bits >> (i * 16 + (x >> 1) * 8)) & 1u ? s[i][n][x] : -INFINITY;
  };
  // the reference of the weights in log2 units; renewed when a score passes it by kRenew + kLift
  auto renew = [&] {
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float top = fmaxf(fmaxf(s[0][n][x], s[0][n][x + 2]), fmaxf(s[1][n][x], s[1][n][x + 2]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        top = fmaxf(top - kLift<KIND>, t.m[n][x]);
        const float fade = top == -INFINITY ? 1.f : ex2_approx(t.m[n][x] - top);
        t.m[n][x] = top;
        t.l[n][x] *= fade;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          t.o[n][j][x] *= fade;
          t.o[n][j][x + 2] *= fade;
        }
      }
  };
  if constexpr (kBlocks) {
    // A key's score gets the log of its value's scale: weights are then those of the stored numbers, and none is
    // beyond what the reference allows.  s becomes the score over the reference at once (any number is far over the
    // one that a row starts from, so that it is renewed).
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float ks = pow2_bits(exponent_at(exps, i)), lv = static_cast<float>(exponent_at(exps, 2 + i));
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
          const F2 sum = add2({s[i][n][x], s[i][n][x + 1]}, {s2[i][n][x], s2[i][n][x + 1]});
          s2[i][n][x] = sum.x;
          s2[i][n][x + 1] = sum.y;
          const F2 over = fma2(sum, {t.scale[n][0] * ks, t.scale[n][1] * ks}, {lv - t.m[n][0], lv - t.m[n][1]});
          s[i][n][x] = over.x;
          s[i][n][x + 1] = over.y;
        }
    }
    if (!whole) hide();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) top = fmaxf(top, s[i][n][x]);
    if (__any_sync(0xFFFFFFFFu, top > kRenew + kLift<KIND>)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float ks = pow2_bits(exponent_at(exps, i)), lv = static_cast<float>(exponent_at(exps, 2 + i));
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[i][n][x] = fmaf(s2[i][n][x], t.scale[n][x & 1] * ks, lv);
      }
      if (!whole) hide();
      renew();
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[i][n][x] -= t.m[n][x & 1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[i][n][x] = (s[i][n][x] + s2[i][n][x]) * t.scale[n][x & 1];
    if (!whole) hide();
    bool pass = false;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) pass |= s[i][n][x] > t.m[n][x & 1] + (kRenew + kLift<KIND>);
    if (__any_sync(0xFFFFFFFFu, pass)) renew();
  }
  // P^T as the B operand [16 keys x 8 heads].  fp16 P (beside an e4m3 cache) keeps 11 bits; bf16 P would
  // keep 8 and be off by as much as the rounded output, so it is cut there and its remainder goes through a
  // second product with the same values.
  uint32_t pb[2][NB][2], rest[2][NB][2];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const float m0 = t.m[n][0] == -INFINITY ? 0.f : t.m[n][0], m1 = t.m[n][1] == -INFINITY ? 0.f : t.m[n][1];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float e[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        e[x] = ex2_approx(kBlocks ? s[i][n][x] : s[i][n][x] - (x & 1 ? m1 : m0));
        if constexpr (!kBlocks) t.l[n][x & 1] += e[x];
      }
      if constexpr (kBlocks) {
        const float iv = pow2_bits(-exponent_at(exps, 2 + i));
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
          const F2 l = fma2({e[x], e[x + 1]}, {iv, iv}, {t.l[n][0], t.l[n][1]});
          t.l[n][0] = l.x;
          t.l[n][1] = l.y;
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t w;
        if constexpr (k8) {
          const __half2 f = __floats2half2_rn(e[2 * x], e[2 * x + 1]);
          w = *reinterpret_cast<const uint32_t*>(&f);
        } else {
          w = __byte_perm(__float_as_uint(e[2 * x]), __float_as_uint(e[2 * x + 1]), 0x7632);  // upper halves
          rest[i][n][x] = movm_trans(pack_bf16x2(left_over(e[2 * x], __uint_as_float(w << 16)),
                                                 left_over(e[2 * x + 1], __uint_as_float(w & 0xFFFF0000u))));
        }
        pb[i][n][x] = movm_trans(w);
      }
    }
  }
  // O^T += V^T P^T.  Hidden keys' values are cleared: 0 * NaN is no 0.
  // bf16: matrices (keys 0-7, piece 2j), (keys 0-7, 2j+1), (keys 8-15, 2j), (keys 8-15, 2j+1);
  // e4m3: matrices (keys 0-7, 8-15) x (pieces 2j, 2j+1), of which a lane gets channels 2c, 2c+1 (c = lane / 4)
  // of keys 2t, 2t+1: row r of the product's tile is channel 2r, row r + 8 channel 2r + 1
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};  // keys 2t, 2t+1 and 8 further
    if (!whole) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t b = seen >> (i * 16 + x * 8 + (lane & 3) * 2);
        keep[x] = (b & 1u ? 0xFFFFu : 0u) | (b & 2u ? 0xFFFF0000u : 0u);
      }
    }
#pragma unroll
    for (int j = 0; j < kValues; ++j) {
      uint32_t w[4] = {v[j][0], v[j][1], v[j][2], v[j][3]};
      if (i == 0) ldsm4t(v[j], piece_at<D, KIND>(v_at, 16 + key, 2 * j + piece));
      if constexpr (!k8) {
        if (!whole) {
          w[0] &= keep[0];
          w[1] &= keep[0];
          w[2] &= keep[1];
          w[3] &= keep[1];
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          mma16816<false>(t.o[n][j], w, rest[i][n][0], rest[i][n][1]);
          mma16816<false>(t.o[n][j], w, pb[i][n][0], pb[i][n][1]);
        }
      } else {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t f[4];
          widen<KIND, true>(w[2 * x], f[0], f[1]);
          widen<KIND, true>(w[2 * x + 1], f[2], f[3]);
          if (!whole) {
            f[0] &= keep[0];
            f[1] &= keep[0];
            f[2] &= keep[1];
            f[3] &= keep[1];
          }
#pragma unroll
          for (int n = 0; n < NB; ++n) mma16816<true>(t.o[n][2 * j + x], f, pb[i][n][0], pb[i][n][1]);
        }
      }
    }
  }
}

// Channel of accumulator x (0 or 2: rows lane / 4 and 8 further) of tile j.
template <int KIND>
__device__ __forceinline__ int channel_of(int j, int x, int lane) {
  return KIND != kBf16 ? j * 16 + (lane >> 2) * 2 + (x >> 1) : j * 16 + (lane >> 2) + (x >> 1) * 8;
}

struct RowAt {
  __nv_bfloat16* o;  // first head of the row
  float* lse;
  int heads;         // of the row
  int h;             // key-value head
};
template <int NB>
__device__ __forceinline__ RowAt row_at(const DecodeArgs& a, int row) {
  const DecodeParams& p = a.p;
  const auto [b, h, chunk] = row_index(a, row);
  const int head = h * a.group + chunk * 8 * NB;
  return {p.o + b * p.os.seq + head * p.os.head,
          p.lse ? p.lse + static_cast<int64_t>(b) * p.H_q + head : nullptr,
          min(8 * NB, a.group - chunk * 8 * NB), h};
}
template <int KIND>
__device__ __forceinline__ float value_scale(const DecodeArgs& a, int h) {
  return KIND == kE4m3 ? __ldg(a.p.c.v_scale + h) : 1.f;
}

// 1 / l, 0 for a row that saw nothing (l = 0 and O = 0: the output is 0)
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float natural_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, int KIND, int NB>
__device__ __forceinline__ void compute(const DecodeArgs& a, char* smem, uint32_t ring, uint32_t meta,
                                        uint32_t bars, uint32_t exps, int pair, int first_row, const WaitCtl& wait, int lane) {
  using C = Cfg<D, KIND, NB>;
  State<D, KIND, NB> t;
  // the next row's queries, on their way while the last tile of a row is computed (the first row's, while
  // its first tile comes); 16 heads' would take the registers of the accumulators
  constexpr bool kAhead = NB == 1;
  uint32_t ahead[kAhead ? D / 16 : 1][2];
  int ahead_row = first_row;
  if constexpr (kAhead) read_q<D, KIND>(a, first_row, 0, lane, ahead);
  int4* heads = reinterpret_cast<int4*>(smem + C::kOffHead) + 2 * pair;
  bool starts = false;
  for (int done = 0;; ++done) {
    const int stage = done % C::kStages;
    const uint32_t full = bars + stage * 16;
    if (!warp_wait(wait, full, (done / C::kStages) & 1, 4)) return;
    const uint4 x = ld_shared_v4(meta + stage * 16);
    const int row = static_cast<int>(x.x), flags = static_cast<int>(x.z);
    if (row < 0) return;
    if (flags & kFirst) {
      starts = flags & kStarts;
      if constexpr (kAhead) {
        if (ahead_row == row) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            t.q[0][i][0] = ahead[i][0];
            t.q[0][i][1] = ahead[i][1];
          }
        } else {
          read_q<D, KIND>(a, row, 0, lane, t.q[0]);
        }
      } else {
#pragma unroll
        for (int n = 0; n < NB; ++n) read_q<D, KIND>(a, row, n, lane, t.q[n]);
      }
      scale_q<D, KIND, NB>(a, row, lane, t.q, t.scale);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        t.m[n][0] = t.m[n][1] = kLowest<KIND>;
        t.l[n][0] = t.l[n][1] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) t.o[n][j][i] = 0.f;
      }
    }
    if constexpr (kAhead) {
      ahead_row = flags & kLast ? static_cast<int>(x.w) : -1;
      if (ahead_row >= 0) read_q<D, KIND>(a, ahead_row, 0, lane, ahead);
    }
    const uint32_t k_at = ring + stage * C::kStage;
    uint32_t e = 0;
    if constexpr (KIND >= kE4m3Block) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(e) : "r"(exps + stage * 4));
    compute_tile<D, KIND, NB>(t, k_at, k_at + C::kMatrix, x.y, e, lane);
    __syncwarp();
    if (lane == 0) mbar_arrive(full + 8);
    if (!(flags & kLast)) continue;

    // the sums so far are per lane: over the 8 lanes of a column
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) t.l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, t.l[n][i], d);
    if (starts && (flags & kEnds)) {  // the whole row
      const RowAt r = row_at<NB>(a, row);
      const float v_scale = value_scale<KIND>(a, r.h);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const float i0 = inverse(t.l[n][0]) * v_scale, i1 = inverse(t.l[n][1]) * v_scale;
        const int h0 = n * 8 + (lane & 3) * 2;
        if constexpr (KIND != kBf16) {
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const int c = channel_of<KIND>(j, 0, lane);
            if (h0 < r.heads)
              *reinterpret_cast<uint32_t*>(r.o + h0 * a.p.os.head + c) = pack_bf16x2(t.o[n][j][0] * i0, t.o[n][j][2] * i0);
            if (h0 + 1 < r.heads)
              *reinterpret_cast<uint32_t*>(r.o + (h0 + 1) * a.p.os.head + c) = pack_bf16x2(t.o[n][j][1] * i1, t.o[n][j][3] * i1);
          }
        } else {  // [channel][head pair] to [head][channel pair]
          const int h = n * 8 + (lane >> 2);
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int x2 = 0; x2 < 2; ++x2) {
              const uint32_t w = movm_trans(pack_bf16x2(t.o[n][j][2 * x2] * i0, t.o[n][j][2 * x2 + 1] * i1));
              if (h < r.heads)
                *reinterpret_cast<uint32_t*>(r.o + h * a.p.os.head + j * 16 + x2 * 8 + (lane & 3) * 2) = w;
            }
        }
        if (r.lse && lane < 4) {
          if (h0 < r.heads) r.lse[h0] = natural_lse(t.m[n][0], t.l[n][0]);
          if (h0 + 1 < r.heads) r.lse[h0 + 1] = natural_lse(t.m[n][1], t.l[n][1]);
        }
      }
      continue;
    }
    // a part: of a row begun before this warp's run (slot 0, its first part), or of one carried on
    // (slot 1, its last part: nothing will come into the ring any more)
    const int slot = starts ? 1 : 0;
    float* f = slot ? reinterpret_cast<float*>(smem + pair * C::kStages * C::kStage)
                    : reinterpret_cast<float*>(smem + C::kOffPiece + pair * C::kPiece);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int h0 = n * 8 + (lane & 3) * 2;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f[(h0 + (i & 1)) * C::kHeadPitch + channel_of<KIND>(j, i, lane)] = t.o[n][j][i];
      if (lane < 4) {
        float* ml = f + C::kHeads * C::kHeadPitch;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ml[h0 + i] = t.m[n][i];
          ml[C::kHeads + h0 + i] = t.l[n][i];
        }
      }
    }
    if (lane == 0)
      heads[slot] = make_int4(row, (starts ? kStarts : 0) | (flags & kEnds), flags >> kFlagBits, 1);
  }
}

// Joins the CTA's parts, row by row: 16 threads a head, D / 16 channels a thread.  Parts lie in the order of
// the keys; the first of a row says whether the row starts in this CTA, the last whether it ends here.
template <int D, int KIND, int NB>
__device__ __forceinline__ void join_warps(const DecodeArgs& a, char* smem, int tid) {
  using C = Cfg<D, KIND, NB>;
  constexpr int N = D / 16;
  const int lane = tid & 31, c0 = (tid & 15) * 4;  // channels c0 .. c0+3 of each 64
  const int4 mine = lane < 2 * C::kPairs ? reinterpret_cast<const int4*>(smem + C::kOffHead)[lane] : make_int4(0, 0, 0, 0);
  uint32_t left = __ballot_sync(0xFFFFFFFFu, mine.w);
  int carried = 0, carried_row = 0;
  auto part_of = [&](int s) {
    return s & 1 ? reinterpret_cast<const float*>(smem + (s >> 1) * C::kStages * C::kStage)
                 : reinterpret_cast<const float*>(smem + C::kOffPiece + (s >> 1) * C::kPiece);
  };
  while (left) {
    const int i = __ffs(left) - 1, row = __shfl_sync(0xFFFFFFFFu, mine.x, i);
    const uint32_t parts = __ballot_sync(0xFFFFFFFFu, mine.w && mine.x == row);
    left &= ~parts;
    const bool starts = __shfl_sync(0xFFFFFFFFu, mine.y, i) & kStarts;
    const bool ends = __shfl_sync(0xFFFFFFFFu, mine.y, 31 - __clz(parts)) & kEnds;
    if (starts && !ends) {
      carried = __shfl_sync(0xFFFFFFFFu, mine.z, i);
      carried_row = row;
    }
    const RowAt r = row_at<NB>(a, row);
    const Part out = part_at<D>(a.p.workspace, C::kHeads, blockIdx.x, starts ? 1 : 0);
#pragma unroll 1
    for (int h = tid >> 4; h < r.heads; h += 2 * C::kPairs) {
      float m = -INFINITY, l = 0.f, o[N];
#pragma unroll
      for (int c = 0; c < N; ++c) o[c] = 0.f;
      // a warp holds one part of a row at most
      float pm[C::kPairs], pl[C::kPairs];
      const float* from[C::kPairs];
#pragma unroll
      for (int x = 0; x < C::kPairs; ++x) {
        const uint32_t which = (parts >> (2 * x)) & 3u;
        from[x] = part_of(2 * x + (which >> 1)) + h * C::kHeadPitch + c0;
        const float* ml = part_of(2 * x + (which >> 1)) + C::kHeads * C::kHeadPitch + h;
        pm[x] = which ? ml[0] : -INFINITY;
        pl[x] = which ? ml[C::kHeads] : 0.f;
        m = fmaxf(m, pm[x]);
      }
      const float zero = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int x = 0; x < C::kPairs; ++x) {
        if (((parts >> (2 * x)) & 3u) == 0) continue;
        const float w = ex2_approx(pm[x] - zero);
        l += pl[x] * w;
#pragma unroll
        for (int g = 0; g < N / 4; ++g) {
          const float4 y = *reinterpret_cast<const float4*>(from[x] + g * 64);
          o[4 * g] += y.x * w;
          o[4 * g + 1] += y.y * w;
          o[4 * g + 2] += y.z * w;
          o[4 * g + 3] += y.w * w;
        }
      }
      if (starts && ends) {
        const float inv = inverse(l) * value_scale<KIND>(a, r.h);
#pragma unroll
        for (int g = 0; g < N / 4; ++g)
          *reinterpret_cast<uint2*>(r.o + h * a.p.os.head + g * 64 + c0) =
              make_uint2(pack_bf16x2(o[4 * g] * inv, o[4 * g + 1] * inv),
                         pack_bf16x2(o[4 * g + 2] * inv, o[4 * g + 3] * inv));
        if (r.lse && (tid & 15) == 0) r.lse[h] = natural_lse(m, l);
      } else {
#pragma unroll
        for (int g = 0; g < N / 4; ++g)
          *reinterpret_cast<float4*>(out.o + h * D + g * 64 + c0) =
              make_float4(o[4 * g], o[4 * g + 1], o[4 * g + 2], o[4 * g + 3]);
        if ((tid & 15) == 0) {
          out.m[h] = m;
          out.l[h] = l;
        }
      }
    }
  }
  if (tid == 0) reinterpret_cast<int4*>(a.p.workspace)[blockIdx.x] = make_int4(carried, carried_row, 0, 0);
}

template <int D, int KIND, int NB, bool WINDOW>
__global__ void __launch_bounds__(Cfg<D, KIND, NB>::kThreads, 1)
    decode_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D, KIND, NB>;
  extern __shared__ __align__(1024) char smem[];  // the swizzled tiles need the alignment
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc);
  // per thread, the cost before its units, and the tiles and the length of its last one; borrowed until the search is done
  int* before = reinterpret_cast<int*>(smem + C::kOffPiece);
  int* tiles_of = before + C::kThreads;
  let_next_start();
  if ((base & 1023u) != 0) {
    wait_for_previous();
    if (tid == 0) {
      set_status(a.p.c.status, kDevBadMeta, 0x1ff);
      reinterpret_cast<int4*>(a.p.workspace)[blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  if (tid < C::kPairs * C::kStages) {
    mbar_init(base + C::kOffBars + tid * 16, 1);
    mbar_init(base + C::kOffBars + tid * 16 + 8, 1);
  }
  if (tid < 2 * C::kPairs) reinterpret_cast<int4*>(smem + C::kOffHead)[tid] = make_int4(0, 0, 0, 0);
  if (tid == 0) {
    *abort_flag = 0;
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  fence_barrier_init();
  wait_for_previous();

  if (KIND == kE4m3 && tid * 32 < a.p.c.H_kv) {  // the scales are wanted at the start and at the end of a row
    asm volatile("prefetch.global.L1 [%0];" ::"l"(a.p.c.k_scale + tid * 32));
    asm volatile("prefetch.global.L1 [%0];" ::"l"(a.p.c.v_scale + tid * 32));
  }
  // cost of all units: each thread adds up a run of them, then a scan over the threads
  const int per = (a.units + C::kThreads - 1) / C::kThreads;
  const int u0 = min(tid * per, a.units), u1 = min(u0 + per, a.units);
  int mine = 0, tiles = 0, len = 0;
#pragma unroll 1
  for (int u = u0; u < u1; ++u) {
    tiles = unit_tiles<WINDOW>(a, u, true, len);
    mine += row_cost(tiles) * a.rows;
    if (tiles == 0 && u % a.ctas == static_cast<int>(blockIdx.x)) {  // nothing visible: zeros
#pragma unroll 1
      for (int m = 0; m < a.rows; ++m) {
        const RowAt r = row_at<NB>(a, u * a.rows + m);
#pragma unroll 1
        for (int h = 0; h < r.heads; ++h) {
#pragma unroll 1
          for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(r.o + h * a.p.os.head + c) = make_uint4(0, 0, 0, 0);
          if (r.lse) r.lse[h] = -INFINITY;
        }
      }
    }
  }
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, sum, d);
    if (lane >= d) sum += x;
  }
  int* len_of = tiles_of + C::kThreads;
  int* warp_sum = len_of + C::kThreads;
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < C::kThreads / 32; ++w) {
    const int x = warp_sum[w];
    total += x;
    if (w < warp) sum += x;
  }
  before[tid] = sum - mine;
  tiles_of[tid] = tiles;
  len_of[tid] = len;
  __syncthreads();
  // the place of a cost below the total: the last thread with no more before its units, then its unit
  auto locate = [&](int at) {
    int n = 0;
#pragma unroll
    for (int t = 0; t < C::kThreads; t += 32) n += before[t + lane] <= at;
    const int t = __reduce_add_sync(0xFFFFFFFFu, n) - 1;
    Place x{t * per, 0, 0, len_of[t], tiles_of[t]};
    int from = before[t];
    if (per > 1)
#pragma unroll 1
      for (;; ++x.u) {
        x.tiles = unit_tiles<WINDOW>(a, x.u, false, x.len);
        const int cost = row_cost(x.tiles) * a.rows;
        if (at < from + cost || x.u + 1 >= a.units) break;
        from += cost;
      }
    x.m = (at - from) / row_cost(x.tiles);
    x.c = at - from - x.m * row_cost(x.tiles);
    return x;
  };
  const int run = max((total + a.ctas - 1) / a.ctas, a.min_run);  // of a CTA
  int cta0 = min(static_cast<int64_t>(run) * blockIdx.x, static_cast<int64_t>(total));
  int cta1 = min(static_cast<int64_t>(cta0) + run, static_cast<int64_t>(total));
  if (a.whole_rows) {  // ends go to the nearest end of a row
    int* bounds = warp_sum;  // the sums have been read
    if (warp < 2) {
      int at = warp ? cta1 : cta0;
      if (at < total) {
        const Place x = locate(at);
        const int cost = row_cost(x.tiles);
        at += 2 * x.c > cost ? cost - x.c : -x.c;
      }
      if (lane == 0) bounds[warp] = at;
    }
    __syncthreads();
    cta0 = bounds[0];
    cta1 = bounds[1];
  }
  const int share = (cta1 - cta0 + C::kPairs - 1) / C::kPairs;  // of a warp
  const int pair = warp & (C::kPairs - 1);
  const int at = min(cta0 + pair * share, cta1);
  const int until = min(static_cast<uint32_t>(at) + share, static_cast<uint32_t>(cta1));  // the sum may pass 2^31
  Place place{0, 0, 0, 0, 0};
  if (at < until) place = locate(at);
  __syncthreads();

  const WaitCtl wait{abort_flag, a.p.c.status, a.wait_ns};
  const uint32_t ring = base + pair * C::kStages * C::kStage;
  const uint32_t meta = base + C::kOffMeta + pair * C::kStages * 16;
  const uint32_t bars = base + C::kOffBars + pair * C::kStages * 16;
  const uint32_t exps = base + C::kOffExps + pair * C::kStages * 4;
  int fetched = 0, rest = 0;
  if constexpr (C::kPairs == 8) {
    if (warp >= C::kPairs) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
  }
  if (at < until) {
    if (warp >= C::kPairs) {
      Walk w;
      w.u = place.u;
      w.m = place.m;
      w.c = place.c;
      w.plan = make_plan<WINDOW>(a, w.u, place.len, place.tiles, lane);
      w.pos = at;
      w.end = until;
      fetched = fetch<D, KIND, NB, WINDOW>(a, &kmap, &vmap, w, ring, meta, bars, exps, run, wait, lane, rest);
    } else {
      compute<D, KIND, NB>(a, smem, ring, meta, bars, exps, pair, place.u * a.rows + place.m, wait, lane);
    }
  }
  __syncthreads();
  if (*abort_flag) {  // the outputs are undefined; the second kernel must not follow what is not there
    // copies in flight end by themselves, and the CTA must not exit before they have
    for (int i = rest; i < fetched; ++i)
      mbar_wait_drain(bars + (i % C::kStages) * 16, (i / C::kStages) & 1, a.p.c.status, 3);
    if (tid == 0) reinterpret_cast<int4*>(a.p.workspace)[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  if (tid < 32 * C::kPairs) join_warps<D, KIND, NB>(a, smem, tid);
}

// Joins the parts of a row that several CTAs hold: CTA x's header says how many there are, its own
// second part first, then the first parts of the CTAs behind it.  One block a head, one thread a channel.
template <int D, int KIND, int NB>
__global__ void __launch_bounds__(D, (NB == 1 ? 512 : 1024) / D) join_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int kHeads = 8 * NB;
  constexpr int kAtOnce = 16;  // parts whose loads are in flight
  const int h = blockIdx.y;
  float pm[kAtOnce], pl[kAtOnce], po[kAtOnce];
  auto load = [&](int i, int at, bool in) {
    const Part x = part_at<D>(a.p.workspace, kHeads, blockIdx.x + at, at == 0);
    pm[i] = in ? x.m[h] : -INFINITY;
    pl[i] = in ? x.l[h] : 0.f;
    po[i] = in ? x.o[h * D + threadIdx.x] : 0.f;
  };
  wait_for_previous();
  // Most rows have two parts: asked for together with the header (1.3 us less for batches of up to 8 heads a row; with
  // 16, the many blocks that have no row would ask for more than that saves).
  constexpr bool kEarly = NB == 1;
  const int4 head = reinterpret_cast<const int4*>(a.p.workspace)[blockIdx.x];
  if constexpr (kEarly) {
    load(0, 0, true);
    load(1, 1, static_cast<int>(blockIdx.x) + 1 < a.ctas);
  }
  const int n = min(head.x, a.ctas - static_cast<int>(blockIdx.x));
  if (n < 2) return;
  const RowAt r = row_at<NB>(a, head.y);
  if (h >= r.heads) return;
  const float v_scale = value_scale<KIND>(a, r.h);
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int i0 = 0; i0 < n; i0 += kAtOnce) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (!kEarly || i >= 2 || i0 > 0) load(i, i0 + i, i0 + i < n);
    float top = m;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, pm[i]);
    const float zero = top == -INFINITY ? 0.f : top, fade = ex2_approx(m - zero);
    m = top;
    l *= fade;
    o *= fade;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float w = ex2_approx(pm[i] - zero);
      l += pl[i] * w;
      o += po[i] * w;
    }
  }
  r.o[h * a.p.os.head + threadIdx.x] = __float2bfloat16(o * inverse(l) * v_scale);
  if (r.lse && threadIdx.x == 0) r.lse[h] = natural_lse(m, l);
}

template <int D, int KIND, int NB, bool WINDOW>
int launch(DecodeArgs& a, int dev, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  using C = Cfg<D, KIND, NB>;
  // Where no row can have more than 4 tiles a warp pair, rows stay whole: the second kernel, 2 to 3 us on
  // the GPU and a launch, costs more than the few tiles by which runs then differ.
  a.whole_rows = a.most_tiles <= 4 * C::kPairs;
  static std::atomic<bool> allowed[kMaxDevices];  // the shared memory it needs
  if (dev >= kMaxDevices || !allowed[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(decode_kernel<D, KIND, NB, WINDOW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem) != cudaSuccess)
      return -1;
    if (dev < kMaxDevices) allowed[dev].store(true, std::memory_order_relaxed);
  }
  return launch_after(decode_kernel<D, KIND, NB, WINDOW>, dim3(a.ctas), C::kThreads, C::kSmem, stream, a, k, v) &&
                 (a.whole_rows || launch_after(join_kernel<D, KIND, NB>, dim3(a.ctas, a.group < C::kHeads ? a.group : C::kHeads), D,
                              0, stream, a))
             ? 0
             : -1;
}

template <int KIND, bool WINDOW>
int launch_shape(DecodeArgs& a, int dev, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  if (a.heads == 8)
    return a.p.c.d == 128 ? launch<128, KIND, 1, WINDOW>(a, dev, k, v, stream) : launch<64, KIND, 1, WINDOW>(a, dev, k, v, stream);
  return a.p.c.d == 128 ? launch<128, KIND, 2, WINDOW>(a, dev, k, v, stream) : launch<64, KIND, 2, WINDOW>(a, dev, k, v, stream);
}

}  // namespace

template <int KIND>
int launch_decode_kind(DecodeArgs& a, int dev, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  return a.p.window ? launch_shape<KIND, true>(a, dev, k, v, stream) : launch_shape<KIND, false>(a, dev, k, v, stream);
}

}  // namespace cm
