// Host side of cm_attn_decode: the plan of a call that does not depend on lengths, and the tensor maps.  The kernels are
// in attn_decode.cuh.
#include <atomic>

#include "attn_decode.h"
#include "tma_host.h"

namespace cm {
namespace {

// 3-D map of a pool: [pages][heads * page size][d], boxes of `rows` keys x 128 bytes (64 where a row
// is no longer), swizzled by that width.
bool make_pool_map(CUtensorMap* map, const void* base, const KvView& c, int64_t page_bytes) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const int item = c.kind == kBf16 ? 2 : 1, P = 1 << c.log2_page, row = c.d * item;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(c.H_kv) * P,
                              static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(page_bytes)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>((row < 128 ? row : 128) / item),
                             static_cast<cuuint32_t>(P < kTileKeys ? P : kTileKeys), 1};
  const cuuint32_t steps[3] = {1, 1, 1};
  return enc(map, item == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
             row < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count(int dev) {
  static std::atomic<int> known[kMaxDevices];
  int n = dev < kMaxDevices ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return -1;
    if (dev < kMaxDevices) known[dev].store(n, std::memory_order_relaxed);
  }
  return n < kMaxCtas ? n : kMaxCtas;
}

// Heads of a row: 8 where a group has no more, else 16 (a larger group takes several rows, whose
// second reading of the keys comes from L2).
int heads_of(int group) { return group <= 8 ? 8 : 16; }

}  // namespace

size_t decode_workspace_bytes(int, int H_q, int H_kv, int d) {
  return kMaxCtas * 16 + static_cast<size_t>(kMaxCtas) * 2 * heads_of(H_q / H_kv) * (d + 2) * 4;
}

static int64_t table_tiles(const DecodeParams& p) {
  return ((static_cast<int64_t>(p.sel ? p.sel_max : p.c.max_pages) << p.c.log2_page) + kTileKeys - 1) / kTileKeys;
}

static int64_t most_tiles(const DecodeParams& p) {
  const int64_t room = table_tiles(p);
  if (!p.window) return room;
  // a window that starts inside a tile takes one more
  const int64_t seen = (int64_t{p.sinks} + kTileKeys - 1) / kTileKeys + (int64_t{p.window} + kTileKeys - 1) / kTileKeys + 1;
  return seen < room ? seen : room;
}

bool decode_fits(const DecodeParams& p) {
  const int group = p.H_q / p.c.H_kv, heads = heads_of(group);
  const int64_t rows = static_cast<int64_t>(p.c.B) * p.c.H_kv * ((group + heads - 1) / heads);
  return rows * (most_tiles(p) + kRowCost) < (1LL << 31) - kMaxCtas;  // the kernel adds less than its grid to the sum
}

int launch_attn_decode(const DecodeParams& p, uint64_t wait_ns, cudaStream_t stream) {
  DecodeArgs a;
  a.p = p;
  a.group = p.H_q / p.c.H_kv;
  const int heads = heads_of(a.group);
  a.heads = heads;
  a.chunks = (a.group + heads - 1) / heads;
  a.units = p.sel ? p.c.B * p.c.H_kv : p.c.B;
  a.rows = p.sel ? a.chunks : p.c.H_kv * a.chunks;
  a.by_chunks = make_divisor(a.chunks);
  a.by_heads = make_divisor(p.c.H_kv);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  a.ctas = sm_count(dev);
  a.min_run = 4 + kRowCost;
  a.most_tiles = most_tiles(p);
  a.wait_ns = wait_ns;
  if (a.ctas < 1) return -1;
  CUtensorMap k, v;
  if (!make_pool_map(&k, p.c.k, p.c, p.c.k_page_bytes) || !make_pool_map(&v, p.c.v, p.c, p.c.v_page_bytes))
    return -1;
  switch (p.c.kind) {
    case kBf16: return launch_decode_kind<kBf16>(a, dev, k, v, stream);
    case kE4m3: return launch_decode_kind<kE4m3>(a, dev, k, v, stream);
    case kE4m3Block: return launch_decode_kind<kE4m3Block>(a, dev, k, v, stream);
    case kInt8Block: return launch_decode_kind<kInt8Block>(a, dev, k, v, stream);
  }
  return -1;
}

}  // namespace cm
