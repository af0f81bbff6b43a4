// Internal interface of the serving kernels (append, decode, page selection): what the C ABI
// (api_decode.cu) hands to their launchers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace cm {

// Limit of each bounded wait inside the kernels (cm_set_wait_limit_ns; kept in api.cu).
uint64_t wait_limit_ns();

// The cache and the sequences of a call (cm_kv_cache and cm_kv_seqs, checked).
struct KvView {
  char* k;
  char* v;
  int64_t k_page_bytes, v_page_bytes;  // distance of two pages
  const float* k_scale;                // [H_kv], e4m3 only
  const float* v_scale;
  int8_t* summary;                     // [num_pages][H_kv][2][d]
  float* summary_scale;                // [num_pages][H_kv]
  int32_t* status;
  const int32_t* table;                // [B][max_pages]
  const int32_t* lens;                 // [B]
  int num_pages, log2_page, H_kv, d, e4m3;
  int B, max_pages;
};

struct Strides {
  int64_t seq, head, token;  // elements
};

struct AppendParams {
  KvView c;
  const __nv_bfloat16 *k, *v, *q;
  __nv_bfloat16 *q_out, *k_out;
  Strides ks, vs, qs, qos, kos;
  const int32_t *cu_new, *n_new;
  int n_tokens, max_new, H_q;
  int rot_dim, interleaved, rope_len;
  const float* rope;
  int32_t* new_lens;
};
// Blocks that go by page (with summaries); the rest of the grid is below 2^30.
int64_t append_page_blocks(const AppendParams& p);
int launch_kv_append(const AppendParams& p, cudaStream_t stream);

struct DecodeParams {
  KvView c;
  const int32_t* itab;  // forward Interval Table [B][NI][S][2], or nullptr
  int NI, S;
  const int32_t* sel;   // [B][H_kv][sel_max] with nsel [B][H_kv], or nullptr
  const int32_t* nsel;
  int sel_max;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  Strides qs, os;
  float* lse;           // [B][H_q] or nullptr
  int H_q;
  float scale;
  void* workspace;
};
// Whether the call's work counts (rows of tiles of 32 keys) stay within 31 bits.
bool decode_fits(const DecodeParams& p);
size_t decode_workspace_bytes(int B, int H_q, int H_kv, int d);
int launch_attn_decode(const DecodeParams& p, uint64_t wait_ns, cudaStream_t stream);

struct SelectParams {
  KvView c;
  const __nv_bfloat16* q;
  Strides qs;
  int H_q, keep_first, keep_last, sel_max;
  int32_t* sel;
  int32_t* nsel;
  float* scores;  // workspace [B][H_kv][score_pitch(max_pages)]
};
// scores of a row, padded so that every row starts on 16 bytes
__host__ __device__ constexpr int score_pitch(int max_pages) { return (max_pages + 3) & ~3; }
int launch_select_pages(const SelectParams& p, cudaStream_t stream);

// Launches that follow one another in a serving step (append, scores, selection, attention, joining)
// are a few microseconds each: every kernel lets the next one's blocks start early and waits for
// the one before it to complete, memory included, before it reads or writes anything in memory.
template <class F, class... A>
bool launch_after(F* kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute overlap;
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- device helpers shared by the kernels ---------------------------------------------------

// Power of two 2^e, e within the normal range, by its bits.
__device__ __forceinline__ float pow2_bits(int e) { return __int_as_float((e + 127) << 23); }

// e of the smallest power of two with a <= 127 * 2^e, held to [-50, 50] (a >= 0; infinities give
// 50).  With a = m * 2^x, m in [1, 2): 127 * 2^e = 1.984375 * 2^(e + 6), so e = x - 6, or x - 5 for
// m > 1.984375 = 0x3F.. mantissa bits 0x7E0000.
__device__ __forceinline__ int scale_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = static_cast<int>(u >> 23) - 127 - 6 + ((u & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  return min(max(e, -50), 50);
}

}  // namespace cm
