/*
 * cm.h -- C ABI of the descriptor-guided masked attention library (libcm.so).
 *
 * The operations follow "CompileMask: Bridging the Gap Between Expressiveness and Efficiency in
 * Attention Masking":
 *   - section 3.2 (MaskSpec, Regions with a row guard and a visibility rule) and section 3.2.2
 *     (symbolic lowering: AST, DNF normalisation, interval extraction, canonicalisation)
 *       -> cm_compile_spec / cm_spec_* (offline, host only);
 *   - section 3.3 and 3.3.1 (online preprocess kernel evaluating the compiled endpoints against
 *     batch metadata; Execution Descriptor = Interval Table padded with zero-length intervals
 *     plus 2-bit Tile-State Bitmaps; separate forward and backward descriptors)
 *       -> cm_descriptor_sizes / cm_build_descriptor;
 *   - section 3.3.2 (descriptor-guided attention: skip empty tiles, run full tiles unmasked,
 *     check partial tiles against the endpoints with unsigned arithmetic, -inf before the
 *     online softmax) and section 4.4 (unsigned visible-interval check)
 *       -> cm_attn_fwd / cm_attn_bwd.
 *
 * Conventions shared by every entry point
 *   - Every pointer named "device" must point to memory of the current CUDA device.  The library
 *     allocates no device memory: the caller owns every buffer and must keep it alive until the
 *     work queued on `stream` has finished.  The only heap object the library owns is the host
 *     cm_spec returned by cm_compile_spec (free it with cm_spec_free).
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Device work is queued on it and
 *     the call returns without waiting; nothing runs on the CPU in place of a kernel.
 *   - Return value: CM_OK (0) or a negative CM_ERR_* code.  Arguments are validated on the host
 *     before anything is queued; a call that fails validation queues nothing.  Errors detected on
 *     the device (bad segment metadata, a bounded wait that expired) are recorded in the
 *     descriptor's status word and reported by cm_get_status.
 *   - Tensors Q, K, V, O, dO, dQ, dK, dV are bf16, contiguous, layout [B][H][S][d].  The LSE is
 *     fp32 [B][H][S] in natural log.  Row i of a descriptor is a query row (forward) or a key
 *     column (backward).
 *   - Supported shapes: d in {64, 128}; S a positive multiple of 128; tile = 128; at most 2^24
 *     heads (CM_ERR_UNSUPPORTED above that).
 */
#ifndef CM_H_
#define CM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CM_API __attribute__((visibility("default")))

enum {
  CM_OK = 0,
  CM_ERR_PARSE = -1,        /* spec text does not parse or uses an unsupported form */
  CM_ERR_INVALID_ARG = -2,  /* null pointer, bad size, descriptor/shape mismatch */
  CM_ERR_UNSUPPORTED = -3,  /* valid request outside the supported shapes (d, S, tile, limits) */
  CM_ERR_CUDA = -4,         /* a CUDA runtime call or launch failed */
  CM_ERR_TIMEOUT = -5,      /* device status: a bounded wait inside a kernel expired */
  CM_ERR_DEVICE_CHECK = -6, /* device status: segment metadata failed validation */
  CM_ERR_DESC_MISMATCH = -7 /* device status: the backward descriptor's Tile-State Bitmap is not
                               the transpose of the forward one (the two MaskSpecs do not
                               describe the same mask) */
};

/* Opaque compiled MaskSpec (host memory, owned by the caller after cm_compile_spec). */
typedef struct cm_spec cm_spec;

/* Per-batch metadata (section 1 / 2.2: sequence lengths and segment boundaries).
 *   seg  device int32 [B][nseg_max + 1]: seg[b][0] = 0, strictly increasing up to
 *        seg[b][nseg[b]] = S; entries after nseg[b] are ignored.
 *   nseg device int32 [B]: segment count of each sample, 1 <= nseg[b] <= nseg_max. */
typedef struct cm_meta {
  const int32_t* seg;
  const int32_t* nseg;
  int32_t nseg_max;
} cm_meta;

/* Execution Descriptor (section 3.3.1), forward and backward halves.  All buffers are device
 * memory allocated by the caller with the sizes from cm_descriptor_sizes.
 *   form    CM_FORM_VISIBLE (the paper's representation): the Interval Tables hold each row's
 *           visible intervals, ni_f / ni_b = the specs' interval counts.  CM_FORM_MASKED (the
 *           representation section 4.4 compares it with): they hold the maximal runs of
 *           invisible indices of each row in increasing order, ni_f / ni_b = the specs' counts
 *           + 1.  The bitmaps and schedules are the same in both forms.
 *   itab_f  int32 [B][ni_f][S][2]  (start, end) of each visible key interval of query row i,
 *           half open; unused slots and empty intervals are (0, 0)
 *   bm_f    uint32 [B][S/tile][ceil((S/tile)/16)]  2 bits per (q-tile, k-tile):
 *           0 empty, 1 partial, 2 full; k-tile t at bits 2*(t % 16) of word t / 16
 *   itab_b  int32 [B][ni_b][S][2]  visible query intervals of key column j
 *   bm_b    uint32 [B][S/tile][ceil((S/tile)/16)]  (k-tile, q-tile) states
 *   sched_f int32 [B * S/tile]  forward work order: (b << 16 | q_tile), most tiles first
 *   sched_b int32 [B * S/tile]  backward work order: (b << 16 | k_tile), most tiles first
 *   status  int32 [2 + 2 * (S/tile + 1) + 6]  device error word (first element), then the
 *           preprocess kernel's grid barrier and schedule histograms, then the work queues of
 *           the three attention kernels (a next-item counter and a finished-CTA counter each,
 *           returned to zero by the last CTA of every launch); cleared by cm_build_descriptor.
 *           Attention calls that use one descriptor must therefore run one after another (one
 *           stream, or ordered by events), never at the same time. */
#define CM_FORM_VISIBLE 0
#define CM_FORM_MASKED 1
typedef struct cm_descriptor {
  int32_t B, S, tile, ni_f, ni_b, form;
  int32_t* itab_f;
  uint32_t* bm_f;
  int32_t* itab_b;
  uint32_t* bm_b;
  int32_t* sched_f;
  int32_t* sched_b;
  int32_t* status;
} cm_descriptor;

/* ---- offline compiler (host only; section 3.2.2) ------------------------------------------- */

/* Parse and lower a MaskSpec.  Text: one Region per line,
 *     region <guard> : <rule>
 * <guard> is `all` or a boolean expression of the row index i; <rule> is a boolean expression
 * over i and the other index j (&&, ||, !, comparisons < <= > >= == !=).  Integer terms: i, j,
 * S, nseg, integer constants, + - and multiplication by a constant, % by a positive constant
 * (non-negative remainder), min(a, b), max(a, b),
 * seg_idx(e), seg_start(e), seg_end(e), seg_start_at(k), seg_end_at(k).  Lines starting with '#'
 * are comments.  Regions are tried in order; the first whose guard holds applies to the row.
 * On success *out receives a new cm_spec.  On CM_ERR_PARSE a message is written to err (if
 * err_len > 0). */
CM_API int cm_compile_spec(const char* text, cm_spec** out, char* err, size_t err_len);

/* Free a spec from cm_compile_spec (NULL is ignored). */
CM_API void cm_spec_free(cm_spec* spec);

/* The compiler-derived interval count (max slots over the Regions), section 3.3.1. */
CM_API int cm_spec_num_intervals(const cm_spec* spec, int* ni_max);

/* Human-readable lowered form (Regions, slot endpoints, slot conditions) written to buf as a
 * NUL-terminated string; *needed (if not NULL) receives the full length + 1.  Host only. */
CM_API int cm_spec_describe(const cm_spec* spec, char* buf, size_t len, size_t* needed);

/* CUDA C++ source of the mask-specific preprocess kernel (section 3.1: the compiler generates a
 * mask-specific preprocess kernel) of a (forward, backward) pair of specs: their two row
 * evaluators and the shared kernel body "descriptor_core.cuh", which the library carries in
 * itself; one launch of it builds both halves of the descriptor and both schedules.  Written to
 * buf as a NUL-terminated string; *needed (if not NULL) receives the full length + 1.  Host
 * only. */
CM_API int cm_descriptor_kernel_source(const cm_spec* fwd, const cm_spec* bwd, char* buf,
                                       size_t len, size_t* needed);

/* Whether the pair's generated kernel can run.  load = 0: compile it with NVRTC only (host only,
 * no GPU needed).  load = 1: compile it and load it into the current device context, which is
 * what cm_build_descriptor does on its first call with the pair (the result, good or bad, is kept
 * with the forward spec; compiling takes a few tenths of a second).  Returns CM_OK on success,
 * CM_ERR_UNSUPPORTED when NVRTC (libnvrtc.so.13) cannot be opened, CM_ERR_CUDA when compiling or
 * loading failed.  The NVRTC log or the failing step goes to log as a NUL-terminated string (log
 * may be NULL). */
CM_API int cm_descriptor_kernel_status(const cm_spec* fwd, const cm_spec* bwd, int load, char* log,
                                       size_t log_len);

/* cm_descriptor_kernel_source / _status with `spec` as both the forward and the backward spec
 * (one spec's generated code on its own). */
CM_API int cm_spec_kernel_source(const cm_spec* spec, char* buf, size_t len, size_t* needed);
CM_API int cm_spec_kernel_status(const cm_spec* spec, int load, char* log, size_t log_len);

/* ---- online descriptor construction (sections 3.3, 3.3.1) ---------------------------------- */

/* Byte sizes of the descriptor buffers, in the order itab_f, bm_f, itab_b, bm_b, sched_f,
 * sched_b, status, for the given form (CM_FORM_VISIBLE or CM_FORM_MASKED).  tile must be 128.
 * Use the status size as given: the status word may be followed by counters of the preprocess
 * kernel. */
CM_API int cm_descriptor_sizes(const cm_spec* fwd, const cm_spec* bwd, int B, int S, int tile,
                               int form, size_t sizes[7]);

/* Which descriptor kernel cm_build_descriptor runs, for the whole process:
 * CM_PREPROCESS_GENERATED (default): the generated kernel of the (forward, backward) spec pair;
 *   if it cannot be compiled or loaded (see cm_descriptor_kernel_status), the generic kernel runs
 *   instead;
 * CM_PREPROCESS_GENERIC: the generic kernel, which interprets the compiled endpoint programs.
 * Either way one cooperative launch builds both halves and both schedules.
 * Both are GPU kernels and build identical descriptors.  Returns CM_ERR_INVALID_ARG for any other
 * mode.  Not synchronised with builds in flight on other host threads. */
#define CM_PREPROCESS_GENERATED 0
#define CM_PREPROCESS_GENERIC 1
CM_API int cm_set_preprocess_mode(int mode);

/* Queue the preprocess kernel that evaluates both specs against `meta` and fills `desc`: a
 * memset of desc->status (the status word and the kernel's counters), then one cooperative
 * launch (all its blocks resident at once; they meet at one grid barrier before the schedules
 * are written).  desc->B, S, tile, form, ni_f, ni_b must match the specs and sizes; its
 * pointers must be set.  Asynchronous on `stream`. */
CM_API int cm_build_descriptor(const cm_spec* fwd, const cm_spec* bwd, const cm_meta* meta,
                               int B, int S, cm_descriptor* desc, void* stream);

/* ---- descriptor-guided attention (section 3.3.2) -------------------------------------------- */

/* Form of the attention kernels' partial-tile check, for the whole process (full and empty
 * tiles never run one; the forms of section 4.4's ablation plus the default):
 * CM_CHECK_UNSIGNED: per score, for each stored interval [s, e) one subtraction and one unsigned
 *   comparison, (uint32)(x - s) < (uint32)(e - s) (the paper's test);
 * CM_CHECK_TWO_COMPARE: per score, s <= x && x < e for each stored interval;
 * CM_CHECK_RANGE_MASK (default): per row and 32 indices, each stored interval becomes a range
 *   of bits of a 32-bit mask (clamped unsigned differences), and each score tests one bit.
 * With a CM_FORM_MASKED descriptor an index is visible iff it lies in none of the stored
 * intervals.  All forms give the same results.  Returns CM_ERR_INVALID_ARG for any other mode.
 * Not synchronised with launches in flight on other host threads. */
#define CM_CHECK_UNSIGNED 0
#define CM_CHECK_TWO_COMPARE 1
#define CM_CHECK_RANGE_MASK 3
CM_API int cm_set_interval_check(int mode);

/* Forward: o = softmax(scale * q k^T masked by desc) v; lse = natural-log row sums.
 * q, k, v, o: device bf16 [B][H][S][d]; lse: device fp32 [B][H][S].  The mask is shared by
 * all heads of a sample.  A row with no visible key gets o = 0 and lse = -inf. */
CM_API int cm_attn_fwd(const cm_descriptor* desc, const void* q, const void* k, const void* v,
                       void* o, float* lse, int B, int H, int S, int d, float scale,
                       void* stream);

/* Workspace bytes cm_attn_bwd needs: per-row D = rowsum(dO * O) and LSE * log2(e), fp32 (8 bytes
 * per row of B*H*S, each array rounded up to 256 bytes). */
CM_API int cm_attn_bwd_workspace_size(int B, int H, int S, int d, size_t* bytes);

/* Backward: dq, dk, dv (device bf16 [B][H][S][d]) of sum(o * dO) given the forward's o and lse.
 * Section 3.3: each traversal direction has its own descriptor.  Two kernels, the stages below
 * in this order: dQ along query tiles with the forward half of the descriptor (itab_f, bm_f,
 * sched_f), which also writes D and LSE * log2(e) into the workspace, then dK and dV along key
 * tiles with the backward half (itab_b, bm_b, sched_b), which read them.  Every output element is written exactly
 * once (no atomics), so results are deterministic.  `workspace` (device, >= the size above,
 * 16-byte aligned) is overwritten.  Every argument is checked before the first stage is queued.
 * The dK/dV stage also checks on the device that bm_b is the transpose of bm_f and records
 * CM_ERR_DESC_MISMATCH in the status word when it is not (the computation still runs). */
CM_API int cm_attn_bwd(const cm_descriptor* desc, const void* q, const void* k, const void* v,
                       const void* o, const float* lse, const void* d_o, void* dq, void* dk,
                       void* dv, void* workspace, size_t workspace_bytes, int B, int H, int S,
                       int d, float scale, void* stream);

/* The stages of cm_attn_bwd, for callers that queue or time them one by one.  cm_attn_bwd queues
 * cm_attn_bwd_dq, then cm_attn_bwd_dkdv, on one stream with one workspace.
 *   cm_attn_bwd_dq        dq along query tiles with the forward descriptor; reads q, k, v, o, lse,
 *                         d_o (device, layouts as above) and writes the workspace: per row of
 *                         every query tile that sees at least one key, -D = -sum_c dO[c] * O[c]
 *                         and -LSE * log2(e) (-inf for a row that sees nothing), fp32;
 *   cm_attn_bwd_dkdv      dk, dv along key tiles with the backward descriptor (section 3.3);
 *                         reads q, k, v, d_o and the workspace written by cm_attn_bwd_dq (or by
 *                         cm_attn_bwd_prologue) earlier on the same stream;
 *   cm_attn_bwd_prologue  writes the whole workspace (every row) from o, lse and d_o alone, for
 *                         callers that run cm_attn_bwd_dkdv without cm_attn_bwd_dq.
 * Same argument rules and error codes as cm_attn_bwd. */
CM_API int cm_attn_bwd_prologue(const void* o, const float* lse, const void* d_o, void* workspace,
                                size_t workspace_bytes, int B, int H, int S, int d,
                                void* stream);
CM_API int cm_attn_bwd_dkdv(const cm_descriptor* desc, const void* q, const void* k,
                            const void* v, const void* d_o, void* dk, void* dv,
                            const void* workspace, size_t workspace_bytes, int B, int H, int S,
                            int d, float scale, void* stream);
CM_API int cm_attn_bwd_dq(const cm_descriptor* desc, const void* q, const void* k, const void* v,
                          const void* o, const float* lse, const void* d_o, void* dq,
                          void* workspace, size_t workspace_bytes, int B, int H, int S, int d,
                          float scale, void* stream);

/* Limit of every bounded wait inside the attention kernels, for the whole process, in ns
 * (0 restores the default of 2 s; at most 60 s, else CM_ERR_INVALID_ARG).  A wait that reaches it
 * makes its CTA stop: the CTA waits for the copies and MMAs it already issued, records
 * CM_ERR_TIMEOUT in the status word (cm_get_status) and exits, leaving the outputs of the work
 * items it had not finished unwritten (the call's outputs are then undefined); the context and
 * the descriptor stay usable.  This is a diagnostic hook: a very small limit makes ordinary waits
 * expire, which tests the time-out path without a fault.  Not synchronised with launches in
 * flight on other host threads.  (The pages describe no failure handling; this is the library's
 * own.)  cm_attn_decode's waits are bounded by it too; it records CM_ERR_TIMEOUT in the cache's status
 * word (cm_kv_status). */
CM_API int cm_set_wait_limit_ns(unsigned long long ns);

/* ---- backward without a workspace (no counterpart in the paper) ---------------------------- */

/* Size of the library's built-in backward scratch array (32 MiB per GPU that loads libcm.so). */
#define CM_NOALLOC_SCRATCH_BYTES (32u << 20)

/* Same computation and arguments as cm_attn_bwd, minus the workspace, for callers that cannot
 * allocate device memory themselves: plugins whose host framework owns all device memory, or
 * latency-critical threads that must not call cudaMalloc (it can synchronise the device).  The
 * scratch comes from a fixed file-scope device array inside the library instead, so this call
 * allocates nothing.
 *   - Limit: the workspace cm_attn_bwd_workspace_size reports must fit CM_NOALLOC_SCRATCH_BYTES
 *     (B*H*S <= 4,194,304 rows); larger problems return CM_ERR_UNSUPPORTED and queue
 *     nothing.
 *   - The array's device address is looked up (cudaGetSymbolAddress) on the first call on each
 *     device, with that device current; make that first call before any stream capture.
 *   - The array is held by every GPU that loads the library until the process exits.
 *   - All calls share the one array per device, and it keeps the previous call's contents.
 *     Each call first rewrites the part it reads (8 bytes per row of B*H*S: D and
 *     LSE * log2(e)), so nothing needs clearing.  Calls whose work overlaps on the GPU, e.g. on
 *     two streams, race on it: order them on one stream. */
CM_API int cm_attn_bwd_noalloc(const cm_descriptor* desc, const void* q, const void* k,
                               const void* v, const void* o, const float* lse, const void* d_o,
                               void* dq, void* dk, void* dv, int B, int H, int S, int d,
                               float scale, void* stream);

/* ---- serving: a paged key-value cache (no counterpart in the paper) ------------------------- */

/* Generated tokens, one at a time: their keys and values go into a cache made of pages
 * (cm_kv_append), and each new token attends to the cache (cm_attn_decode), under the mask of the
 * prompt's descriptor where one is given, or to pages that a cheap score selects for it
 * (cm_select_pages).  Beside the conventions above:
 *   - "lens" is the number of tokens a sequence holds; token p of sequence b is row
 *     p % page_size of page page_table[b][p / page_size].
 *   - Index arrays are read on the device, so a captured graph can be replayed with new lengths
 *     and page tables.  Values that would lead out of bounds (a page number outside
 *     [0, num_pages), a length beyond the table) are not followed: the kernel records
 *     CM_ERR_DEVICE_CHECK in the cache's status word and skips what they name, as each entry
 *     point says.
 *   - Keys past a sequence's length, and keys that a mask hides, are never used: whatever their
 *     memory holds (NaN and infinities too) does not reach an output.
 *   - An infinite value of a key that is used makes its channel of o infinite (NaN beside the other
 *     infinity), and a NaN makes it NaN; the other channels do not change.  Weights are held in fp32: one
 *     below 2^-110 of a row's largest may count as 0, and 0 times an infinity is NaN.  Weights of at
 *     most 1 times values are summed before the division: beside a bf16 cache, where a row's keys times
 *     the largest |v| pass 2^127, an output may overflow.
 *   - Beside 8-bit caches weights are rounded to fp16: to 11 bits each, and below 2^-21 of the row's largest to 2^-32 of
 *     that.  With block scales this holds for the products of weights and their values' scales. */

#define CM_KV_BF16 0
#define CM_KV_E4M3 1
#define CM_KV_E4M3_BLOCK 2
#define CM_KV_INT8_BLOCK 3

/* The cache.  All pointers are device memory of the caller, 16-byte aligned but the scales, the
 * summary scales and the status word (4 bytes).
 *   k, v         [num_pages][H_kv][page_size][d] of the type `dtype` names: bf16, or e4m3 with one
 *                positive fp32 scale per head (value = stored * scale).  Pages may lie apart:
 *                page n starts at n * k_page_stride (v_page_stride) elements, a multiple of 16
 *                bytes and at least H_kv * page_size * d.
 *                CM_KV_E4M3_BLOCK and CM_KV_INT8_BLOCK: e4m3, or whole numbers in 8 bits, with a scale for each
 *                block of 16 consecutive tokens (those of a page from a multiple of 16 on) and head.
 *   k_scale, v_scale  fp32 [H_kv] for CM_KV_E4M3, fp32 [num_pages][H_kv][page_size / 16] for the block types
 *                (written by cm_kv_append: positive powers of two within 2^-32 .. 2^32; any other number there counts as
 *                the power of two that its exponent says, held to that range), NULL for bf16.
 *   summary      int8 [num_pages][H_kv][2][d] and summary_scale fp32 [num_pages][H_kv], both or
 *                neither (NULL): per page, head and channel the largest key, then the smallest,
 *                over the tokens the page holds, in units of summary_scale.  With a = the largest
 *                magnitude of any channel's two, summary_scale is the smallest power of two 2^e
 *                with a <= 127 * 2^e, e held to [-50, 50]; the largest keys are rounded up, the
 *                smallest down, and held to [-127, 127].  NaN keys are passed over.
 *                Maintained by cm_kv_append, read by cm_select_pages.
 *   status       int32: 0, or the first device error; zeroed by the caller when it makes the
 *                cache, read and zeroed by cm_kv_status.
 * page_size is 16, 32, 64 or 128; d 64 or 128; H_kv at most 1024; num_pages * H_kv * page_size
 * below 2^40. */
typedef struct cm_kv_cache {
  int32_t num_pages, page_size, H_kv, d, dtype;
  int64_t k_page_stride, v_page_stride;
  void* k;
  void* v;
  const float* k_scale;
  const float* v_scale;
  int8_t* summary;
  float* summary_scale;
  int32_t* status;
} cm_kv_cache;

/* The sequences of a call: page_table device int32 [B][max_pages], lens device int32 [B].
 * Entries of the table past a sequence's tokens may hold anything.  B at most 32767; max_pages *
 * page_size at most 2^27; for cm_attn_decode, with n the keys a table (or a selection) has room for and
 * one row for up to 16 query heads of a key-value head, rows * (ceil(n / 32) + 2) below 2^31 - 320, where
 * rows = B * H_kv * ceil(H_q / H_kv / 16). */
typedef struct cm_kv_seqs {
  int32_t B, max_pages;
  const int32_t* page_table;
  const int32_t* lens;
} cm_kv_seqs;

/* New tokens of cm_kv_append: bf16 tensors whose last axis (d) is contiguous, with strides in
 * elements for {sequence, head, token}, each a multiple of 8.
 *   k, v    H_kv heads; q (may be NULL) H_q heads, rotated into q_out; k_out (may be NULL) receives
 *           the rotated keys.  q_out may be q, and k_out k, with the same strides; otherwise
 *           outputs overlap nothing else, nor themselves (an output's strides are at least d
 *           along every axis of more than one entry; inputs may be expanded, strides of 0).
 *   cu_new  packed tokens: device int32 [B + 1], ascending, sequence b's are tokens cu_new[b] .. cu_new[b+1]-1
 *           of n_tokens (the sequence strides are not used).  NULL: padded tokens, sequence b's
 *           are tokens 0 .. n_new[b]-1 of n_tokens; n_new (device int32 [B]) NULL: all n_tokens.
 *   max_new the most tokens any sequence appends in this call (host), at most n_tokens.
 *   rope    fp32 [rope_len][rot_dim / 2][2]: cosine and sine of each position's angles.  The first
 *           rot_dim channels (a multiple of 16, at most d; 0: no rotation, rope NULL) are rotated
 *           in pairs (i, i + rot_dim / 2), or (2i, 2i + 1) if interleaved:
 *           (x, y) -> (x cos - y sin, y cos + x sin), every product and sum rounded to fp32 once.
 *   new_lens device int32 [B] (may be NULL; no part of lens, n_new, cu_new or granted): receives lens[b] + the tokens
 *           appended.
 *   granted packed tokens only: device int32 [B] (may be NULL: all), the tokens that each sequence may append, as
 *           cm_kv_reserve gives them.  Sequence b appends the first granted[b] of its own, which must be 0 to all of them;
 *           the others count as tokens of no sequence.  (Padded tokens say the same by n_new.) */
typedef struct cm_kv_new {
  const void* k;
  const void* v;
  const void* q;
  void* q_out;
  void* k_out;
  int64_t k_stride[3], v_stride[3], q_stride[3], q_out_stride[3], k_out_stride[3];
  const int32_t* cu_new;
  const int32_t* n_new;
  int32_t n_tokens, max_new, H_q;
  int32_t rot_dim, interleaved, rope_len;
  const float* rope;
  int32_t* new_lens;
  const int32_t* granted;
} cm_kv_new;

/* Append: token i of sequence b gets position p = lens[b] + i; its key and query are rotated to p
 * and rounded to bf16, its key and value stored in the cache (e4m3: the bf16 value divided by the
 * head's scale, rounded to nearest, held to +-448), and the summaries of the pages it touches
 * are made anew from all the tokens these then hold.  lens is read only.
 * Block types: with a the largest magnitude of a call's new keys (values) in a block (NaN passed over), 2^e is the
 * smallest power of two with a <= 448 * 2^e (e4m3) or a <= 127 * 2^e (int8), e held to [-32, 32].  A block without
 * earlier tokens (none at a position below lens[b]) gets it as its scale; one that has some gets the larger of it and its
 * own, and where that is larger its earlier tokens become round(stored * old / new).  New tokens are stored as
 * round(x / scale), held to +-448 or +-127; halves go to even; a NaN is kept by e4m3 and becomes 0 in int8.  So what
 * a block holds depends on how many calls its tokens came in, by these roundings alone.  No calibration goes before, and an outlier
 * costs 16 tokens of one head their precision.
 * A sequence whose length or token count is out of range (lens[b] < 0, more than max_new tokens,
 * tokens outside n_tokens, granted[b] below 0 or above its tokens, positions past the table or rope_len) appends nothing (new_lens[b] =
 * lens[b]), and tokens of a page outside the pool are left out (their q_out and k_out are written);
 * both record CM_ERR_DEVICE_CHECK.  Tokens of no sequence, and their outputs, are left alone.
 * Sequences must not append to a page they share. */
CM_API int cm_kv_append(const cm_kv_cache* cache, const cm_kv_seqs* seqs, const cm_kv_new* tok,
                        void* stream);

/* Workspace bytes of cm_attn_decode (device, 16-byte aligned, contents irrelevant before and
 * after the call; calls whose work may overlap need one each). */
CM_API int cm_attn_decode_workspace_size(int B, int H_q, int H_kv, int d, size_t* bytes);

/* Attention of one new token per sequence, the last of its lens[b] tokens:
 * o[b][h] = softmax_j(scale * q[b][h] . k[j]) v[j] over the visible j < lens[b], of key-value head
 * h / (H_q / H_kv).  q, o: bf16 [B][H_q][d] with strides in elements for {sequence, head}, multiples
 * of 8; lse: fp32 [B][H_q] in natural log, or NULL.  H_q is a multiple of H_kv.  (Beside an 8-bit cache,
 * channels of q below 2^-31 of their head's largest lose bits; beside block types all do, where the head's largest times
 * scale passes 2^108.)  o may be q with the same strides; otherwise
 * outputs overlap nothing else, nor themselves (o_stride at least d).
 *   desc  NULL: every token is visible.  Else a descriptor of B samples with S >= lens[b] in the
 *         CM_FORM_VISIBLE form: the token sees what row lens[b] - 1 of the forward half says, cut
 *         at lens[b].  One built for the prompt's MaskSpec with room for the tokens to come (the
 *         last segment ending at S) serves the prompt and every token after it.
 *   sel   NULL, or device int32 [B][H_kv][sel_max] with nsel device int32 [B][H_kv]: only the pages
 *         sel[b][g][0 .. nsel[b][g]-1] (places in the sequence's table, ascending; nsel is held to
 *         [0, sel_max]) are attended to.  Not together with desc.
 * A row with no visible key, or whose visible keys all score -inf, gets o = 0 and lse = -inf, and
 * so does a sequence whose length is below 0, beyond the table or beyond
 * desc->S (with CM_ERR_DEVICE_CHECK); a page outside the pool, or a selected page that is not above the
 * entry before it or is past the sequence, is skipped (same).  A visible key
 * whose score is NaN or +inf makes its head's o and lse NaN.
 * The sums of a row are split over the keys in a way that depends on all the batch's lengths; the
 * same call gives the same bits every time. */
CM_API int cm_attn_decode(const cm_kv_cache* cache, const cm_kv_seqs* seqs,
                          const cm_descriptor* desc, const int32_t* sel, const int32_t* nsel,
                          int sel_max, const void* q, const int64_t q_stride[2], void* o,
                          const int64_t o_stride[2], float* lse, int H_q, float scale,
                          void* workspace, size_t workspace_bytes, void* stream);

/* The same under a sliding window with a few first tokens that stay visible (sinks): the token at
 * position p = lens[b] - 1 sees the positions j < sinks and p - window < j <= p (window >= 1, sinks >= 0).
 * Arguments, results and errors as for cm_attn_decode, without a descriptor's limit on the length.  The
 * page table's entries of pages that hold no visible key are not read, so those pages may be anybody's.  (With n of
 * cm_kv_seqs' limit at most the keys that sinks and window can cover.)  For prompts and training the same
 * mask is a MaskSpec, "region i < W + A : j <= i" then "region all : j < A || (j > i - W && j <= i)" for a
 * window W and A sinks. */
CM_API int cm_attn_decode_window(const cm_kv_cache* cache, const cm_kv_seqs* seqs, int window,
                                 int sinks, const void* q, const int64_t q_stride[2], void* o,
                                 const int64_t o_stride[2], float* lse, int H_q, float scale,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of cm_select_pages (rules as for cm_attn_decode's). */
CM_API int cm_select_pages_workspace_size(int B, int H_kv, int max_pages, size_t* bytes);

/* For every sequence and key-value head, the sel_max pages whose summaries promise the largest
 * scores for the new token's queries.  With f from the largest |q| of a query head as e is from a
 * page's keys, x = rint(q / 2^f) (halves to even, held to [-127, 127]) and
 *   score(page) = max over the group's query heads of
 *                 2^(e + f) * sum_c (x_c > 0 ? x_c * largest_c : x_c * smallest_c),
 * which is exact: whole numbers, scaled by powers of two.  The first keep_first and the last
 * keep_last pages of the sequence come before all others (keep_first + keep_last <= sel_max); the
 * rest by score, the lowest page first among equals.  sel [B][H_kv][sel_max] receives them in
 * ascending order, -1 behind the last, nsel [B][H_kv] their number: all pages of a sequence that
 * holds no more than sel_max.  q as in cm_attn_decode; a summary of a page outside the pool
 * counts as the lowest score, a length out of range selects nothing (both with
 * CM_ERR_DEVICE_CHECK).  sel_max at most 8192; max_pages at most 32768. */
CM_API int cm_select_pages(const cm_kv_cache* cache, const cm_kv_seqs* seqs, const void* q,
                           const int64_t q_stride[2], int H_q, int keep_first, int keep_last,
                           int32_t* sel, int32_t* nsel, int sel_max, void* workspace,
                           size_t workspace_bytes, void* stream);

/* Wait for `stream`, then read the cache's status word and zero it: CM_OK or the first error
 * recorded since it was last zeroed (CM_ERR_DEVICE_CHECK, CM_ERR_TIMEOUT; CM_ERR_CUDA if the wait
 * or a copy itself failed). */
CM_API int cm_kv_status(const cm_kv_cache* cache, void* stream);

/* The pages of a pool and the page tables that are made of them, on the device: cm_kv_reserve takes pages
 * for the tokens to come out of a list of free ones, cm_kv_release puts them back.  A step of a serving
 * loop is reserve, append (cm_kv_append with n_new = granted, or packed tokens with granted beside cu_new), attention, release;
 * nothing of it is read on the host, so it can be captured into one graph.
 *   num_pages, page_size, B, max_pages  as in cm_kv_cache and cm_kv_seqs (same limits)
 *   window, sinks  window 0: sequences keep all their pages until they end.  Else pages that hold no token
 *                  which a token to come sees under cm_attn_decode_window(window, sinks) are given back.
 *   page_table     device int32 [B][max_pages], as in cm_kv_seqs
 *   free_pages     device int32 [num_pages]: the numbers of the free pages, as many as the state says
 *   status         device int32: 0, or the first device error (cm_kv_pages_status)
 * State, device int32 [B + 1][2], 8-byte aligned: for sequence b the pages {lo, hi} that it owns, which are the entries
 * [0, f) and [max(lo, f), hi) of its row below hi, with f = ceil(sinks / page_size); in row B {free pages, 0}.  Both
 * calls read `state` and write all of `new_state` (memory that is no part of what the call reads, as `granted`); the next call goes on from there, so the calls on one pool
 * run one after another (one stream, or ordered by events).  A new pool starts
 * with all pages in free_pages, {0, 0} for every sequence and {num_pages, 0}. */
typedef struct cm_kv_pages {
  int32_t num_pages, page_size, B, max_pages, window, sinks;
  int32_t* page_table;
  int32_t* free_pages;
  int32_t* status;
} cm_kv_pages;

/* Pages for the tokens that each sequence is about to append behind its lens[b], counted as in cm_kv_new
 * (cu_new, n_new, n_tokens, max_new): its row gets the pages it lacks, from the end of the list, in
 * the order of the sequences.  From the first sequence on for which too few are left, sequences that need a page get none.
 *   granted  device int32 [B] (may be NULL): the tokens that may be appended, all of a
 *            sequence's or 0.  A row that was granted nothing keeps its entries, which may name pages that are another
 *            sequence's by now, so an append that does not heed `granted` would write there.
 *   slots    device int64, [n_tokens] for packed tokens, [B][n_tokens] for padded ones (may be NULL): each new token's
 *            place in the pool, page * page_size + row; -1 where none was granted.  Places of no token are left alone.
 * A sequence whose length, token count or state is out of range (as in cm_kv_append; lo * page_size <= lens[b] <= hi *
 * page_size, hi <= max_pages), and every sequence behind one at which cu_new falls, gets nothing, keeps its state and its slots are
 * not written; a number in the list or the table
 * that names no page becomes -1 in the row, and -1 in slots.  Both record CM_ERR_DEVICE_CHECK.  Entries of a row below hi are not changed, and
 * entries of the list not at all. */
CM_API int cm_kv_reserve(const cm_kv_pages* pages, const int32_t* state, int32_t* new_state,
                         const int32_t* lens, const int32_t* cu_new, const int32_t* n_new, int n_tokens,
                         int max_new, int32_t* granted, int64_t* slots, void* stream);

/* Pages back into the list, behind its end, in the order of the sequences and of their rows: all that a sequence with
 * done[b] != 0 owns (done: device int32 [B], may be NULL), and under a window, of the others, those that lie wholly
 * before the position lens[b] - window but not among the first f.  The rows keep their entries, which
 * are no longer the sequence's: a call that reads them reads what the page's new owner put there (attention under the same window does not).
 * After its end a row of the table is ready for another sequence with lens[b] = 0.
 * Lengths must not fall behind a release by more than what the window still covers.  A sequence whose state is out of
 * range, or under a window its length (beyond hi * page_size), keeps its state and gives nothing back; a number that names no page goes into the list as it is
 * (cm_kv_reserve will not hand it out), and pages beyond num_pages in the list are dropped; these record
 * CM_ERR_DEVICE_CHECK. */
CM_API int cm_kv_release(const cm_kv_pages* pages, const int32_t* state, int32_t* new_state,
                         const int32_t* lens, const int32_t* done, void* stream);

/* cm_kv_status of the pool's status word. */
CM_API int cm_kv_pages_status(const cm_kv_pages* pages, void* stream);

/* ---- status --------------------------------------------------------------------------------- */

/* Wait for `stream`, then read desc->status: CM_OK, CM_ERR_TIMEOUT, CM_ERR_DEVICE_CHECK or
 * CM_ERR_DESC_MISMATCH, the first error recorded since cm_build_descriptor cleared the word
 * (CM_ERR_CUDA if the wait or copy itself failed). */
CM_API int cm_get_status(const cm_descriptor* desc, void* stream);

/* Static description of a CM_* code. */
CM_API const char* cm_error_string(int code);

#ifdef __cplusplus
}
#endif

#endif /* CM_H_ */
