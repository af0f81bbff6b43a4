// C ABI of the serving entry points: the paged key-value cache (declarations in include/cm.h).
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "../../include/cm.h"
#include "kv_cache.h"
#include "ptx.cuh"

namespace {

constexpr int kMaxHeads = 16384;
constexpr int kMaxB = 32767;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool good_ptr(const void* p) { return p && aligned(p, 16); }
bool good_ints(const void* p) { return p && aligned(p, 4); }

int check_cache(const cm_kv_cache* c) {
  if (!c || c->num_pages < 1 || c->H_kv < 1) return CM_ERR_INVALID_ARG;
  if (c->dtype != CM_KV_BF16 && c->dtype != CM_KV_E4M3) return CM_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return CM_ERR_UNSUPPORTED;
  if ((c->d != 64 && c->d != 128) || c->H_kv > 1024) return CM_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->num_pages) * c->H_kv >= (1LL << 40) / c->page_size)
    return CM_ERR_UNSUPPORTED;
  if (!good_ptr(c->k) || !good_ptr(c->v) || !good_ints(c->status)) return CM_ERR_INVALID_ARG;
  const int item = c->dtype == CM_KV_E4M3 ? 1 : 2;
  const int64_t page = static_cast<int64_t>(c->H_kv) * c->page_size * c->d;
  for (const int64_t s : {c->k_page_stride, c->v_page_stride}) {
    if (s < page || (s * item) % 16 != 0) return CM_ERR_INVALID_ARG;
    if (s >= (1LL << 38)) return CM_ERR_UNSUPPORTED;  // strides of a tensor map end at 2^40 bytes
  }
  if (c->dtype == CM_KV_E4M3 ? !(good_ints(c->k_scale) && good_ints(c->v_scale))
                             : (c->k_scale || c->v_scale))
    return CM_ERR_INVALID_ARG;
  if ((c->summary != nullptr) != (c->summary_scale != nullptr)) return CM_ERR_INVALID_ARG;
  if (c->summary && (!good_ptr(c->summary) || !good_ints(c->summary_scale)))
    return CM_ERR_INVALID_ARG;
  return CM_OK;
}

int check_seqs(const cm_kv_cache* c, const cm_kv_seqs* s) {
  if (!s || s->B < 1 || s->max_pages < 1) return CM_ERR_INVALID_ARG;
  if (s->B > kMaxB || static_cast<int64_t>(s->max_pages) * c->page_size > (1LL << 27))
    return CM_ERR_UNSUPPORTED;
  if (!good_ints(s->page_table) || !good_ints(s->lens)) return CM_ERR_INVALID_ARG;
  return CM_OK;
}

int check_both(const cm_kv_cache* c, const cm_kv_seqs* s) {
  const int rc = check_cache(c);
  return rc != CM_OK ? rc : check_seqs(c, s);
}

bool good_strides(const int64_t* s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i] % 8 != 0 || s[i] < 0) return false;
  return true;
}

// Whether an output's rows of d elements lie apart along every axis that has more than one entry.
bool rows_apart(const int64_t* s, const int64_t* entries, int n, int d) {
  for (int i = 0; i < n; ++i)
    if (entries[i] > 1 && s[i] < d) return false;
  return true;
}

bool same_strides(const int64_t* a, const int64_t* b) {
  return a[0] == b[0] && a[1] == b[1] && a[2] == b[2];
}

cm::KvView view(const cm_kv_cache* c, const cm_kv_seqs* s) {
  cm::KvView v;
  const int item = c->dtype == CM_KV_E4M3 ? 1 : 2;
  v.k = static_cast<char*>(c->k);
  v.v = static_cast<char*>(c->v);
  v.k_page_bytes = c->k_page_stride * item;
  v.v_page_bytes = c->v_page_stride * item;
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.summary = c->summary;
  v.summary_scale = c->summary_scale;
  v.status = c->status;
  v.table = s->page_table;
  v.lens = s->lens;
  v.num_pages = c->num_pages;
  v.log2_page = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  v.H_kv = c->H_kv;
  v.d = c->d;
  v.e4m3 = c->dtype == CM_KV_E4M3;
  v.B = s->B;
  v.max_pages = s->max_pages;
  return v;
}

cm::Strides strides3(const int64_t* s) { return {s[0], s[1], s[2]}; }

int check_heads(int H_q, int H_kv) {
  if (H_q < 1 || H_q % H_kv != 0) return CM_ERR_INVALID_ARG;
  return H_q > kMaxHeads ? CM_ERR_UNSUPPORTED : CM_OK;
}

}  // namespace

extern "C" {

CM_API int cm_kv_append(const cm_kv_cache* cache, const cm_kv_seqs* seqs, const cm_kv_new* t,
                        void* stream) {
  int rc = check_both(cache, seqs);
  if (rc != CM_OK) return rc;
  if (!t) return CM_ERR_INVALID_ARG;
  const bool none = t->n_tokens == 0;  // tensors without elements may have no memory
  if (!none && (!good_ptr(t->k) || !good_ptr(t->v))) return CM_ERR_INVALID_ARG;
  if (!good_strides(t->k_stride, 3) || !good_strides(t->v_stride, 3)) return CM_ERR_INVALID_ARG;
  if ((t->q != nullptr) != (t->q_out != nullptr)) return CM_ERR_INVALID_ARG;
  if (t->q && !none) {
    if (!good_ptr(t->q) || !good_ptr(t->q_out) || t->H_q < 1) return CM_ERR_INVALID_ARG;
    if (t->H_q > kMaxHeads) return CM_ERR_UNSUPPORTED;
    if (!good_strides(t->q_stride, 3) || !good_strides(t->q_out_stride, 3))
      return CM_ERR_INVALID_ARG;
    if (t->q == t->q_out && !same_strides(t->q_stride, t->q_out_stride)) return CM_ERR_INVALID_ARG;
  }
  if (t->k_out && !none) {
    if (!good_ptr(t->k_out) || !good_strides(t->k_out_stride, 3)) return CM_ERR_INVALID_ARG;
    if (t->k_out == t->k && !same_strides(t->k_stride, t->k_out_stride)) return CM_ERR_INVALID_ARG;
  }
  if (!none) {
    const int64_t seqs_apart = t->cu_new ? 1 : seqs->B;
    const int64_t q_rows[3] = {seqs_apart, t->H_q, t->n_tokens};
    const int64_t k_rows[3] = {seqs_apart, cache->H_kv, t->n_tokens};
    if ((t->q_out && !rows_apart(t->q_out_stride, q_rows, 3, cache->d)) ||
        (t->k_out && !rows_apart(t->k_out_stride, k_rows, 3, cache->d)))
      return CM_ERR_INVALID_ARG;
  }
  if (t->n_tokens < 0 || t->max_new < 0 || t->max_new > t->n_tokens) return CM_ERR_INVALID_ARG;
  if (t->cu_new ? (t->n_new || !good_ints(t->cu_new)) : (t->n_new && !good_ints(t->n_new)))
    return CM_ERR_INVALID_ARG;
  if (!t->cu_new && !t->n_new && t->max_new != t->n_tokens) return CM_ERR_INVALID_ARG;
  if (t->rot_dim < 0 || t->rot_dim > cache->d || t->rot_dim % 16 != 0) return CM_ERR_INVALID_ARG;
  if (t->rot_dim ? (!good_ptr(t->rope) || t->rope_len < 1) : t->rope != nullptr)
    return CM_ERR_INVALID_ARG;
  if (t->new_lens && (!good_ints(t->new_lens) || t->new_lens == seqs->lens))
    return CM_ERR_INVALID_ARG;
  if ((t->cu_new ? t->n_tokens : static_cast<int64_t>(seqs->B) * t->max_new) > (1LL << 30))
    return CM_ERR_UNSUPPORTED;
  cm::AppendParams p;
  p.c = view(cache, seqs);
  p.k = static_cast<const __nv_bfloat16*>(t->k);
  p.v = static_cast<const __nv_bfloat16*>(t->v);
  p.q = static_cast<const __nv_bfloat16*>(t->q);
  p.q_out = static_cast<__nv_bfloat16*>(t->q_out);
  p.k_out = static_cast<__nv_bfloat16*>(t->k_out);
  p.ks = strides3(t->k_stride);
  p.vs = strides3(t->v_stride);
  p.qs = strides3(t->q_stride);
  p.qos = strides3(t->q_out_stride);
  p.kos = strides3(t->k_out_stride);
  p.cu_new = t->cu_new;
  p.n_new = t->n_new;
  p.n_tokens = t->n_tokens;
  p.max_new = t->max_new;
  p.H_q = t->q ? t->H_q : 0;
  p.rot_dim = t->rot_dim;
  p.interleaved = t->interleaved;
  p.rope_len = t->rope_len;
  p.rope = t->rope;
  p.new_lens = t->new_lens;
  if (cm::append_page_blocks(p) > (1LL << 30)) return CM_ERR_UNSUPPORTED;
  return cm::launch_kv_append(p, static_cast<cudaStream_t>(stream)) == 0 ? CM_OK : CM_ERR_CUDA;
}

CM_API int cm_attn_decode_workspace_size(int B, int H_q, int H_kv, int d, size_t* bytes) {
  if (!bytes || B < 1 || H_kv < 1) return CM_ERR_INVALID_ARG;
  const int rc = check_heads(H_q, H_kv);
  if (rc != CM_OK) return rc;
  if (B > kMaxB || H_kv > 1024 || (d != 64 && d != 128)) return CM_ERR_UNSUPPORTED;
  *bytes = cm::decode_workspace_bytes(B, H_q, H_kv, d);
  return CM_OK;
}

CM_API int cm_attn_decode(const cm_kv_cache* cache, const cm_kv_seqs* seqs,
                          const cm_descriptor* desc, const int32_t* sel, const int32_t* nsel,
                          int sel_max, const void* q, const int64_t q_stride[2], void* o,
                          const int64_t o_stride[2], float* lse, int H_q, float scale,
                          void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_both(cache, seqs);
  if (rc != CM_OK) return rc;
  rc = check_heads(H_q, cache->H_kv);
  if (rc != CM_OK) return rc;
  if (!good_ptr(q) || !good_ptr(o) || !q_stride || !o_stride || !good_strides(q_stride, 2) ||
      !good_strides(o_stride, 2) || (lse && !aligned(lse, 4)) || !std::isfinite(scale))
    return CM_ERR_INVALID_ARG;
  const int64_t o_rows[2] = {seqs->B, H_q};
  if (!rows_apart(o_stride, o_rows, 2, cache->d)) return CM_ERR_INVALID_ARG;
  if ((sel != nullptr) != (nsel != nullptr) || (sel && desc)) return CM_ERR_INVALID_ARG;
  if (sel && (!good_ints(sel) || !good_ints(nsel) || sel_max < 1)) return CM_ERR_INVALID_ARG;
  if (sel && sel_max > 8192) return CM_ERR_UNSUPPORTED;
  if (desc) {
    if (desc->B != seqs->B || desc->S < 1 || desc->ni_f < 1 || desc->ni_f > 8 || !desc->itab_f ||
        !aligned(desc->itab_f, 16))
      return CM_ERR_INVALID_ARG;
    if (desc->form != CM_FORM_VISIBLE) return CM_ERR_UNSUPPORTED;
  }
  size_t need = 0;
  rc = cm_attn_decode_workspace_size(seqs->B, H_q, cache->H_kv, cache->d, &need);
  if (rc != CM_OK) return rc;
  if (!good_ptr(workspace) || workspace_bytes < need) return CM_ERR_INVALID_ARG;
  cm::DecodeParams p;
  p.c = view(cache, seqs);
  p.itab = desc ? desc->itab_f : nullptr;
  p.NI = desc ? desc->ni_f : 1;
  p.S = desc ? desc->S : 0;
  p.sel = sel;
  p.nsel = nsel;
  p.sel_max = sel ? sel_max : 0;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.qs = {q_stride[0], q_stride[1], 0};
  p.os = {o_stride[0], o_stride[1], 0};
  p.lse = lse;
  p.H_q = H_q;
  p.scale = scale;
  p.workspace = workspace;
  if (!cm::decode_fits(p)) return CM_ERR_UNSUPPORTED;
  return cm::launch_attn_decode(p, cm::wait_limit_ns(), static_cast<cudaStream_t>(stream)) == 0
             ? CM_OK
             : CM_ERR_CUDA;
}

CM_API int cm_select_pages_workspace_size(int B, int H_kv, int max_pages, size_t* bytes) {
  if (!bytes || B < 1 || H_kv < 1 || max_pages < 1) return CM_ERR_INVALID_ARG;
  if (B > kMaxB || H_kv > 1024 || max_pages > 32768) return CM_ERR_UNSUPPORTED;
  *bytes = static_cast<size_t>(B) * H_kv * cm::score_pitch(max_pages) * 4;
  return CM_OK;
}

CM_API int cm_select_pages(const cm_kv_cache* cache, const cm_kv_seqs* seqs, const void* q,
                           const int64_t q_stride[2], int H_q, int keep_first, int keep_last,
                           int32_t* sel, int32_t* nsel, int sel_max, void* workspace,
                           size_t workspace_bytes, void* stream) {
  int rc = check_both(cache, seqs);
  if (rc != CM_OK) return rc;
  if (!cache->summary) return CM_ERR_INVALID_ARG;
  rc = check_heads(H_q, cache->H_kv);
  if (rc != CM_OK) return rc;
  if (!good_ptr(q) || !q_stride || !good_strides(q_stride, 2)) return CM_ERR_INVALID_ARG;
  if (!good_ints(sel) || !good_ints(nsel) || sel_max < 1) return CM_ERR_INVALID_ARG;
  if (sel_max > 8192 || seqs->max_pages > 32768) return CM_ERR_UNSUPPORTED;
  if (keep_first < 0 || keep_last < 0 || keep_first > sel_max || keep_last > sel_max - keep_first)
    return CM_ERR_INVALID_ARG;
  size_t need = 0;
  rc = cm_select_pages_workspace_size(seqs->B, cache->H_kv, seqs->max_pages, &need);
  if (rc != CM_OK) return rc;
  if (!good_ptr(workspace) || workspace_bytes < need) return CM_ERR_INVALID_ARG;
  cm::SelectParams p;
  p.c = view(cache, seqs);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.qs = {q_stride[0], q_stride[1], 0};
  p.H_q = H_q;
  p.keep_first = keep_first;
  p.keep_last = keep_last;
  p.sel_max = sel_max;
  p.sel = sel;
  p.nsel = nsel;
  p.scores = static_cast<float*>(workspace);
  return cm::launch_select_pages(p, static_cast<cudaStream_t>(stream)) == 0 ? CM_OK : CM_ERR_CUDA;
}

CM_API int cm_kv_status(const cm_kv_cache* cache, void* stream) {
  if (!cache || !good_ints(cache->status)) return CM_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t v = 0;
  if (cudaMemcpyAsync(&v, cache->status, 4, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return CM_ERR_CUDA;
  if (v == 0) return CM_OK;
  if (cudaMemsetAsync(cache->status, 0, 4, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return CM_ERR_CUDA;
  return (v >> 16) == cm::kDevTimeout ? CM_ERR_TIMEOUT : CM_ERR_DEVICE_CHECK;
}

}  // extern "C"
