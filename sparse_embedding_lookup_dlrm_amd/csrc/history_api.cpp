// C ABI of dlrm_history.h: argument validation on the host, then kernel launches on the
// caller's stream. Every check runs before the first HIP call, so a rejected call touches
// neither the device nor any output.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "history.h"

namespace {

using namespace dlrm;

constexpr int64_t kI32Max = 0x7fffffffLL;
// What kernels count in int32, with room for a tile or a grid's step past the last one.
constexpr int64_t kMostCounted = kI32Max - (1 << 17);

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int bytes_of(int dtype) { return dtype == DLRM_F32 ? 4 : dtype == DLRM_F16 || dtype == DLRM_BF16 ? 2 : 0; }

int from_hip(hipError_t e) { return e == hipSuccess ? DLRM_OK : DLRM_E_HIP; }

// Sizes that every call takes.
int check_heads(int64_t n, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t dtype, bool cache) {
  if (n < 0 || n >= kI32Max || q_heads < 0 || kv_heads < 1) return DLRM_E_INVAL;
  if (static_cast<int64_t>(q_heads) + kv_heads > 65535) return DLRM_E_UNSUPPORTED;
  if (bytes_of(dtype) == 0 || (cache && dtype == DLRM_F32)) return DLRM_E_UNSUPPORTED;
  if (dim != 32 && dim != 64 && dim != 128 && dim != 256) return DLRM_E_UNSUPPORTED;
  return DLRM_OK;
}

// A tensor of heads: 16-byte aligned, and so is every head of it.
int check_tensor(const void* p, int64_t stride, int64_t head_stride, int dtype, int64_t n) {
  if (n > 0 && !p) return DLRM_E_INVAL;
  const int64_t per16 = 16 / bytes_of(dtype);
  if (!aligned(p, 16) || stride % per16 || head_stride % per16) return DLRM_E_ALIGN;
  return DLRM_OK;
}

int check_rotation(int64_t n, int32_t dim, int32_t rot, const int32_t* positions, int64_t pos_stride, int32_t axes,
                   const int32_t* sections, const float* inv_freq, int32_t interleaved, Rotation* r) {
  memset(r, 0, sizeof(*r));
  if (rot < 0 || rot > dim) return DLRM_E_INVAL;
  if (rot % 16 != 0) return DLRM_E_UNSUPPORTED;
  r->rot = rot;
  r->interleaved = interleaved != 0;
  if (rot == 0) return DLRM_OK;
  if (!inv_freq || !sections || (n > 0 && !positions) || axes < 1) return DLRM_E_INVAL;
  if (axes > DLRM_MAX_AXES) return DLRM_E_UNSUPPORTED;
  if (!aligned(positions, 4) || !aligned(inv_freq, 4)) return DLRM_E_ALIGN;
  int64_t sum = 0;
  for (int i = 0; i < axes; ++i) {
    if (sections[i] < 0) return DLRM_E_INVAL;
    sum += sections[i];
    if (sum > rot / 2) return DLRM_E_INVAL;
    r->section_end[i] = static_cast<int32_t>(sum);
  }
  if (sum != rot / 2) return DLRM_E_INVAL;
  r->positions = positions;
  r->pos_stride = pos_stride;
  r->inv_freq = inv_freq;
  r->axes = axes;
  return DLRM_OK;
}

int check_norm(const float* w_q, const float* w_k, float eps) {
  if (!aligned(w_q, 4) || !aligned(w_k, 4)) return DLRM_E_ALIGN;
  if ((w_q || w_k) && !(eps >= 0.f && eps < INFINITY)) return DLRM_E_INVAL;
  return DLRM_OK;
}

int check_paged(int64_t n, int32_t seqs, int32_t kv_heads, int32_t dim, int dtype, const int32_t* q_offsets,
                const int32_t* kv_lens, const int32_t* page_table, int64_t table_stride, int32_t table_width,
                int32_t page, int64_t num_pages, int64_t page_stride, int64_t head_stride, const void* k_cache,
                const void* v_cache, int32_t* status, Paged* p) {
  if (seqs < 0 || (n > 0 && (!q_offsets || (seqs > 0 && !kv_lens)))) return DLRM_E_INVAL;
  if (table_width < 0 || table_stride < 0 || num_pages < 0 || num_pages > kI32Max)
    return DLRM_E_INVAL;
  if (n > 0 && seqs > 0 && table_width > 0 && !page_table) return DLRM_E_INVAL;
  if (n > 0 && num_pages > 0 && (!k_cache || !v_cache)) return DLRM_E_INVAL;
  if (page < 16 || page > 65536 || (page & (page - 1))) return DLRM_E_UNSUPPORTED;
  // entries and sequences
  if (static_cast<int64_t>(table_width) * page > kMostCounted || seqs > kMostCounted) return DLRM_E_UNSUPPORTED;
  const int64_t per16 = 16 / bytes_of(dtype);
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || page_stride % per16 || head_stride % per16) return DLRM_E_ALIGN;
  if (!aligned(q_offsets, 4) || !aligned(kv_lens, 4) || !aligned(page_table, 4) || !aligned(status, 4))
    return DLRM_E_ALIGN;
  // heads and pages that overlap
  if (head_stride < static_cast<int64_t>(page) * dim && kv_heads > 1) return DLRM_E_INVAL;
  if (page_stride < (kv_heads - 1) * head_stride + static_cast<int64_t>(page) * dim && num_pages > 1)
    return DLRM_E_INVAL;
  p->q_offsets = q_offsets;
  p->kv_lens = kv_lens;
  p->page_table = page_table;
  p->table_stride = table_stride;
  p->table_width = table_width;
  p->seqs = seqs;
  p->page_shift = __builtin_ctz(page);
  p->num_pages = num_pages;
  p->page_stride = page_stride;
  p->head_stride = head_stride;
  p->status = status;
  return DLRM_OK;
}

#define TRY(call)                \
  do {                           \
    const int rc_ = (call);      \
    if (rc_ != DLRM_OK) return rc_; \
  } while (0)

// Sizes of the attention, shared with its workspace query.
int check_attn(int64_t n, int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t causal, int32_t window,
               int32_t max_q, int32_t max_kv) {
  TRY(check_heads(n, q_heads, kv_heads, dim, DLRM_BF16, true));
  if (q_heads < 1 || q_heads % kv_heads != 0) return DLRM_E_INVAL;
  if (seqs < 0 || window < 0 || (window > 0 && !causal) || max_q < 0 || max_kv < 0) return DLRM_E_INVAL;
  // rows and sequences
  if (q_heads / kv_heads > 1024 || n * q_heads > kMostCounted || seqs > kMostCounted) return DLRM_E_UNSUPPORTED;
  return DLRM_OK;
}

}  // namespace

extern "C" {

int dlrm_qk_norm_rope(int64_t n, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t rot, int32_t dtype,
                      const void* q, int64_t q_stride, int64_t q_head_stride, const void* k, int64_t k_stride,
                      int64_t k_head_stride, const int32_t* positions, int64_t pos_stride, int32_t axes,
                      const int32_t* sections, const float* inv_freq, const float* w_q, const float* w_k, float eps,
                      int32_t interleaved, void* q_out, void* k_out, void* stream) {
  NormRopeArgs a;
  memset(&a, 0, sizeof(a));
  TRY(check_heads(n, q_heads, kv_heads, dim, dtype, false));
  if (q_heads < 1 || (n > 0 && (!q_out || !k_out)) || !w_q != !w_k) return DLRM_E_INVAL;
  TRY(check_rotation(n, dim, rot, positions, pos_stride, axes, sections, inv_freq, interleaved, &a.rope));
  TRY(check_norm(w_q, w_k, eps));
  TRY(check_tensor(q, q_stride, q_head_stride, dtype, n));
  TRY(check_tensor(k, k_stride, k_head_stride, dtype, n));
  if (!aligned(q_out, 16) || !aligned(k_out, 16)) return DLRM_E_ALIGN;
  a.n = n; a.q_heads = q_heads; a.kv_heads = kv_heads; a.dim = dim; a.dtype = dtype;
  a.q = {q, q_stride, q_head_stride};
  a.k = {k, k_stride, k_head_stride};
  a.w_q = w_q; a.w_k = w_k; a.eps = eps; a.q_out = q_out; a.k_out = k_out;
  return from_hip(launch_norm_rope(a, static_cast<hipStream_t>(stream)));
}

int dlrm_qk_norm_rope_bwd_workspace_bytes(int64_t n, int32_t dim, int32_t norm, size_t* bytes) {
  if (!bytes) return DLRM_E_INVAL;
  TRY(check_heads(n, 1, 1, dim, DLRM_F32, false));
  *bytes = norm_rope_bwd_workspace(n, dim, norm != 0);
  return DLRM_OK;
}

int dlrm_qk_norm_rope_bwd(int64_t n, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t rot, int32_t dtype,
                          const void* d_q_out, int64_t dq_stride, int64_t dq_head_stride, const void* d_k_out,
                          int64_t dk_stride, int64_t dk_head_stride, const void* q, int64_t q_stride,
                          int64_t q_head_stride, const void* k, int64_t k_stride, int64_t k_head_stride,
                          const int32_t* positions, int64_t pos_stride, int32_t axes, const int32_t* sections,
                          const float* inv_freq, const float* w_q, const float* w_k, float eps, int32_t interleaved,
                          void* d_q, void* d_k, float* d_w_q, float* d_w_k, void* workspace, size_t ws_bytes,
                          void* stream) {
  NormRopeBwdArgs a;
  memset(&a, 0, sizeof(a));
  TRY(check_heads(n, q_heads, kv_heads, dim, dtype, false));
  if (q_heads < 1 || (n > 0 && (!d_q || !d_k)) || !w_q != !w_k) return DLRM_E_INVAL;
  TRY(check_rotation(n, dim, rot, positions, pos_stride, axes, sections, inv_freq, interleaved, &a.rope));
  TRY(check_norm(w_q, w_k, eps));
  TRY(check_tensor(d_q_out, dq_stride, dq_head_stride, dtype, n));
  TRY(check_tensor(d_k_out, dk_stride, dk_head_stride, dtype, n));
  if (!aligned(d_q, 16) || !aligned(d_k, 16)) return DLRM_E_ALIGN;
  if (w_q) {
    TRY(check_tensor(q, q_stride, q_head_stride, dtype, n));
    TRY(check_tensor(k, k_stride, k_head_stride, dtype, n));
    if (!d_w_q || !d_w_k) return DLRM_E_INVAL;
    if (!aligned(d_w_q, 4) || !aligned(d_w_k, 4)) return DLRM_E_ALIGN;
    const size_t need = norm_rope_bwd_workspace(n, dim, true);
    if (ws_bytes < need) return DLRM_E_WORKSPACE;
    if (need > 0 && !workspace) return DLRM_E_INVAL;
    if (!aligned(workspace, 256)) return DLRM_E_ALIGN;
  }
  a.n = n; a.q_heads = q_heads; a.kv_heads = kv_heads; a.dim = dim; a.dtype = dtype;
  a.dq_out = {d_q_out, dq_stride, dq_head_stride};
  a.dk_out = {d_k_out, dk_stride, dk_head_stride};
  a.q = {q, q_stride, q_head_stride};
  a.k = {k, k_stride, k_head_stride};
  a.w_q = w_q; a.w_k = w_k; a.eps = eps; a.d_q = d_q; a.d_k = d_k; a.d_w_q = d_w_q; a.d_w_k = d_w_k;
  a.partials = static_cast<float*>(workspace);
  return from_hip(launch_norm_rope_bwd(a, static_cast<hipStream_t>(stream)));
}

int dlrm_kv_append(int64_t n, int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t rot, int32_t dtype,
                   const void* q, int64_t q_stride, int64_t q_head_stride, const void* k, int64_t k_stride,
                   int64_t k_head_stride, const void* v, int64_t v_stride, int64_t v_head_stride,
                   const int32_t* positions, int64_t pos_stride, int32_t axes, const int32_t* sections,
                   const float* inv_freq, const float* w_q, const float* w_k, float eps, int32_t interleaved,
                   const int32_t* q_offsets, const int32_t* kv_lens, const int32_t* page_table, int64_t table_stride,
                   int32_t table_width, int32_t page, int64_t num_pages, int64_t cache_page_stride,
                   int64_t cache_head_stride, void* k_cache, void* v_cache, void* q_out, int32_t* status,
                   void* stream) {
  NormRopeArgs a;
  memset(&a, 0, sizeof(a));
  TRY(check_heads(n, q_heads, kv_heads, dim, dtype, true));
  if (q_heads > 0 && (!w_q != !w_k || (n > 0 && !q_out))) return DLRM_E_INVAL;
  if (q_heads == 0 && (q || q_out || w_q)) return DLRM_E_INVAL;
  TRY(check_rotation(n, dim, rot, positions, pos_stride, axes, sections, inv_freq, interleaved, &a.rope));
  TRY(check_norm(w_q, w_k, eps));
  if (q_heads > 0) TRY(check_tensor(q, q_stride, q_head_stride, dtype, n));
  TRY(check_tensor(k, k_stride, k_head_stride, dtype, n));
  TRY(check_tensor(v, v_stride, v_head_stride, dtype, n));
  if (!aligned(q_out, 16)) return DLRM_E_ALIGN;
  TRY(check_paged(n, seqs, kv_heads, dim, dtype, q_offsets, kv_lens, page_table, table_stride, table_width, page,
                  num_pages, cache_page_stride, cache_head_stride, k_cache, v_cache, status, &a.paged));
  a.n = n; a.q_heads = q_heads; a.kv_heads = kv_heads; a.dim = dim; a.dtype = dtype;
  a.q = {q, q_stride, q_head_stride};
  a.k = {k, k_stride, k_head_stride};
  a.v = {v, v_stride, v_head_stride};
  a.w_q = w_q; a.w_k = w_k; a.eps = eps; a.q_out = q_out;
  a.k_cache = k_cache; a.v_cache = v_cache;
  return from_hip(launch_kv_append(a, static_cast<hipStream_t>(stream)));
}

int dlrm_paged_attn_workspace_bytes(int64_t n, int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t dim,
                                    int32_t causal, int32_t window, int32_t max_q, int32_t max_kv, size_t* bytes) {
  if (!bytes) return DLRM_E_INVAL;
  TRY(check_attn(n, seqs, q_heads, kv_heads, dim, causal, window, max_q, max_kv));
  *bytes = attn_workspace(n, seqs, q_heads, kv_heads, dim, causal, window, max_q, max_kv);
  return DLRM_OK;
}

int dlrm_paged_attn(int64_t n, int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t dtype,
                    const void* q, int64_t q_stride, int64_t q_head_stride, const void* k_cache, const void* v_cache,
                    int32_t page, int64_t num_pages, int64_t cache_page_stride, int64_t cache_head_stride,
                    const int32_t* q_offsets, const int32_t* kv_lens, const int32_t* page_table, int64_t table_stride,
                    int32_t table_width, int32_t causal, int32_t window, float scale, int32_t max_q, int32_t max_kv,
                    void* out, float* lse, void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  TRY(check_attn(n, seqs, q_heads, kv_heads, dim, causal, window, max_q, max_kv));
  if (bytes_of(dtype) != 2) return DLRM_E_UNSUPPORTED;
  if (!(scale > 0.f && scale < INFINITY) || (n > 0 && !out)) return DLRM_E_INVAL;
  TRY(check_tensor(q, q_stride, q_head_stride, dtype, n));
  TRY(check_paged(n, seqs, kv_heads, dim, dtype, q_offsets, kv_lens, page_table, table_stride, table_width, page,
                  num_pages, cache_page_stride, cache_head_stride, k_cache, v_cache, status, &a.paged));
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 256)) return DLRM_E_ALIGN;
  const size_t need = attn_workspace(n, seqs, q_heads, kv_heads, dim, causal, window, max_q, max_kv);
  if (ws_bytes < need) return DLRM_E_WORKSPACE;
  if (need > 0 && !workspace) return DLRM_E_INVAL;
  a.n = n; a.q_heads = q_heads; a.kv_heads = kv_heads; a.dim = dim; a.dtype = dtype;
  a.q = {q, q_stride, q_head_stride};
  a.k_cache = k_cache; a.v_cache = v_cache;
  a.causal = causal != 0; a.window = window; a.max_q = max_q; a.max_kv = max_kv; a.scale = scale;
  a.out = out; a.lse = lse; a.workspace = workspace;
  return from_hip(launch_paged_attn(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
