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

// bytes: of a cache's element.
int check_paged(int64_t n, int32_t seqs, int32_t kv_heads, int32_t dim, const int32_t* q_offsets,
                const int32_t* kv_lens, const int32_t* page_table, int64_t table_stride, int32_t table_width,
                int32_t page, int64_t num_pages, int64_t page_stride, int64_t head_stride, const void* k_cache,
                const void* v_cache, int32_t* status, Paged* p, int bytes = 2) {
  if (seqs < 0 || (n > 0 && (!q_offsets || (seqs > 0 && !kv_lens)))) return DLRM_E_INVAL;
  if (table_width < 0 || table_stride < 0 || num_pages < 0 || num_pages > kI32Max)
    return DLRM_E_INVAL;
  if (n > 0 && seqs > 0 && table_width > 0 && !page_table) return DLRM_E_INVAL;
  if (n > 0 && num_pages > 0 && (!k_cache || !v_cache)) return DLRM_E_INVAL;
  if (page < 16 || page > 65536 || (page & (page - 1))) return DLRM_E_UNSUPPORTED;
  // entries and sequences
  if (static_cast<int64_t>(table_width) * page > kMostCounted || seqs > kMostCounted) return DLRM_E_UNSUPPORTED;
  const int64_t per16 = 16 / bytes;
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

// The scales of an 8-bit cache: two bytes a block, blocks of a head and page contiguous.
int check_scales(int64_t n, int32_t kv_heads, int32_t page, int64_t num_pages, const uint8_t* scales,
                 int64_t page_stride, int64_t head_stride) {
  if (n > 0 && num_pages > 0 && !scales) return DLRM_E_INVAL;
  if (!aligned(scales, 2) || page_stride % 2 || head_stride % 2) return DLRM_E_ALIGN;
  const int64_t own = 2 * (page / DLRM_KV_BLOCK);
  if (kv_heads > 1 && head_stride < own) return DLRM_E_INVAL;
  if (num_pages > 1 && page_stride < (kv_heads - 1) * head_stride + own) return DLRM_E_INVAL;
  return DLRM_OK;
}

// Arguments of the append that both caches share; bytes: of a cache's element.
int check_append(int64_t n, int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t rot, int32_t dtype,
                 const Heads& q, const Heads& k, const Heads& v, const int32_t* positions, int64_t pos_stride,
                 int32_t axes, const int32_t* sections, const float* inv_freq, const float* w_q, const float* w_k,
                 float eps, int32_t interleaved, const int32_t* q_offsets, const int32_t* kv_lens,
                 const int32_t* page_table, int64_t table_stride, int32_t table_width, int32_t page, int64_t num_pages,
                 int64_t cache_page_stride, int64_t cache_head_stride, void* k_cache, void* v_cache, int bytes,
                 void* q_out, int32_t* status, NormRopeArgs* a) {
  memset(a, 0, sizeof(*a));
  TRY(check_heads(n, q_heads, kv_heads, dim, dtype, true));
  if (q_heads > 0 && (!w_q != !w_k || (n > 0 && !q_out))) return DLRM_E_INVAL;
  if (q_heads == 0 && (q.ptr || q_out || w_q)) return DLRM_E_INVAL;
  TRY(check_rotation(n, dim, rot, positions, pos_stride, axes, sections, inv_freq, interleaved, &a->rope));
  TRY(check_norm(w_q, w_k, eps));
  if (q_heads > 0) TRY(check_tensor(q.ptr, q.stride, q.head_stride, dtype, n));
  TRY(check_tensor(k.ptr, k.stride, k.head_stride, dtype, n));
  TRY(check_tensor(v.ptr, v.stride, v.head_stride, dtype, n));
  if (!aligned(q_out, 16)) return DLRM_E_ALIGN;
  TRY(check_paged(n, seqs, kv_heads, dim, q_offsets, kv_lens, page_table, table_stride, table_width, page, num_pages,
                  cache_page_stride, cache_head_stride, k_cache, v_cache, status, &a->paged, bytes));
  a->n = n; a->q_heads = q_heads; a->kv_heads = kv_heads; a->dim = dim; a->dtype = dtype;
  a->q = q; a->k = k; a->v = v;
  a->w_q = w_q; a->w_k = w_k; a->eps = eps; a->q_out = q_out;
  a->k_cache = k_cache; a->v_cache = v_cache;
  return DLRM_OK;
}

// What assignment and release of pages share.
int check_pages(int32_t seqs, int32_t users, const int32_t* who, const int32_t* held, const int32_t* held_out,
                const int32_t* tables, int64_t table_stride, int32_t table_width, int32_t page,
                const int32_t* free_pages, int64_t num_pages, const int32_t* count, const int32_t* count_out,
                const void* workspace, size_t ws_bytes, const int32_t* status) {
  if (seqs < 0 || users < 0 || table_width < 0 || num_pages < 0 || num_pages > kI32Max) return DLRM_E_INVAL;
  if (page < 16 || page > 65536 || (page & (page - 1))) return DLRM_E_UNSUPPORTED;
  if (static_cast<int64_t>(table_width) * page > kMostCounted || seqs > kMostCounted) return DLRM_E_UNSUPPORTED;
  if (!who && seqs > users) return DLRM_E_INVAL;
  if (table_stride < 0 || (users > 1 && table_stride < table_width)) return DLRM_E_INVAL;
  if (!count || !count_out || (num_pages > 0 && !free_pages)) return DLRM_E_INVAL;
  if (seqs > 0 && users > 0 && (!held || !held_out || (table_width > 0 && !tables))) return DLRM_E_INVAL;
  if (!aligned(who, 4) || !aligned(held, 4) || !aligned(held_out, 4) || !aligned(tables, 4) ||
      !aligned(free_pages, 4) || !aligned(count, 4) || !aligned(count_out, 4) || !aligned(status, 4) ||
      !aligned(workspace, 256))
    return DLRM_E_ALIGN;
  if (ws_bytes < pages_workspace(seqs)) return DLRM_E_WORKSPACE;
  if (!workspace) return DLRM_E_INVAL;
  // lengths in place and the count beside it, or the other way round, would be half a step
  if (users > 0 && (held == held_out) != (count == count_out)) return DLRM_E_INVAL;
  return DLRM_OK;
}

// A buffer of a call: its address, its bytes, and whether the call writes it.
struct Buffer {
  const void* at;
  uint64_t bytes;
  bool written;
};

// Whether no buffer that is written shares a byte with another one.
bool apart(const Buffer* b, int count) {
  for (int i = 0; i < count; ++i)
    for (int j = i + 1; j < count; ++j) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(b[i].at), y = reinterpret_cast<uintptr_t>(b[j].at);
      if (!x || !y || !(b[i].written || b[j].written)) continue;
      if (x <= y ? y - x < b[i].bytes && b[j].bytes > 0 : x - y < b[j].bytes && b[i].bytes > 0) return false;
    }
  return true;
}

// The buffers of an assignment or release: the kernels read lengths and users again after they wrote others, so
// nothing but the two lengths and the two counts may be one.
int check_page_buffers(const PagesArgs& a, bool assign, size_t ws_bytes) {
  const uint64_t seqs = a.seqs, users = a.users, width = a.table_width;
  const uint64_t rows = users > 1 ? users - 1 : 0, step = users > 1 ? a.table_stride : 0;
  uint64_t table_bytes;
  if (__builtin_mul_overflow(rows, step, &table_bytes) || table_bytes > (uint64_t(1) << 60)) return DLRM_E_INVAL;
  table_bytes = users > 0 ? 4 * (table_bytes + width) : 0;
  const bool held_apart = a.held != a.held_out, count_apart = a.count != a.count_out;
  const Buffer all[] = {{a.lens, 4 * seqs, false},
                        {a.who, 4 * seqs, false},
                        {held_apart ? a.held : nullptr, 4 * users, false},
                        {a.held_out, 4 * users, true},
                        {count_apart ? a.count : nullptr, 4, false},
                        {a.count_out, 4, true},
                        {a.tables, table_bytes, assign},
                        {a.free_pages, 4 * static_cast<uint64_t>(a.num_pages), !assign},
                        {a.workspace, ws_bytes, true},
                        {a.status, 4, true},
                        {a.q_offsets, 4 * (seqs + 1), true},
                        {a.kv_lens, 4 * seqs, true},
                        {a.page_table, 4 * seqs * static_cast<uint64_t>(a.out_width), true},
                        {a.slots, 8 * static_cast<uint64_t>(a.n), true},
                        {a.positions, 4 * static_cast<uint64_t>(a.n), true}};
  return apart(all, sizeof(all) / sizeof(all[0])) ? DLRM_OK : DLRM_E_INVAL;
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
  TRY(check_append(n, seqs, q_heads, kv_heads, dim, rot, dtype, {q, q_stride, q_head_stride}, {k, k_stride, k_head_stride},
                   {v, v_stride, v_head_stride}, positions, pos_stride, axes, sections, inv_freq, w_q, w_k, eps,
                   interleaved, q_offsets, kv_lens, page_table, table_stride, table_width, page, num_pages,
                   cache_page_stride, cache_head_stride, k_cache, v_cache, 2, q_out, status, &a));
  return from_hip(launch_kv_append(a, static_cast<hipStream_t>(stream)));
}

int dlrm_kv_append_q8(int64_t n, int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t rot,
                      int32_t dtype, const void* q, int64_t q_stride, int64_t q_head_stride, const void* k,
                      int64_t k_stride, int64_t k_head_stride, const void* v, int64_t v_stride, int64_t v_head_stride,
                      const int32_t* positions, int64_t pos_stride, int32_t axes, const int32_t* sections,
                      const float* inv_freq, const float* w_q, const float* w_k, float eps, int32_t interleaved,
                      const int32_t* q_offsets, const int32_t* kv_lens, const int32_t* page_table,
                      int64_t table_stride, int32_t table_width, int32_t page, int64_t num_pages,
                      int64_t cache_page_stride, int64_t cache_head_stride, void* k_cache, void* v_cache,
                      uint8_t* kv_scales, int64_t scale_page_stride, int64_t scale_head_stride, void* q_out,
                      int32_t* status, void* stream) {
  NormRopeArgs a;
  TRY(check_append(n, seqs, q_heads, kv_heads, dim, rot, dtype, {q, q_stride, q_head_stride}, {k, k_stride, k_head_stride},
                   {v, v_stride, v_head_stride}, positions, pos_stride, axes, sections, inv_freq, w_q, w_k, eps,
                   interleaved, q_offsets, kv_lens, page_table, table_stride, table_width, page, num_pages,
                   cache_page_stride, cache_head_stride, k_cache, v_cache, 1, q_out, status, &a));
  TRY(check_scales(n, kv_heads, page, num_pages, kv_scales, scale_page_stride, scale_head_stride));
  a.kv_scales = kv_scales; a.scale_page_stride = scale_page_stride; a.scale_head_stride = scale_head_stride;
  return from_hip(launch_kv_append_q8(a, static_cast<hipStream_t>(stream)));
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
  TRY(check_paged(n, seqs, kv_heads, dim, q_offsets, kv_lens, page_table, table_stride, table_width, page,
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

int dlrm_paged_attn_q8_workspace_bytes(int64_t n, int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t dim,
                                       int32_t causal, int32_t window, int32_t max_q, int32_t max_kv, size_t* bytes) {
  if (!bytes) return DLRM_E_INVAL;
  TRY(check_attn(n, seqs, q_heads, kv_heads, dim, causal, window, max_q, max_kv));
  *bytes = attn_q8_workspace(n, seqs, q_heads, kv_heads, dim, causal, window, max_q, max_kv);
  return DLRM_OK;
}

int dlrm_paged_attn_q8(int64_t n, int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t dtype,
                       const void* q, int64_t q_stride, int64_t q_head_stride, const void* k_cache,
                       const void* v_cache, int32_t page, int64_t num_pages, int64_t cache_page_stride,
                       int64_t cache_head_stride, const uint8_t* kv_scales, int64_t scale_page_stride,
                       int64_t scale_head_stride, const int32_t* q_offsets, const int32_t* kv_lens,
                       const int32_t* page_table, int64_t table_stride, int32_t table_width, int32_t causal,
                       int32_t window, float scale, int32_t max_q, int32_t max_kv, void* out, float* lse,
                       void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  TRY(check_attn(n, seqs, q_heads, kv_heads, dim, causal, window, max_q, max_kv));
  if (bytes_of(dtype) != 2) return DLRM_E_UNSUPPORTED;
  if (!(scale > 0.f && scale < INFINITY) || (n > 0 && !out)) return DLRM_E_INVAL;
  TRY(check_tensor(q, q_stride, q_head_stride, dtype, n));
  TRY(check_paged(n, seqs, kv_heads, dim, q_offsets, kv_lens, page_table, table_stride, table_width, page, num_pages,
                  cache_page_stride, cache_head_stride, k_cache, v_cache, status, &a.paged, 1));
  TRY(check_scales(n, kv_heads, page, num_pages, kv_scales, scale_page_stride, scale_head_stride));
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 256)) return DLRM_E_ALIGN;
  const size_t need = attn_q8_workspace(n, seqs, q_heads, kv_heads, dim, causal, window, max_q, max_kv);
  if (ws_bytes < need) return DLRM_E_WORKSPACE;
  if (need > 0 && !workspace) return DLRM_E_INVAL;
  a.n = n; a.q_heads = q_heads; a.kv_heads = kv_heads; a.dim = dim; a.dtype = dtype;
  a.q = {q, q_stride, q_head_stride};
  a.k_cache = k_cache; a.v_cache = v_cache;
  a.kv_scales = kv_scales; a.scale_page_stride = scale_page_stride; a.scale_head_stride = scale_head_stride;
  a.causal = causal != 0; a.window = window; a.max_q = max_q; a.max_kv = max_kv; a.scale = scale;
  a.out = out; a.lse = lse; a.workspace = workspace;
  return from_hip(launch_paged_attn_q8(a, static_cast<hipStream_t>(stream)));
}

int dlrm_pages_workspace_bytes(int32_t seqs, size_t* bytes) {
  if (!bytes || seqs < 0) return DLRM_E_INVAL;
  if (seqs > kMostCounted) return DLRM_E_UNSUPPORTED;
  *bytes = pages_workspace(seqs);
  return DLRM_OK;
}

int dlrm_pages_assign(int64_t n, int32_t seqs, int32_t users, const int32_t* new_lens, const int32_t* who,
                      const int32_t* held, int32_t* held_out, int32_t* tables, int64_t table_stride,
                      int32_t table_width, int32_t page, const int32_t* free_pages, int64_t num_pages,
                      const int32_t* free_count, int32_t* count_out, int32_t* q_offsets, int32_t* kv_lens,
                      int32_t* page_table, int32_t out_width, int64_t* slots, int32_t* positions, void* workspace,
                      size_t ws_bytes, int32_t* status, void* stream) {
  PagesArgs a;
  memset(&a, 0, sizeof(a));
  if (n < 0 || n >= kI32Max || out_width < 0 || out_width > table_width) return DLRM_E_INVAL;
  TRY(check_pages(seqs, users, who, held, held_out, tables, table_stride, table_width, page, free_pages, num_pages,
                  free_count, count_out, workspace, ws_bytes, status));
  if (!q_offsets || (seqs > 0 && (!new_lens || !kv_lens || (out_width > 0 && !page_table)))) return DLRM_E_INVAL;
  if (!aligned(new_lens, 4) || !aligned(q_offsets, 4) || !aligned(kv_lens, 4) || !aligned(page_table, 4) ||
      !aligned(slots, 8) || !aligned(positions, 4))
    return DLRM_E_ALIGN;
  a.n = n; a.num_pages = num_pages; a.table_stride = table_stride;
  a.seqs = seqs; a.users = users; a.page_shift = __builtin_ctz(page);
  a.table_width = table_width; a.out_width = out_width;
  a.lens = new_lens; a.who = who; a.held = held; a.count = free_count;
  a.tables = tables; a.free_pages = const_cast<int32_t*>(free_pages); a.held_out = held_out; a.count_out = count_out;
  a.q_offsets = q_offsets; a.kv_lens = kv_lens; a.page_table = page_table; a.positions = positions; a.slots = slots;
  a.workspace = workspace; a.status = status;
  TRY(check_page_buffers(a, true, pages_workspace(seqs)));
  return from_hip(launch_pages_assign(a, static_cast<hipStream_t>(stream)));
}

int dlrm_pages_release(int32_t seqs, int32_t users, const int32_t* keep, const int32_t* who, const int32_t* held,
                       int32_t* held_out, const int32_t* tables, int64_t table_stride, int32_t table_width,
                       int32_t page, int32_t* free_pages, int64_t num_pages, const int32_t* free_count,
                       int32_t* count_out, void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
  PagesArgs a;
  memset(&a, 0, sizeof(a));
  TRY(check_pages(seqs, users, who, held, held_out, tables, table_stride, table_width, page, free_pages, num_pages,
                  free_count, count_out, workspace, ws_bytes, status));
  if (!aligned(keep, 4)) return DLRM_E_ALIGN;
  a.num_pages = num_pages; a.table_stride = table_stride;
  a.seqs = seqs; a.users = users; a.page_shift = __builtin_ctz(page); a.table_width = table_width;
  a.lens = keep; a.who = who; a.held = held; a.count = free_count;
  a.tables = const_cast<int32_t*>(tables); a.free_pages = free_pages; a.held_out = held_out; a.count_out = count_out;
  a.workspace = workspace; a.status = status;
  TRY(check_page_buffers(a, false, pages_workspace(seqs)));
  return from_hip(launch_pages_release(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
