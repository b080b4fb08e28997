// Host-side interface between the C ABI of dlrm_history.h (history_api.cpp) and its kernel
// launchers (norm_rope.hip, kv_append_q8.hip, paged_attn.hip, paged_attn_q8.hip, pages.hip).
// Plain C++: no device code.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "dlrm_history.h"

namespace dlrm {

// A tensor [n][heads][dim]: address and strides in elements.
struct Heads {
  const void* ptr;
  int64_t stride, head_stride;
};

// Paged cache and the sequences of a call.
struct Paged {
  const int32_t* q_offsets;
  const int32_t* kv_lens;
  const int32_t* page_table;
  int64_t table_stride;
  int32_t table_width, seqs;
  int32_t page_shift;
  int64_t num_pages, page_stride, head_stride;
  int32_t* status;
};

struct Rotation {
  const int32_t* positions;
  int64_t pos_stride;
  const float* inv_freq;
  int32_t section_end[DLRM_MAX_AXES];  // first pair past each axis; the last one is rot / 2
  int32_t axes, rot, interleaved;
};

struct NormRopeArgs {
  int64_t n;
  int32_t q_heads, kv_heads, dim, dtype;
  Heads q, k, v;
  Rotation rope;
  const float *w_q, *w_k;
  float eps;
  void *q_out, *k_out;
  // append: k and v go to the cache instead of k_out
  Paged paged;
  void *k_cache, *v_cache;
  // the 8-bit cache: two bytes a block of 16 entries
  uint8_t* kv_scales;
  int64_t scale_page_stride, scale_head_stride;
};

struct NormRopeBwdArgs {
  int64_t n;
  int32_t q_heads, kv_heads, dim, dtype;
  Heads dq_out, dk_out, q, k;
  Rotation rope;
  const float *w_q, *w_k;
  float eps;
  void *d_q, *d_k;
  float *d_w_q, *d_w_k;
  float* partials;
};

hipError_t launch_norm_rope(const NormRopeArgs& a, hipStream_t s);
hipError_t launch_kv_append(const NormRopeArgs& a, hipStream_t s);
hipError_t launch_kv_append_q8(const NormRopeArgs& a, hipStream_t s);
size_t norm_rope_bwd_workspace(int64_t n, int dim, bool norm);
hipError_t launch_norm_rope_bwd(const NormRopeBwdArgs& a, hipStream_t s);

struct AttnArgs {
  int64_t n;
  int32_t q_heads, kv_heads, dim, dtype;
  Heads q;
  const void *k_cache, *v_cache;
  Paged paged;
  int32_t causal, window, max_q, max_kv;
  float scale;
  void* out;
  float* lse;
  void* workspace;
  // the 8-bit cache: two bytes a block of 16 entries
  const uint8_t* kv_scales;
  int64_t scale_page_stride, scale_head_stride;
};

size_t attn_workspace(int64_t n, int seqs, int q_heads, int kv_heads, int dim, int causal, int window, int max_q,
                      int max_kv);
hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t s);
size_t attn_q8_workspace(int64_t n, int seqs, int q_heads, int kv_heads, int dim, int causal, int window, int max_q,
                         int max_kv);
hipError_t launch_paged_attn_q8(const AttnArgs& a, hipStream_t s);

// Pages handed out and taken back.
struct PagesArgs {
  int64_t n, num_pages, table_stride;
  int32_t seqs, users, page_shift, table_width, out_width;
  const int32_t *lens, *who, *held;  // lens: new entries, or those to keep
  const int32_t* count;
  int32_t *tables, *free_pages, *held_out, *count_out;
  int32_t *q_offsets, *kv_lens, *page_table, *positions;
  int64_t* slots;
  void* workspace;
  int32_t* status;
};

size_t pages_workspace(int seqs);
hipError_t launch_pages_assign(const PagesArgs& a, hipStream_t s);
hipError_t launch_pages_release(const PagesArgs& a, hipStream_t s);

}  // namespace dlrm
