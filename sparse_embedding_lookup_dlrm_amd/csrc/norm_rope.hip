// Norms of queries and keys per head with the position rotation in the same pass, their
// backward, and the append of keys and values to a paged cache.
//
//   y = x w / sqrt(mean(x^2) + eps), then (a, b) -> (a cos - b sin, a sin + b cos) on each pair
//
// Bound by memory: a token's heads are read once and written once. A head's pairs need one
// angle each, the same for all heads of a token, so a workgroup takes the cosines and sines of
// its tokens into LDS first (one evaluation per token and pair) and then walks the heads. The
// angle is formed in fp64 and reduced to a part of a turn before it is rounded: at position
// 100,000 an fp32 angle would be off by 4e-3 radians.
#include "rope_device.h"

namespace dlrm {
namespace {

constexpr int kMaxTokens = 4;  // tokens of a workgroup

// The first sequence with good offsets that holds a token, by the whole wave, or -1. For offsets that do not
// ascend, where the search of find_slots can end elsewhere.
__device__ __forceinline__ int scan_sequences(const Paged& p, int lo, int hi, int token) {
  const int lane = threadIdx.x & (kWave - 1);
  for (long long s0 = 0; s0 < p.seqs; s0 += kWave) {
    const long long s = s0 + lane;
    bool holds = false;
    if (s < p.seqs) {
      const int a = p.q_offsets[s], b = p.q_offsets[s + 1];
      holds = a >= lo && b <= hi && a <= token && token < b;
    }
    const unsigned long long found = __ballot(holds);
    if (found) return static_cast<int>(s0) + __builtin_ctzll(found);
  }
  return -1;
}

// Cache slots of tokens t0 .. t0 + count, one wave each, the last wave first: the first ones have the
// angles to form. A sequence's offsets are good if they ascend between the first and the last one of all.
template <int D>
__device__ __forceinline__ void find_slots(const Paged& p, long long n, long long t0, int count, long long* slots) {
  const int lane = threadIdx.x & (kWave - 1);
  for (int t = kThreads / kWave - 1 - threadIdx.x / kWave; t < count; t += kThreads / kWave) {
    const int token = static_cast<int>(t0) + t;
    const int first_of_all = p.q_offsets[0], last_of_all = p.q_offsets[p.seqs];
    int seq = wave_upper_bound(p.q_offsets, p.seqs + 1, token) - 1;
    long long slot = -1;
    if (token >= first_of_all && token < last_of_all) {  // else the token is in no sequence
      const int lo = first_of_all > 0 ? first_of_all : 0, hi = last_of_all < n ? last_of_all : static_cast<int>(n);
      bool bad = seq < 0 || seq >= p.seqs;
      int last = 0;
      if (!bad) {
        const int first = p.q_offsets[seq];
        last = p.q_offsets[seq + 1];
        bad = first < lo || last > hi || token < first || token >= last;
      }
      if (bad) {
        if (lane == 0) flag(p.status, DLRM_STATUS_BAD_OFFSETS);
        seq = scan_sequences(p, lo, hi, token);
        if (seq >= 0) last = p.q_offsets[seq + 1];
      }
      const int held = seq < 0 ? -1 : p.kv_lens[seq];
      const long long room = static_cast<long long>(p.table_width) << p.page_shift;
      const long long at = static_cast<long long>(held) - last + token;
      bad = at < 0 || at >= room || held < 0 || held > room;
      if (bad) {
        if (lane == 0) flag(p.status, DLRM_STATUS_BAD_OFFSETS);
      } else {
        const int page = p.page_table[seq * p.table_stride + (at >> p.page_shift)];
        if (page < 0 || page >= p.num_pages) {
          if (lane == 0) flag(p.status, DLRM_STATUS_BAD_PAGE);
        } else {
          slot = page * p.page_stride + (at & ((1LL << p.page_shift) - 1)) * D;
        }
      }
    }
    if (lane == 0) slots[t] = slot;
  }
}

template <int DT, int D, bool APPEND>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(NormRopeArgs a, long long from, int per_group) {
  __shared__ float2 cs[kMaxTokens * D / 2];
  __shared__ long long slots[APPEND ? kMaxTokens : 1];
  const long long t0 = from + static_cast<long long>(blockIdx.x) * per_group;
  const int count = static_cast<int>(a.n - t0 < per_group ? a.n - t0 : per_group);
  constexpr int G = Split<DT, D>::groups;
  const int after_q = G - count * a.q_heads % G, after_k = after_q + G - count * a.kv_heads % G;
  Walk<DT, D, true> q(a, a.q, a.q_heads, a.w_q, t0, count, 0);
  Walk<DT, D, true> k(a, a.k, a.kv_heads, a.w_k, t0, count, after_q);
  if constexpr (APPEND) {
    Walk<DT, D, false> v(a, a.v, a.kv_heads, nullptr, t0, count, after_k);
    angles(a.rope, t0, count, cs);
    find_slots<D>(a.paged, a.n, t0, count, slots);
    __syncthreads();
    q.run(a, cs, a.q_out, nullptr);
    k.run(a, cs, a.k_cache, slots);
    v.run(a, cs, a.v_cache, slots);
  } else {
    angles(a.rope, t0, count, cs);
    __syncthreads();
    q.run(a, cs, a.q_out, nullptr);
    k.run(a, cs, a.k_out, nullptr);
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
constexpr int kBwdGroups = 1024;  // workgroups that share the tokens; one row of partial weight gradients each
constexpr int kBwdTokens = 4;     // tokens whose angles are held at once

// One kind of head of the workgroup's tokens. (With loads an item ahead, or the next tokens' angles formed
// beside, the kernel takes 166 registers and more, three waves to a SIMD instead of four: 104 .. 114 us for
// the training batch against 100.)
template <int DT, int D, bool Far>
__device__ __forceinline__ void walk_bwd(const NormRopeBwdArgs& a, const Heads& dy, const Heads& x, int heads,
                                         const float* w, long long t0, int count, const float2* cs, void* out,
                                         float* dw) {
  using S = Split<DT, D>;
  constexpr int V = S::V;
  const int lane = threadIdx.x % S::lanes;
  const S split(lane, a.rope.rot, a.rope.interleaved);
  float wv[2 * V];
  if (w) {
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) wv[i] = w[split.at[i / V] + i % V];
  }
  const int pairs = a.rope.rot / 2;
  for (Items it(threadIdx.x / S::lanes, S::groups, heads); it.t < count; it.next()) {
    const int t = it.t, h = it.h;
    const char* from = head_at<DT>(dy, t0 + t, h);
    float g[2 * V];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      widen<DT>(get<Far>(from + split.at[i] * Storage<DT>::bytes), g + i * V);
    rotate<DT, D>(g, cs + t * pairs, split, a.rope.interleaved, -1.f);
    if (w) {
      const char* in = head_at<DT>(x, t0 + t, h);
      float u[2 * V];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        widen<DT>(get<Far>(in + split.at[i] * Storage<DT>::bytes), u + i * V);
      float sq = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) {
        sq = fmaf(u[i], u[i], sq);
        dot = fmaf(g[i] * wv[i], u[i], dot);
      }
      sq = group_sum<S::lanes>(sq);
      dot = group_sum<S::lanes>(dot);
      const float r = rsqrtf(sq * (1.f / D) + a.eps);
      const float mean = dot * r * (1.f / D);  // mean of g w u r
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) {
        u[i] *= r;
        dw[i] = fmaf(g[i], u[i], dw[i]);
        g[i] = r * (g[i] * wv[i] - u[i] * mean);
      }
    }
    char* to = static_cast<char*>(out) + ((t0 + t) * heads + h) * D * Storage<DT>::bytes;
#pragma unroll
    for (int i = 0; i < 2; ++i) put(to + split.at[i] * Storage<DT>::bytes, narrow<DT>(g + i * V));
  }
}

// Sums dw over the groups of the workgroup into row[D], in a fixed order.
template <int DT, int D>
__device__ __forceinline__ void join(const Rotation& rope, const float* dw, float* lds, float* row) {
  using S = Split<DT, D>;
  constexpr int V = S::V;
  const int lane = threadIdx.x % S::lanes;
  const S split(lane, rope.rot, rope.interleaved);
  __syncthreads();  // lds is free again
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) {
    float v = dw[i];
#pragma unroll
    for (int m = S::lanes; m < kWave; m *= 2) v += __shfl_xor(v, m);  // lanes that hold the same element
    if (threadIdx.x % kWave < S::lanes) lds[threadIdx.x / kWave * D + split.at[i / V] + i % V] = v;
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kThreads) row[d] = lds[d] + lds[D + d] + lds[2 * D + d] + lds[3 * D + d];
}

template <int DT, int D, bool Far>
__global__ __launch_bounds__(kThreads) void norm_rope_bwd_kernel(NormRopeBwdArgs a) {
  constexpr int V = Storage<DT>::per16;
  __shared__ float2 cs[kBwdTokens * D / 2];
  __shared__ float lds[kThreads / kWave * D];
  float dq[2 * V] = {}, dk[2 * V] = {};
  const long long step = static_cast<long long>(gridDim.x) * kBwdTokens;
  for (long long t0 = static_cast<long long>(blockIdx.x) * kBwdTokens; t0 < a.n; t0 += step) {
    const int count = static_cast<int>(a.n - t0 < kBwdTokens ? a.n - t0 : kBwdTokens);
    __syncthreads();  // the angles of the tokens before are no longer read
    angles(a.rope, t0, count, cs);
    __syncthreads();
    walk_bwd<DT, D, Far>(a, a.dq_out, a.q, a.q_heads, a.w_q, t0, count, cs, a.d_q, dq);
    walk_bwd<DT, D, Far>(a, a.dk_out, a.k, a.kv_heads, a.w_k, t0, count, cs, a.d_k, dk);
  }
  if (a.w_q) {
    float* row = a.partials + static_cast<long long>(blockIdx.x) * 2 * D;
    join<DT, D>(a.rope, dq, lds, row);
    join<DT, D>(a.rope, dk, lds, row + D);
  }
}

// Columns of the partial weight gradients [rows][2 D] summed in a fixed order, in fp64: 32 columns to a
// workgroup, 32 threads to a column (1024 rows: 4 us; with eight threads and no loads ahead it was 38).
constexpr int kDwThreads = 1024;
__global__ __launch_bounds__(kDwThreads) void norm_rope_dw_kernel(const float* __restrict__ partials, int rows, int dim,
                                                                  float* d_w_q, float* d_w_k) {
  __shared__ double lds[kDwThreads / 32][33];
  const int c = threadIdx.x % 32, col = blockIdx.x * 32 + c, part = threadIdx.x / 32;
  double sum = 0.;
#pragma unroll 8
  for (int r = part; r < rows; r += kDwThreads / 32) sum += partials[static_cast<long long>(r) * 2 * dim + col];
  lds[part][c] = sum;
  __syncthreads();
  // 32 lanes to a column
  double v = lds[c][part];
#pragma unroll
  for (int m = 1; m < 32; m *= 2) v += __shfl_xor(v, m, 32);
  const int to = blockIdx.x * 32 + part;
  if (c == 0) (to < dim ? d_w_q + to : d_w_k + (to - dim))[0] = static_cast<float>(v);
}

// Tokens of a workgroup: as many as leave four workgroups to each CU, so that the angles of a
// token are shared by all its heads and small calls still spread over the chip.
int tokens_per_group(long long n) {
  const long long t = n / 1024;
  return static_cast<int>(t < 1 ? 1 : t > kMaxTokens ? kMaxTokens : t);
}

template <int DT, int D, bool APPEND>
hipError_t run(const NormRopeArgs& a, hipStream_t s) {
  const int per = tokens_per_group(a.n);
  // a grid has fewer than 2^32 threads: 2^23 workgroups to a launch
  constexpr long long kMostGroups = 1 << 23;
  for (long long from = 0; from < a.n; from += kMostGroups * per) {
    const long long left = (a.n - from + per - 1) / per;
    hipLaunchKernelGGL((norm_rope_kernel<DT, D, APPEND>),
                       dim3(static_cast<unsigned>(left < kMostGroups ? left : kMostGroups)), dim3(kThreads), 0, s, a,
                       from, per);
  }
  return hipGetLastError();
}

template <int DT, bool APPEND>
hipError_t run_dim(const NormRopeArgs& a, hipStream_t s) {
  switch (a.dim) {
    case 32: return run<DT, 32, APPEND>(a, s);
    case 64: return run<DT, 64, APPEND>(a, s);
    case 128: return run<DT, 128, APPEND>(a, s);
    default: return run<DT, 256, APPEND>(a, s);
  }
}

int bwd_groups(long long n) {
  const long long g = (n + kBwdTokens - 1) / kBwdTokens;
  return static_cast<int>(g < kBwdGroups ? g : kBwdGroups);
}

template <int DT, int D>
hipError_t run_bwd(const NormRopeBwdArgs& a, hipStream_t s) {
  const int groups = bwd_groups(a.n);
  // Inputs of more than the 256 MB of the last cache are read past the caches (16384 tokens of 40 heads of 128,
  // 335 MB: 94 us against 100); smaller ones may still lie there from the kernels that made them (8192 tokens,
  // 168 MB: 48 us against 52 if they do, 56 against 53 if not).
  const double read = static_cast<double>(a.n) * (a.q_heads + a.kv_heads) * D * Storage<DT>::bytes * (a.w_q ? 2 : 1);
  if (groups > 0 && read > 256e6)
    hipLaunchKernelGGL((norm_rope_bwd_kernel<DT, D, true>), dim3(groups), dim3(kThreads), 0, s, a);
  else if (groups > 0)
    hipLaunchKernelGGL((norm_rope_bwd_kernel<DT, D, false>), dim3(groups), dim3(kThreads), 0, s, a);
  if (a.w_q)
    hipLaunchKernelGGL(norm_rope_dw_kernel, dim3(2 * D / 32), dim3(kDwThreads), 0, s, a.partials, groups, D, a.d_w_q,
                       a.d_w_k);
  return hipGetLastError();
}

template <int DT>
hipError_t run_bwd_dim(const NormRopeBwdArgs& a, hipStream_t s) {
  switch (a.dim) {
    case 32: return run_bwd<DT, 32>(a, s);
    case 64: return run_bwd<DT, 64>(a, s);
    case 128: return run_bwd<DT, 128>(a, s);
    default: return run_bwd<DT, 256>(a, s);
  }
}

}  // namespace

hipError_t launch_norm_rope(const NormRopeArgs& a, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  switch (a.dtype) {
    case DLRM_F32: return run_dim<DLRM_F32, false>(a, s);
    case DLRM_F16: return run_dim<DLRM_F16, false>(a, s);
    default: return run_dim<DLRM_BF16, false>(a, s);
  }
}

hipError_t launch_kv_append(const NormRopeArgs& a, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  return a.dtype == DLRM_F16 ? run_dim<DLRM_F16, true>(a, s) : run_dim<DLRM_BF16, true>(a, s);
}

size_t norm_rope_bwd_workspace(int64_t n, int dim, bool norm) {
  return norm ? static_cast<size_t>(bwd_groups(n)) * 2 * dim * sizeof(float) : 0;
}

hipError_t launch_norm_rope_bwd(const NormRopeBwdArgs& a, hipStream_t s) {
  switch (a.dtype) {
    case DLRM_F32: return run_bwd_dim<DLRM_F32>(a, s);
    case DLRM_F16: return run_bwd_dim<DLRM_F16>(a, s);
    default: return run_bwd_dim<DLRM_BF16>(a, s);
  }
}

}  // namespace dlrm
