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
#include "history_device.h"

namespace dlrm {
namespace {

constexpr int kThreads = 256;

// A head of D elements is D / (2 V) lanes of two 16-byte pieces (V elements each), chosen so that the
// pairs of the rotation lie in one lane and each piece of neighbouring lanes is contiguous. Pairs of
// neighbours: the two halves of the head. Pairs (j, j + rot / 2): lane p < rot / (2 V) holds pairs V p ..
// V p + V - 1, the other lanes the halves of what is not rotated.
template <int DT, int D>
struct Split {
  static constexpr int V = Storage<DT>::per16;
  static constexpr int lanes = D / (2 * V);  // per head: 2 .. 32
  static constexpr int groups = kThreads / lanes;
  int at[2];        // first element of each piece
  int pair[2];      // first pair of each piece (of both, unless neighbours)
  bool rotated[2];

  __device__ __forceinline__ Split(int lane, int rot, bool interleaved) {
    const int turned = interleaved ? 0 : rot / (2 * V), from = interleaved ? 0 : rot;
    if (lane < turned) {
      at[0] = lane * V;
      at[1] = rot / 2 + lane * V;
      pair[0] = pair[1] = lane * V;
      rotated[0] = rotated[1] = true;
    } else {
      at[0] = from + (lane - turned) * V;
      at[1] = at[0] + (D - from) / 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        pair[i] = at[i] / 2;
        rotated[i] = interleaved && at[i] < rot;
      }
    }
  }
};

// A 16-byte piece of a result, stored past the caches. Other inputs each time, past and through them: training
// batch 60 us and 64, half of it 29 and 32, append of chunks 67 and 72. Calls of fewer tokens take as long either
// way, also with the attention that reads the results next: append and attention of 96 tokens 104 us and 105, of
// 4 x 1024 205 and 202, of 8 x 2048 760 and 767. (The backward alone would be faster through them: 94 us and 89.)
__device__ __forceinline__ void put(char* to, const uint4& v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4*>(to));
}

// A 16-byte piece of an input; Far: past the caches.
template <bool Far>
__device__ __forceinline__ uint4 get(const char* from) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  if constexpr (!Far) return *reinterpret_cast<const uint4*>(from);
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// cos and sin of the angles of tokens t0 .. t0 + count, [count][rot / 2] pairs in LDS.
__device__ __forceinline__ void angles(const Rotation& r, long long t0, int count, float2* cs) {
  const int pairs = r.rot / 2;
  if (pairs == 0) return;
  for (int i = threadIdx.x; i < count * pairs; i += kThreads) {
    const int t = i / pairs, j = i - t * pairs;
    int axis = 0;
    while (j >= r.section_end[axis]) ++axis;  // the last section ends at pairs
    const double turn = static_cast<double>(r.positions[axis * r.pos_stride + t0 + t]) *
                        static_cast<double>(r.inv_freq[j]) * 0.15915494309189535;
    float s, c;
    sincospif(static_cast<float>(2.0 * (turn - rint(turn))), &s, &c);
    cs[i] = make_float2(c, s);
  }
}

// x: V elements of piece 0, then V of piece 1; cs: the token's pairs. dir = 1 turns by the angles, -1
// turns back.
template <int DT, int D>
__device__ __forceinline__ void rotate(float* x, const float2* cs, const Split<DT, D>& split, bool interleaved,
                                       float dir) {
  constexpr int V = Split<DT, D>::V;
  if (interleaved) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (!split.rotated[p]) continue;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        float* y = x + p * V + 2 * i;
        const float2 w = cs[split.pair[p] + i];
        const float c = w.x, s = dir * w.y, a = y[0], b = y[1];
        y[0] = a * c - b * s;
        y[1] = a * s + b * c;
      }
    }
  } else if (split.rotated[0]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 w = cs[split.pair[0] + i];
      const float c = w.x, s = dir * w.y, a = x[i], b = x[V + i];
      x[i] = a * c - b * s;
      x[V + i] = a * s + b * c;
    }
  }
}

template <int DT>
__device__ __forceinline__ const char* head_at(const Heads& x, long long token, int head) {
  return static_cast<const char*>(x.ptr) + (token * x.stride + head * x.head_stride) * Storage<DT>::bytes;
}

// The (token, head) items of a workgroup's tokens, one to a group of lanes, groups apart.
struct Items {
  int t, h;
  const int heads, dt, dh;
  __device__ __forceinline__ Items(int group, int groups, int heads_)
      : t(group / heads_), h(group - t * heads_), heads(heads_), dt(groups / heads_), dh(groups - dt * heads_) {}
  __device__ __forceinline__ void next() {
    t += dt;
    h += dh;
    if (h >= heads) {
      h -= heads;
      ++t;
    }
  }
};

// One kind of head (queries, keys or values) of the workgroup's tokens. `before` shifts which group of
// lanes begins: the keys begin where the queries ended, so that in a small call each kind has groups of
// its own. The first item and the weights are asked for when the walk is made, before the workgroup has
// its angles and slots, and every further item while the one before it is worked on.
template <int DT, int D, bool TURN>
struct Walk {
  using S = Split<DT, D>;
  static constexpr int V = S::V;
  const Heads x;
  const int heads, count;
  const long long t0;
  Items it;
  const int lane;
  const S split;
  const bool norm;
  float wv[TURN ? 2 * V : 1];
  uint4 piece[2];

  __device__ __forceinline__ void load(int t, int h) {
    const char* from = head_at<DT>(x, t0 + t, h);
#pragma unroll
    for (int i = 0; i < 2; ++i) piece[i] = *reinterpret_cast<const uint4*>(from + split.at[i] * Storage<DT>::bytes);
  }

  __device__ __forceinline__ Walk(const NormRopeArgs& a, const Heads& x_, int heads_, const float* w, long long t0_,
                                  int count_, int before)
      : x(x_), heads(heads_), count(heads_ ? count_ : 0), t0(t0_),
        it((threadIdx.x / S::lanes + before) % S::groups, S::groups, heads_ ? heads_ : 1), lane(threadIdx.x % S::lanes),
        split(lane, TURN ? a.rope.rot : 0, a.rope.interleaved), norm(w != nullptr) {
    if (it.t >= count) return;
    load(it.t, it.h);
    if constexpr (TURN) {
      if (norm) {
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) wv[i] = w[split.at[i / V] + i % V];
      }
    }
  }

  // Without slots the result goes to out, contiguous [n][heads][D]; else to the cache: slots holds the
  // element offset of each token's slot in head 0 of its page, or -1 for a token that is not stored.
  __device__ __forceinline__ void run(const NormRopeArgs& a, const float2* cs, void* out, const long long* slots) {
    const int pairs = a.rope.rot / 2;
    while (it.t < count) {
      const int t = it.t, h = it.h;
      uint4 now[2] = {piece[0], piece[1]};
      it.next();
      if (it.t < count) load(it.t, it.h);
      if constexpr (TURN) {
        float y[2 * V];
        widen<DT>(now[0], y);
        widen<DT>(now[1], y + V);
        if (norm) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 2 * V; ++i) sum = fmaf(y[i], y[i], sum);
          sum = group_sum<S::lanes>(sum);
          const float r = rsqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
          for (int i = 0; i < 2 * V; ++i) y[i] = y[i] * r * wv[i];
        }
        rotate<DT, D>(y, cs + t * pairs, split, a.rope.interleaved, 1.f);
        now[0] = narrow<DT>(y);
        now[1] = narrow<DT>(y + V);
      }
      char* to;
      if (slots) {
        const long long slot = slots[t];
        if (slot < 0) continue;
        to = static_cast<char*>(out) + (slot + h * a.paged.head_stride) * Storage<DT>::bytes;
      } else {
        to = static_cast<char*>(out) + ((t0 + t) * heads + h) * D * Storage<DT>::bytes;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) put(to + split.at[i] * Storage<DT>::bytes, now[i]);
    }
  }
};

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
