// Append of keys and values to a paged cache of 8-bit codes, the keys normed and rotated on the way, and norm and
// rotation of the queries in the same launch.
//
// A block of 16 entries of a head has one power of two, 2^(b - 127), for its keys and one for its values. With A the
// largest finite |x| of the new entries in it, b is the smallest for which A <= 448 x 2^(b - 127), 448 = 1.75 x 2^8
// being the largest code: the biased exponent of A less 8, and one more if its significand is above 1.75. A block
// that holds older entries keeps its b where that is larger; else their codes are rounded again to the new one. The
// scale is a power of two, so that this second rounding only shortens codes that become subnormal: a code of k
// significant bits stays as it is as long as it keeps them.
//
// A wave takes the block of one head: 16 entries in registers, one maximum, and the codes. Blocks that new entries
// touch are known on the device only, so each sequence has a fixed number of workgroups that take its blocks in turn.
//
// Bound by memory: 11937 tokens of 12 users, 32 + 2 x 8 heads of 128 fp16: 62 us for 269 MB, 4.3 TB/s (the queries, 195
// MB, would take 36 at the rate of the 16-bit append; keys and values wait for their blocks' maxima between load and
// store, with 12 waves on a CU).
#include "rope_device.h"

namespace dlrm {
namespace {

constexpr int kBlock = DLRM_KV_BLOCK;
constexpr int kWaves = kThreads / kWave;
constexpr int kQueryTokens = 4;  // most tokens of a workgroup of the queries

// How a call is cut: for the keys and values `lanes` workgroups to a sequence that take its blocks in turn, times
// `parts` that share the heads; then workgroups of the queries, `per` tokens to each step.
struct AppendGrid {
  long long query_steps, units;  // steps of all workgroups; lanes x sequences x parts
  int query_groups, unit_groups, per, lanes, parts;
};

// Eight fp32 values as codes, and back. The conversion rounds to nearest even, what is not finite to NaN.
__device__ __forceinline__ uint2 to_codes(const float* x) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
  return make_uint2(lo, hi);
}
__device__ __forceinline__ void from_codes(const uint2& codes, float* x) {
  const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], true);
    x[4 * i] = a[0];
    x[4 * i + 1] = a[1];
    x[4 * i + 2] = b[0];
    x[4 * i + 3] = b[1];
  }
}

// The byte of a block whose largest finite element is `top`.
__device__ __forceinline__ int scale_byte(float top) {
  const uint32_t bits = __float_as_uint(top);
  const int b = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return b < 1 ? 1 : b;
}

// A block of a sequence: entries first .. first + 16, of which [from, to) are new and those before `from` are older.
struct Unit {
  int first, from, to;
  long long token;  // of entry `from`
  long long at;     // bytes: entry `first` of head 0
  long long scale;  // its scales of head 0
};

// The block of one head, by a wave (of heads of 32: by half a wave). Key: normed and rotated.
template <int DT, int D, bool KEY>
struct BlockTask {
  using S = Split<DT, D>;
  static constexpr int V = S::V, Lanes = S::lanes;
  static constexpr int Slots = kWave / Lanes;              // entries of a pass
  static constexpr int Side = Slots > kBlock ? Slots / kBlock : 1;  // heads side by side
  static constexpr int Passes = Slots < kBlock ? kBlock / Slots : 1;
  const NormRopeArgs& a;
  const S split;
  const int slot;
  uint4 raw[Passes][2];

  __device__ __forceinline__ explicit BlockTask(const NormRopeArgs& a_)
      : a(a_), split(threadIdx.x % Lanes, KEY ? a_.rope.rot : 0, a_.rope.interleaved),
        slot(threadIdx.x % kWave / Lanes % kBlock) {}

  // The new entry of this lane in pass p, counted from the first. A lane without one takes its neighbour's, which
  // changes no maximum, and stores nothing: a load within a branch would be waited for at its end.
  __device__ __forceinline__ int entry(const Unit& u, int p) const {
    const int e = u.first + p * Slots + slot;
    return (e < u.from ? u.from : e < u.to ? e : u.to - 1) - u.from;
  }

  __device__ __forceinline__ void load(const Unit& u, int head) {
#pragma unroll
    for (int p = 0; p < Passes; ++p) {
      const char* x = head_at<DT>(KEY ? a.k : a.v, u.token + entry(u, p), head);
#pragma unroll
      for (int i = 0; i < 2; ++i) raw[p][i] = *reinterpret_cast<const uint4*>(x + split.at[i] * Storage<DT>::bytes);
    }
  }

  __device__ __forceinline__ void store(const Unit& u, int head, const float2* cs) {
    uint8_t* scale = a.kv_scales + u.scale + head * a.scale_head_stride + (KEY ? 0 : 1);
    const int had = u.from > u.first ? *scale : 0;
    float y[Passes][2 * V], top = 0.f;
    float wv[KEY ? 2 * V : 1];
    const bool norm = KEY && a.w_k;
    if constexpr (KEY) {
      if (norm) {
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) wv[i] = a.w_k[split.at[i / V] + i % V];
      }
    }
#pragma unroll
    for (int p = 0; p < Passes; ++p) {
      widen<DT>(raw[p][0], y[p]);
      widen<DT>(raw[p][1], y[p] + V);
      if constexpr (KEY)
        norm_turn<DT, D>(y[p], wv, norm, a.eps, cs + entry(u, p) * (a.rope.rot / 2), split, a.rope.interleaved);
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) {
        const float x = fabsf(y[p][i]);
        top = fmaxf(top, x < INFINITY ? x : 0.f);
      }
    }
#pragma unroll
    for (int m = 1; m < kWave / Side; m *= 2) top = fmaxf(top, __shfl_xor(top, m));
    const int need = scale_byte(top), b = need > had ? need : had;
    const float up = ldexpf(1.f, 127 - b), again = ldexpf(1.f, had - b);
    uint8_t* to = static_cast<uint8_t*>(KEY ? a.k_cache : a.v_cache) + u.at + head * a.paged.head_stride;
#pragma unroll
    for (int p = 0; p < Passes; ++p) {
      const int in = p * Slots + slot, e = u.first + in;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint2* place = reinterpret_cast<uint2*>(to + in * D + split.at[i]);
        if (e < u.from) {
          if (b == had) continue;
          float x[8];
          from_codes(*place, x);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] *= again;
          *place = to_codes(x);
        } else if (e < u.to) {
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = y[p][i * V + k] * up;
          *place = to_codes(x);
        }
      }
    }
    if (threadIdx.x % (kWave / Side) == 0) *scale = static_cast<uint8_t>(b);
  }
};

template <int DT, int D>
__device__ __forceinline__ void append_unit(const NormRopeArgs& a, const AppendGrid& grid, long long unit, float2* cs) {
  const Paged& pg = a.paged;
  const int part = static_cast<int>(unit % grid.parts);
  const int seq = static_cast<int>(unit / grid.parts % pg.seqs), lane = static_cast<int>(unit / grid.parts / pg.seqs);
  const int first_of_all = pg.q_offsets[0], last_of_all = pg.q_offsets[pg.seqs];
  const int first = pg.q_offsets[seq], last = pg.q_offsets[seq + 1], held = pg.kv_lens[seq];
  const long long room = static_cast<long long>(pg.table_width) << pg.page_shift;
  int bad = 0, tokens = last - first;
  if (first < 0 || first < first_of_all || last < first || last > last_of_all || last > a.n) {
    bad = DLRM_STATUS_BAD_OFFSETS;
    tokens = 0;
  } else if (tokens > 0 && (held < 0 || held > room)) {
    bad = DLRM_STATUS_BAD_OFFSETS;
    tokens = 0;
  } else if (tokens > held) {  // those before the first entry are not stored
    bad = DLRM_STATUS_BAD_OFFSETS;
    tokens = held;
  }
  if (bad && threadIdx.x == 0) flag(pg.status, bad);
  if (tokens == 0) return;
  const int from = held - tokens, blocks = (held - 1) / kBlock - from / kBlock + 1;
  using Key = BlockTask<DT, D, true>;
  using Value = BlockTask<DT, D, false>;
  constexpr int Side = Key::Side;
  // the heads of values and then of keys, in turn over the waves (and their halves) of the parts
  const int wave = threadIdx.x / kWave, half = threadIdx.x % kWave / (kWave / Side);
  const int mine = (part * kWaves + wave) * Side + half, step = grid.parts * kWaves * Side;

  for (int i = lane; i < blocks; i += grid.lanes) {
    Unit u;
    u.first = (from / kBlock + i) * kBlock;
    u.from = u.first > from ? u.first : from;
    u.to = held < u.first + kBlock ? held : u.first + kBlock;
    u.token = last - held + u.from;
    const int page = pg.page_table[seq * pg.table_stride + (u.first >> pg.page_shift)];
    if (page < 0 || page >= pg.num_pages) {
      if (threadIdx.x == 0) flag(pg.status, DLRM_STATUS_BAD_PAGE);
      continue;
    }
    const int in_page = u.first & ((1 << pg.page_shift) - 1);
    u.at = page * pg.page_stride + static_cast<long long>(in_page) * D;
    u.scale = page * a.scale_page_stride + in_page / kBlock * 2;
    Value value(a);
    int task = mine;
    for (; task < a.kv_heads; task += step) {
      value.load(u, task);
      value.store(u, task, nullptr);
    }
    __syncthreads();  // the angles of the block before are no longer read
    angles(a.rope, u.token, u.to - u.from, cs);
    __syncthreads();
    Key key(a);
    for (; task < 2 * a.kv_heads; task += step) {
      key.load(u, task - a.kv_heads);
      key.store(u, task - a.kv_heads, cs);
    }
  }
}

template <int DT, int D>
__global__ __launch_bounds__(kThreads) void kv_append_q8_kernel(NormRopeArgs a, AppendGrid grid) {
  __shared__ float2 cs[kBlock * D / 2];
  // keys and values first: their workgroups take longer
  if (blockIdx.x < grid.unit_groups) {
    for (long long unit = blockIdx.x; unit < grid.units; unit += grid.unit_groups) {
      __syncthreads();
      append_unit<DT, D>(a, grid, unit, cs);
    }
    return;
  }
  for (long long step = blockIdx.x - grid.unit_groups; step < grid.query_steps; step += grid.query_groups) {
    const long long t0 = step * grid.per;
    const int count = static_cast<int>(a.n - t0 < grid.per ? a.n - t0 : grid.per);
    Walk<DT, D, true> q(a, a.q, a.q_heads, a.w_q, t0, count, 0);
    __syncthreads();  // the angles of the tokens before are no longer read
    angles(a.rope, t0, count, cs);
    __syncthreads();
    q.run(a, cs, a.q_out, nullptr);
  }
}

// A grid has fewer than 2^32 threads; what is past these many workgroups is done in turn.
constexpr long long kMostGroups = 1 << 22;

AppendGrid append_grid(const NormRopeArgs& a) {
  AppendGrid g;
  const long long seqs = a.paged.seqs > 0 ? a.paged.seqs : 1;
  const long long per = a.n / 1024;
  g.per = static_cast<int>(per < 1 ? 1 : per > kQueryTokens ? kQueryTokens : per);
  g.query_steps = a.q_heads > 0 ? (a.n + g.per - 1) / g.per : 0;
  g.query_groups = static_cast<int>(g.query_steps < kMostGroups ? g.query_steps : kMostGroups);
  // Workgroups of a sequence: twice the blocks that sequences have on average, more where there are few, and no more
  // than blocks it can have. Those that find none cost as well (chunks of 12 users, with queries before keys: 64 us, 72
  // with twice as many in parts, 88 with four times). That is made for lengths that are alike: where one is far above
  // the average its blocks wait in turn (a chunk of 2048 beside 95 single events 74 us, alone 30; one of 16384 beside
  // 127 of them 514, alone 62).
  const long long most = a.n / kBlock + 2, average = 2 * (a.n / (kBlock * seqs) + 1), fill = 512 / seqs;
  long long lanes = average > fill ? average : fill;
  if (lanes > most) lanes = most;
  g.lanes = static_cast<int>(lanes < 1 ? 1 : lanes);
  const long long blocks = a.n / kBlock + seqs;  // about as many as have work
  const int side = a.dim == 32 ? 2 : 1, apart = (2 * a.kv_heads + kWaves * side - 1) / (kWaves * side);
  const long long parts = 1024 / blocks;
  g.parts = static_cast<int>(parts < 1 ? 1 : parts < apart ? parts : apart);
  g.units = a.paged.seqs > 0 ? g.lanes * seqs * g.parts : 0;
  g.unit_groups = static_cast<int>(g.units < kMostGroups ? g.units : kMostGroups);
  return g;
}

template <int DT>
hipError_t run_dim(const NormRopeArgs& a, hipStream_t s) {
  const AppendGrid g = append_grid(a);
  const dim3 grid(g.query_groups + g.unit_groups);
  if (grid.x == 0) return hipSuccess;
  switch (a.dim) {
    case 32: hipLaunchKernelGGL((kv_append_q8_kernel<DT, 32>), grid, dim3(kThreads), 0, s, a, g); break;
    case 64: hipLaunchKernelGGL((kv_append_q8_kernel<DT, 64>), grid, dim3(kThreads), 0, s, a, g); break;
    case 128: hipLaunchKernelGGL((kv_append_q8_kernel<DT, 128>), grid, dim3(kThreads), 0, s, a, g); break;
    default: hipLaunchKernelGGL((kv_append_q8_kernel<DT, 256>), grid, dim3(kThreads), 0, s, a, g);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append_q8(const NormRopeArgs& a, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  return a.dtype == DLRM_F16 ? run_dim<DLRM_F16>(a, s) : run_dim<DLRM_BF16>(a, s);
}

}  // namespace dlrm
