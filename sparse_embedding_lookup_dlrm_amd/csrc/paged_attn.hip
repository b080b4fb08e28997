// Attention of new tokens over a paged cache.
//
// For one head of the cache, the `group` query heads that read it and the new tokens of a
// sequence form rows, row = token * group + head in group. With c = scale log2(e), scores
// s = q . k and a running maximum m and sum l per row:
//     m' = max(m, max s),  p = 2^(c (s - m')),  l' = l 2^(c (m - m')) + sum p,
//     O' = O 2^(c (m - m')) + sum p v,          out = O / l,   lse = scale m + ln l.
//
// Scores are formed transposed, S^T = K Q^T, by 16x16x32 matrix instructions. Their result holds
// four entries of one row in each lane, which is what the second product O^T = V^T P^T takes as
// its right operand when the order of the 32 entries in the sum is chosen to fit (lane group g
// takes entries 4g .. 4g+3 of both halves): the weights never leave the lane, and m, l and the
// rescale of O are one value per lane.
#include "history_device.h"

namespace dlrm {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// fp16 weights are held times 2^8: a weight below 2^-14 of the largest would otherwise be
// subnormal and lose bits. bf16 has the exponent range of fp32.
template <int DT>
constexpr float kLift = DT == DLRM_F16 ? 8.f : 0.f;

template <int DT>
__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  if constexpr (DT == DLRM_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// Whether one of the two 16-bit values of a dword is infinite or NaN.
template <int DT>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  constexpr uint32_t e = DT == DLRM_BF16 ? 0x7f80u : 0x7c00u;
  return (w & e) == e || (w >> 16 & e) == e;
}

// A sequence of the call: its tokens and its history, checked.
struct Seq {
  int first, tokens, held;  // first token of the call, new tokens, entries (0 .. page table's room)
};

__device__ __forceinline__ Seq load_seq(const Paged& p, long long n, int seq) {
  Seq s;
  const int a = p.q_offsets[seq], b = p.q_offsets[seq + 1];
  const int held = p.kv_lens[seq], room = p.table_width << p.page_shift;
  const bool bad = a < 0 || b < a || b > n;
  s.first = bad ? 0 : a;
  s.tokens = bad ? 0 : b - a;
  s.held = held < 0 ? 0 : held > room ? room : held;
  if (s.held > 0 && p.num_pages == 0) {  // nothing to read
    s.held = 0;
    if (threadIdx.x == 0) flag(p.status, DLRM_STATUS_BAD_PAGE);
    return s;
  }
  if ((bad || s.held != held) && threadIdx.x == 0) flag(p.status, DLRM_STATUS_BAD_OFFSETS);
  return s;
}

// Entries [lo, hi) that a token sees.
struct Span {
  int lo, hi;
};

__device__ __forceinline__ Span seen_by(const Seq& s, int token, int causal, int window) {
  if (!causal) return {0, s.held};
  const long long at = static_cast<long long>(s.held) - s.tokens + token;
  const long long hi = at + 1, lo = window ? at - window + 1 : 0;
  return {static_cast<int>(lo > 0 ? lo : 0), static_cast<int>(hi > 0 ? hi : 0)};
}

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;

// ---------------------------------------------------------------------------
// Rows kernel: 16 RT rows of one head to a workgroup, the four waves take the 32-entry tiles of
// the history in turn and join their (m, l, O) through LDS at the end. Keys and values go from
// global memory to registers: each is used once. A lane takes D / 16 neighbouring elements of
// eight values' rows, so that a load instruction covers whole rows, and the transposition that
// the second product needs is 16-bit permutations in registers.
// ---------------------------------------------------------------------------
// How a call is cut: q_tiles tiles of rows per sequence and head, splits parts of a tile's entries.
struct Cut {
  int q_tiles, splits, part;  // part: entries of a part, unless the history is longer than announced
  long long units;            // workgroups' worth of work: sequences x tiles x parts x heads
  float* o;                   // [splits][n][q_heads][dim], not yet divided by the sums
  float2* ml;                 // [n][q_heads][splits]: maximum and sum
};

// Entries that the rows [row0, row_end) of a sequence see between them, and their parts.
struct Reach {
  int tok0, tok1;
  int lo, hi;          // some row sees these
  int all_lo, all_hi;  // every row sees these
  int first, part, parts;
  __device__ __forceinline__ Reach(const Seq& s, long long row0, long long row_end, int group, int causal, int window,
                                   const Cut& cut) {
    tok0 = static_cast<int>(row0 / group);
    tok1 = static_cast<int>((row_end - 1) / group);
    const Span s0 = seen_by(s, tok0, causal, window), s1 = seen_by(s, tok1, causal, window);
    lo = s0.lo;
    hi = s1.hi;
    all_lo = s1.lo;
    all_hi = s0.hi;
    first = lo & ~31;
    const int span = hi > first ? hi - first : 0;
    part = cut.part;
    if (span > static_cast<long long>(part) * cut.splits) part = static_cast<int>(((static_cast<long long>(span) + cut.splits - 1) / cut.splits + 31) & ~31LL);
    parts = span > part ? static_cast<int>((static_cast<long long>(span) + part - 1) / part) : 1;
  }
};

// Eight elements of a row's result, x still to be divided by the sum; a row that saw nothing is zero.
template <int DT>
__device__ __forceinline__ void finish(const AttnArgs& a, long long to, int at, float* x, float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int d = 0; d < 8; ++d) x[d] *= inv;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + to * a.dim + at) = narrow<DT>(x);
  if (at == 0 && a.lse) a.lse[to] = l == 0.f ? -INFINITY : fmaf(m, a.scale, logf(l) - kLift<DT> * kLn2);
}

template <int DT, int D, int RT>
__global__ __launch_bounds__(kThreads) void attn_rows_kernel(AttnArgs a, Cut cut) {
  constexpr int F = D / 32;           // k steps of the first product
  constexpr int E = D / 16;           // elements of a value row that a lane takes, and 16-wide pieces of O
  constexpr int Rows = 16 * RT;
  constexpr int Pitch = D + 4;        // floats; a row of O in LDS
  __shared__ float lds_o[kWaves][16 * Pitch];
  __shared__ float2 lds_ml[kWaves][Rows];
  const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int group = a.q_heads / a.kv_heads;
  const float c = a.scale * kLog2e;
  const Paged& pg = a.paged;
  const int page_mask = (1 << pg.page_shift) - 1;

  for (long long unit = blockIdx.x; unit < cut.units; unit += gridDim.x) {
    const int head = static_cast<int>(unit % a.kv_heads);
    long long rest = unit / a.kv_heads;
    const int split = static_cast<int>(rest % cut.splits);
    rest /= cut.splits;
    const int seq = static_cast<int>(rest / cut.q_tiles);
    const Seq sq = load_seq(pg, a.n, seq);
    const long long rows = static_cast<long long>(sq.tokens) * group;
    const uint16_t* kh = static_cast<const uint16_t*>(a.k_cache) + head * pg.head_stride;
    const uint16_t* vh = static_cast<const uint16_t*>(a.v_cache) + head * pg.head_stride;
    const int32_t* table = pg.page_table + seq * pg.table_stride;

    for (long long row0 = rest % cut.q_tiles * Rows; row0 < rows; row0 += static_cast<long long>(cut.q_tiles) * Rows) {
      const long long row_end = row0 + Rows < rows ? row0 + Rows : rows;
      const Reach rc(sq, row0, row_end, group, a.causal, a.window, cut);
      if (split >= rc.parts) continue;
      const int tok0 = rc.tok0, tok1 = rc.tok1, lo = rc.lo;
      const int k_first = rc.first + split * rc.part;
      const int hi = rc.hi < k_first + rc.part ? rc.hi : k_first + rc.part;

      u32x4 qf[RT][F];
      int row_lo[RT], row_hi[RT], row_tok[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const long long row = row0 + rt * 16 + c16;
        row_lo[rt] = row_hi[rt] = 0;
        row_tok[rt] = -1;
#pragma unroll
        for (int f = 0; f < F; ++f) qf[rt][f] = u32x4{0, 0, 0, 0};
        if (row < row_end) {
          const int tok = static_cast<int>(row / group), gi = static_cast<int>(row - static_cast<long long>(tok) * group);
          const Span s = seen_by(sq, tok, a.causal, a.window);
          row_lo[rt] = s.lo;
          row_hi[rt] = s.hi;
          row_tok[rt] = tok;
          const uint16_t* q = static_cast<const uint16_t*>(a.q.ptr) + (sq.first + tok) * a.q.stride +
                              (head * group + gi) * a.q.head_stride + g * 8;
#pragma unroll
          for (int f = 0; f < F; ++f) qf[rt][f] = *reinterpret_cast<const u32x4*>(q + f * 32);
        }
      }

      float m[RT], l[RT];
      f32x4 o[RT][E];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        m[rt] = -INFINITY;
        l[rt] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[rt][e] = f32x4{0, 0, 0, 0};
      }

      // Two 16-entry halves of a tile: where they are, and whether their pages are good. Past the end
      // and in place of a bad page another page of the cache is read and masked.
      struct Tile {
        long long at[2];
        bool good[2];
      };
      const auto look_up = [&](int k0) {
        Tile t;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int key = k0 + 16 * i < hi ? k0 + 16 * i : hi - 1;
          const int page = table[key >> pg.page_shift];
          t.good[i] = page >= 0 && page < pg.num_pages;
          if (!t.good[i] && k0 + 16 * i + 16 > lo && lane == 0) flag(pg.status, DLRM_STATUS_BAD_PAGE);
          t.at[i] = (t.good[i] ? page : 0) * pg.page_stride + (key & page_mask & ~15) * D;
        }
        return t;
      };
      u32x4 kf[2][F];
      uint32_t v[8][E / 2];
      const auto load_keys = [&](const Tile& t) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int f = 0; f < F; ++f)
            kf[i][f] = *reinterpret_cast<const u32x4*>(kh + t.at[i] + (c16 * D + g * 8) + f * 32);
      };
      const auto load_values = [&](const Tile& t) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          __builtin_memcpy(v[j], __builtin_assume_aligned(vh + t.at[j / 4] + (4 * g * D + c16 * E) + j % 4 * D,
                                                          E >= 8 ? 16 : 2 * E), 2 * E);
      };

      // The next tile's keys are asked for as soon as this tile's are used, its values likewise, so
      // that a wave has a tile of loads on the way all the time without a second set of registers.
      const int k_begin = k_first + 32 * wave;
      Tile tile, next;
      if (k_begin < hi) {
        tile = look_up(k_begin);
        load_keys(tile);
        load_values(tile);
      }
      for (int k0 = k_begin; k0 < hi; k0 += 32 * kWaves) {
        const int k_next = k0 + 32 * kWaves;
        if (k_next < hi) next = look_up(k_next);
        f32x4 sc[RT][2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            sc[rt][t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int f = 0; f < F; ++f) sc[rt][t] = mfma16<DT>(kf[t][f], qf[rt][f], sc[rt][t]);
          }
        if (k_next < hi) load_keys(next);

        u32x4 pw[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          f32x4(&s)[2] = sc[rt];
          float top = -INFINITY;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int key = k0 + 16 * t + 4 * g + r;
              if (!tile.good[t] || key < row_lo[rt] || key >= row_hi[rt] || key >= hi) s[t][r] = -INFINITY;
              top = fmaxf(top, s[t][r]);
            }
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(top, __shfl_xor(top, 32));
          const float next = fmaxf(m[rt], top);
          const float base = next == -INFINITY ? 0.f : next * c - kLift<DT>;
          const float keep = exp2f(m[rt] == -INFINITY ? -INFINITY : (m[rt] - next) * c);
          m[rt] = next;
          float p[8], sum = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            p[i] = exp2f(fmaf(s[i / 4][i % 4], c, -base));
            sum += p[i];
          }
          l[rt] = fmaf(l[rt], keep, sum);
#pragma unroll
          for (int e = 0; e < E; ++e) o[rt][e] *= keep;
#pragma unroll
          for (int i = 0; i < 4; ++i) pw[rt][i] = pack2<DT>(p[2 * i], p[2 * i + 1]);
        }

        // values that no row sees are zero, whatever they hold
        if (k0 < lo || k0 + 32 > hi || !tile.good[0] || !tile.good[1]) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int key = k0 + 16 * (j / 4) + 4 * g + j % 4;
            if (key < lo || key >= hi || !tile.good[j / 4]) {
#pragma unroll
              for (int i = 0; i < E / 2; ++i) v[j][i] = 0;
            }
          }
        }

        // entries that only some rows see: if one holds an infinity or NaN, the second product runs
        // token by token, with what the token does not see set to zero, and only the token's own rows
        // take the sum
        bool apart = false;
        if (tok1 > tok0 && (k0 < rc.all_lo || k0 + 32 > rc.all_hi)) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < E / 2; ++i) apart |= not_finite<DT>(v[j][i]);
          apart = __ballot(apart) != 0;
        }
        for (int tok = apart ? tok0 : tok1; tok <= tok1; ++tok) {
          uint32_t see[8];
          const Span s = seen_by(sq, tok, a.causal, a.window);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int key = k0 + 16 * (j / 4) + 4 * g + j % 4;
            see[j] = !apart || (key >= s.lo && key < s.hi) ? 0xffffffffu : 0;
          }
#pragma unroll
          for (int e = 0; e < E; ++e) {
            u32x4 vt;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              vt[i] = __builtin_amdgcn_perm(v[2 * i + 1][e / 2] & see[2 * i + 1], v[2 * i][e / 2] & see[2 * i],
                                            e % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              const f32x4 sum = mfma16<DT>(vt, pw[rt], o[rt][e]);
              if (!apart || row_tok[rt] == tok) o[rt][e] = sum;
            }
          }
        }
        if (k_next < hi) {
          load_values(next);
          tile = next;
        }
      }

      // join the waves
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        l[rt] += __shfl_xor(l[rt], 16);
        l[rt] += __shfl_xor(l[rt], 32);
        if (g == 0) lds_ml[wave][rt * 16 + c16] = make_float2(m[rt], l[rt]);
      }
      __syncthreads();
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, lds_ml[w][rt * 16 + c16].x);
        const float keep = m[rt] == -INFINITY ? 0.f : exp2f((m[rt] - top) * c);
        // lane (g, c16) holds elements 4 E g .. 4 E (g + 1) of its row, E at a time
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int e = 0; e < E; ++e) lds_o[wave][c16 * Pitch + (4 * g + r) * E + e] = o[rt][e][r] * keep;
        __syncthreads();
        constexpr int Pieces = D / 8;
        for (int i = threadIdx.x; i < 16 * Pieces; i += kThreads) {
          const int r16 = i / Pieces, at = i % Pieces * 8;
          const long long row = row0 + rt * 16 + r16;
          if (row >= row_end) continue;
          float mt = -INFINITY, lt = 0.f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) mt = fmaxf(mt, lds_ml[w][rt * 16 + r16].x);
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            const float2 ml = lds_ml[w][rt * 16 + r16];
            lt += ml.y * (ml.x == -INFINITY ? 0.f : exp2f((ml.x - mt) * c));
          }
          float x[8];
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            x[d] = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) x[d] += lds_o[w][r16 * Pitch + at + d];
          }
          const int tok = static_cast<int>(row / group), gi = static_cast<int>(row - static_cast<long long>(tok) * group);
          const long long to = static_cast<long long>(sq.first + tok) * a.q_heads + head * group + gi;
          if (rc.parts == 1) {
            finish<DT>(a, to, at, x, mt, lt);
          } else {
            float* p = cut.o + (split * a.n * a.q_heads + to) * D + at;
            *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
            if (at == 0) cut.ml[to * cut.splits + split] = make_float2(mt, lt);
          }
        }
        __syncthreads();
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Joins the parts of split histories: a workgroup to a row, D / 8 lanes to a part.
// ---------------------------------------------------------------------------
constexpr int kMaxSplits = 512;

template <int DT, int D>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnArgs a, Cut cut, int tile_rows) {
  constexpr int Lanes = D / 8, Slots = kThreads / Lanes;
  __shared__ float weight[kMaxSplits];
  __shared__ float red[kWaves];
  __shared__ float lds_o[kWaves][D];
  const int group = a.q_heads / a.kv_heads;
  const float c = a.scale * kLog2e;
  const long long units = cut.units / cut.splits;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  for (long long unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int head = static_cast<int>(unit % a.kv_heads);
    const long long rest = unit / a.kv_heads;
    const Seq sq = load_seq(a.paged, a.n, static_cast<int>(rest / cut.q_tiles));
    const long long rows = static_cast<long long>(sq.tokens) * group;
    for (long long row0 = rest % cut.q_tiles * tile_rows; row0 < rows;
         row0 += static_cast<long long>(cut.q_tiles) * tile_rows) {
      const long long row_end = row0 + tile_rows < rows ? row0 + tile_rows : rows;
      const Reach rc(sq, row0, row_end, group, a.causal, a.window, cut);
      if (rc.parts == 1) continue;
      for (long long row = row0 + blockIdx.y; row < row_end; row += gridDim.y) {
        const int tok = static_cast<int>(row / group), gi = static_cast<int>(row - static_cast<long long>(tok) * group);
        const long long to = static_cast<long long>(sq.first + tok) * a.q_heads + head * group + gi;
        const float2* ml = cut.ml + to * cut.splits;
        float m = -INFINITY;
        for (int i = threadIdx.x; i < rc.parts; i += kThreads) m = fmaxf(m, ml[i].x);
        for (int d = 1; d < kWave; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
        if (lane == 0) red[wave] = m;
        __syncthreads();
        m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        float l = 0.f;
        for (int i = threadIdx.x; i < rc.parts; i += kThreads) {
          const float2 p = ml[i];
          const float w = p.x == -INFINITY ? 0.f : exp2f((p.x - m) * c);
          weight[i] = w;
          l = fmaf(p.y, w, l);
        }
        for (int d = 1; d < kWave; d *= 2) l += __shfl_xor(l, d);
        __syncthreads();  // red was read
        if (lane == 0) red[wave] = l;
        __syncthreads();
        l = red[0] + red[1] + red[2] + red[3];
        const int at = threadIdx.x % Lanes * 8;
        float x[8] = {};
        const long long step = a.n * a.q_heads * D;
        const float* o = cut.o + to * D + at;
#pragma unroll 4
        for (int i = threadIdx.x / Lanes; i < rc.parts; i += Slots) {
          const float4 u = *reinterpret_cast<const float4*>(o + i * step);
          const float4 v = *reinterpret_cast<const float4*>(o + i * step + 4);
          const float w = weight[i];
          x[0] = fmaf(u.x, w, x[0]); x[1] = fmaf(u.y, w, x[1]); x[2] = fmaf(u.z, w, x[2]); x[3] = fmaf(u.w, w, x[3]);
          x[4] = fmaf(v.x, w, x[4]); x[5] = fmaf(v.y, w, x[5]); x[6] = fmaf(v.z, w, x[6]); x[7] = fmaf(v.w, w, x[7]);
        }
#pragma unroll
        for (int d = 0; d < 8; ++d) {
#pragma unroll
          for (int s = Lanes; s < kWave; s *= 2) x[d] += __shfl_xor(x[d], s);
          if (lane < Lanes) lds_o[wave][at + d] = x[d];
        }
        __syncthreads();
        if (threadIdx.x < Lanes) {
#pragma unroll
          for (int d = 0; d < 8; ++d) x[d] = lds_o[0][at + d] + lds_o[1][at + d] + lds_o[2][at + d] + lds_o[3][at + d];
          finish<DT>(a, to, at, x, m, l);
        }
        __syncthreads();
      }
    }
  }
}

// Sizes of a call's cut. A tile of one token's rows is bound by memory and its history is split into
// parts of at least kPart entries until there are kWanted workgroups: 16 for each place on the chip, so
// that histories of unequal length even out (64 histories of up to 16k entries: 270 us against 380 with
// 2048; one of 131k: 33.6 us with parts of 1024, 35.3 with 512, 39.7 with 256).
constexpr int kWanted = 8192, kPart = 1024;

Cut cut_rows(int rows_per_tile, long long max_rows, int seqs, int kv_heads, int causal, int window, int max_q,
             int max_kv) {
  Cut c;
  const long long tiles = max_rows > rows_per_tile ? (max_rows + rows_per_tile - 1) / rows_per_tile : 1;
  c.q_tiles = static_cast<int>(tiles);
  const long long whole = tiles * seqs * kv_heads;
  long long span = max_kv > 0 ? max_kv : 1;
  if (causal && window && span > static_cast<long long>(window) + max_q + 32) span = static_cast<long long>(window) + max_q + 32;
  long long splits = tiles > 1 ? 1 : kWanted / (whole > 0 ? whole : 1);
  const long long most = (span + kPart - 1) / kPart;
  splits = splits < 1 ? 1 : splits > most ? most : splits;
  if (splits > kMaxSplits) splits = kMaxSplits;
  c.splits = static_cast<int>(splits);
  c.part = static_cast<int>(((span + splits - 1) / splits + 31) & ~31LL);
  c.units = whole * splits;
  c.o = nullptr;
  c.ml = nullptr;
  return c;
}

constexpr size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

size_t cut_bytes(const Cut& c, int64_t n, int q_heads, int dim) {
  if (c.splits == 1) return 0;
  const size_t rows = static_cast<size_t>(n) * q_heads * c.splits;
  return round256(rows * dim * sizeof(float)) + rows * sizeof(float2);
}

constexpr long long kMaxGrid = 1 << 22;

template <int DT, int D, int RT>
hipError_t run_rows(const AttnArgs& a, hipStream_t s) {
  const long long rows = static_cast<long long>(a.max_q) * (a.q_heads / a.kv_heads);
  Cut cut = cut_rows(16 * RT, rows, a.paged.seqs, a.kv_heads, a.causal, a.window, a.max_q, a.max_kv);
  cut.o = static_cast<float*>(a.workspace);
  cut.ml = reinterpret_cast<float2*>(static_cast<char*>(a.workspace) +
                                     round256(static_cast<size_t>(a.n) * a.q_heads * cut.splits * D * sizeof(float)));
  hipLaunchKernelGGL((attn_rows_kernel<DT, D, RT>),
                     dim3(static_cast<unsigned>(cut.units < kMaxGrid ? cut.units : kMaxGrid)), dim3(kThreads), 0, s, a,
                     cut);
  if (cut.splits > 1) {
    const long long units = cut.units / cut.splits;
    hipLaunchKernelGGL((attn_join_kernel<DT, D>),
                       dim3(static_cast<unsigned>(units < kMaxGrid ? units : kMaxGrid),
                            static_cast<unsigned>(rows < 1 ? 1 : rows < 16 * RT ? rows : 16 * RT)),
                       dim3(kThreads), 0, s, a, cut, 16 * RT);
  }
  return hipGetLastError();
}

template <int DT, int D>
hipError_t run(const AttnArgs& a, hipStream_t s) {
  return run_rows<DT, D, 1>(a, s);
}

template <int DT>
hipError_t run_dim(const AttnArgs& a, hipStream_t s) {
  switch (a.dim) {
    case 32: return run<DT, 32>(a, s);
    case 64: return run<DT, 64>(a, s);
    case 128: return run<DT, 128>(a, s);
    default: return run<DT, 256>(a, s);
  }
}

}  // namespace

size_t attn_workspace(int64_t n, int seqs, int q_heads, int kv_heads, int dim, int causal, int window, int max_q,
                      int max_kv) {
  if (n == 0 || seqs == 0) return 0;
  return cut_bytes(cut_rows(16, static_cast<long long>(max_q) * (q_heads / kv_heads), seqs, kv_heads, causal, window,
                            max_q, max_kv),
                   n, q_heads, dim);
}

hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t s) {
  if (a.n == 0 || a.paged.seqs == 0) return hipSuccess;
  return a.dtype == DLRM_F16 ? run_dim<DLRM_F16>(a, s) : run_dim<DLRM_BF16>(a, s);
}

}  // namespace dlrm
