// What the attention kernels of the 16-bit and the 8-bit cache share: sequences and what their tokens see,
// how a call is cut, matrix instructions, and the join of split histories.
//
// For one head of the cache, the `group` query heads that read it and the new tokens of a
// sequence form rows, row = token * group + head in group. With c = scale log2(e), scores
// s = q . k and a running maximum m and sum l per row:
//     m' = max(m, max s),  p = 2^(c (s - m')),  l' = l 2^(c (m - m')) + sum p,
//     O' = O 2^(c (m - m')) + sum p v,          out = O / l,   lse = scale m + ln l.
#pragma once

#include <type_traits>

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

// The 8-bit cache: e4m3 codes, and for each block of 16 entries of a head a byte b for the keys and one for the
// values, whose codes stand for code x 2^(b - 127).
constexpr int kScaleBlock = 16;

// Two values of a dword of codes (the low or the high half) in the 16-bit type; exact within its range. The
// instruction takes the power of two from the exponent of its scale.
template <int DT, bool HIGH>
__device__ __forceinline__ uint32_t widen_codes(uint32_t codes, float scale) {
  if constexpr (DT == DLRM_BF16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, HIGH));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, HIGH));
}

// The scales of keys and of values from the two bytes of a block.
__device__ __forceinline__ float key_scale(int bytes) { return __uint_as_float((bytes & 0xff) << 23); }
__device__ __forceinline__ float value_scale(int bytes) { return __uint_as_float((bytes >> 8 & 0xff) << 23); }

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ f32x16 mfma32(const u32x4& a, const u32x4& b, const f32x16& c) {
  if constexpr (DT == DLRM_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// Tiles of the tile kernels lie in LDS in rows of D 16-bit elements, D / 8 pieces of 16 bytes; piece c of entry r
// lies at place c ^ swizzle(r). Keys are read as rows (32 entries, the same piece): neighbours differ in every place
// bit.
template <int D>
__device__ __forceinline__ int key_swizzle(int r) {
  return D == 32 ? r >> 1 & 3 : D == 64 ? r & 7 : r & 15;
}
// Values are read as blocks of 4 entries x 2 (or, with the neighbouring lanes, 4) pieces.
template <int D>
__device__ __forceinline__ int value_swizzle(int r) {
  return D == 32 ? r & 2 : D == 64 ? (r & 1) << 2 | (r & 2) : (r & 1) << 2 | (r & 2) | (r & 2) << 2;
}

// All bits of those of the two 16-bit values of a dword that are infinite or NaN.
template <int DT>
__device__ __forceinline__ uint32_t not_finite_halves(uint32_t w) {
  constexpr uint32_t e = DT == DLRM_BF16 ? 0x7f80u : 0x7c00u;
  return ((w & e) == e ? 0xffffu : 0u) | ((w >> 16 & e) == e ? 0xffff0000u : 0u);
}

// A word that is the same for the whole wave, read by the scalar unit: no wait for it holds up vector
// loads on the way. Nothing writes the arrays read so while a kernel runs.
__device__ __forceinline__ int scalar_load(const int32_t* p, long long i) {
  return ((const __attribute__((address_space(4))) int32_t*)p)[i];
}

// A sequence of the call: its tokens and its history, checked.
struct Seq {
  int first, tokens, held;  // first token of the call, new tokens, entries (0 .. page table's room)
};

__device__ __forceinline__ Seq load_seq(const Paged& p, long long n, int seq) {
  Seq s;
  const int a = scalar_load(p.q_offsets, seq), b = scalar_load(p.q_offsets, seq + 1LL);
  const int first = scalar_load(p.q_offsets, 0), last = scalar_load(p.q_offsets, p.seqs);
  const int held = scalar_load(p.kv_lens, seq), room = p.table_width << p.page_shift;
  const bool bad = a < 0 || a < first || b < a || b > last || b > n;
  s.first = bad ? 0 : a;
  s.tokens = bad ? 0 : b - a;
  s.held = held < 0 ? 0 : held > room ? room : held;
  if ((bad || s.held != held) && threadIdx.x == 0) flag(p.status, DLRM_STATUS_BAD_OFFSETS);
  if (p.num_pages == 0) {  // nothing to read; the last token would see the last entry
    if (s.held > 0 && s.tokens > 0 && threadIdx.x == 0) flag(p.status, DLRM_STATUS_BAD_PAGE);
    s.held = 0;
  }
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

// The larger of a lane and the one 32 away.
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The same within pairs of sixteen lanes.
__device__ __forceinline__ float max_quarters(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add_quarters(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// How a call is cut: q_tiles tiles of rows per sequence and head, splits parts of a tile's entries. The
// grid is heads x (tiles x parts) x sequences. A sequence of fewer tiles than there are places for them has up to
// `spread` parts in their stead, if that is more and its rows have room.
//
// Sums of parts lie in rows of dim elements: with splits > 1 splits x n x q_heads of them, [split][token][head];
// behind these, with a spread, spare x kv_heads rows for each sequence, [split][token of the sequence][head].
struct Cut {
  int q_tiles, splits, part;  // part: entries of a part, unless the history is longer than announced
  int spread, spare;          // spare: rows of a head that a sequence has for the sums of its spread
  float* o;                   // sums, not yet divided
  float2* ml;                 // maximum and sum of each: [token][head][split], like the rows in bytes
  // Parts that a sequence of so many rows may have, in tiles of tile_rows.
  __device__ __forceinline__ int parts_of(int rows, int tile_rows) const {
    if (spread <= splits || rows <= 0) return splits;
    const int places = places_of(rows, tile_rows);
    int most = places < spread ? places : spread;
    if (most > splits && rows * most > spare) most = spare / rows;
    return most > splits ? most : splits;
  }
  // Workgroups of a head for each tile of such a sequence.
  __device__ __forceinline__ int places_of(int rows, int tile_rows) const {
    return q_tiles * splits / ((rows - 1) / tile_rows + 1);
  }
};

// Where the parts of a sequence that may have so many are: row r of the sequence's (token, head) and part `split`.
struct Sums {
  long long first, step, first_ml;
  int per;
  __device__ __forceinline__ Sums(const AttnArgs& a, const Cut& cut, const Seq& s, int seq, int may) : per(may) {
    if (may > cut.splits) {
      const long long all = cut.splits > 1 ? cut.splits * a.n * a.q_heads : 0;
      first = first_ml = all + static_cast<long long>(seq) * cut.spare * a.kv_heads;
      step = static_cast<long long>(s.tokens) * a.q_heads;
    } else {
      first = static_cast<long long>(s.first) * a.q_heads;
      first_ml = first * cut.splits;
      step = a.n * a.q_heads;
    }
  }
  __device__ __forceinline__ long long row(int r, int split) const { return first + split * step + r; }
  __device__ __forceinline__ long long ml(int r) const { return first_ml + static_cast<long long>(r) * per; }
};

constexpr int kLeastPart = 512;  // entries of a part that a sequence of few rows is spread to

// Entries that the rows [row0, row_end) of a sequence see between them, and their parts.
struct Reach {
  int tok0, tok1;
  int lo, hi;          // some row sees these
  int all_lo, all_hi;  // every row sees these
  int first, part, parts;
  __device__ __forceinline__ Reach(const Seq& s, int row0, int row_end, int group, int causal, int window,
                                   const Cut& cut, int may) {  // may: most parts
    tok0 = row0 / group;
    tok1 = (row_end - 1) / group;
    const Span s0 = seen_by(s, tok0, causal, window), s1 = seen_by(s, tok1, causal, window);
    lo = s0.lo;
    hi = s1.hi;
    all_lo = s1.lo;
    all_hi = s0.hi;
    first = lo & ~31;
    const int span = hi > first ? hi - first : 0;
    part = may > cut.splits && cut.part > kLeastPart ? kLeastPart : cut.part;
    // spans stay below 2^31 - 2^17, so the sums below fit 32 bits
    if (span > static_cast<long long>(part) * may)
      part = ((static_cast<uint32_t>(span) + may - 1) / static_cast<uint32_t>(may) + 63) & ~63u;
    parts = span > part ? (static_cast<uint32_t>(span) + part - 1) / static_cast<uint32_t>(part) : 1;
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

// The sequence that comes `at`-th if those with the most entries to a workgroup come first, where a wave can look at
// all of them (up to 64); else the at-th. Equal ones keep their order. tile_rows: rows of a tile. Counted are the
// workgroups that a sequence has, up to 16 to a tile, also where its parts are fewer (candidates: 23.5 us, by parts
// 25.8).
__device__ __forceinline__ int longest_first(const AttnArgs& a, const Cut& cut, int at, int tile_rows) {
  const Paged& p = a.paged;
  if (p.seqs > kWave) return at;
  const int lane = threadIdx.x & (kWave - 1), i = lane < p.seqs ? lane : 0, group = a.q_heads / a.kv_heads;
  const int held = p.kv_lens[i], tokens = p.q_offsets[i + 1] - p.q_offsets[i];  // bad ones count as they may
  const int seen = a.window > 0 && held > a.window ? a.window : held;
  const bool some = lane < p.seqs && tokens > 0 && tokens <= a.n;
  const int places = some ? cut.places_of(tokens * group, tile_rows) : 1, parts = places < 16 ? places : 16;
  const int work = some && seen > 0 ? seen / (parts > cut.splits ? parts : cut.splits) + 1 : lane < p.seqs ? 0 : -1;
  int before = 0;
  for (int j = 0; j < p.seqs; ++j) {
    const int other = __builtin_amdgcn_readlane(work, j);
    before += other > work || (other == work && j < lane);
  }
  return __builtin_ctzll(__ballot(lane < p.seqs && before == at));
}

template <int D>
constexpr int kPitch = D + 4;  // floats; a row of O in LDS

// The end of a workgroup of the rows kernels: joins its four waves' maxima, sums and O of 16 rows, lane (g, c16) with
// elements 4 E g .. 4 E (g + 1) of row c16, E = D / 16 at a time, and writes the rows' results or their part.
template <int DT, int D>
__device__ __forceinline__ void join_waves(const AttnArgs& a, const Cut& cut, const Reach& rc, const Seq& sq, int row0,
                                           int row_end, int group, int head, int split, float m, float l,
                                           const f32x4 (&o)[D / 16], float (*lds_o)[16 * kPitch<D>],
                                           float2 (*lds_ml)[16]) {
  constexpr int E = D / 16, Rows = 16, Pitch = kPitch<D>;
  const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const float c = a.scale * kLog2e;
  l = add_halves(add_quarters(l));
  if (g == 0) lds_ml[wave][c16] = make_float2(m, l);
  __syncthreads();
  float top = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, lds_ml[w][c16].x);
  const float keep = m == -INFINITY ? 0.f : exp2f((m - top) * c);
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int e = 0; e < E; ++e) lds_o[wave][c16 * Pitch + (4 * g + r) * E + e] = o[e][r] * keep;
  __syncthreads();
  constexpr int Pieces = D / 8;
  for (int i = threadIdx.x; i < Rows * Pieces; i += kThreads) {
    const int r16 = i / Pieces, at = i % Pieces * 8;
    const int out_row = row0 + r16;
    if (out_row >= row_end) continue;
    float mt = -INFINITY, lt = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mt = fmaxf(mt, lds_ml[w][r16].x);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float2 ml = lds_ml[w][r16];
      lt += ml.y * (ml.x == -INFINITY ? 0.f : exp2f((ml.x - mt) * c));
    }
    float x[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      x[d] = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) x[d] += lds_o[w][r16 * Pitch + at + d];
    }
    const int tok = out_row / group, gi = out_row - tok * group;
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
}

// ---------------------------------------------------------------------------
// Joins the parts of split histories: D / 8 lanes to a row, eight elements each. Slots > 1: the parts of
// a row are shared between that many groups of lanes (a workgroup to a row), which is quicker where
// there are many parts and so few rows. Spread: sequences of few rows may have more parts than the others; without it the
// kernel does not ask (candidates over the 8-bit cache: 23.2 us, 23.4 if it did).
// ---------------------------------------------------------------------------
constexpr int kMaxSplits = 512;

template <int DT, int D, int Slots, bool Spread>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnArgs a, Cut cut, int tile_rows) {
  constexpr int Lanes = D / 8, Rows = kThreads / (Lanes * Slots);
  __shared__ float lds_x[Slots > 1 ? Slots : 1][D];
  __shared__ float2 lds_ml[Slots];
  const int group = a.q_heads / a.kv_heads;
  const float c = a.scale * kLog2e;
  const int at = threadIdx.x % Lanes * 8, slot = threadIdx.x / Lanes % Slots;
  for (int seq = blockIdx.y; seq < a.paged.seqs; seq += gridDim.y) {
    const Seq sq = load_seq(a.paged, a.n, seq);
    const int rows = sq.tokens * a.q_heads, may = Spread ? cut.parts_of(sq.tokens * group, tile_rows) : cut.splits;
    if (may == 1) continue;
    const Sums sums(a, cut, sq, seq, may);
    for (long long first = static_cast<long long>(blockIdx.x) * Rows; first < rows;
         first += static_cast<long long>(gridDim.x) * Rows) {
      const int row = static_cast<int>(first) + threadIdx.x / (Lanes * Slots);
      if (row >= rows) continue;  // with Slots > 1 there is one row, and no thread leaves it
      const int tok = row / a.q_heads, in_head = tok * group + (row - tok * a.q_heads) % group;
      const int row0 = in_head / tile_rows * tile_rows, in_all = sq.tokens * group;
      const Reach rc(sq, row0, in_all - row0 > tile_rows ? row0 + tile_rows : in_all, group, a.causal, a.window, cut,
                     may);
      if (rc.parts == 1) continue;
      const long long to = static_cast<long long>(sq.first) * a.q_heads + row;
      const float2* ml = cut.ml + sums.ml(row);
      const float* o = cut.o + sums.row(row, 0) * D + at;
      const long long step = sums.step * D;
      float m = -INFINITY, l = 0.f, x[8] = {};
#pragma unroll 4
      for (int i = slot; i < rc.parts; i += Slots) m = fmaxf(m, ml[i].x);
#pragma unroll 4
      for (int i = slot; i < rc.parts; i += Slots) {
        const float4 u = *reinterpret_cast<const float4*>(o + i * step);
        const float4 v = *reinterpret_cast<const float4*>(o + i * step + 4);
        const float2 p = ml[i];
        const float w = p.x == -INFINITY ? 0.f : exp2f((p.x - m) * c);
        l = fmaf(p.y, w, l);
        x[0] = fmaf(u.x, w, x[0]); x[1] = fmaf(u.y, w, x[1]); x[2] = fmaf(u.z, w, x[2]); x[3] = fmaf(u.w, w, x[3]);
        x[4] = fmaf(v.x, w, x[4]); x[5] = fmaf(v.y, w, x[5]); x[6] = fmaf(v.z, w, x[6]); x[7] = fmaf(v.w, w, x[7]);
      }
      if constexpr (Slots == 1) {
        finish<DT>(a, to, at, x, m, l);
      } else {
        __syncthreads();  // the row before was read
#pragma unroll
        for (int d = 0; d < 8; ++d) lds_x[slot][at + d] = x[d];
        if (at == 0) lds_ml[slot] = make_float2(m, l);
        __syncthreads();
        if (slot == 0) {
          for (int i = 1; i < Slots; ++i) m = fmaxf(m, lds_ml[i].x);
          l = 0.f;
#pragma unroll
          for (int d = 0; d < 8; ++d) x[d] = 0.f;
          for (int i = 0; i < Slots; ++i) {
            const float2 p = lds_ml[i];
            const float w = p.x == -INFINITY ? 0.f : exp2f((p.x - m) * c);
            l = fmaf(p.y, w, l);
#pragma unroll
            for (int d = 0; d < 8; ++d) x[d] = fmaf(lds_x[i][at + d], w, x[d]);
          }
          finish<DT>(a, to, at, x, m, l);
        }
      }
    }
  }
}

template <int DT, int D, int Slots, bool Spread>
void join(const AttnArgs& a, const Cut& cut, int tile_rows, hipStream_t s) {
  constexpr int Rows = kThreads / (D / 8 * Slots);
  const long long rows = static_cast<long long>(a.max_q) * a.q_heads, groups = (rows + Rows - 1) / Rows;
  // where only sequences of few rows are in parts, the workgroups of all others would come for nothing (16384 of
  // them: 25 us, 1024: 6)
  const long long most = cut.splits > 1 ? 65535 : 256;
  const unsigned x = static_cast<unsigned>(groups < 1 ? 1 : groups < most ? groups : most);
  const unsigned y = static_cast<unsigned>(a.paged.seqs < 65535 / 8 ? a.paged.seqs : 65535 / 8);
  hipLaunchKernelGGL((attn_join_kernel<DT, D, Slots, Spread>), dim3(x, y), dim3(kThreads), 0, s, a, cut, tile_rows);
}

// Rows of a tile: 16 for the rows kernel (one wave's matrix instruction), 128 for the tile kernel.
int tile_rows(long long max_rows) { return max_rows <= 16 ? 16 : 32 * kWaves; }

constexpr size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// Rows of sums of a call.
long long sum_rows(const Cut& c, int64_t n, int seqs, int q_heads, int kv_heads) {
  return (c.splits > 1 ? c.splits * n * q_heads : 0) +
         (c.spread > c.splits ? static_cast<long long>(seqs) * c.spare * kv_heads : 0);
}

size_t cut_bytes(const Cut& c, int64_t n, int seqs, int q_heads, int kv_heads, int dim) {
  const size_t rows = static_cast<size_t>(sum_rows(c, n, seqs, q_heads, kv_heads));
  return rows == 0 ? 0 : round256(rows * dim * sizeof(float)) + rows * sizeof(float2);
}

// The kernel of a call that is cut into tiles of `tile` rows and into parts, and their join. Spread: the kernel knows
// of sequences with more parts than the others.
template <int DT, int D, bool Spread>
hipError_t launch_cut(const AttnArgs& a, Cut cut, int tile, void (*kernel)(AttnArgs, Cut), int threads, hipStream_t s) {
  const long long rows = static_cast<long long>(a.max_q) * (a.q_heads / a.kv_heads);
  cut.o = static_cast<float*>(a.workspace);
  const size_t sums = static_cast<size_t>(sum_rows(cut, a.n, a.paged.seqs, a.q_heads, a.kv_heads));
  cut.ml = reinterpret_cast<float2*>(static_cast<char*>(a.workspace) + round256(sums * D * sizeof(float)));
  const unsigned seqs = a.paged.seqs < 65535 ? a.paged.seqs : 65535;
  hipLaunchKernelGGL(kernel, dim3(a.kv_heads, cut.q_tiles * cut.splits, seqs), dim3(threads), 0, s, a, cut);
  const long long all_rows = rows * a.kv_heads * a.paged.seqs;
  if (cut.splits > 16 && all_rows <= 512)
    join<DT, D, kThreads / (D / 8), false>(a, cut, tile, s);
  else if (Spread && cut.spread > cut.splits)
    join<DT, D, 1, Spread>(a, cut, tile, s);
  else if (cut.splits > 1)
    join<DT, D, 1, false>(a, cut, tile, s);
  return hipGetLastError();
}

}  // namespace
}  // namespace dlrm
