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
template <int DT, int D, int RT>
__global__ __launch_bounds__(kThreads) void attn_rows_kernel(AttnArgs a, int q_tiles, long long units) {
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

  for (long long unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int head = static_cast<int>(unit % a.kv_heads);
    const long long rest = unit / a.kv_heads;
    const int seq = static_cast<int>(rest / q_tiles);
    const Seq sq = load_seq(pg, a.n, seq);
    const long long rows = static_cast<long long>(sq.tokens) * group;
    const uint16_t* kh = static_cast<const uint16_t*>(a.k_cache) + head * pg.head_stride;
    const uint16_t* vh = static_cast<const uint16_t*>(a.v_cache) + head * pg.head_stride;
    const int32_t* table = pg.page_table + seq * pg.table_stride;

    for (long long row0 = rest % q_tiles * Rows; row0 < rows; row0 += static_cast<long long>(q_tiles) * Rows) {
      const long long row_end = row0 + Rows < rows ? row0 + Rows : rows;
      const int tok0 = static_cast<int>(row0 / group), tok1 = static_cast<int>((row_end - 1) / group);
      // entries that some row of the tile sees, and that all of them see
      const Span s0 = seen_by(sq, tok0, a.causal, a.window), s1 = seen_by(sq, tok1, a.causal, a.window);
      const int lo = s0.lo, hi = s1.hi, all_lo = s1.lo, all_hi = s0.hi;

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

      for (int k0 = (lo & ~31) + 32 * wave; k0 < hi; k0 += 32 * kWaves) {
        u32x4 kf[2][F];
        uint32_t v[8][E / 2];
        bool have[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int key = k0 + 16 * t;
          have[t] = false;
          if (key < hi) {
            const int page = table[key >> pg.page_shift];
            have[t] = page >= 0 && page < pg.num_pages;
            if (!have[t] && lane == 0) flag(pg.status, DLRM_STATUS_BAD_PAGE);
            if (have[t]) {
              const long long at = page * pg.page_stride + (key & page_mask) * D;
              const uint16_t* kp = kh + at + c16 * D + g * 8;
              const uint16_t* vp = vh + at + 4 * g * D + c16 * E;
#pragma unroll
              for (int f = 0; f < F; ++f) kf[t][f] = *reinterpret_cast<const u32x4*>(kp + f * 32);
#pragma unroll
              for (int j = 0; j < 4; ++j) __builtin_memcpy(v[4 * t + j], __builtin_assume_aligned(vp + j * D, E >= 8 ? 16 : 2 * E), 2 * E);
            }
          }
          if (!have[t]) {
#pragma unroll
            for (int f = 0; f < F; ++f) kf[t][f] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < E / 2; ++i) v[4 * t + j][i] = 0;
          }
        }

        // values that no row sees are zero, whatever they hold
        if (k0 < lo || k0 + 32 > hi) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int key = k0 + 16 * (j / 4) + 4 * g + j % 4;
            if (key < lo || key >= hi) {
#pragma unroll
              for (int i = 0; i < E / 2; ++i) v[j][i] = 0;
            }
          }
        }

        u32x4 pw[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          f32x4 s[2];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            s[t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int f = 0; f < F; ++f) s[t] = mfma16<DT>(kf[t][f], qf[rt][f], s[t]);
          }
          float top = -INFINITY;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int key = k0 + 16 * t + 4 * g + r;
              if (!have[t] || key < row_lo[rt] || key >= row_hi[rt]) s[t][r] = -INFINITY;
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

        // entries that only some rows see: if one holds an infinity or NaN, the second product runs
        // token by token, with what the token does not see set to zero, and only the token's own rows
        // take the sum
        bool apart = false;
        if (tok1 > tok0 && (k0 < all_lo || k0 + 32 > all_hi)) {
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
          const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
          for (int d = 0; d < 8; ++d) x[d] *= inv;
          const int tok = static_cast<int>(row / group), gi = static_cast<int>(row - static_cast<long long>(tok) * group);
          const long long to = static_cast<long long>(sq.first + tok) * a.q_heads + head * group + gi;
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + to * D + at) = narrow<DT>(x);
          if (at == 0 && a.lse) a.lse[to] = lt == 0.f ? -INFINITY : fmaf(mt, a.scale, logf(lt) - kLift<DT> * kLn2);
        }
        __syncthreads();
      }
    }
  }
}

template <int DT, int D, int RT>
hipError_t run_rows(const AttnArgs& a, hipStream_t s) {
  const long long rows = static_cast<long long>(a.max_q) * (a.q_heads / a.kv_heads);
  const long long tiles = rows > 16 * RT ? (rows + 16 * RT - 1) / (16 * RT) : 1;
  const long long units = tiles * a.paged.seqs * a.kv_heads;
  const long long most = 1 << 22;
  hipLaunchKernelGGL((attn_rows_kernel<DT, D, RT>), dim3(static_cast<unsigned>(units < most ? units : most)),
                     dim3(kThreads), 0, s, a, static_cast<int>(tiles), units);
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

size_t attn_workspace(int64_t, int, int, int, int, int, int, int, int) { return 0; }

hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t s) {
  if (a.n == 0 || a.paged.seqs == 0) return hipSuccess;
  return a.dtype == DLRM_F16 ? run_dim<DLRM_F16>(a, s) : run_dim<DLRM_BF16>(a, s);
}

}  // namespace dlrm
