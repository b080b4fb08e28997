// Attention of new tokens over a paged cache of 16-bit values (formulas in attn_device.h).
//
// Scores are formed transposed, S^T = K Q^T, by 16x16x32 matrix instructions. Their result holds
// four entries of one row in each lane, which is what the second product O^T = V^T P^T takes as
// its right operand when the order of the 32 entries in the sum is chosen to fit (lane group g
// takes entries 4g .. 4g+3 of both halves): the weights never leave the lane, and m, l and the
// rescale of O are one value per lane.
#include "attn_tile.h"

namespace dlrm {
namespace {

// ---------------------------------------------------------------------------
// Rows kernel: 16 rows of one head to a workgroup, the four waves take the tiles of 32 entries of the
// history in turn and join their (m, l, O) through LDS at the end. Bound by memory: keys and values go from
// global memory to registers, each is used once. A lane takes D / 16 neighbouring elements of four values'
// rows of each 16, so that a load instruction covers whole rows, and the transposition that the second
// product needs is 16-bit permutations in registers.
// A wave has a tile of loads on the way all the time: the next tile's keys are asked for as soon as this
// one's are used, its values likewise, without a second set of registers. Tiles of 32 entries: 64 of heads of
// 64 and 32 leave fewer waves (63 us against 61 for 64 histories of up to 16k), 16 of heads of 256 keep two
// waves to a SIMD but half the loads on the way (151 us against 134 for 64 of up to 8k).
// ---------------------------------------------------------------------------
template <int DT, int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void attn_rows_kernel(AttnArgs a, Cut cut) {
  constexpr int TT = 2;          // blocks of 16 entries to a tile
  constexpr int K = 16 * TT;
  constexpr int F = D / 32;      // k steps of the first product
  constexpr int E = D / 16;      // elements of a value row that a lane takes, and 16-wide pieces of O
  constexpr int Rows = 16;
  constexpr int Ahead = 64 / TT; // tiles whose pages a wave holds
  __shared__ float lds_o[kWaves][Rows * kPitch<D>];
  __shared__ float2 lds_ml[kWaves][Rows];
  const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int group = a.q_heads / a.kv_heads;
  const float c = a.scale * kLog2e;
  const Paged& pg = a.paged;
  const int page_mask = (1 << pg.page_shift) - 1;
  const int head = blockIdx.x, split = blockIdx.y % cut.splits;
  const uint16_t* kh = static_cast<const uint16_t*>(a.k_cache) + head * pg.head_stride + (c16 * D + g * 8);
  const uint16_t* vh = static_cast<const uint16_t*>(a.v_cache) + head * pg.head_stride + (4 * g * D + c16 * E);

  for (int seq = blockIdx.z; seq < pg.seqs; seq += gridDim.z) {
    const Seq sq = load_seq(pg, a.n, seq);
    const int rows = sq.tokens * group;
    const int32_t* table = pg.page_table + seq * pg.table_stride;

    for (long long first_row = static_cast<long long>(blockIdx.y / cut.splits) * Rows; first_row < rows;
         first_row += static_cast<long long>(cut.q_tiles) * Rows) {
      const int row0 = static_cast<int>(first_row), row_end = rows - row0 > Rows ? row0 + Rows : rows;
      const Reach rc(sq, row0, row_end, group, a.causal, a.window, cut);
      if (split >= rc.parts) continue;
      const int k_first = rc.first + split * rc.part;
      const int hi = rc.hi - k_first < rc.part ? rc.hi : k_first + rc.part;
      const int k_begin = k_first + K * wave;

      // Pages of the blocks of this wave's next Ahead tiles, one to a lane; past the end: of the last entry.
      const auto key_of = [&](int k0, int block) { return k0 + block / TT * (K * kWaves) + block % TT * 16; };
      const auto look_up = [&](int k0) {
        const int key = key_of(k0, lane);
        return table[(key < hi ? key : hi - 1) >> pg.page_shift];
      };
      const auto good_pages = [&](int k0, int page) {  // bit i: the page of block i is good
        const bool good = static_cast<uint32_t>(page) < static_cast<uint32_t>(pg.num_pages);
        const int key = key_of(k0, lane);
        if (!good && key < hi && key + 16 > rc.lo) flag(pg.status, DLRM_STATUS_BAD_PAGE);
        return __ballot(good);
      };
      int pages = 0;
      if (k_begin < hi) pages = look_up(k_begin);

      u32x4 qf[F];
#pragma unroll
      for (int f = 0; f < F; ++f) qf[f] = u32x4{0, 0, 0, 0};
      const int row = row0 + c16;
      int row_lo = 0, row_hi = 0, row_tok = -1;
      if (row < row_end) {
        row_tok = row / group;
        const int gi = row - row_tok * group;
        const Span s = seen_by(sq, row_tok, a.causal, a.window);
        row_lo = s.lo;
        row_hi = s.hi;
        const uint16_t* q = static_cast<const uint16_t*>(a.q.ptr) + (sq.first + row_tok) * a.q.stride +
                            (head * group + gi) * a.q.head_stride + g * 8;
#pragma unroll
        for (int f = 0; f < F; ++f) qf[f] = *reinterpret_cast<const u32x4*>(q + f * 32);
      }

      float m = -INFINITY, l = 0.f;
      f32x4 o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = f32x4{0, 0, 0, 0};

      // Where the blocks of a tile are, in elements, and whether their pages are good. Past the end and in
      // place of a bad page another page of the cache is read and masked.
      struct Tile {
        long long at[TT];
        int good;
      };
      uint64_t good64 = 0;
      const auto find = [&](int k0, int index) {
        Tile t;
        t.good = static_cast<int>(good64 >> (index * TT)) & ((1 << TT) - 1);
#pragma unroll
        for (int i = 0; i < TT; ++i) {
          const int key = k0 + 16 * i < hi ? k0 + 16 * i : hi - 1;
          const int page = t.good >> i & 1 ? __builtin_amdgcn_readlane(pages, index * TT + i) : 0;
          t.at[i] = page * pg.page_stride + (key & page_mask & ~15) * D;
        }
        return t;
      };
      u32x4 kf[TT][F];
      uint32_t v[4 * TT][E / 2];
      const auto load_keys = [&](const Tile& t) {
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
          for (int f = 0; f < F; ++f) kf[i][f] = *reinterpret_cast<const u32x4*>(kh + t.at[i] + f * 32);
      };
      const auto load_values = [&](const Tile& t) {
#pragma unroll
        for (int j = 0; j < 4 * TT; ++j)
          __builtin_memcpy(v[j], __builtin_assume_aligned(vh + t.at[j / 4] + j % 4 * D, E >= 8 ? 16 : 2 * E), 2 * E);
      };

      // One tile at k0; with More, the loads of the next one at its places.
      const auto work = [&](int k0, const Tile& tile, const Tile& next, auto more) {
        constexpr bool More = decltype(more)::value;
        f32x4 s[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          s[t] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int f = 0; f < F; ++f) s[t] = mfma16<DT>(kf[t][f], qf[f], s[t]);
        }
        if constexpr (More) load_keys(next);
        const bool edge = k0 < rc.all_lo || k0 + K > rc.all_hi || k0 + K > hi || tile.good != (1 << TT) - 1;
        if (edge) {
#pragma unroll
          for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int key = k0 + 16 * t + 4 * g + r;
              if (!(tile.good >> t & 1) || key < row_lo || key >= row_hi || key >= hi) s[t][r] = -INFINITY;
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) top = fmaxf(top, s[t][r]);
        const float now = fmaxf(m, max_halves(max_quarters(top)));
        // O and l stay relative to an older maximum until a row's grows by 2^8 (fp16, with its lift: 2^7)
        if (__any((now - m) * c > (DT == DLRM_F16 ? 7.f : 8.f))) {
          const float keep = m == -INFINITY ? 0.f : exp2f((m - now) * c);
          m = now;
          l *= keep;
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] *= keep;
        }
        const float base = m == -INFINITY ? 0.f : m * c - kLift<DT>;
        uint32_t pw[TT][2];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          float p[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) p[r] = __builtin_amdgcn_exp2f(fmaf(s[t][r], c, -base));
          l += (p[0] + p[1]) + (p[2] + p[3]);
          pw[t][0] = pack2<DT>(p[0], p[1]);
          pw[t][1] = pack2<DT>(p[2], p[3]);
        }

        // Entries that no row sees are zero, whatever they hold. If one that only some rows see holds an
        // infinity or NaN, the second product runs token by token, with what the token does not see set to
        // zero, and only the token's own rows take the sum.
        bool apart = false;
        if (edge) {
#pragma unroll
          for (int j = 0; j < 4 * TT; ++j) {
            const int key = k0 + 16 * (j / 4) + 4 * g + j % 4;
            const bool none = key < rc.lo || key >= hi || !(tile.good >> (j / 4) & 1);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
              if (none) v[j][i] = 0;
              apart |= not_finite_halves<DT>(v[j][i]) != 0;
            }
          }
          apart = rc.tok1 > rc.tok0 && __any(apart);
        }
        const auto product = [&](auto seen, bool mine) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const uint32_t pick = e % 2 ? 0x07060302u : 0x05040100u;
            f32x4 sum = o[e];
#pragma unroll
            for (int t = 0; t < TT; t += 2) {
              u32x4 vt;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int j = 4 * t + 2 * i;
                vt[i] = __builtin_amdgcn_perm(v[j + 1][e / 2] & seen(j + 1), v[j][e / 2] & seen(j), pick);
              }
              sum = mfma16<DT>(vt, u32x4{pw[t][0], pw[t][1], pw[t + 1][0], pw[t + 1][1]}, sum);
            }
            if (mine) o[e] = sum;
          }
        };
        if (!apart) {
          product([](int) { return 0xffffffffu; }, true);
        } else {
#pragma unroll 1
          for (int tok = rc.tok0; tok <= rc.tok1; ++tok) {
            const Span sp = seen_by(sq, tok, a.causal, a.window);
            product([&](int j) {
              const int key = k0 + 16 * (j / 4) + 4 * g + j % 4;
              return key >= sp.lo && key < sp.hi ? 0xffffffffu : 0u;
            }, row_tok == tok);
          }
        }
        if constexpr (More) load_values(next);
      };

      if (k_begin < hi) {
        good64 = good_pages(k_begin, pages);
        int index = 0;
        Tile tile = find(k_begin, 0);
        load_keys(tile);
        load_values(tile);
        int k0 = k_begin;
        for (; k0 + K * kWaves < hi; k0 += K * kWaves) {
          const int k_next = k0 + K * kWaves;
          if (++index == Ahead) {
            index = 0;
            pages = look_up(k_next);
            good64 = good_pages(k_next, pages);
          }
          const Tile next = find(k_next, index);
          work(k0, tile, next, std::true_type{});
          tile = next;
        }
        work(k0, tile, tile, std::false_type{});
      }

      join_waves<DT, D>(a, cut, rc, sq, row0, row_end, group, head, split, m, l, o, lds_o, lds_ml);
      __syncthreads();
    }
  }
}

// Where the workgroups of a call would not fill the chip, or histories may be of unequal length, every
// history is split into parts.
// Rows kernel: parts of 256 KB of keys and as much of values (64 histories of up to 16k entries of 128: 220 us in 17
// parts, 222 in 9, 231 in 33), smaller ones of 512 entries where that leaves fewer than 256 workgroups, and 16k
// workgroups. One history of 131k and two heads: 30 us in 129 parts, 29 in 65, 32 in 257, 36 in 511.
// Tile kernel: twice as many workgroups as there are places, in parts of 512 entries, and of heads below 256 up to
// four times as many in parts of 1024 (13 sequences of up to 83 tokens over up to 24k: 57 us in 19 parts, 69 in 11,
// 63 in 31), of which more than 20 cost more than they give (3 sequences of up to 352 tokens over up to 37k: 76 us
// in 19 parts, 81 in 21, 92 in 37). 24 sequences of up to 257 x 1500: 21 us in 3 parts, 27 in one; 8 sequences of
// 32 tokens over up to 32k: 49 us in 33 parts, 61 in 15, as many as places; but 208 working workgroups of 256-wide
// heads, one to a CU: 80 us unsplit, 120 in two parts and 94 in three, since the parts wait for a place and their
// sums are written and read.
// The number of parts, and of tiles of a sequence, is made odd last: workgroups go to the XCDs in turn, and with 16
// parts of 4 heads the first parts of all sequences, the ones that short histories fill, would meet on the same four
// of eight (64 histories of up to 8k, 256-wide heads: 180 us, with 17 parts 134 us). There may so be one part more
// than the limits above say, and parts may be shorter: 513 entries make three of 192.
//
// The parts' sums take n x q_heads rows each. Where these rows are more than the hints and the sequences have tiles
// for (max_q too small, or tokens past the last sequence), the number of parts is bounded so that the sums take at
// most four times what they can with right hints: 1.6 GB for heads of 256, half of it for half of the width.
Cut cut_call(long long all_rows, long long max_rows, int seqs, int kv_heads, int dim, int causal, int window, int max_q,
             int max_kv) {
  Cut c;
  const int rows = tile_rows(max_rows);
  long long tiles = max_rows > rows ? (max_rows + rows - 1) / rows : 1;
  if (tiles > 65535) tiles = 65535;  // a workgroup takes further tiles in turn
  c.q_tiles = static_cast<int>(tiles);
  const long long whole = tiles * seqs * kv_heads;
  long long span = max_kv > 0 ? max_kv : 1;
  if (span > 0x7fffffffLL - (1 << 17)) span = 0x7fffffffLL - (1 << 17);  // no history is longer
  const long long seen = static_cast<long long>(window) + max_q + 32;
  if (causal && window && span > seen) span = seen;
  long long splits;
  const long long units = whole > 0 ? whole : 1;
  const long long held = (all_rows + rows - 1) / rows, busy = held > units ? held : units;  // tiles of all rows
  if (rows == 16) {
    const long long least = 131072 / dim, fill = 256 / units, finest = (span + 511) / 512, most = 16384 / units;
    splits = (span + least - 1) / least;
    if (splits < fill) splits = fill < finest ? fill : finest;
    if (splits > most) splits = most;
    if (splits > 4 * 16384 / busy) splits = 4 * 16384 / busy;
  } else {
    const long long places = dim == 256 ? 256 : dim == 128 ? 512 : 768, finest = (span + 511) / 512;
    splits = 2 * places / units;
    if (splits > finest) splits = finest;
    const long long coarse = 4 * places / units < span / 1024 ? 4 * places / units : span / 1024;
    if (dim < 256 && splits < coarse) splits = coarse < 20 ? coarse : splits < 20 ? 20 : splits;
    if (splits > 4 * 4 * places / busy) splits = 4 * 4 * places / busy;
  }
  if (splits < 1) splits = 1;
  if (splits > 1) splits |= 1;
  if (tiles > 1) c.q_tiles = static_cast<int>(tiles |= 1);
  if (splits > kMaxSplits) splits = kMaxSplits - 1;
  if (splits > 65535 / tiles) splits = 65535 / tiles;
  c.splits = static_cast<int>(splits);
  c.part = static_cast<int>(((span + splits - 1) / splits + 63) & ~63LL);
  c.o = nullptr;
  c.ml = nullptr;
  return c;
}

template <int DT, int D>
hipError_t run(const AttnArgs& a, hipStream_t s) {
  const long long rows = static_cast<long long>(a.max_q) * (a.q_heads / a.kv_heads);
  const Cut cut = cut_call(a.n * a.q_heads, rows, a.paged.seqs, a.kv_heads, D, a.causal, a.window, a.max_q, a.max_kv);
  return launch_cut<DT, D>(a, cut, attn_rows_kernel<DT, D>, attn_tile_kernel<DT, D, false>, kTileThreads<D>, s);
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
  const long long rows = static_cast<long long>(max_q) * (q_heads / kv_heads);
  return cut_bytes(cut_call(n * q_heads, rows, seqs, kv_heads, dim, causal, window, max_q, max_kv), n, q_heads, dim);
}

hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t s) {
  if (a.n == 0 || a.paged.seqs == 0) return hipSuccess;
  return a.dtype == DLRM_F16 ? run_dim<DLRM_F16>(a, s) : run_dim<DLRM_BF16>(a, s);
}

}  // namespace dlrm
