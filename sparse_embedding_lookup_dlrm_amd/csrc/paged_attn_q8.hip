// Attention of new tokens over a paged cache of 8-bit codes (formulas in attn_device.h): e4m3 codes with a power of
// two for each block of 16 entries of a head, one for the keys and one for the values.
//
// Codes are widened to the 16-bit type of the queries, which is exact, by an instruction that takes two of them and
// their scale, so that the matrix products, the softmax and the joins are those of the 16-bit cache.
#include "attn_device.h"

namespace dlrm {
namespace {

// ---------------------------------------------------------------------------
// Rows kernel: 16 rows of one head to a workgroup, as for the 16-bit cache: the four waves take the tiles of the
// history in turn, a wave's next tile is on the way from global memory to registers while one is worked on, and the
// waves join their (m, l, O) through LDS at the end. Scores are formed transposed, S^T = K Q^T, so that the weights
// are the second product's right operand where they lie: lane (g, c16) holds entries 4 g .. 4 g + 3 of each block of
// 16. The order of the elements in a score's sum is free: a lane takes 16 neighbouring codes of a key, which serve
// two steps of the product, and the queries are read to fit. Of the values it takes D / 16 neighbouring codes of its
// entries; a byte permutation of two entries' words gives the pairs of two elements, one widening each.
//
// Bound by memory: 64 histories of up to 16k entries, 32 / 8 heads of 128, 625 MB: 121 us, 5.2 TB/s (16-bit cache
// 214). A third wave on each SIMD changes nothing (152 registers are room for it), tiles of 64 entries spill (205 us
// of the whole call instead of 130); vector units are busy 30 % of the time, matrix units 8 %. A second form of the
// product, token by token for NaN that only some rows see, took 22 registers more (133 us).
// ---------------------------------------------------------------------------
template <int DT, int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void attn_rows_q8_kernel(AttnArgs a, Cut cut) {
  constexpr int TT = D >= 128 ? 2 : 4;  // blocks of 16 entries to a tile
  constexpr int K = 16 * TT;
  constexpr int F = D / 32;       // k steps of the first product
  constexpr int Chunk = D == 32 ? 8 : 16, Chunks = D / (4 * Chunk);  // codes of a key that a lane takes at once
  constexpr int E = D / 16;       // codes of a value that a lane takes, and 16-wide pieces of O
  constexpr int VW = (E + 3) / 4;  // their words
  constexpr int Rows = 16;
  constexpr int Ahead = 64 / TT;  // tiles whose pages a wave holds
  __shared__ float lds_o[kWaves][Rows * kPitch<D>];
  __shared__ float2 lds_ml[kWaves][Rows];
  const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int group = a.q_heads / a.kv_heads;
  const float c = a.scale * kLog2e;
  const Paged& pg = a.paged;
  const int page_mask = (1 << pg.page_shift) - 1;
  const int head = blockIdx.x, split = blockIdx.y % cut.splits;
  const uint8_t* kh = static_cast<const uint8_t*>(a.k_cache) + head * pg.head_stride + (c16 * D + g * Chunk);
  const uint8_t* value_head = static_cast<const uint8_t*>(a.v_cache) + head * pg.head_stride;
  const uint8_t* vh = value_head + (4 * g * D + c16 * E);
  const uint8_t* sh = a.kv_scales + head * a.scale_head_stride;

  for (int seq = blockIdx.z; seq < pg.seqs; seq += gridDim.z) {
    const Seq sq = load_seq(pg, a.n, seq);
    const int rows = sq.tokens * group;
    const int32_t* table = pg.page_table + seq * pg.table_stride;

    for (long long first_row = static_cast<long long>(blockIdx.y / cut.splits) * Rows; first_row < rows;
         first_row += static_cast<long long>(cut.q_tiles) * Rows) {
      const int row0 = static_cast<int>(first_row), row_end = rows - row0 > Rows ? row0 + Rows : rows;
      const Reach rc(sq, row0, row_end, group, a.causal, a.window, cut, cut.splits);
      if (split >= rc.parts) continue;
      const int k_first = rc.first + split * rc.part;
      const int hi = rc.hi - k_first < rc.part ? rc.hi : k_first + rc.part;
      const int k_begin = k_first + K * wave;

      // Pages of the blocks of this wave's next Ahead tiles, one to a lane, and their scales; past the end: of the
      // last entry.
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
      const auto look_up_scales = [&](int k0, int page, uint64_t good) {
        const int key = key_of(k0, lane), from = good >> lane & 1 ? page : 0;
        return static_cast<int>(*reinterpret_cast<const uint16_t*>(
            sh + from * a.scale_page_stride + ((key < hi ? key : hi - 1) & page_mask) / kScaleBlock * 2));
      };
      int pages = 0;
      if (k_begin < hi) pages = look_up(k_begin);

      u32x4 qf[F];
#pragma unroll
      for (int f = 0; f < F; ++f) qf[f] = u32x4{0, 0, 0, 0};
      const int row = row0 + c16;
      int row_lo = 0, row_hi = 0;
      if (row < row_end) {
        const int tok = row / group, gi = row - tok * group;
        const Span s = seen_by(sq, tok, a.causal, a.window);
        row_lo = s.lo;
        row_hi = s.hi;
        const uint16_t* q = static_cast<const uint16_t*>(a.q.ptr) + (sq.first + tok) * a.q.stride +
                            (head * group + gi) * a.q.head_stride + g * Chunk;
#pragma unroll
        for (int f = 0; f < F; ++f)
          qf[f] = *reinterpret_cast<const u32x4*>(q + f * 8 / Chunk * 4 * Chunk + f * 8 % Chunk);
      }

      float m = -INFINITY, l = 0.f;
      f32x4 o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = f32x4{0, 0, 0, 0};

      // Where the blocks of a tile are, and whether their pages are good. Past the end and in place of a bad page
      // another page of the cache is read and masked.
      struct Tile {
        long long at[TT];
        int good;
      };
      uint64_t good64 = 0;
      int scales = 0;
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
      uint32_t kf[TT][Chunks][Chunk / 4];
      uint32_t v[4 * TT][VW];
      const auto load_keys = [&](const Tile& t) {
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
          for (int f = 0; f < Chunks; ++f)
            __builtin_memcpy(kf[i][f], __builtin_assume_aligned(kh + t.at[i] + f * 4 * Chunk, Chunk), Chunk);
      };
      const auto load_values = [&](const Tile& t) {
#pragma unroll
        for (int j = 0; j < 4 * TT; ++j) {
          const uint8_t* from = vh + t.at[j / 4] + j % 4 * D;
          if constexpr (E == 2)
            v[j][0] = *reinterpret_cast<const uint16_t*>(from);
          else
            __builtin_memcpy(v[j], __builtin_assume_aligned(from, E), E);
        }
      };

      // One tile at k0 with the scales `two`; with More, the loads of the next one at its places.
      const auto work = [&](int k0, const Tile& tile, const int (&two)[TT], const Tile& next, auto more) {
        constexpr bool More = decltype(more)::value;
        f32x4 s[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          s[t] = f32x4{0, 0, 0, 0};
          const float scale = key_scale(two[t]);
#pragma unroll
          for (int f = 0; f < F; ++f) {
            const uint32_t* w = &kf[t][f * 8 / Chunk][f * 8 % Chunk / 4];
            s[t] = mfma16<DT>(u32x4{widen_codes<DT, false>(w[0], scale), widen_codes<DT, true>(w[0], scale),
                                    widen_codes<DT, false>(w[1], scale), widen_codes<DT, true>(w[1], scale)},
                              qf[f], s[t]);
          }
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
        // Weights go to the product in its type, half a step off: the matrix unit takes both operands in it. Relative to
        // 64 bits, results are 2.3e-3 off in bf16 and 2.4e-4 in fp16, their own rounding included; with fp32 weights
        // 1.7e-3 and 2.0e-4. The sum l is of the weights as they were.
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

        // Entries that no row sees are zero, whatever they and their scale hold. What only some rows see and is NaN
        // (or a value that fp16 does not hold) counts as zero in the product, and is added after it to the rows that
        // see it.
        float vs[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) vs[t] = value_scale(two[t]);
        bool special = false;
        if (edge) {
          const bool apart = rc.tok1 > rc.tok0;
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const int first = k0 + 16 * t;
            if (first + 16 <= rc.lo || first >= hi || !(tile.good >> t & 1)) vs[t] = 1.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int j = 4 * t + r, key = first + 4 * g + r;
              const bool none = key < rc.lo || key >= hi || !(tile.good >> t & 1);
#pragma unroll
              for (int i = 0; i < VW; ++i) {
                if (none) v[j][i] = 0;
                const uint32_t odd = __builtin_amdgcn_perm(not_finite_halves<DT>(widen_codes<DT, true>(v[j][i], vs[t])),
                                                           not_finite_halves<DT>(widen_codes<DT, false>(v[j][i], vs[t])),
                                                           0x06040200u);
                if (apart && odd) {
                  v[j][i] &= ~odd;
                  special = true;
                }
              }
            }
            if (apart && (two[t] >> 8 & 0xff) == 0xff) vs[t] = 1.f;  // zeros under a scale of NaN would be NaN
          }
          special = __any(special);
        }
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const uint32_t pick = e % 4 ? 0x07030602u : 0x05010400u;
#pragma unroll
          for (int t = 0; t < TT; t += 2) {
            u32x4 v0, v1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 4 * t + 2 * i;
              const uint32_t codes = __builtin_amdgcn_perm(v[j + 1][e / 4], v[j][e / 4], pick);
              v0[i] = widen_codes<DT, false>(codes, vs[j / 4]);
              v1[i] = widen_codes<DT, true>(codes, vs[j / 4]);
            }
            const u32x4 p = {pw[t][0], pw[t][1], pw[t + 1][0], pw[t + 1][1]};
            o[e] = mfma16<DT>(v0, p, o[e]);
            o[e + 1] = mfma16<DT>(v1, p, o[e + 1]);
          }
        }
        if (special) {
#pragma unroll 1
          for (int e0 = 0; e0 < K; ++e0) {
            const int key = k0 + e0;
            const int page = key < hi ? scalar_load(table, key >> pg.page_shift) : -1;
            if (page < 0 || page >= pg.num_pages) continue;
            const int in = key & page_mask;
            const uint8_t* from = value_head + page * pg.page_stride + static_cast<long long>(in) * D + 4 * g * E;
            const float scale = value_scale(sh[page * a.scale_page_stride + in / kScaleBlock * 2 + 1] << 8);
            const bool mine = key >= row_lo && key < row_hi;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int e = 0; e < E; ++e) {  // lane (g, c16) holds element (4 g + r) E + e of its row
                const uint32_t u = widen_codes<DT, false>(from[r * E + e], scale) & 0xffffu;
                const float x = DT == DLRM_BF16 ? bf16_lo(u) : f16_lo(u);
                o[e][r] += mine && not_finite_halves<DT>(u) ? x : 0.f;
              }
          }
        }
        if constexpr (More) load_values(next);
      };

      if (k_begin < hi) {
        good64 = good_pages(k_begin, pages);
        int index = 0;
        Tile tile = find(k_begin, 0);
        scales = look_up_scales(k_begin, pages, good64);
        load_keys(tile);
        load_values(tile);
        int two[TT];
        const auto pick_scales = [&] {
#pragma unroll
          for (int i = 0; i < TT; ++i) two[i] = __builtin_amdgcn_readlane(scales, index * TT + i);
        };
        int k0 = k_begin;
        for (; k0 + K * kWaves < hi; k0 += K * kWaves) {
          const int k_next = k0 + K * kWaves;
          pick_scales();
          if (++index == Ahead) {
            index = 0;
            pages = look_up(k_next);
            good64 = good_pages(k_next, pages);
            scales = look_up_scales(k_next, pages, good64);
          }
          const Tile next = find(k_next, index);
          work(k0, tile, two, next, std::true_type{});
          tile = next;
        }
        pick_scales();
        work(k0, tile, two, tile, std::false_type{});
      }

      join_waves<DT, D>(a, cut, rc, sq, row0, row_end, group, head, split, m, l, o, lds_o, lds_ml);
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// Tile kernel: 128 rows of one head to a workgroup, 32 to a wave, tiles of 64 entries in LDS that every wave reads
// all of. Products are 32x32x16: the score of row lane % 32 with entries 8 i + 4 h + j (h = lane / 32, i, j = 0 .. 3)
// lies in one lane, which again is the second product's right operand as it stands; its left operand V^T is read by
// the transposing LDS load: sixteen lanes take a block of 4 entries x 16 elements and get one element of the 4
// entries each.
//
// Codes are widened on their way to LDS, once for the workgroup and not by each of its waves: a wave brings 16
// entries of a tile, loaded while the tile before is worked on, in pieces of 8 codes that become 16 bytes.
//
// 4 sequences of up to 2048 tokens over up to 8192, 32 / 8 heads of 128: 338-352 us on five cards, 836-871 TFLOP/s, at
// 1.94 GHz, to which the clock falls under this load (16-bit cache, same inputs: 447, without parts for sequences of few
// rows and without their order). Matrix units are busy 41 % of the time that a CU has work, vector units 52 %; a CU has
// work 78 % of the kernel's clocks. 256 registers are 13 too few, which spill (48 bytes of scratch a lane). Left out:
// widening 13 us (of 411 then), the pieces to LDS 40, these and the loads 80. Tiles of 128 entries and 256 rows to a
// workgroup: 430-468 us, for jobs are fewer and longer; the jobs of all sequences in order of length: as long, and 5 us
// more for short calls. Heads of 256: a wave holds all of O, one to a SIMD, and works on 32 entries at once with 4
// pieces read ahead, 35 registers spilled: 102-106 us for 12 sequences of up to 513 tokens with a window of 1024; with 8
// pieces ahead, more of whose registers spill, 127-133, with two waves for the same rows, each with half of O, 120-157
// (16-bit cache, which has no codes to hold, 86).
// ---------------------------------------------------------------------------
template <int DT, int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void attn_tile_q8_kernel(AttnArgs a, Cut cut) {
  constexpr int K = 16 * kWaves;    // entries of a tile: a wave brings 16, which lie in one page
  constexpr int Q = D / 16;         // steps of the first product, and of the second, for 32 entries
  constexpr int C = D / 32;         // 32-wide pieces of O
  constexpr int P = D / 8;          // pieces of a row
  constexpr int T = D == 256 ? 1 : 2;  // blocks of 32 entries worked on at once
  constexpr int Loads = 16 * D / (kWave * 8);  // of a wave's keys, and of its values
  constexpr int Rows = 32 * kWaves;
  constexpr int Ahead = 64 / kWaves;           // tiles whose pages a wave holds
  static_assert(2 * Loads == Q, "a piece goes to LDS beside each matrix instruction of the first scores");
  __shared__ __align__(16) uint16_t lds_k[2][K * D];
  __shared__ __align__(16) uint16_t lds_v[2][K * D];
  const int lane = threadIdx.x & (kWave - 1), h = lane >> 5, c32 = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int group = a.q_heads / a.kv_heads;
  const float c = a.scale * kLog2e;
  const Paged& pg = a.paged;
  const int page_mask = (1 << pg.page_shift) - 1;
  const int head = blockIdx.x;
  const char* kh = static_cast<const char*>(a.k_cache) + head * pg.head_stride;
  const char* vh = static_cast<const char*>(a.v_cache) + head * pg.head_stride;
  const uint8_t* sh = a.kv_scales + head * a.scale_head_stride;

  for (int at_seq = blockIdx.z; at_seq < pg.seqs; at_seq += gridDim.z) {
    const int seq = longest_first(a, cut, at_seq, Rows);
    const Seq sq = load_seq(pg, a.n, seq);
    const int rows = sq.tokens * group;
    const int32_t* table = pg.page_table + seq * pg.table_stride;

    // the last rows of a causal chunk see the most: they start first
    const int may = cut.parts_of(rows, Rows), split = blockIdx.y % may, step = gridDim.y / may;
    for (int tile = (rows + Rows - 1) / Rows - 1 - blockIdx.y / may; tile >= 0; tile -= step) {
      const int row0 = tile * Rows, row_end = rows - row0 > Rows ? row0 + Rows : rows;
      const Reach rc(sq, row0, row_end, group, a.causal, a.window, cut, may);
      if (split >= rc.parts) continue;
      const int k_first = rc.first + split * rc.part;
      const int hi = rc.hi - k_first < rc.part ? rc.hi : k_first + rc.part;
      // what this wave's rows see: some of them [w_lo, w_hi), all of them [w_all_lo, w_all_hi)
      const int w0 = row0 + 32 * wave, w1 = w0 + 32 < row_end ? w0 + 32 : row_end;
      int w_lo = 0, w_hi = 0, w_all_lo = 0, w_all_hi = 0;
      if (w0 < w1) {
        const Span s0 = seen_by(sq, w0 / group, a.causal, a.window);
        const Span s1 = seen_by(sq, (w1 - 1) / group, a.causal, a.window);
        w_lo = s0.lo;
        w_hi = s1.hi;
        w_all_lo = s1.lo;
        w_all_hi = s0.hi;
      }
      const int row = w0 + c32;
      int row_lo = 0, row_hi = 0;
      long long to = 0;  // row of the output
      u32x4 qf[Q];
#pragma unroll
      for (int s = 0; s < Q; ++s) qf[s] = u32x4{0, 0, 0, 0};
      if (row < w1) {
        const int tok = row / group, gi = row - tok * group;
        const Span s = seen_by(sq, tok, a.causal, a.window);
        row_lo = s.lo;
        row_hi = s.hi;
        to = static_cast<long long>(sq.first + tok) * a.q_heads + head * group + gi;
        const uint16_t* q = static_cast<const uint16_t*>(a.q.ptr) + (sq.first + tok) * a.q.stride +
                            (head * group + gi) * a.q.head_stride + h * 8;
#pragma unroll
        for (int i = 0; i < Q; ++i) qf[i] = *reinterpret_cast<const u32x4*>(q + i * 16);
      }

      float m = -INFINITY, l = 0.f;
      f32x16 o[C];
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.f;

      // Pages of 64 blocks of 16 entries (Ahead tiles) at a time, one to a lane, read as many tiles ahead, and their
      // scales; past the end: of the last entry.
      const auto look_up = [&](int k0) {
        const int key = k0 + 16 * lane;
        return table[(key < hi ? key : hi - 1) >> pg.page_shift];
      };
      int pages = 0, pages_next = 0, scales = 0, at = 0;
      uint64_t good64 = 0;  // bit i: the page of block i is good
      const auto next_pages = [&](int k0) {  // the tile at k0 is the first of the next Ahead
        pages = pages_next;
        const bool good = static_cast<uint32_t>(pages) < static_cast<uint32_t>(pg.num_pages);
        if (!good && k0 + 16 * lane < hi && k0 + 16 * lane + 16 > rc.lo) flag(pg.status, DLRM_STATUS_BAD_PAGE);
        good64 = __ballot(good);
        pages_next = look_up(k0 + Ahead * K < hi ? k0 + Ahead * K : k0);
        const int key = k0 + 16 * lane, known = (key < hi ? key : hi - 1) & page_mask;
        scales = *reinterpret_cast<const uint16_t*>(sh + (good ? pages : 0) * a.scale_page_stride +
                                                    known / kScaleBlock * 2);
      };
      // This wave's 16 entries of the tile at k0, block kWaves at + wave of the pages at hand: a contiguous piece of
      // the cache. Past the end and in place of a bad page other entries are read, and masked.
      uint2 raw[2][Loads];
      const auto fetch_tile = [&](int k0) {
        const int key = k0 + 16 * wave, known = key < hi ? key : hi - 1, block = kWaves * at + wave;
        const int page = good64 >> block & 1 ? __builtin_amdgcn_readlane(pages, block) : 0;
        const long long from = page * pg.page_stride + (known & page_mask & ~15) * D + lane * 8;
#pragma unroll
        for (int i = 0; i < Loads; ++i) {
          raw[0][i] = *reinterpret_cast<const uint2*>(kh + from + i * kWave * 8);
          raw[1][i] = *reinterpret_cast<const uint2*>(vh + from + i * kWave * 8);
        }
      };
      float put_scale[2] = {1.f, 1.f};  // of the keys and values in registers
      const auto put_scales = [&] {
        const int two = __builtin_amdgcn_readlane(scales, kWaves * at + wave);
        put_scale[0] = key_scale(two);
        put_scale[1] = value_scale(two);
      };
      // Piece n of what the registers hold goes to LDS. Sixteen lanes fill places of all banks (with 16 codes a lane
      // it is every other place of a row of values, 18 % of the time in conflicts).
      const auto put_one = [&](int n, int buf) {
        const int value = n / Loads, i = n % Loads, r = (i * kWave + lane) / P, piece = lane % P;
        uint16_t* rows16 = (value ? lds_v[buf] : lds_k[buf]) + (16 * wave + r) * D;
        uint2 w = raw[value][i];
        asm volatile("" : "+v"(w.x), "+v"(w.y));  // widened here, not ahead of the branches that come to this
        const float scale = put_scale[value];
        *reinterpret_cast<uint4*>(rows16 + (piece ^ (value ? value_swizzle<D>(r) : key_swizzle<D>(r))) * 8) =
            make_uint4(widen_codes<DT, false>(w.x, scale), widen_codes<DT, true>(w.x, scale),
                       widen_codes<DT, false>(w.y, scale), widen_codes<DT, true>(w.y, scale));
      };
      constexpr int kAllGood = (1 << (K / 16)) - 1;

      __syncthreads();  // the tiles of the rows before are no longer read
      int good_next = 0;
      if (k_first < hi) {
        pages_next = look_up(k_first);
        next_pages(k_first);
        fetch_tile(k_first);
        put_scales();
#pragma unroll
        for (int n = 0; n < Q; ++n) put_one(n, 0);
        good_next = static_cast<int>(good64) & kAllGood;
        if (k_first + K < hi) {
          at = 1;
          fetch_tile(k_first + K);
        }
      }
      for (int k0 = k_first, buf = 0; k0 < hi; k0 += K, buf ^= 1) {
        __syncthreads();  // this tile is in LDS, and the other one is no longer read
        const int good = good_next;
        // The next tile, in registers, goes to LDS between the matrix instructions of the first scores (past the last
        // tile: what the registers hold, for nobody); then the one after it is asked for.
        if (k0 + K < hi) {
          put_scales();
          good_next = static_cast<int>(good64 >> (kWaves * at)) & kAllGood;
        }
        const auto fetch_next = [&] {
          if (k0 + 2 * K < hi) {
            at = (at + 1) % Ahead;
            if (at == 0) next_pages(k0 + 2 * K);
            fetch_tile(k0 + 2 * K);
          }
        };
        // A tile that some rows do not see whole: a value that is infinite or NaN would reach the rows that
        // do not see it as 0 x inf, so it counts as zero in the product, and is added after it to the rows
        // that see it.
        bool special = false;
        if (k0 < rc.all_lo || k0 + K > rc.all_hi || k0 + K > hi || good != kAllGood) {
          bool found = false;
#pragma unroll 4
          for (int i = 0; i < K * P / kThreads; ++i) {
            uint4* piece = reinterpret_cast<uint4*>(lds_v[buf]) + i * kThreads + threadIdx.x;
            uint4 w = *piece;
            const uint4 odd = make_uint4(not_finite_halves<DT>(w.x), not_finite_halves<DT>(w.y),
                                         not_finite_halves<DT>(w.z), not_finite_halves<DT>(w.w));
            if (odd.x | odd.y | odd.z | odd.w) {
              *piece = make_uint4(w.x & ~odd.x, w.y & ~odd.y, w.z & ~odd.z, w.w & ~odd.w);
              found = true;
            }
          }
          special = __syncthreads_or(found) != 0;
        }

        if (k0 >= w_hi || k0 + K <= w_lo) {  // this wave's rows see none of these entries
#pragma unroll
          for (int n = 0; n < Q; ++n) put_one(n, buf ^ 1);
          fetch_next();
        } else {
          // pieces of keys and values are read KW and VW ahead of the matrix unit
          constexpr int KW = Q > 8 ? 4 : Q < 8 ? Q : 8, VW = KW;
          const auto key_frag = [&](int b0, int n) {  // block b0 + n % T of 32 entries, step n / T
            const int r = 32 * (b0 + n % T) + c32, place = (n / T * 2 + h) ^ key_swizzle<D>(r);
            return *reinterpret_cast<const u32x4*>(lds_k[buf] + r * D + place * 8);
          };
          // V^T of 16 entries (step n / C) and 32 elements (piece n % C): entries 4 h .. and 8 + 4 h .. of the step
          const auto value_frag = [&](int b0, int n) {
            u32x4 w;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int r = 32 * b0 + 16 * (n / C) + 8 * k + 4 * h + (lane & 15) / 4;
              const int place = (n % C * 4 + (lane >> 4 & 1) * 2 + (lane >> 1 & 1)) ^ value_swizzle<D>(r);
              const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (__attribute__((address_space(3))) s16x4*)(lds_v[buf] + r * D + place * 8 + (lane & 1) * 4));
              const uint2 u = __builtin_bit_cast(uint2, x);
              w[2 * k] = u.x;
              w[2 * k + 1] = u.y;
            }
            return w;
          };
          const auto mask = [&](f32x16& s, int b) {  // block b of 32 entries
            const int e0 = k0 + 32 * b;
            if (e0 < w_all_lo || e0 + 32 > w_all_hi || e0 + 32 > hi || (good >> (2 * b) & 3) != 3) {
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                const int e = 8 * (r / 4) + 4 * h + r % 4, key = e0 + e;
                if (key < row_lo || key >= row_hi || key >= hi || !(good >> (2 * b + e / 16) & 1)) s[r] = -INFINITY;
              }
            }
          };
#pragma unroll
          for (int b0 = 0; b0 < 2; b0 += T) {
            u32x4 kf[KW], vf[VW];
#pragma unroll
            for (int n = 0; n < KW; ++n) kf[n] = key_frag(b0, n);
            // the blocks' chains in turn: a matrix instruction waits for the one before it in its sum
            f32x16 s[T];
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
              for (int r = 0; r < 16; ++r) s[t][r] = 0.f;
#pragma unroll
            for (int n = 0; n < T * Q; ++n) {
              s[n % T] = mfma32<DT>(kf[n % KW], qf[n / T], s[n % T]);
              if (n + KW < T * Q) kf[n % KW] = key_frag(b0, n + KW);
              if (b0 == 0 && n < Q) put_one(n, buf ^ 1);
              if (b0 == 0 && n == Q - 1) fetch_next();
            }
#pragma unroll
            for (int n = 0; n < VW; ++n) vf[n] = value_frag(b0, n);
#pragma unroll
            for (int t = 0; t < T; ++t) mask(s[t], b0 + t);
            float tops[4] = {s[0][0], s[0][1], s[0][2], s[0][3]};
#pragma unroll
            for (int r = 4; r < 16 * T; ++r) tops[r % 4] = fmaxf(tops[r % 4], s[r / 16][r % 16]);
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            const float next = fmaxf(m, max_halves(top));
            // O and l stay relative to an older maximum until a row's grows by 2^8: weights are then at most
            // 2^8 (fp16: 2^15 with its lift)
            if (__any((next - m) * c > (DT == DLRM_F16 ? 7.f : 8.f))) {
              const float keep = m == -INFINITY ? 0.f : exp2f((m - next) * c);
              m = next;
              l *= keep;
#pragma unroll
              for (int i = 0; i < C; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[i][r] *= keep;
            }
            const float base = m == -INFINITY ? 0.f : m * c - kLift<DT>;
            float sum[4] = {};
            u32x4 pw[2 * T];  // weights of 16 entries each, in the product's type as in the rows kernel
            const auto weigh = [&](int pair) {
              const int r = 2 * (pair % 8);
              const float p_0 = __builtin_amdgcn_exp2f(fmaf(s[pair / 8][r], c, -base));
              const float p_1 = __builtin_amdgcn_exp2f(fmaf(s[pair / 8][r + 1], c, -base));
              sum[r % 4] += p_0;
              sum[r % 4 + 1] += p_1;
              pw[pair / 4][pair % 4] = pack2<DT>(p_0, p_1);
            };
            // the product of 16 entries beside the weights of the next 16
#pragma unroll
            for (int pair = 0; pair < 4; ++pair) weigh(pair);
#pragma unroll
            for (int n = 0; n < 2 * T * C; ++n) {
              o[n % C] = mfma32<DT>(vf[n % VW], pw[n / C], o[n % C]);
              if (n + VW < 2 * T * C) vf[n % VW] = value_frag(b0, n + VW);
              if (n < (2 * T - 1) * C) {
#pragma unroll
                for (int k = n % C * 4 / C; k < (n % C + 1) * 4 / C; ++k) weigh(4 * (n / C + 1) + k);
              }
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          }
        }

        if (special) {
#pragma unroll 1
          for (int e = 0; e < K; ++e) {
            const int key = k0 + e;
            const int page = key < hi ? scalar_load(table, key >> pg.page_shift) : -1;
            if (page < 0 || page >= pg.num_pages) continue;
            const char* v = vh + page * pg.page_stride + static_cast<long long>(key & page_mask) * D + 4 * h;
            const float scale =
                value_scale(sh[page * a.scale_page_stride + (key & page_mask) / kScaleBlock * 2 + 1] << 8);
            const bool mine = key >= row_lo && key < row_hi;
#pragma unroll
            for (int i = 0; i < 4 * C; ++i) {
              const uint32_t codes = *reinterpret_cast<const uint32_t*>(v + 8 * i);
              const uint32_t w[2] = {widen_codes<DT, false>(codes, scale), widen_codes<DT, true>(codes, scale)};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t u = w[j / 2] >> (j % 2 * 16) & 0xffffu;
                const float x = DT == DLRM_BF16 ? bf16_lo(u) : f16_lo(u);
                o[i / 4][4 * (i % 4) + j] += mine && not_finite_halves<DT>(u) ? x : 0.f;
              }
            }
          }
        }
      }

      l = add_halves(l);
      if (row < w1) {
        const bool part = rc.parts > 1;
        const Sums sums(a, cut, sq, seq, may);
        const int in_seq = static_cast<int>(to - static_cast<long long>(sq.first) * a.q_heads);
        const float inv = part ? 1.f : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int at_d = 32 * i + 8 * q + 4 * h;
            const float x0 = o[i][4 * q] * inv, x1 = o[i][4 * q + 1] * inv, x2 = o[i][4 * q + 2] * inv,
                        x3 = o[i][4 * q + 3] * inv;
            if (part)
              *reinterpret_cast<float4*>(cut.o + sums.row(in_seq, split) * D + at_d) = make_float4(x0, x1, x2, x3);
            else
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to * D + at_d) =
                  make_uint2(pack2<DT>(x0, x1), pack2<DT>(x2, x3));
          }
        if (h == 0) {
          if (part)
            cut.ml[sums.ml(in_seq) + split] = make_float2(m, l);
          else if (a.lse)
            a.lse[to] = l == 0.f ? -INFINITY : fmaf(m, a.scale, logf(l) - kLift<DT> * kLn2);
        }
      }
    }
  }
}

// Where the workgroups of a call would not fill the chip, or histories may be of unequal length, every history is split
// into parts, by the rules for the 16-bit cache and with what was measured for them, places included: heads of 64 count
// 768 workgroups, of which this kernel's registers hold 512 (177, two waves to a SIMD). Measured for this cache are the
// rows kernel's parts, of 256 KB of keys, which are twice the entries (64 histories of up to 16k entries of 128: 128 us
// in 9 parts, 130 in 17), and the spread below.
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
    const long long least = 262144 / dim, fill = 256 / units, finest = (span + 511) / 512, most = 16384 / units;
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
  // Sequences of few rows beside those of many: up to 16 parts, less in calls of many rows (one of 8192 tokens and 127
  // of one: 1533 us in 3, 1588 in 16), and none where that gives no history more. Their sums take no more room than
  // twice the result in fp32, or 32 MB where that is less, and all sums no more than a million rows. The room is shared
  // out evenly (12 chunks of 256-wide heads: 102 us, with half of it 118); a sequence needs at most what its tiles and
  // parts fill. A single one is taken to have the n tokens of the call.
  const long long finest = (span + kLeastPart - 1) / kLeastPart, least_room = (8LL << 20) / dim;
  const long long filled = static_cast<long long>(c.q_tiles) * c.splits * rows;
  long long parts = (1LL << 20) / (all_rows > 0 ? all_rows : 1), left = 1LL << 20;
  if (parts > 16) parts = 16;
  if (parts > finest) parts = finest;
  if (c.splits > 1) left -= all_rows * c.splits;
  long long room = 2 * all_rows > least_room ? 2 * all_rows : least_room;
  room = (room < left ? room : left) / (static_cast<long long>(seqs) * kv_heads);
  if (room > filled) room = filled;
  const bool alone = seqs == 1 && all_rows / kv_heads > filled / (c.splits + 1);
  const bool spread = rows > 16 && tiles > 1 && parts > c.splits && room > c.splits && !alone;
  c.spread = spread ? static_cast<int>(parts) : 0;
  c.spare = spread ? static_cast<int>(room) : 0;
  c.o = nullptr;
  c.ml = nullptr;
  return c;
}

template <int DT, int D>
hipError_t run(const AttnArgs& a, hipStream_t s) {
  const long long rows = static_cast<long long>(a.max_q) * (a.q_heads / a.kv_heads);
  const Cut cut = cut_call(a.n * a.q_heads, rows, a.paged.seqs, a.kv_heads, D, a.causal, a.window, a.max_q, a.max_kv);
  const int tile = tile_rows(rows);
  if (tile == 16) return launch_cut<DT, D, false>(a, cut, tile, attn_rows_q8_kernel<DT, D>, kThreads, s);
  return launch_cut<DT, D, true>(a, cut, tile, attn_tile_q8_kernel<DT, D>, kThreads, s);
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

size_t attn_q8_workspace(int64_t n, int seqs, int q_heads, int kv_heads, int dim, int causal, int window, int max_q,
                         int max_kv) {
  if (n == 0 || seqs == 0) return 0;
  const long long rows = static_cast<long long>(max_q) * (q_heads / kv_heads);
  return cut_bytes(cut_call(n * q_heads, rows, seqs, kv_heads, dim, causal, window, max_q, max_kv), n, seqs, q_heads,
                   kv_heads, dim);
}

hipError_t launch_paged_attn_q8(const AttnArgs& a, hipStream_t s) {
  if (a.n == 0 || a.paged.seqs == 0) return hipSuccess;
  return a.dtype == DLRM_F16 ? run_dim<DLRM_F16>(a, s) : run_dim<DLRM_BF16>(a, s);
}

}  // namespace dlrm
