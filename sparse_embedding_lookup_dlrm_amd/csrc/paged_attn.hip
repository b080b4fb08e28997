// Attention of new tokens over a paged cache of 16-bit values (formulas in attn_device.h).
//
// Scores are formed transposed, S^T = K Q^T, by 16x16x32 matrix instructions. Their result holds
// four entries of one row in each lane, which is what the second product O^T = V^T P^T takes as
// its right operand when the order of the 32 entries in the sum is chosen to fit (lane group g
// takes entries 4g .. 4g+3 of both halves): the weights never leave the lane, and m, l and the
// rescale of O are one value per lane.
#include "attn_device.h"

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
      const Reach rc(sq, row0, row_end, group, a.causal, a.window, cut, cut.splits);
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

// ---------------------------------------------------------------------------
// Tile kernel: 128 rows of one head to a workgroup, 32 to a wave. Tiles of K entries go straight
// from global memory to LDS (16 bytes a lane), one tile ahead, and every wave reads all of a tile.
// The products are 32x32x16: the score of row lane % 32 with entries 8 i + 4 h + j (h = lane / 32,
// i, j = 0 .. 3) lies in one lane, which again is the second product's right operand as it stands.
// Its left operand V^T is read by the transposing LDS load: sixteen lanes take a block of 4 entries
// x 16 elements and get one element of the 4 entries each.
//
// A row of D elements is D / 8 pieces of 16 bytes; piece c of entry r lies at place c ^ swizzle(r),
// so that the lanes that LDS serves together fall on different banks. The copy to LDS writes places
// in order and picks the piece for each.
//
// Long chunks are bound by the matrix and the vector units, which are rarely at work at once. A tile takes a wave 32
// matrix instructions of 32 clocks (D = 128) and 188 vector ones, about 890 clocks of the softmax, of the 2280 clocks
// that its SIMD has for it: the matrix units are at 45 %. Four chunks of up to 2048 new tokens over up to 8192
// entries, 32 heads of 128: 278 us, 963 TFLOP/s; the matrix instructions alone take 198 us, everything else 181. LDS
// is at 23 %: its reads left out save 14 us, the copies to it 29. Short histories and windows wait for a workgroup's
// tiles in a row (24 sequences of up to 257 x 1500: 17 us, 208 workgroups of heads of 256 with a window of 1024: 80).
// Two blocks of 32 rows to a wave halve the LDS reads, but leave one wave to a SIMD, whose exponentials then stand
// beside idle matrix units: 357 .. 550 us. Scores of the next tile formed beside this one's exponentials: 307 .. 335
// us, for the registers. Priorities around the matrix instructions: no difference.
// ---------------------------------------------------------------------------
constexpr int kTileKeys = 64;

// N copies of 16 bytes a lane to LDS: copy i brings from `from` + off[i] + 1024 i, lane j's bytes to
// `to` + 1024 i + 16 j; from and to are the same in every lane. Written out because after the builtin
// the compiler holds every LDS read back until the copy has landed, also reads of the other tile. No
// register receives anything; the kernel itself waits (wait_copies) before the barrier that publishes
// the tile. The offset of the instruction counts on both sides. m0, which holds the LDS address, is the compiler's:
// each block puts back what it found there.
template <int N>
__device__ __forceinline__ void copy16(const char* from, const uint32_t (&off)[N], const uint16_t* to) {
  const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (const __attribute__((address_space(3))) uint16_t*)to));
  uint32_t m0;
  if constexpr (N == 1)
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\t"
                 "s_mov_b32 m0, %0"
                 : "=&s"(m0) : "s"(lds), "v"(off[0]), "s"(from) : "memory");
  else if constexpr (N == 2)
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %4\n\t"
                 "global_load_lds_dwordx4 %3, %4 offset:0x400\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0) : "s"(lds), "v"(off[0]), "v"(off[1]), "s"(from) : "memory");
  else
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %6\n\t"
                 "global_load_lds_dwordx4 %3, %6 offset:0x400\n\tglobal_load_lds_dwordx4 %4, %6 offset:0x800\n\t"
                 "global_load_lds_dwordx4 %5, %6 offset:0xc00\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0) : "s"(lds), "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "s"(from) : "memory");
}

// Waits for this wave's copies to LDS (vmcnt 0, the other counts open); a barrier makes those of the
// other waves visible too. The builtin tells the compiler that its own loads are in as well.
__device__ __forceinline__ void wait_copies() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70);
  asm volatile("" ::: "memory");
}

// Heads of 256 elements take two waves for the same 32 rows, each with half of O: all of it beside the
// queries would leave one wave to a SIMD, and nothing to run while it waits. Both form all scores.
template <int D>
constexpr int kHalves = D == 256 ? 2 : 1;
template <int D>
constexpr int kTileThreads = kThreads * kHalves<D>;

template <int DT, int D>
__global__ __launch_bounds__(kTileThreads<D>, 2) void attn_tile_kernel(AttnArgs a, Cut cut) {
  constexpr int K = kTileKeys;
  constexpr int T = D == 256 ? 1 : K / 32;  // 32-entry blocks of scores held at once
  constexpr int Part = 32 * T;       // entries worked on at once
  constexpr int Q = D / 16;          // steps of the first product
  constexpr int H = kHalves<D>;
  constexpr int C = D / 32 / H;      // 32-wide pieces of O
  constexpr int P = D / 8;           // pieces of a row
  constexpr int Rows = 32 * kWaves;
  constexpr int CopyRows = kWave / P;  // entries that a wave copies at once, 16 bytes a lane
  constexpr int Copy = 16 / CopyRows;  // copies for the 16 entries that a wave brings of each tile
  static_assert(K == 16 * kWaves, "a wave brings 16 entries, which lie in one page");
  __shared__ __align__(16) uint16_t lds_k[2][K * D];
  __shared__ __align__(16) uint16_t lds_v[2][K * D];
  const int lane = threadIdx.x & (kWave - 1), h = lane >> 5, c32 = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave % kWaves);
  const int half = __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);  // of O
  const int group = a.q_heads / a.kv_heads;
  const float c = a.scale * kLog2e;
  const Paged& pg = a.paged;
  const int page_mask = (1 << pg.page_shift) - 1;
  // what this lane copies: byte offsets in the 16 entries, less the copy's own 1024 i. They repeat after
  // four entries (values) or sixteen (keys).
  constexpr int Group = Copy < 4 ? Copy : 4;
  uint32_t copy_k[Copy / Group][Group], copy_v[Group];
#pragma unroll
  for (int i = 0; i < Copy; ++i) {
    const int r = i * CopyRows + lane / P;
    copy_k[i / Group][i % Group] = 2 * (lane / P * D + (lane % P ^ key_swizzle<D>(r)) * 8);
    if (i < Group) copy_v[i] = 2 * (lane / P * D + (lane % P ^ value_swizzle<D>(r)) * 8);
  }

  const int head = blockIdx.x, split = blockIdx.y % cut.splits;
  for (int seq = blockIdx.z; seq < pg.seqs; seq += gridDim.z) {
    const Seq sq = load_seq(pg, a.n, seq);
    const int rows = sq.tokens * group;
    const uint16_t* kh = static_cast<const uint16_t*>(a.k_cache) + head * pg.head_stride;
    const uint16_t* vh = static_cast<const uint16_t*>(a.v_cache) + head * pg.head_stride;
    const int32_t* table = pg.page_table + seq * pg.table_stride;

    // the last rows of a causal chunk see the most: they start first
    for (long long first_row = static_cast<long long>(cut.q_tiles - 1 - blockIdx.y / cut.splits) * Rows;
         first_row < rows; first_row += static_cast<long long>(cut.q_tiles) * Rows) {
      const int row0 = static_cast<int>(first_row), row_end = rows - row0 > Rows ? row0 + Rows : rows;
      const Reach rc(sq, row0, row_end, group, a.causal, a.window, cut, cut.splits);
      if (split >= rc.parts) continue;
      const int k_first = rc.first + split * rc.part;
      const int hi = rc.hi - k_first < rc.part ? rc.hi : k_first + rc.part;
      // what this wave's rows see: some of them [w_lo, w_hi), all of them [w_all_lo, w_all_hi)
      const int w0 = row0 + 32 * wave, w1 = w0 + 32 < row_end ? w0 + 32 : row_end;
      int tok0 = 0, tok1 = -1, w_lo = 0, w_hi = 0, w_all_lo = 0, w_all_hi = 0;
      if (w0 < w1) {
        tok0 = w0 / group;
        tok1 = (w1 - 1) / group;
        const Span s0 = seen_by(sq, tok0, a.causal, a.window), s1 = seen_by(sq, tok1, a.causal, a.window);
        w_lo = s0.lo;
        w_hi = s1.hi;
        w_all_lo = s1.lo;
        w_all_hi = s0.hi;
      }
      const int row = w0 + c32;
      int row_lo = 0, row_hi = 0, row_tok = -1;
      long long to = 0;  // row of the output
      u32x4 qf[Q];
#pragma unroll
      for (int s = 0; s < Q; ++s) qf[s] = u32x4{0, 0, 0, 0};
      if (row < w1) {
        row_tok = row / group;
        const int gi = row - row_tok * group;
        const Span s = seen_by(sq, row_tok, a.causal, a.window);
        row_lo = s.lo;
        row_hi = s.hi;
        to = static_cast<long long>(sq.first + row_tok) * a.q_heads + head * group + gi;
        const uint16_t* q = static_cast<const uint16_t*>(a.q.ptr) + (sq.first + row_tok) * a.q.stride +
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

      // Pages of 64 blocks of 16 entries (16 tiles) at a time, one to a lane, read 16 tiles ahead; past
      // the end: of the last entry.
      const auto look_up = [&](int k0) {
        const int key = k0 + 16 * lane;
        return table[(key < hi ? key : hi - 1) >> pg.page_shift];
      };
      // Bit i: the page of block i is good.
      const auto good_pages = [&](int k0, int page) {
        const bool good = static_cast<uint32_t>(page) < static_cast<uint32_t>(pg.num_pages);
        if (!good && k0 + 16 * lane < hi && k0 + 16 * lane + 16 > rc.lo) flag(pg.status, DLRM_STATUS_BAD_PAGE);
        return __ballot(good);
      };
      // Brings this wave's 16 entries of the tile at k0, block 4 at + wave of the pages at hand, to LDS.
      // Past the end and in place of a bad page other entries of the cache are read, and masked.
      const auto copy_tile = [&](int k0, int pages, uint64_t good, int at, int buf) {
        const int key = k0 + 16 * wave, known = key < hi ? key : hi - 1;
        const int block = 4 * at + wave;
        const int page = good >> block & 1 ? __builtin_amdgcn_readlane(pages, block) : 0;
        const long long from = 2 * (page * pg.page_stride + (known & page_mask & ~15) * D);
        const char* kp = reinterpret_cast<const char*>(kh) + from;
        const char* vp = reinterpret_cast<const char*>(vh) + from;
#pragma unroll
        for (int i = 0; i < Copy / Group; ++i) {
          if (H == 1 || half == 0) copy16(kp + i * 4096, copy_k[i], lds_k[buf] + 16 * wave * D + i * 2048);
          if (H == 1 || half == 1) copy16(vp + i * 4096, copy_v, lds_v[buf] + 16 * wave * D + i * 2048);
        }
      };
      constexpr int kAllGood = (1 << (K / 16)) - 1;

      __syncthreads();  // the tiles of the rows before are no longer read
      int pages = 0, pages_next = 0, at = 0, good_next = 0;
      uint64_t good64 = 0;
      if (k_first < hi) {
        pages = look_up(k_first);
        pages_next = look_up(k_first + 16 * K < hi ? k_first + 16 * K : k_first);
        good64 = good_pages(k_first, pages);
        copy_tile(k_first, pages, good64, 0, 0);
        good_next = static_cast<int>(good64) & kAllGood;
      }
      for (int k0 = k_first, buf = 0; k0 < hi; k0 += K, buf ^= 1) {
        wait_copies();
        __syncthreads();  // this tile is in LDS, and the other one is no longer read
        const int good = good_next;
        if (k0 + K < hi) {
          at = (at + 1) & 15;
          if (at == 0) {
            pages = pages_next;
            good64 = good_pages(k0 + K, pages);
            pages_next = look_up(k0 + 17 * K < hi ? k0 + 17 * K : k0);
          }
          copy_tile(k0 + K, pages, good64, at, buf ^ 1);
          good_next = static_cast<int>(good64 >> (4 * at)) & kAllGood;
        }
        // A tile that some rows do not see whole: a value that is infinite or NaN would reach the rows that
        // do not see it as 0 x inf, so it counts as zero in the product, and is added after it to the rows
        // that see it.
        bool special = false;
        if (k0 < rc.all_lo || k0 + K > rc.all_hi || k0 + K > hi || good != kAllGood) {
          bool found = false;
#pragma unroll
          for (int i = 0; i < K * P / (kThreads * H); ++i) {
            uint4* piece = reinterpret_cast<uint4*>(lds_v[buf]) + i * kThreads * H + threadIdx.x;
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

        // pieces of keys and values are read KW and VW ahead of the matrix unit
        constexpr int KW = Q < 8 ? Q : 8, VW = 2 * T * C < 8 ? 2 * T * C : 8;
#pragma unroll 1
        for (int p0 = 0; p0 < K; p0 += Part) {
          if (k0 + p0 >= w_hi || k0 + p0 + Part <= w_lo) continue;  // this wave's rows see none of these entries
          const auto key_frag = [&](int t, int i) {
            const int r = p0 + 32 * t + c32, place = (2 * i + h) ^ key_swizzle<D>(r);
            return *reinterpret_cast<const u32x4*>(lds_k[buf] + r * D + place * 8);
          };
          f32x16 s[T];
          u32x4 kf[KW];
#pragma unroll
          for (int i = 0; i < KW; ++i) kf[i] = key_frag(i / Q, i % Q);
#pragma unroll
          for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[t][r] = 0.f;
#pragma unroll
            for (int i = 0; i < Q; ++i) {
              const int n = t * Q + i, ahead = n + KW;
              s[t] = mfma32<DT>(kf[n % KW], qf[i], s[t]);
              if (ahead < T * Q) kf[n % KW] = key_frag(ahead / Q, ahead % Q);
            }
          }
          const int part0 = k0 + p0, part1 = part0 + Part;
          if (part0 < w_all_lo || part1 > w_all_hi || part1 > hi || good != kAllGood) {
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                const int e = p0 + 32 * t + 8 * (r / 4) + 4 * h + r % 4, key = k0 + e;
                if (key < row_lo || key >= row_hi || key >= hi || !(good >> (e / 16) & 1)) s[t][r] = -INFINITY;
              }
          }

          // V^T of 16 entries (step) and 32 elements (piece): entries 4 h .. and 8 + 4 h .. of the step
          const auto value_frag = [&](int step, int piece) {
            u32x4 w;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int r = p0 + 16 * step + 8 * n + 4 * h + (lane & 15) / 4;
              const int place =
                  ((half * C + piece) * 4 + (lane >> 4 & 1) * 2 + (lane >> 1 & 1)) ^ value_swizzle<D>(r);
              const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (__attribute__((address_space(3))) s16x4*)(lds_v[buf] + r * D + place * 8 + (lane & 1) * 4));
              const uint2 u = __builtin_bit_cast(uint2, x);
              w[2 * n] = u.x;
              w[2 * n + 1] = u.y;
            }
            return w;
          };
          u32x4 vf[VW];
#pragma unroll
          for (int i = 0; i < VW; ++i) vf[i] = value_frag(i / C, i % C);

          float top = s[0][0];
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[t][r]);
          top = max_halves(top);
          const float next = fmaxf(m, top);
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
          u32x4 pw[2 * T];
          float sum[4] = {};
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 16; r += 2) {
              const float p_0 = __builtin_amdgcn_exp2f(fmaf(s[t][r], c, -base));
              const float p_1 = __builtin_amdgcn_exp2f(fmaf(s[t][r + 1], c, -base));
              sum[r % 4] += p_0;
              sum[r % 4 + 1] += p_1;
              pw[2 * t + r / 8][r % 8 / 2] = pack2<DT>(p_0, p_1);
            }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);

#pragma unroll
          for (int n = 0; n < 2 * T * C; ++n) {
            o[n % C] = mfma32<DT>(vf[n % VW], pw[n / C], o[n % C]);
            if (n + VW < 2 * T * C) vf[n % VW] = value_frag((n + VW) / C, (n + VW) % C);
          }
        }

        if (special) {
#pragma unroll 1
          for (int e = 0; e < K; ++e) {
            const int key = k0 + e;
            const int page = key < hi ? scalar_load(table, key >> pg.page_shift) : -1;
            if (page < 0 || page >= pg.num_pages) continue;
            const uint16_t* v =
                vh + page * pg.page_stride + static_cast<long long>(key & page_mask) * D + half * 32 * C + 4 * h;
            const bool mine = key >= row_lo && key < row_hi;
#pragma unroll
            for (int i = 0; i < 4 * C; ++i) {
              const uint2 w = *reinterpret_cast<const uint2*>(v + 8 * i);
              const uint32_t u[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float x = DT == DLRM_BF16 ? bf16_lo(u[j]) : f16_lo(u[j]);
                o[i / 4][4 * (i % 4) + j] += mine && not_finite_halves<DT>(u[j]) ? x : 0.f;
              }
            }
          }
        }
      }

      l = add_halves(l);
      if (row < w1) {
        const bool part = rc.parts > 1;
        const float inv = part ? 1.f : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int at = half * 32 * C + 32 * i + 8 * q + 4 * h;
            const float x0 = o[i][4 * q] * inv, x1 = o[i][4 * q + 1] * inv, x2 = o[i][4 * q + 2] * inv,
                        x3 = o[i][4 * q + 3] * inv;
            if (part)
              *reinterpret_cast<float4*>(cut.o + (split * a.n * a.q_heads + to) * D + at) = make_float4(x0, x1, x2, x3);
            else
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to * D + at) =
                  make_uint2(pack2<DT>(x0, x1), pack2<DT>(x2, x3));
          }
        if (h == 0 && half == 0) {
          if (part)
            cut.ml[to * cut.splits + split] = make_float2(m, l);
          else if (a.lse)
            a.lse[to] = l == 0.f ? -INFINITY : fmaf(m, a.scale, logf(l) - kLift<DT> * kLn2);
        }
      }
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
  c.spread = c.spare = 0;
  c.o = nullptr;
  c.ml = nullptr;
  return c;
}

template <int DT, int D>
hipError_t run(const AttnArgs& a, hipStream_t s) {
  const long long rows = static_cast<long long>(a.max_q) * (a.q_heads / a.kv_heads);
  const Cut cut = cut_call(a.n * a.q_heads, rows, a.paged.seqs, a.kv_heads, D, a.causal, a.window, a.max_q, a.max_kv);
  const int tile = tile_rows(rows);
  if (tile == 16) return launch_cut<DT, D, false>(a, cut, tile, attn_rows_kernel<DT, D>, kThreads, s);
  return launch_cut<DT, D, false>(a, cut, tile, attn_tile_kernel<DT, D>, kTileThreads<D>, s);
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
  return cut_bytes(cut_call(n * q_heads, rows, seqs, kv_heads, dim, causal, window, max_q, max_kv), n, seqs, q_heads,
                   kv_heads, dim);
}

hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t s) {
  if (a.n == 0 || a.paged.seqs == 0) return hipSuccess;
  return a.dtype == DLRM_F16 ? run_dim<DLRM_F16>(a, s) : run_dim<DLRM_BF16>(a, s);
}

}  // namespace dlrm
