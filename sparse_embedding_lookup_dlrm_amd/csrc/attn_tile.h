// The tile kernel of the attention over a paged cache, for calls of more than 16 rows a head.
#pragma once

#include "attn_device.h"

namespace dlrm {
namespace {

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

// Keys are read as rows (32 entries, the same piece): neighbours differ in every place bit.
template <int D>
__device__ __forceinline__ int key_swizzle(int r) {
  return D == 32 ? r >> 1 & 3 : D == 64 ? r & 7 : r & 15;
}
// Values are read as blocks of 4 entries x 2 (or, with the neighbouring lanes, 4) pieces.
template <int D>
__device__ __forceinline__ int value_swizzle(int r) {
  return D == 32 ? r & 2 : D == 64 ? (r & 1) << 2 | (r & 2) : (r & 1) << 2 | (r & 2) | (r & 2) << 2;
}

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

// Q8: the cache holds 8-bit codes. A wave then takes its 16 entries of a tile through registers, loaded while the
// tile two before is worked on, and widens them on their way to LDS: once for the workgroup, not once for each of its
// waves.
template <int DT, int D, bool Q8>
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
    using Stored = std::conditional_t<Q8, uint8_t, uint16_t>;
    const Stored* kh = static_cast<const Stored*>(a.k_cache) + head * pg.head_stride;
    const Stored* vh = static_cast<const Stored*>(a.v_cache) + head * pg.head_stride;
    const uint8_t* sh = Q8 ? a.kv_scales + head * a.scale_head_stride : nullptr;
    const int32_t* table = pg.page_table + seq * pg.table_stride;

    // the last rows of a causal chunk see the most: they start first
    for (long long first_row = static_cast<long long>(cut.q_tiles - 1 - blockIdx.y / cut.splits) * Rows;
         first_row < rows; first_row += static_cast<long long>(cut.q_tiles) * Rows) {
      const int row0 = static_cast<int>(first_row), row_end = rows - row0 > Rows ? row0 + Rows : rows;
      const Reach rc(sq, row0, row_end, group, a.causal, a.window, cut);
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

      // 8-bit codes: this wave's 16 entries of a tile, a contiguous piece of the cache, in registers. Chunk bytes a
      // lane and load, which are one or two pieces of 16 bytes in LDS.
      constexpr int Chunk = D == 32 ? 8 : 16, Loads = 16 * D / (kWave * Chunk);
      uint32_t raw[3 - H][Q8 ? Loads : 1][4];  // keys and values, or this half's
      int scales = 0;  // of the blocks whose pages are at hand, one to a lane
      const auto look_up_scales = [&](int k0, int page, uint64_t good) {
        const int key = k0 + 16 * lane, known = (key < hi ? key : hi - 1) & page_mask;
        const int from = good >> lane & 1 ? page : 0;
        return static_cast<int>(
            *reinterpret_cast<const uint16_t*>(sh + from * a.scale_page_stride + known / kScaleBlock * 2));
      };
      const auto fetch_tile = [&](int k0, int pages, uint64_t good, int at) {
        const int key = k0 + 16 * wave, known = key < hi ? key : hi - 1;
        const int block = 4 * at + wave;
        const int page = good >> block & 1 ? __builtin_amdgcn_readlane(pages, block) : 0;
        const long long from = page * pg.page_stride + (known & page_mask & ~15) * D + lane * Chunk;
#pragma unroll
        for (int i = 0; i < Loads; ++i) {
          const uint8_t* first = reinterpret_cast<const uint8_t*>(H == 1 || half == 0 ? kh : vh);
          __builtin_memcpy(raw[0][i], __builtin_assume_aligned(first + from + i * kWave * Chunk, Chunk), Chunk);
          if constexpr (H == 1)
            __builtin_memcpy(raw[1][i], __builtin_assume_aligned(
                reinterpret_cast<const uint8_t*>(vh) + from + i * kWave * Chunk, Chunk), Chunk);
        }
      };
      const auto put_piece = [&](uint16_t* to, const uint32_t* codes, float scale) {
        *reinterpret_cast<uint4*>(to) =
            make_uint4(widen_codes<DT, false>(codes[0], scale), widen_codes<DT, true>(codes[0], scale),
                       widen_codes<DT, false>(codes[1], scale), widen_codes<DT, true>(codes[1], scale));
      };
      const auto put_tile = [&](int at, int buf) {
        const int two = __builtin_amdgcn_readlane(scales, 4 * at + wave);
        const float ks = key_scale(two), vs = value_scale(two);
#pragma unroll
        for (int i = 0; i < Loads; ++i) {
          const int r = (i * kWave + lane) * Chunk / D, piece = (i * kWave + lane) * Chunk % D / 8;
#pragma unroll
          for (int j = 0; j < Chunk / 8; ++j) {
            const int to = (16 * wave + r) * D;
            if (H == 1 || half == 0)
              put_piece(lds_k[buf] + to + ((piece + j) ^ key_swizzle<D>(r)) * 8, raw[0][i] + 2 * j, ks);
            if (H == 1 || half == 1)
              put_piece(lds_v[buf] + to + ((piece + j) ^ value_swizzle<D>(r)) * 8, raw[2 - H][i] + 2 * j, vs);
          }
        }
      };

      __syncthreads();  // the tiles of the rows before are no longer read
      int pages = 0, pages_next = 0, at = 0, good_next = 0;
      uint64_t good64 = 0;
      const auto next_pages = [&](int k0) {  // the tile at k0 is the first of the next 16
        pages = pages_next;
        good64 = good_pages(k0, pages);
        pages_next = look_up(k0 + 16 * K < hi ? k0 + 16 * K : k0);
        if constexpr (Q8) scales = look_up_scales(k0, pages, good64);
      };
      if constexpr (Q8) {
        if (k_first < hi) {
          pages_next = look_up(k_first);
          next_pages(k_first);
          fetch_tile(k_first, pages, good64, 0);
          put_tile(0, 0);
          good_next = static_cast<int>(good64) & kAllGood;
          if (k_first + K < hi) {
            at = 1;
            fetch_tile(k_first + K, pages, good64, 1);
          }
        }
      } else if (k_first < hi) {
        pages = look_up(k_first);
        pages_next = look_up(k_first + 16 * K < hi ? k_first + 16 * K : k_first);
        good64 = good_pages(k_first, pages);
        copy_tile(k_first, pages, good64, 0, 0);
        good_next = static_cast<int>(good64) & kAllGood;
      }
      for (int k0 = k_first, buf = 0; k0 < hi; k0 += K, buf ^= 1) {
        if constexpr (!Q8) wait_copies();
        __syncthreads();  // this tile is in LDS, and the other one is no longer read
        const int good = good_next;
        if constexpr (Q8) {
          if (k0 + K < hi) {
            put_tile(at, buf ^ 1);
            good_next = static_cast<int>(good64 >> (4 * at)) & kAllGood;
            if (k0 + 2 * K < hi) {
              at = (at + 1) & 15;
              if (at == 0) next_pages(k0 + 2 * K);
              fetch_tile(k0 + 2 * K, pages, good64, at);
            }
          }
        } else if (k0 + K < hi) {
          at = (at + 1) & 15;
          if (at == 0) next_pages(k0 + K);
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
            const Stored* v =
                vh + page * pg.page_stride + static_cast<long long>(key & page_mask) * D + half * 32 * C + 4 * h;
            const bool mine = key >= row_lo && key < row_hi;
            float vs = 0.f;
            if constexpr (Q8)
              vs = value_scale(sh[page * a.scale_page_stride + (key & page_mask) / kScaleBlock * 2 + 1] << 8);
#pragma unroll
            for (int i = 0; i < 4 * C; ++i) {
              uint2 w;
              if constexpr (Q8) {
                const uint32_t codes = *reinterpret_cast<const uint32_t*>(v + 8 * i);
                w = make_uint2(widen_codes<DT, false>(codes, vs), widen_codes<DT, true>(codes, vs));
              } else {
                w = *reinterpret_cast<const uint2*>(v + 8 * i);
              }
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

}  // namespace
}  // namespace dlrm
