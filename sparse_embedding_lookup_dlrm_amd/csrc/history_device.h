// Device helpers shared by the kernels of dlrm_history.h: 16-byte pieces of heads as fp32,
// rounding back, sums over a group of lanes, and the sequence a token belongs to.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "history.h"

namespace dlrm {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Two fp32 values rounded to nearest even into one dword.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const f32x2 v = {a, b};
  if constexpr (DT == DLRM_BF16)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  else
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// The elements of a 16-byte piece (4 of fp32, 8 of the 16-bit types) as fp32, and back.
template <int DT>
__device__ __forceinline__ void widen(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == DLRM_F32) {
      x[i] = __uint_as_float(w[i]);
    } else if constexpr (DT == DLRM_BF16) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    } else {
      x[2 * i] = f16_lo(w[i]);
      x[2 * i + 1] = f16_hi(w[i]);
    }
  }
}

template <int DT>
__device__ __forceinline__ uint4 narrow(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == DLRM_F32)
      w[i] = __float_as_uint(x[i]);
    else
      w[i] = pack2<DT>(x[2 * i], x[2 * i + 1]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, 0xf, 0xf, true));
}

// Sum over aligned groups of N lanes (2 .. 32), the same in every lane of the group.
template <int N>
__device__ __forceinline__ float group_sum(float x) {
  static_assert(N >= 2 && N <= 32, "group of lanes");
  x += dpp<0xB1>(x);                             // lane ^ 1
  if constexpr (N >= 4) x += dpp<0x4E>(x);       // lane ^ 2
  if constexpr (N >= 8) x += dpp<0x141>(x);      // the other four of eight (mirrored)
  if constexpr (N >= 16) x += dpp<0x140>(x);     // the other eight of sixteen (mirrored)
  if constexpr (N >= 32) x += __uint_as_float(__builtin_amdgcn_ds_swizzle(__float_as_uint(x), 0x401F));  // lane ^ 16
  return x;
}

// Number of entries of off[0 .. count) that are <= x (off ascending), found by the whole wave: up to 256
// entries are looked at at once, more in parts: each step splits the range into 64 with one load per
// lane. Never reads outside off[0 .. count), also where off is not ascending.
__device__ __forceinline__ int wave_upper_bound(const int32_t* __restrict__ off, int count, int x) {
  int lo = 0, len = count;  // entries before lo are <= x, entries from lo + len on are > x
  const int lane = threadIdx.x & (kWave - 1);
  while (len > 4 * kWave) {
    const int step = (len + kWave - 1) / kWave;
    const long long i = static_cast<long long>(lane) * step + step - 1;  // last entry of this lane's part
    const bool below = i < len && off[lo + i] <= x;
    const int parts = __builtin_popcountll(__ballot(below));  // whole parts that are <= x
    const long long skip = static_cast<long long>(parts) * step;
    lo += static_cast<int>(skip);
    len = static_cast<int>(skip + step - 1 < len ? step - 1 : len - skip);
  }
  int v[4], found = lo;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = lane + k * kWave < len ? off[lo + lane + k * kWave] : 0x7fffffff;
#pragma unroll
  for (int k = 0; k < 4; ++k) found += __builtin_popcountll(__ballot(lane + k * kWave < len && v[k] <= x));
  return found;
}

}  // namespace dlrm
