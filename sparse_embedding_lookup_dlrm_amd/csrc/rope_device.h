// Norm of queries and keys per head and their position rotation, for the kernels that do it on the way: into new
// tensors, a 16-bit cache or an 8-bit one.
//
//   y = x w / sqrt(mean(x^2) + eps), then (a, b) -> (a cos - b sin, a sin + b cos) on each pair
//
// Bound by memory: a token's heads are read once and written once. A head's pairs need one
// angle each, the same for all heads of a token, so a workgroup takes the cosines and sines of
// its tokens into LDS first (one evaluation per token and pair) and then walks the heads. The
// angle is formed in fp64 and reduced to a part of a turn before it is rounded: at position
// 100,000 an fp32 angle would be off by 4e-3 radians.
#pragma once

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

// Norm of a head, if there is one, and its rotation; wv: the weights of this lane's elements.
template <int DT, int D>
__device__ __forceinline__ void norm_turn(float* y, const float* wv, bool norm, float eps, const float2* cs,
                                          const Split<DT, D>& split, bool interleaved) {
  constexpr int V = Split<DT, D>::V;
  if (norm) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) sum = fmaf(y[i], y[i], sum);
    sum = group_sum<Split<DT, D>::lanes>(sum);
    const float r = rsqrtf(sum * (1.f / D) + eps);
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) y[i] = y[i] * r * wv[i];
  }
  rotate<DT, D>(y, cs, split, interleaved, 1.f);
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
        norm_turn<DT, D>(y, wv, norm, a.eps, cs + t * pairs, split, a.rope.interleaved);
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

}  // namespace
}  // namespace dlrm
