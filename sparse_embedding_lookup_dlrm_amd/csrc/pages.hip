// Pages of the history cache, handed out and taken back on the device.
//
// Assignment: with had = ceil(held / page) and has = ceil((held + new) / page) of each sequence, the
// sequences take has - had pages each from the end of the free list, one after the other, so an exclusive
// sum of those over the sequences says where each begins. Release: pages ceil(keep / page) .. had - 1 go to
// the end of the free list, in order.
//
// A call changes all of its sequences or nothing, so one workgroup first looks at all of them (plan): checks,
// the two sums, and whether a user appears twice, which it finds by letting every sequence write its number
// into its user's length and look whether it is still there. The second kernel (fill) writes what is long: page
// tables, slots and positions, with a workgroup for each sequence and part.
//
// Both kernels wait for a few loads in a row and a launch: one event each for 64 users, 1024 pages to a row, 3.5 + 3.9
// us; chunks of 300 users, 300k tokens (4 MB) 4.9 + 6.2; 256 histories of up to 65536 entries dropped 4.0 + 4.7.
#include "history_device.h"

namespace dlrm {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr long long kI32Top = 0x7fffffffLL;

// What the plan tells the fill, in the workspace.
struct Plan {
  int32_t ok, count;  // whether the call is carried out, and the free pages before it
  int32_t at[1];      // [seqs]: pages moved for the sequences before this one; release: [seqs] entries held before
};

// Entries that a release leaves of h.
__device__ __forceinline__ int kept(const PagesArgs& a, long long s, int h) {
  const int keep = a.lens ? a.lens[s] : 0;
  return keep < h ? keep : h;
}

__device__ __forceinline__ long long clamped(long long x) { return x < kI32Top ? x : kI32Top; }

// Exclusive sums of x and y over the threads of the workgroup; the totals come back in sum_x and sum_y.
__device__ __forceinline__ void scan_two(long long& x, long long& y, long long& sum_x, long long& sum_y,
                                         long long (*lds)[kPlanThreads / kWave]) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
  const long long own_x = x, own_y = y;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const long long u = __shfl_up(x, o, kWave), v = __shfl_up(y, o, kWave);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  if (lane == kWave - 1) {
    lds[0][wave] = x;
    lds[1][wave] = y;
  }
  __syncthreads();
  x -= own_x;
  y -= own_y;
  sum_x = sum_y = 0;
  for (int w = 0; w < waves; ++w) {
    if (w < wave) {
      x += lds[0][w];
      y += lds[1][w];
    }
    sum_x += lds[0][w];
    sum_y += lds[1][w];
  }
  __syncthreads();
}

// The call's decision: every sequence checked, summed up and looked for twice.
template <bool ASSIGN>
__device__ __forceinline__ void plan_call(const PagesArgs& a) {
  __shared__ long long lds[2][kPlanThreads / kWave];
  Plan* plan = static_cast<Plan*>(a.workspace);
  const int seqs = a.seqs;
  const long long room = static_cast<long long>(ASSIGN ? a.out_width : a.table_width) << a.page_shift;
  const long long held_room = static_cast<long long>(a.table_width) << a.page_shift;
  const int free_now = *a.count;
  const auto pages_of = [&](long long entries) { return (entries + (1LL << a.page_shift) - 1) >> a.page_shift; };
  const auto user_of = [&](long long s) { return a.who ? a.who[s] : static_cast<int>(s); };

  int bad = 0;
  long long tokens = 0, pages = 0;
  for (long long base = 0; base < seqs; base += blockDim.x) {
    const long long s = base + threadIdx.x;
    long long m = 0, moved = 0;
    if (s < seqs) {
      const int u = user_of(s);
      long long h = 0;
      m = a.lens ? a.lens[s] : 0;
      if (m < 0) {
        bad |= DLRM_STATUS_BAD_OFFSETS;
        m = 0;
      }
      if (static_cast<uint32_t>(u) >= static_cast<uint32_t>(a.users)) {
        bad |= DLRM_STATUS_BAD_USER;
      } else {
        const int raw = a.held[u];
        if (a.held_out != a.held) a.held_out[u] = raw;
        h = raw;
        if (h < 0 || h > held_room) {
          bad |= DLRM_STATUS_BAD_OFFSETS;
          h = 0;
        }
      }
      if constexpr (ASSIGN) {
        if (h + m > room) bad |= DLRM_STATUS_NO_ROOM;
        moved = pages_of(h + m) - pages_of(h);
        a.kv_lens[s] = static_cast<int32_t>(h);
      } else {
        moved = pages_of(h) - pages_of(m < h ? m : h);
        plan->at[static_cast<long long>(seqs) + s] = static_cast<int32_t>(h);
        m = 0;
      }
    }
    long long sum_m, sum_moved;
    scan_two(m, moved, sum_m, sum_moved, lds);
    if (s < seqs) {
      if constexpr (ASSIGN) a.q_offsets[s] = static_cast<int32_t>(clamped(tokens + m));
      plan->at[s] = static_cast<int32_t>(clamped(pages + moved));
    }
    tokens += sum_m;
    pages += sum_moved;
  }
  if (threadIdx.x == 0) {
    if (free_now < 0 || free_now > a.num_pages) bad |= DLRM_STATUS_BAD_PAGE;
    if constexpr (ASSIGN) {
      if (tokens > a.n) bad |= DLRM_STATUS_BAD_OFFSETS;
      if (pages > free_now) bad |= DLRM_STATUS_NO_ROOM;
    } else {
      if (pages + free_now > a.num_pages) bad |= DLRM_STATUS_BAD_PAGE;  // more than there are: some are free already
    }
  }
  if (bad) flag(a.status, bad);
  bool refused = __syncthreads_or(bad) != 0;

  // A user twice: of those that write their number, only one finds it.
  const auto counts = [&](long long s) { return !ASSIGN || a.lens[s] > 0; };
  if (!refused) {
    for (long long s = threadIdx.x; s < seqs; s += blockDim.x)
      if (counts(s)) a.held_out[user_of(s)] = ~static_cast<int32_t>(s);
    __syncthreads();
    bool twice = false;
    for (long long s = threadIdx.x; s < seqs; s += blockDim.x)
      twice |= counts(s) && a.held_out[user_of(s)] != ~static_cast<int32_t>(s);
    if (twice) flag(a.status, DLRM_STATUS_BAD_USER);
    refused = __syncthreads_or(twice) != 0;
    for (long long s = threadIdx.x; s < seqs; s += blockDim.x) {
      if (!counts(s)) continue;
      int32_t now;
      if constexpr (ASSIGN) {
        now = a.kv_lens[s] + (refused ? 0 : a.lens[s]);
        a.kv_lens[s] = now;
      } else {
        now = plan->at[static_cast<long long>(seqs) + s];
        if (!refused) now = kept(a, s, now);
      }
      a.held_out[user_of(s)] = now;
    }
  }
  if (ASSIGN && refused)
    for (long long s = threadIdx.x; s < seqs; s += blockDim.x) a.q_offsets[s] = 0;
  if (threadIdx.x == 0) {
    if constexpr (ASSIGN) a.q_offsets[seqs] = refused ? 0 : static_cast<int32_t>(tokens);
    plan->ok = !refused;
    plan->count = free_now;
    *a.count_out = refused ? free_now : static_cast<int32_t>(ASSIGN ? free_now - pages : free_now + pages);
  }
}

__global__ __launch_bounds__(kPlanThreads) void assign_plan_kernel(PagesArgs a) { plan_call<true>(a); }
__global__ __launch_bounds__(kPlanThreads) void release_plan_kernel(PagesArgs a) { plan_call<false>(a); }

// Part `part` of `parts` of sequence s: columns of its page table and its tokens' slots, `threads` at a time.
__device__ __forceinline__ void assign_fill(const PagesArgs& a, long long s, int part, int parts, int thread,
                                            int threads) {
  const Plan* plan = static_cast<const Plan*>(a.workspace);
  const int32_t first = a.q_offsets[s], last = a.q_offsets[s + 1];
  const int now = a.kv_lens[s], held = now - (last - first), page = 1 << a.page_shift;
  const int had = (held + page - 1) >> a.page_shift, has = (now + page - 1) >> a.page_shift;
  const int u = a.who ? a.who[s] : static_cast<int>(s);
  int32_t* own = now > 0 ? a.tables + u * a.table_stride : nullptr;  // a user that does not exist holds nothing
  const int32_t* fresh = a.free_pages + (static_cast<long long>(plan->count) - 1 - plan->at[s] + had);
  const auto page_at = [&](int i) { return i < had ? own[i] : fresh[-static_cast<long long>(i)]; };
  int32_t* row = a.page_table + s * a.out_width;
  for (int i = part * threads + thread; i < a.out_width; i += parts * threads) {
    const int32_t p = i < has ? page_at(i) : -1;
    row[i] = p;
    if (i >= had && i < has) own[i] = p;
  }
  for (long long t = static_cast<long long>(part) * threads + thread; t < last - first;
       t += static_cast<long long>(parts) * threads) {
    const int e = held + static_cast<int>(t);
    if (a.slots) {
      const int p = page_at(e >> a.page_shift);
      const bool good = p >= 0 && p < a.num_pages;
      if (!good) flag(a.status, DLRM_STATUS_BAD_PAGE);
      a.slots[first + t] = good ? (static_cast<int64_t>(p) << a.page_shift) + (e & (page - 1)) : -1;
    }
    if (a.positions) a.positions[first + t] = e;
  }
}

// Tokens past the last sequence.
__device__ __forceinline__ void assign_rest(const PagesArgs& a, long long thread, long long threads) {
  for (long long t = a.q_offsets[a.seqs] + thread; t < a.n; t += threads) {
    if (a.slots) a.slots[t] = -1;
    if (a.positions) a.positions[t] = -1;
  }
}

__global__ __launch_bounds__(kFillThreads) void assign_fill_kernel(PagesArgs a) {
  for (long long s = blockIdx.y; s <= a.seqs; s += gridDim.y) {
    if (s < a.seqs)
      assign_fill(a, s, blockIdx.x, gridDim.x, threadIdx.x, kFillThreads);
    else
      assign_rest(a, static_cast<long long>(blockIdx.x) * kFillThreads + threadIdx.x,
                  static_cast<long long>(gridDim.x) * kFillThreads);
  }
}

// A page outside the cache in a user's row would reach another user by way of the free list: the workgroup that meets
// one puts lengths and count back to what they were, the same from every workgroup that does. What the others copied lies
// past the free pages and means nothing then. So the pages are looked at while they are copied, not ahead of it by the
// one workgroup that plans.
__global__ __launch_bounds__(kFillThreads) void release_fill_kernel(PagesArgs a) {
  const Plan* plan = static_cast<const Plan*>(a.workspace);
  if (!plan->ok) return;
  const int page = 1 << a.page_shift;
  bool bad = false;
  for (long long s = blockIdx.y; s < a.seqs; s += gridDim.y) {
    const int held = plan->at[static_cast<long long>(a.seqs) + s];
    const int stay = (kept(a, s, held) + page - 1) >> a.page_shift, has = (held + page - 1) >> a.page_shift;
    const int u = a.who ? a.who[s] : static_cast<int>(s);
    const int32_t* own = a.tables + u * a.table_stride;
    int32_t* to = a.free_pages + plan->count + (static_cast<long long>(plan->at[s]) - stay);
    for (int i = stay + blockIdx.x * kFillThreads + threadIdx.x; i < has; i += gridDim.x * kFillThreads) {
      const int32_t p = own[i];
      bad |= p < 0 || p >= a.num_pages;
      to[i] = p;
    }
  }
  if (!__syncthreads_or(bad)) return;
  if (bad) flag(a.status, DLRM_STATUS_BAD_PAGE);
  for (long long s = threadIdx.x; s < a.seqs; s += kFillThreads)
    a.held_out[a.who ? a.who[s] : s] = plan->at[static_cast<long long>(a.seqs) + s];
  if (threadIdx.x == 0) *a.count_out = plan->count;
}

// Parts of a sequence: as many as take 1024 columns or tokens each, as long as that leaves 4096 workgroups.
dim3 fill_grid(long long rows, long long longest) {
  const long long y = rows < 65535 ? rows : 65535, most = 4096 / y, want = (longest + 1023) / 1024;
  const long long x = want < most ? want : most;
  return dim3(static_cast<unsigned>(x < 1 ? 1 : x), static_cast<unsigned>(y));
}

// Threads of the plan: one to a sequence.
int plan_threads(int seqs) {
  return seqs >= kPlanThreads ? kPlanThreads : seqs <= kWave ? kWave : (seqs + kWave - 1) & ~(kWave - 1);
}

}  // namespace

size_t pages_workspace(int seqs) { return (sizeof(int32_t) * (2 + 2 * static_cast<size_t>(seqs)) + 255) & ~size_t(255); }

hipError_t launch_pages_assign(const PagesArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(assign_plan_kernel, dim3(1), dim3(plan_threads(a.seqs)), 0, s, a);
  const long long longest = a.out_width > a.n ? a.out_width : a.n;
  const dim3 grid = fill_grid(static_cast<long long>(a.seqs) + 1, longest);
  hipLaunchKernelGGL(assign_fill_kernel, grid, dim3(kFillThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_pages_release(const PagesArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(release_plan_kernel, dim3(1), dim3(plan_threads(a.seqs)), 0, s, a);
  if (a.seqs > 0)
    hipLaunchKernelGGL(release_fill_kernel, fill_grid(a.seqs, a.table_width), dim3(kFillThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace dlrm
