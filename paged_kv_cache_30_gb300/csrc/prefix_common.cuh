// prefix_common.cuh -- what the grids of a decode call with shared tokens agree on: how many
// of a group's tokens are read once for all of its rows, and which CTAs take them.  Each CTA
// of prefix_attn.cu and prefix_own.cu works it out for itself from offsets and lengths, as a grid
// for it alone would cost more than the few dependent reads.
#pragma once
#include <limits.h>

#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {

// Groups in shared memory, from plan_groups.
struct GroupPlan {
  const int *cu, *boxes;  // [groups + 1]; shared 16-key boxes [groups]
  int groups;             // 0: none (all requests are on their own)
  int B;

  __device__ __forceinline__ int first() const { return groups ? cu[0] : 0; }
  __device__ __forceinline__ int end() const { return groups ? cu[groups] : B; }
  // the last group that begins at or before request b (-1: none)
  __device__ __forceinline__ int find(int b) const {
    int lo = -1, hi = groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cu[mid] <= b) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
  // request b's group, from that of a request before it
  __device__ __forceinline__ int next(int g, int b) const {
    while (g + 1 < groups && cu[g + 1] <= b) ++g;
    return g;
  }
  // Boxes that request b of group g shares; of one outside of all groups, more than there
  // are, so that it has none of its own.
  __device__ __forceinline__ int shared(int g, int b) const {
    return groups == 0 ? 0 : g < 0 || b >= cu[groups] ? INT_MAX : boxes[g];
  }
};

// Row blocks of group g's units for a kv head.
__device__ __forceinline__ int blocks_of(const PagedParams& p, const GroupPlan& plan, int g) {
  return ((plan.cu[g + 1] - plan.cu[g]) * p.G + kPrefixRows - 1) / kPrefixRows;
}

constexpr int plan_ints(int groups) { return 3 * (groups + 1); }

// Shared tokens are counted in whole pages, at most one token less than the group's shortest
// request that is not empty (so every row sees all of them, and has at least one token behind
// them), and 0 for a group with fewer than two such requests.  (Boxes are 16 tokens.)
//
// mem: plan_ints(groups) ints; lead, with kLead: groups + 1 ints, which get each group's first
// request that is not empty.  All kThreads threads call it.  Offsets that decrease or leave
// [0, B] raise DEVERR_BAD_ROW (report: by this CTA) and no group counts.
template <int kThreads, bool kLead>
__device__ __forceinline__ GroupPlan plan_groups(const PagedParams& p, const PrefixParams& x, int* mem,
                                                 int* lead, bool report) {
  const int tid = threadIdx.x, B = p.B, n = x.groups;
  int *cu = mem, *least = cu + n + 1, *live = least + n + 1;
  const int per = (B + kThreads - 1) / kThreads, b0 = tid * per, b1 = min(b0 + per, B);
  // asked for together
  const int len0 = b0 < B ? __ldg(p.seq_lens + b0) : 0;
  const int shared0 = tid < n ? __ldg(x.shared_lens + tid) : 0;
  bool bad = false;
  for (int i = tid; i <= n; i += kThreads) {
    const int c = __ldg(x.cu_groups + i);
    bad |= c < 0 || c > B || (i < n && __ldg(x.cu_groups + i + 1) < c);
    cu[i] = c;
    least[i] = INT_MAX;
    live[i] = 0;
    if (kLead) lead[i] = INT_MAX;
  }
  if (__syncthreads_or(bad)) {
    if (report && tid == 0) atomicOr(p.err, DEVERR_BAD_ROW);
    return {cu, least, 0, B};
  }
  GroupPlan plan = {cu, least, n, B};
  // a thread's requests are neighbours: one step a group for each
  int g = plan.find(b0), lo = INT_MAX, cnt = 0, one = 0;
  auto note = [&] {
    if (cnt) {
      atomicMin(least + g, lo);
      atomicAdd(live + g, cnt);
      if (kLead) atomicMin(lead + g, one);
    }
    lo = INT_MAX;
    cnt = 0;
  };
#pragma unroll 1
  for (int b = b0; b <= b1; ++b) {
    const int to = b < b1 ? plan.next(g, b) : n;
    if (to != g) note();
    g = to;
    if (b == b1) break;
    const int L = min(b == b0 ? len0 : __ldg(p.seq_lens + b), p.max_blocks * p.page_size);
    if (g < 0 || b >= cu[n] || L <= 0) continue;
    lo = min(lo, L);
    if (cnt++ == 0) one = b;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const int S = i == tid ? shared0 : __ldg(x.shared_lens + i);
    const int pages = live[i] < 2 ? 0 : min(max(S, 0), least[i] - 1) >> p.page_shift;
    least[i] = pages << (p.page_shift - 4);
  }
  __syncthreads();
  return plan;
}

}  // namespace pkv
