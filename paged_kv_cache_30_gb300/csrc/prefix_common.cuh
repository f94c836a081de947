// prefix_common.cuh -- what the two grids of a decode call with shared tokens agree on:
// how many of a group's tokens are read once for all of its rows, and where the parts of
// a row lie.
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

// Shared tokens are counted in whole boxes of 16, at most one token less than the group's
// shortest request that is not empty (so every row sees all of them, and has at least one
// token behind them), and 0 for a group with fewer than two such requests.
// scratch: 3 (groups + 1) ints.  All kThreads threads call it.  Offsets that decrease or
// leave [0, B] raise DEVERR_BAD_ROW (report: by this CTA) and no group counts.
template <int kThreads>
__device__ __forceinline__ GroupPlan plan_groups(const PagedParams& p, const PrefixParams& x,
                                                 int* scratch, bool report) {
  const int tid = threadIdx.x, B = p.B, n = x.groups;
  int *cu = scratch, *least = cu + n + 1, *live = least + n + 1;
  bool bad = false;
  for (int i = tid; i <= n; i += kThreads) {
    const int c = __ldg(x.cu_groups + i);
    bad |= c < 0 || c > B || (i < n && __ldg(x.cu_groups + i + 1) < c);
    cu[i] = c;
    if (i < n) {
      least[i] = INT_MAX;
      live[i] = 0;
    }
  }
  if (__syncthreads_or(bad)) {
    if (report && tid == 0) atomicOr(p.err, DEVERR_BAD_ROW);
    return {cu, least, 0, B};
  }
  GroupPlan plan = {cu, least, n, B};
  // a thread's requests are neighbours: one step a group for each
  const int per = (B + kThreads - 1) / kThreads, b0 = tid * per, b1 = min(b0 + per, B);
  int g = plan.find(b0), lo = INT_MAX, cnt = 0;
  for (int b = b0; b < b1; ++b) {
    const int to = plan.next(g, b);
    if (to != g && cnt) {
      atomicMin(least + g, lo);
      atomicAdd(live + g, cnt);
    }
    if (to != g) lo = INT_MAX, cnt = 0;
    g = to;
    const int L = min(__ldg(p.seq_lens + b), p.max_blocks * p.page_size);
    if (g < 0 || b >= cu[n] || L <= 0) continue;
    lo = min(lo, L);
    ++cnt;
  }
  if (cnt) {
    atomicMin(least + g, lo);
    atomicAdd(live + g, cnt);
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const int tokens = live[i] < 2 ? 0 : min(max(__ldg(x.shared_lens + i), 0), least[i] - 1);
    least[i] = tokens >> 4;
  }
  __syncthreads();
  return plan;
}

// A row's parts, first to last.  Units of a group are laid end to end in the space of costs:
// kPrefixUnitCost and its boxes each; CTA c takes places [c share, (c + 1) share), whole
// tiles whose first box lies in them, so a unit's parts are those of the CTAs from the one
// that holds the end of its first tile to the one that holds its end.
struct SharedParts {
  const float4 *first_o, *rest_o;    // of row quad 0
  const float2 *first_ml, *rest_ml;
  int64_t first_step, rest_cta;      // from quad to quad; from CTA to CTA
  int n;

  __device__ __forceinline__ const float2* ml(int i) const {
    return i == 0 ? first_ml : rest_ml + (int64_t)i * kPrefixRows;
  }
  __device__ __forceinline__ const float4* o(int i, int quad) const {
    return i == 0 ? first_o + quad * first_step
                  : rest_o + i * rest_cta + (int64_t)quad * kPrefixRows;
  }
  __device__ __forceinline__ const float* at(int i, int d) const {
    return reinterpret_cast<const float*>(o(i, d >> 2)) + (d & 3);
  }
};

// begin: the unit's place; the CTAs that have a part of it
__device__ __forceinline__ int first_cta(int begin, int boxes, int share) {
  return (begin + kPrefixUnitCost + min(boxes, kPrefixTileKeys / 16) - 1) / share;
}
__device__ __forceinline__ int last_cta(int begin, int boxes, int share) {
  return (begin + kPrefixUnitCost + boxes - 1) / share;
}

template <int D>
__device__ __forceinline__ SharedParts shared_parts(const PagedParams& p, const PrefixParams& x,
                                                    int b, int kvh, int h) {
  SharedParts s = {};
  const int4 at = __ldcg(x.info + 2 * b);
  if (at.z == 0) return s;
  const int blocks = __ldcg(x.info + 2 * b + 1).x;
  const int row = (b - at.x) * p.G + h, block = row / kPrefixRows;
  const int begin = at.y + (kvh * blocks + block) * (kPrefixUnitCost + at.z);
  const int c0 = first_cta(begin, at.z, at.w);
  const int64_t rows = (int64_t)p.B * p.G, mine = (int64_t)b * p.G + h;
  s.n = last_cta(begin, at.z, at.w) - c0 + 1;
  s.first_o = x.first_o + kvh * (D / 4) * rows + mine;
  s.first_ml = x.first_ml + kvh * rows + mine;
  s.first_step = rows;
  s.rest_cta = (int64_t)(D / 4) * kPrefixRows;
  s.rest_o = x.rest_o + c0 * s.rest_cta + row % kPrefixRows;
  s.rest_ml = x.rest_ml + (int64_t)c0 * kPrefixRows + row % kPrefixRows;
  return s;
}

}  // namespace pkv
