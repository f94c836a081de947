// pages.cu -- the pages of a paged cache: copying, forking, releasing,
// reserving and compacting them on the device.
//
// State: block_table [rows, W] (row b's logical page j is block_table[b][j]),
// seq_lens [rows], and page_refs [num_pages], the number of table entries that
// name each page (0: free).  Row b owns entries [0, ceil(seq_lens[b] / P)).
// New pages are taken lowest index first, in the order of the call's list, so
// results do not depend on timing.
//
//   fork(p -> c)     c's full pages are p's (refs + 1); a partly filled last page
//                    gets a page of its own, and (source, copy) goes to the list.
//   release(b, n)    entries past ceil(n / P) go (refs - 1, entry -1), length n.
//   reserve(b, n)    entries up to ceil(n / P) come (refs = 1), length n.
//   compact          with n live pages, the k-th live page at or above n moves to
//                    the k-th free page below n: sources and targets are disjoint,
//                    so the copies need no order.
//
// Bound by latency (lists of a few hundred entries) except copying, which is
// bound by memory.
#include <limits.h>

#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// Exclusive scan over the CTA; *total = the sum.
template <typename T>
__device__ T block_scan(T v, T* scratch, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const T s = scratch[lane];
    T t = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T n = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += n;
    }
    scratch[lane] = t - s;
    if (lane == 31) scratch[32] = t;
  }
  __syncthreads();
  const T res = scratch[warp] + incl - v;
  *total = scratch[32];
  __syncthreads();
  return res;
}

__device__ __forceinline__ int pages_of(long long len, int P) { return (int)((len + P - 1) / P); }

// The length of a row, clamped to what its table holds.
__device__ __forceinline__ int row_len(const PageTables& t, int row) {
  const int L = max(t.seq_lens[row], 0);
  if (L > (long long)t.max_blocks * t.page_size) {
    atomicOr(t.err, DEVERR_SEQ_TOO_LONG);
    return t.max_blocks * t.page_size;
  }
  return L;
}

// scratch: [0] free pages found, [8 + i] first rank of entry i, [8 + n + i] pages
// it wants (-1: skipped) or, for fork, the parent's length; [8 + 2n + k] the
// free page of rank k.
//
// Fork (rows = children, other = parents) or reserve (rows, other = new lengths).
template <bool kFork>
__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const PageTables t, const int32_t* rows, const int32_t* other, int n, int* ws) {
  extern __shared__ int tag[];  // [rows] first entry that names the row; then parent marks
  __shared__ int scratch[33];
  __shared__ long long scratch64[33];
  const int tid = threadIdx.x;
  int* parent = tag + t.rows;
  for (int i = tid; i < t.rows; i += kPlanThreads) {
    tag[i] = INT_MAX;
    if (kFork) parent[i] = 0;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int r = rows[i];
    if (r >= 0 && r < t.rows) atomicMin(&tag[r], i);
    if (kFork) {
      const int q = other[i];
      if (q >= 0 && q < t.rows) parent[q] = 1;
    }
  }
  __syncthreads();
  long long run = 0;  // all rows of a table may want all of it
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int need = 0, note = -1;
    if (i < n) {
      const int r = rows[i], o = other[i];
      // each row once; a fork's child is empty and no one's parent
      bool ok = r >= 0 && r < t.rows && tag[r] == i;
      if (kFork) ok = ok && o >= 0 && o < t.rows && !parent[r] && t.seq_lens[r] <= 0;
      if (!ok) {
        atomicOr(t.err, DEVERR_BAD_ROW);
      } else if (kFork) {
        note = row_len(t, o);
        need = note % t.page_size != 0;
      } else {
        const int L = row_len(t, r);
        if (o > (long long)t.max_blocks * t.page_size)
          atomicOr(t.err, DEVERR_SEQ_TOO_LONG);
        else
          note = need = max(pages_of(o, t.page_size) - pages_of(L, t.page_size), 0);
      }
    }
    long long total;
    const long long base = run + block_scan((long long)need, scratch64, &total);
    if (i < n) {
      ws[8 + i] = (int)min(base, (long long)INT_MAX);
      ws[8 + n + i] = note;
    }
    run += total;
  }
  // the free pages of the first `run` ranks, lowest first
  int found = 0;
  for (int p0 = 0; p0 < t.num_pages && found < run; p0 += 4 * kPlanThreads) {
    const int p = p0 + 4 * tid;
    int free4[4], c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      free4[k] = p + k < t.num_pages && t.refs[p + k] == 0;
      c += free4[k];
    }
    int total;
    int at = found + block_scan(c, scratch, &total);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (free4[k]) {
        if (at < run) ws[8 + 2 * n + at] = p + k;
        ++at;
      }
    }
    found += total;
  }
  if (tid == 0) ws[0] = found;
}

__global__ void fork_kernel(const PageTables t, const int32_t* parents, const int32_t* children,
                            int n, int32_t* copy_src, int32_t* copy_dst, const int* ws) {
  const int i = blockIdx.x, tid = threadIdx.x;
  int L = ws[8 + n + i], src = -1, dst = -1;
  if (L >= 0) {
    const int full = L / t.page_size;
    const bool part = L % t.page_size != 0;
    const bool granted = !part || ws[8 + i] < ws[0];
    const int32_t* from = t.bt + parents[i] * t.bt_sb;
    int32_t* to = t.bt + children[i] * t.bt_sb;
    if (part && granted) {
      src = from[full];
      dst = ws[8 + 2 * n + ws[8 + i]];
    }
    for (int j = tid; j < t.max_blocks; j += blockDim.x) {
      int page = -1;
      if (granted && j < full) {
        page = from[j];
        if (page >= 0 && page < t.num_pages)
          atomicAdd(t.refs + page, 1);
        else
          atomicOr(t.err, DEVERR_BAD_BLOCK);
      } else if (j == full) {
        page = dst;
      }
      to[j] = page;
    }
    if (tid == 0) {
      if (dst >= 0) t.refs[dst] = 1;
      if (!granted) atomicOr(t.err, DEVERR_NO_PAGE);
      t.seq_lens[children[i]] = granted ? L : 0;
      if (dst >= 0 && (src < 0 || src >= t.num_pages)) {
        atomicOr(t.err, DEVERR_BAD_BLOCK);
        src = -1;
      }
    }
  }
  if (tid == 0) {
    copy_src[i] = src;
    copy_dst[i] = src < 0 ? -1 : dst;
  }
}

__global__ void release_kernel(const PageTables t, const int32_t* rows, const int32_t* keep) {
  __shared__ int sL;
  const int i = blockIdx.x, tid = threadIdx.x, row = rows[i];
  if (row < 0 || row >= t.rows) {
    if (tid == 0) atomicOr(t.err, DEVERR_BAD_ROW);
    return;
  }
  if (tid == 0) sL = row_len(t, row);
  __syncthreads();
  const int L = sL, k = max(min(keep[i], L), 0);
  // an entry goes once, whoever takes it
  for (int j = pages_of(k, t.page_size) + tid; j < pages_of(L, t.page_size); j += blockDim.x) {
    const int page = atomicExch(t.bt + row * t.bt_sb + j, -1);
    if (page < 0 || page >= t.num_pages) {
      if (page != -1) atomicOr(t.err, DEVERR_BAD_BLOCK);
    } else if (atomicSub(t.refs + page, 1) <= 0) {
      atomicAdd(t.refs + page, 1);
      atomicOr(t.err, DEVERR_BAD_ROW);
    }
  }
  if (tid == 0) atomicMin(t.seq_lens + row, k);
}

__global__ void reserve_kernel(const PageTables t, const int32_t* rows, const int32_t* lens, int n,
                               const int* ws) {
  const int i = blockIdx.x, tid = threadIdx.x, need = ws[8 + n + i];
  if (need < 0) return;
  const int row = rows[i], base = ws[8 + i];
  if (need > 0 && (long long)base + need > ws[0]) {
    if (tid == 0) atomicOr(t.err, DEVERR_NO_PAGE);
    return;
  }
  const int L = row_len(t, row), have = pages_of(L, t.page_size);
  for (int j = tid; j < need; j += blockDim.x) {
    const int page = ws[8 + 2 * n + base + j];
    t.refs[page] = 1;
    t.bt[row * t.bt_sb + have + j] = page;
  }
  __syncthreads();
  if (tid == 0 && lens[i] > L) t.seq_lens[row] = lens[i];
}

// One CTA: the moves, and each page's new index in ws.
__global__ void __launch_bounds__(kPlanThreads)
    compact_kernel(const PageTables t, int32_t* copy_src, int32_t* copy_dst, int n,
                   int32_t* num_moves, int* ws) {
  __shared__ int scratch[33];
  const int tid = threadIdx.x;
  int c = 0, live;
  for (int p = tid; p < t.num_pages; p += kPlanThreads) c += t.refs[p] > 0;
  block_scan(c, scratch, &live);
  int nsrc = 0, ndst = 0;
  for (int p0 = 0; p0 < t.num_pages; p0 += kPlanThreads) {
    const int p = p0 + tid;
    const bool in = p < t.num_pages, used = in && t.refs[p] > 0;
    const int is_src = used && p >= live, is_dst = in && !used && p < live;
    int total_src, total_dst;
    const int at_src = nsrc + block_scan(is_src, scratch, &total_src);
    const int at_dst = ndst + block_scan(is_dst, scratch, &total_dst);
    if (is_src && at_src < n) copy_src[at_src] = p;
    if (is_dst && at_dst < n) copy_dst[at_dst] = p;
    if (in) ws[p] = p;
    nsrc += total_src;
    ndst += total_dst;
  }
  __syncthreads();
  const int moves = min(nsrc, n);
  for (int k = tid; k < n; k += kPlanThreads) {
    if (k < moves) {
      const int s = copy_src[k], d = copy_dst[k];
      t.refs[d] = t.refs[s];
      t.refs[s] = 0;
      ws[s] = d;
    } else {
      copy_src[k] = copy_dst[k] = -1;
    }
  }
  if (tid == 0) *num_moves = moves;
}

__global__ void remap_kernel(const PageTables t, const int* to) {
  const int row = blockIdx.x, used = pages_of(row_len(t, row), t.page_size);
  int32_t* bt = t.bt + row * t.bt_sb;
  for (int j = threadIdx.x; j < used; j += blockDim.x) {
    const int page = bt[j];
    if (page >= 0 && page < t.num_pages)
      bt[j] = to[page];
    else
      atomicOr(t.err, DEVERR_BAD_BLOCK);
  }
}

__global__ void copy_kernel(const __grid_constant__ PagesCopyParams p) {
  const PagesCopyTensor& t = p.t[blockIdx.y];
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const int s = p.src[i], d = p.dst[i];
    if (s < 0 || d < 0) continue;
    if (s >= t.num_pages || d >= t.num_pages) {
      if (threadIdx.x == 0) atomicOr(p.err, DEVERR_BAD_BLOCK);
      continue;
    }
    const uint8_t* from = t.base + s * t.stride;
    uint8_t* to = t.base + d * t.stride;
    for (int64_t k = threadIdx.x * 4; k < t.bytes; k += blockDim.x * 4)
      *reinterpret_cast<uint32_t*>(to + k) = *reinterpret_cast<const uint32_t*>(from + k);
  }
}

}  // namespace

cudaError_t launch_pages_copy(const PagesCopyParams& p, int num_sms, cudaStream_t stream) {
  const int grid = p.n < 8 * num_sms ? p.n : 8 * num_sms;
  copy_kernel<<<dim3(grid, p.num_tensors), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PageTables& t, const int32_t* parents, const int32_t* children,
                              int n, int32_t* copy_src, int32_t* copy_dst, int* scratch,
                              cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_smem_attr_once(plan_kernel<true>, kPagesMaxRows * 8, done);
  if (e != cudaSuccess) return e;
  plan_kernel<true><<<1, kPlanThreads, t.rows * 8, stream>>>(t, children, parents, n, scratch);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  fork_kernel<<<n, 256, 0, stream>>>(t, parents, children, n, copy_src, copy_dst, scratch);
  return cudaGetLastError();
}

cudaError_t launch_pages_release(const PageTables& t, const int32_t* rows, const int32_t* keep,
                                 int n, cudaStream_t stream) {
  release_kernel<<<n, 64, 0, stream>>>(t, rows, keep);
  return cudaGetLastError();
}

cudaError_t launch_pages_reserve(const PageTables& t, const int32_t* rows, const int32_t* lens,
                                 int n, int* scratch, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_smem_attr_once(plan_kernel<false>, kPagesMaxRows * 8, done);
  if (e != cudaSuccess) return e;
  plan_kernel<false><<<1, kPlanThreads, t.rows * 4, stream>>>(t, rows, lens, n, scratch);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  reserve_kernel<<<n, 64, 0, stream>>>(t, rows, lens, n, scratch);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PageTables& t, int32_t* copy_src, int32_t* copy_dst, int n,
                                 int32_t* num_moves, int* scratch, cudaStream_t stream) {
  compact_kernel<<<1, kPlanThreads, 0, stream>>>(t, copy_src, copy_dst, n, num_moves, scratch);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  remap_kernel<<<t.rows, 128, 0, stream>>>(t, scratch);
  return cudaGetLastError();
}

}  // namespace pkv
