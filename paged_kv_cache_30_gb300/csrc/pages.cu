// pages.cu -- the pages of a paged cache: copying, forking, releasing,
// reserving and compacting them on the device.
//
// State: block_table [rows, W] (row b's logical page j is block_table[b][j]),
// seq_lens [rows], and page_refs [num_pages], the number of table entries that
// name each page (0: free).  Row b owns entries [0, ceil(seq_lens[b] / P)); -1 among
// them is a page given back.
// New pages are taken lowest index first, in the order of the call's list, so
// results do not depend on timing.
//
//   fork(p -> c)     c's full pages are p's (refs + 1); a partly filled last page
//                    gets a page of its own, and (source, copy) goes to the list.
//   release(b, n)    entries past ceil(n / P) go (refs - 1, entry -1), length n.
//   trim             entries of pages that a window and first tokens hide go (-1).
//   reserve(b, n)    entries up to ceil(n / P) come (refs = 1), length n.
//   compact          with n live pages, the k-th live page at or above n moves to
//                    the k-th free page below n: sources and targets are disjoint,
//                    so the copies need no order.
//
// Bound by latency (lists of a few hundred entries: launches and two or three
// dependent reads each) except copying, which is bound by memory.  Measured (GB300,
// graph replays): a reservation or fork of a few rows 2.5 to 3 us, a compaction of
// 16384 pages 7 us (three launches; one CTA took 50), copying 4109 pages of 32 KB
// 42.9 us = 6.27 TB/s (the same bytes as one contiguous copy: 40.9).
#include <limits.h>

#include <algorithm>

#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kPlanThreads = 1024;
// Table entries that the planning CTA handles itself: one launch less (about 1 us);
// with more, a CTA for each row is faster (256 forks of 250 entries: 13.8 -> 11.5 us).
constexpr int kOneCtaEntries = 16384;

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
    const T s = lane < (int)(blockDim.x >> 5) ? scratch[lane] : 0;
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

// Bit i: page p + i is free (p a multiple of 16).
__device__ __forceinline__ uint32_t free_pages16(const PageTables& t, int p) {
  uint32_t bits = 0;
  if (p + 16 <= t.num_pages && (reinterpret_cast<uintptr_t>(t.refs) & 15) == 0) {
    const int4* refs = reinterpret_cast<const int4*>(t.refs + p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int4 r = refs[i];
      bits |= (uint32_t)((r.x <= 0) | (r.y <= 0) << 1 | (r.z <= 0) << 2 | (r.w <= 0) << 3) << 4 * i;
    }
  } else {
    for (int i = 0; i < 16; ++i)
      if (p + i < t.num_pages && t.refs[p + i] <= 0) bits |= 1u << i;
  }
  return bits;
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

// Entry i of a fork, by kLanes threads (a warp, or a CTA).
template <int kLanes>
__device__ __forceinline__ void apply_fork(const PageTables& t, const int32_t* children,
                                           const int32_t* parents, int n, int i, int32_t* copy_src,
                                           int32_t* copy_dst, const int* ws) {
  const int lane = threadIdx.x % kLanes, L = ws[8 + n + i];
  int src = -1, dst = -1;
  if (L >= 0) {
    const int full = L / t.page_size, child = children[i];
    const int32_t* from = t.bt + parents[i] * t.bt_sb;
    const bool part = L % t.page_size != 0 && from[full] != -1;
    const bool granted = !part || ws[8 + i] < ws[0];
    int32_t* to = t.bt + child * t.bt_sb;
    if (part && granted) {
      src = from[full];
      dst = ws[8 + 2 * n + ws[8 + i]];
    }
#pragma unroll 4
    for (int j = lane; j < t.max_blocks; j += kLanes) {
      int page = -1;
      if (granted && j < full) {
        page = from[j];
        if (page >= 0 && page < t.num_pages)
          atomicAdd(t.refs + page, 1);
        else if (page != -1)  // a page given back
          atomicOr(t.err, DEVERR_BAD_BLOCK);
      } else if (j == full) {
        page = dst;
      }
      to[j] = page;
    }
    if (lane == 0) {
      if (dst >= 0) t.refs[dst] = 1;
      if (!granted) atomicOr(t.err, DEVERR_NO_PAGE);
      t.seq_lens[child] = granted ? L : 0;
      if (dst >= 0 && (src < 0 || src >= t.num_pages)) {
        atomicOr(t.err, DEVERR_BAD_BLOCK);
        src = -1;
      }
    }
  }
  if (lane == 0) {
    copy_src[i] = src;
    copy_dst[i] = src < 0 ? -1 : dst;
  }
}

// Entry i of a reservation, by kLanes threads.
template <int kLanes>
__device__ __forceinline__ void apply_reserve(const PageTables& t, const int32_t* rows,
                                              const int32_t* lens, int n, int i, const int* ws) {
  const int lane = threadIdx.x % kLanes, need = ws[8 + n + i], base = ws[8 + i];
  if (need < 0) return;
  if (need > 0 && (long long)base + need > ws[0]) {
    if (lane == 0) atomicOr(t.err, DEVERR_NO_PAGE);
    return;
  }
  const int row = rows[i], L = row_len(t, row), have = pages_of(L, t.page_size);
  for (int j = lane; j < need; j += kLanes) {
    const int page = ws[8 + 2 * n + base + j];
    t.refs[page] = 1;
    t.bt[row * t.bt_sb + have + j] = page;
  }
  if (kLanes == 32) __syncwarp(); else __syncthreads();  // every thread has read the length
  if (lane == 0 && lens[i] > L) t.seq_lens[row] = lens[i];
}

// scratch: [0] free pages found, [8 + i] first rank of entry i, [8 + n + i] pages
// it wants (-1: skipped) or, for fork, the parent's length; [8 + 2n + k] the
// free page of rank k.
//
// Fork (rows = children, other = parents) or reserve (rows, other = new lengths):
// which entries get which pages; with `apply` this CTA carries them out too.
template <bool kFork>
__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const PageTables t, const int32_t* rows, const int32_t* other, int n,
                int32_t* copy_src, int32_t* copy_dst, int* ws, bool apply) {
  extern __shared__ int tag[];  // [rows] first entry that names the row; then parent marks
  __shared__ int scratch[33];
  __shared__ long long scratch64[33];
  const int tid = threadIdx.x;
  int* parent = tag + t.rows;
  griddep_wait();
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
        need = note % t.page_size != 0 && t.bt[o * t.bt_sb + note / t.page_size] != -1;
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
  // the free pages of the first `run` ranks, lowest first, 16 a thread
  int found = 0;
  for (int p0 = 0; p0 < t.num_pages && found < run; p0 += 16 * kPlanThreads) {
    const int p = p0 + 16 * tid;
    uint32_t free16 = free_pages16(t, p);
    int total, at = found + block_scan((int)__popc(free16), scratch, &total);
    for (; free16 && at < run; free16 &= free16 - 1) ws[8 + 2 * n + at++] = p + __ffs(free16) - 1;
    found += total;
  }
  if (tid == 0) ws[0] = found;
  if (!apply) return;
  __syncthreads();
  for (int i = tid >> 5; i < n; i += kPlanThreads / 32) {
    if (kFork)
      apply_fork<32>(t, rows, other, n, i, copy_src, copy_dst, ws);
    else
      apply_reserve<32>(t, rows, other, n, i, ws);
  }
}

// Takes entry j of a row and gives its page back; an entry goes once, whoever takes it.
__device__ __forceinline__ void give_back(const PageTables& t, int row, int j) {
  const int page = atomicExch(t.bt + row * t.bt_sb + j, -1);
  if (page < 0 || page >= t.num_pages) {
    if (page != -1) atomicOr(t.err, DEVERR_BAD_BLOCK);
  } else if (atomicSub(t.refs + page, 1) <= 0) {
    atomicAdd(t.refs + page, 1);
    atomicOr(t.err, DEVERR_BAD_ROW);
  }
}

__global__ void release_kernel(const PageTables t, const int32_t* rows, const int32_t* keep) {
  __shared__ int sL;
  griddep_wait();
  const int i = blockIdx.x, tid = threadIdx.x, row = rows[i];
  if (row < 0 || row >= t.rows) {
    if (tid == 0) atomicOr(t.err, DEVERR_BAD_ROW);
    return;
  }
  if (tid == 0) sL = row_len(t, row);
  __syncthreads();
  const int L = sL, k = max(min(keep[i], L), 0);
  for (int j = pages_of(k, t.page_size) + tid; j < pages_of(L, t.page_size); j += blockDim.x)
    give_back(t, row, j);
  if (tid == 0) atomicMin(t.seq_lens + row, k);
}

// Row blockIdx.x: the pages that end at or before its window and begin at or after
// its first tokens.
__global__ void trim_kernel(const PageTables t, int window, int first) {
  griddep_wait();
  const int row = blockIdx.x, L = row_len(t, row), P = t.page_size;
  const int begin = pages_of(first, P), end = (L > window ? L - window : 0) / P;
  for (int j = begin + threadIdx.x; j < end; j += blockDim.x)
    if (t.bt[row * t.bt_sb + j] != -1) give_back(t, row, j);
}

constexpr int kApplyThreads = 128;

template <bool kFork>
__global__ void __launch_bounds__(kApplyThreads)
    apply_kernel(const PageTables t, const int32_t* rows, const int32_t* other, int n,
                 int32_t* copy_src, int32_t* copy_dst, const int* ws) {
  griddep_wait();
  if (kFork)
    apply_fork<kApplyThreads>(t, rows, other, n, blockIdx.x, copy_src, copy_dst, ws);
  else
    apply_reserve<kApplyThreads>(t, rows, other, n, blockIdx.x, ws);
}

// Compaction in three steps over blocks of kBlockPages pages.  With used(p) the
// live pages below p and n = used(num_pages): the live page p >= n is move
// used(p) - used(n), the free page p < n is target p - used(p).
constexpr int kBlockThreads = 256;
constexpr int kBlockPages = 16 * kBlockThreads;

// Live pages of p .. p + 15 as bits.
__device__ __forceinline__ uint32_t live_pages16(const PageTables& t, int p) {
  if (p >= t.num_pages) return 0;
  const uint32_t in = t.num_pages - p >= 16 ? 0xffffu : (1u << (t.num_pages - p)) - 1;
  return ~free_pages16(t, p) & in;
}

// ws[block]: live pages of each block.
__global__ void __launch_bounds__(kBlockThreads) compact_count_kernel(const PageTables t, int* ws) {
  griddep_wait();
  const int p = blockIdx.x * kBlockPages + 16 * threadIdx.x;
  const int c = __popc(live_pages16(t, p));
  __shared__ int sum;
  if (threadIdx.x == 0) sum = 0;
  __syncthreads();
  const int w = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0) atomicAdd(&sum, w);
  __syncthreads();
  if (threadIdx.x == 0) ws[blockIdx.x] = sum;
}

// Lists the moves and targets; ws[blocks + p]: the move of live page p >= n.
__global__ void __launch_bounds__(kBlockThreads)
    compact_list_kernel(const PageTables t, int32_t* copy_src, int32_t* copy_dst, int m,
                        int32_t* num_moves, int* ws) {
  griddep_wait();
  const int tid = threadIdx.x, blocks = gridDim.x;
  __shared__ int sums[3], scratch[33];
  if (tid < 3) sums[tid] = 0;
  __syncthreads();
  // live pages of all blocks, and of the ones before this
  int all = 0, before = 0;
  for (int b = tid; b < blocks; b += kBlockThreads) {
    const int c = ws[b];
    all += c;
    before += b < (int)blockIdx.x ? c : 0;
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  if ((tid & 31) == 0) {
    atomicAdd(&sums[0], all);
    atomicAdd(&sums[1], before);
  }
  __syncthreads();
  const int n = sums[0];
  before = sums[1];
  // used(n): live pages of the blocks before page n's, and of its own below n
  const int nb = n / kBlockPages;
  int below = 0;
  for (int b = tid; b < nb; b += kBlockThreads) below += ws[b];
  {
    const int p = nb * kBlockPages + 16 * tid;
    if (p < n) below += __popc(live_pages16(t, p) & (n - p >= 16 ? 0xffffu : (1u << (n - p)) - 1));
  }
  below = __reduce_add_sync(0xffffffffu, below);
  if ((tid & 31) == 0) atomicAdd(&sums[2], below);
  __syncthreads();
  below = sums[2];
  const int moves = min(n - below, m);

  const int p0 = blockIdx.x * kBlockPages + 16 * tid;
  const uint32_t live = live_pages16(t, p0);
  int total, used = before + block_scan((int)__popc(live), scratch, &total);
  for (int i = 0; i < 16 && p0 + i < t.num_pages; ++i) {
    const int p = p0 + i;
    if (live >> i & 1) {
      if (p >= n) {
        ws[blocks + p] = used - below;
        if (used - below < m) copy_src[used - below] = p;
      }
      ++used;
    } else if (p < n && p - used < m) {
      copy_dst[p - used] = p;
    }
  }
  for (int k = moves + blockIdx.x * kBlockThreads + tid; k < m; k += blocks * kBlockThreads)
    copy_src[k] = copy_dst[k] = -1;
  if (blockIdx.x == 0 && tid == 0) {
    *num_moves = moves;
    ws[blocks + t.num_pages] = n;
  }
}

// CTAs [0, rows): the tables' rows; the others: the counts of the moved pages.
__global__ void __launch_bounds__(kBlockThreads)
    compact_apply_kernel(const PageTables t, const int32_t* copy_src, const int32_t* copy_dst, int m,
                         const int32_t* num_moves, int blocks, const int* ws) {
  griddep_wait();
  const int moves = *num_moves;
  if ((int)blockIdx.x < t.rows) {
    const int n = ws[blocks + t.num_pages];
    const int row = blockIdx.x, used = pages_of(row_len(t, row), t.page_size);
    int32_t* bt = t.bt + row * t.bt_sb;
    for (int j = threadIdx.x; j < used; j += kBlockThreads) {
      const int page = bt[j];
      if (page < 0 || page >= t.num_pages) {
        if (page != -1) atomicOr(t.err, DEVERR_BAD_BLOCK);
      } else if (page >= n) {
        // a page with no count is no one's: its entry stays, as the page does
        const int k = ws[blocks + page];
        if (k >= 0 && k < moves && copy_src[k] == page) bt[j] = copy_dst[k];
      }
    }
  } else {
    for (int k = (blockIdx.x - t.rows) * kBlockThreads + threadIdx.x; k < moves;
         k += (gridDim.x - t.rows) * kBlockThreads) {
      t.refs[copy_dst[k]] = t.refs[copy_src[k]];
      t.refs[copy_src[k]] = 0;
    }
  }
}

// A CTA copies pieces of kCopyPiece bytes of the listed pages of one tensor, eight
// 16-byte loads of a thread in flight (compaction of half of 16384 pages: 53.7 us; with
// four 58.9).
constexpr int kCopyThreads = 128;
constexpr int kCopyLoads = 8;
constexpr int64_t kCopyPiece = kCopyThreads * kCopyLoads * 16;

template <typename V>
__device__ __forceinline__ void copy_piece(uint8_t* to, const uint8_t* from, int64_t bytes) {
  // kCopyLoads loads of a thread are in flight at once
  for (int64_t k0 = threadIdx.x * sizeof(V); k0 < bytes; k0 += kCopyThreads * kCopyLoads * sizeof(V)) {
    V v[kCopyLoads];
#pragma unroll
    for (int i = 0; i < kCopyLoads; ++i) {
      const int64_t k = k0 + i * kCopyThreads * (int64_t)sizeof(V);
      if (k < bytes) v[i] = *reinterpret_cast<const V*>(from + k);
    }
#pragma unroll
    for (int i = 0; i < kCopyLoads; ++i) {
      const int64_t k = k0 + i * kCopyThreads * (int64_t)sizeof(V);
      if (k < bytes) *reinterpret_cast<V*>(to + k) = v[i];
    }
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ PagesCopyParams p) {
  griddep_wait();
  const PagesCopyTensor& t = p.t[blockIdx.y];
  const int64_t pieces = (t.bytes + kCopyPiece - 1) / kCopyPiece;
  const bool wide = ((reinterpret_cast<uintptr_t>(t.base) | t.stride | t.bytes) & 15) == 0;
  for (int64_t u = blockIdx.x; u < pieces * p.n; u += gridDim.x) {
    const int64_t i = pieces == 1 ? u : u / pieces, at = (u - i * pieces) * kCopyPiece;
    const int s = __ldg(p.src + i), d = __ldg(p.dst + i);
    if (s < 0 || d < 0) continue;
    if (s >= t.num_pages || d >= t.num_pages) {
      if (threadIdx.x == 0) atomicOr(p.err, DEVERR_BAD_BLOCK);
      continue;
    }
    const uint8_t* from = t.base + s * t.stride + at;
    uint8_t* to = t.base + d * t.stride + at;
    const int64_t bytes = min(kCopyPiece, (int64_t)(t.bytes - at));
    if (wide)
      copy_piece<uint4>(to, from, bytes);
    else
      copy_piece<uint32_t>(to, from, bytes);
  }
}

// Every kernel here launches as a programmatic dependent and reads nothing of the
// caller's before its wait.
template <typename... P, typename... A>
cudaError_t launch(void (*fn)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, A... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(a)...);
}

}  // namespace

cudaError_t launch_pages_copy(const PagesCopyParams& p, int num_sms, cudaStream_t stream) {
  int64_t units = 0;
  for (int i = 0; i < p.num_tensors; ++i)
    units = std::max(units, (p.t[i].bytes + kCopyPiece - 1) / kCopyPiece * p.n);
  return launch(copy_kernel, dim3((unsigned)std::min<int64_t>(units, 16 * num_sms), p.num_tensors),
                kCopyThreads, 0, stream, p);
}

// One launch when the planning CTA can do the rest too, else two.
template <bool kFork>
static cudaError_t plan_and_apply(const PageTables& t, const int32_t* rows, const int32_t* other,
                                  int n, int32_t* copy_src, int32_t* copy_dst, int* scratch,
                                  cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_smem_attr_once(plan_kernel<kFork>, kPagesMaxRows * 8, done);
  if (e != cudaSuccess) return e;
  const bool apply = (int64_t)n * t.max_blocks <= kOneCtaEntries;
  e = launch(plan_kernel<kFork>, dim3(1), kPlanThreads, t.rows * (kFork ? 8 : 4), stream, t, rows,
             other, n, copy_src, copy_dst, scratch, apply);
  if (e != cudaSuccess || apply) return e;
  return launch(apply_kernel<kFork>, dim3(n), kApplyThreads, 0,
                stream, t, rows, other, n, copy_src, copy_dst, scratch);
}

cudaError_t launch_pages_fork(const PageTables& t, const int32_t* parents, const int32_t* children,
                              int n, int32_t* copy_src, int32_t* copy_dst, int* scratch,
                              cudaStream_t stream) {
  return plan_and_apply<true>(t, children, parents, n, copy_src, copy_dst, scratch, stream);
}

cudaError_t launch_pages_release(const PageTables& t, const int32_t* rows, const int32_t* keep,
                                 int n, cudaStream_t stream) {
  return launch(release_kernel, dim3(n), 64, 0, stream, t, rows, keep);
}

cudaError_t launch_pages_trim(const PageTables& t, int window, int first, cudaStream_t stream) {
  return launch(trim_kernel, dim3(t.rows), 128, 0, stream, t, window, first);
}

cudaError_t launch_pages_reserve(const PageTables& t, const int32_t* rows, const int32_t* lens,
                                 int n, int* scratch, cudaStream_t stream) {
  return plan_and_apply<false>(t, rows, lens, n, nullptr, nullptr, scratch, stream);
}

cudaError_t launch_pages_compact(const PageTables& t, int32_t* copy_src, int32_t* copy_dst, int n,
                                 int32_t* num_moves, int* scratch, cudaStream_t stream) {
  const int blocks = (t.num_pages + kBlockPages - 1) / kBlockPages;
  cudaError_t e = launch(compact_count_kernel, dim3(blocks), kBlockThreads, 0, stream, t, scratch);
  if (e != cudaSuccess) return e;
  e = launch(compact_list_kernel, dim3(blocks), kBlockThreads, 0, stream, t, copy_src, copy_dst, n,
             num_moves, scratch);
  if (e != cudaSuccess) return e;
  const int movers = std::max(1, std::min(64, n / kBlockThreads));
  return launch(compact_apply_kernel, dim3(t.rows + movers), kBlockThreads, 0, stream, t, copy_src,
                copy_dst, n, num_moves, blocks, scratch);
}

}  // namespace pkv
