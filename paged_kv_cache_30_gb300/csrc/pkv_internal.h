// pkv_internal.h -- declarations shared by the host launcher (api.cpp) and the
// kernel translation units.  Not part of the public ABI.
#pragma once
#include <cuda.h>

#include <atomic>
#include <cuda_runtime.h>
#include <stdint.h>

struct pkv_tensor;  // include/pkv.h

namespace pkv {

// Device-side error bits, OR-ed into the workspace error word and read back by
// pkv_check_errors().
enum : int {
  DEVERR_BAD_BLOCK = 1,      // a block-table entry outside [0, num_blocks)
  DEVERR_SEQ_TOO_LONG = 2,   // seq_len needs more pages than the block table holds
  DEVERR_WAIT_TIMEOUT = 4,   // a pipeline wait gave up (the kernel drained and returned)
  DEVERR_ITEM_OVERFLOW = 8,  // more work items than the workspace holds
  DEVERR_QUEUE = 16,         // a CTA drew more items than the launch has (it stopped)
  DEVERR_NO_PAGE = 32,       // the page pool ran out: a row was not forked or extended
  DEVERR_BAD_ROW = 64,       // a bad row list or reference count (the entry was skipped)
};

// Per-device workspace carved out of one allocation (see api.cpp).
struct Workspace {
  void* base = nullptr;
  size_t bytes = 0;
  float* partials = nullptr;  // split partials, reused by both paths
  size_t partial_bytes = 0;
  int* counters = nullptr;    // self-resetting arrival counters
  int64_t num_counters = 0;
  int* sched = nullptr;       // [0] work-queue head (self-resetting)
  int* err = nullptr;         // device error word
  int num_sms = 0;
};

// ---------------------------------------------------------------- GQA --
constexpr int kGqaHeadDim = 128;
constexpr int kGqaGroup = 8;         // query heads per kv head
constexpr int kGqaMaxBatch = 2048;   // requests per call (device-side scheduler table)
constexpr int kGqaPartialFloats = kGqaGroup * kGqaHeadDim;  // O partial of one work item
constexpr int kGqaMlFloats = 2 * kGqaGroup;                 // m[8], l[8] of one work item

struct GqaParams {
  const uint16_t* q;  // bf16 [B, Hq, 128]
  int64_t q_sb, q_sh;
  const int32_t* bt;
  int64_t bt_sb;
  int max_blocks;
  int num_blocks;
  const int32_t* seq_lens;
  const float* sinks;  // [Hq] or null
  uint16_t* out;       // bf16 [B, Hq, 128]
  int64_t o_sb, o_sh;
  float* lse;          // [B, Hq] or null
  int64_t lse_sb, lse_sh;
  int B, Hkv;
  int window;          // <= 0: all keys
  float scale_log2;    // scale * log2(e)
  float scale;
  int cap;             // max splits per (request, kv head)
  int min_pages;       // fewest pages a split may hold
  int target_items;    // desired number of work items per launch
  float* part_o;       // [max_items][8][128]
  float* part_ml;      // [max_items][16]
  int64_t max_items;
  int* counters;       // [B * Hkv] arrival counters of the last merge level
  int* group_counters; // [max_items] arrival counters of split groups (by first item)
  int* sched;
  int* err;
  int cluster;         // > 1: cluster mode with this many splits per cluster (see below)
};

// Launch the GQA decode kernel for page size 16 or 32.  p.cluster <= 1: the
// persistent kernel on `grid` CTAs.  p.cluster = C in [2, 8]: the cluster
// mode, grid (C, B * Hkv) in clusters of C CTAs, CTA r of a cluster taking
// split r of one (request, kv head); the splits merge through distributed
// shared memory (no workspace partials, counters or queue).
cudaError_t launch_gqa_decode(const GqaParams& p, const CUtensorMap& kv_map, int page_size,
                              int grid, cudaStream_t stream);
constexpr int kGqaMaxCluster = 8;
int gqa_ctas_per_sm();

// A validated GQA decode call: kernel parameters (without workspace pointers)
// and the KV-cache tensor map.
struct GqaCall {
  GqaParams p;
  CUtensorMap map;  // CUtensorMap carries its own 64-byte alignment
  int64_t pairs;   // B * Hkv
  int cap_req;     // num_kv_splits as given (0 = library's choice)
  int page_size;
  int device;      // the device holding q (current, and the stream's device)
};

// Defined in api.cpp, for entry points implemented in other files.
// Validates every argument (shapes, dtypes, strides, alignment, overlap of
// outputs with inputs, the device of q against the current device and the
// stream's) and fills `call`; B == 0 returns PKV_OK with call->pairs == 0
// before any CUDA call.
int prepare_gqa_call(const ::pkv_tensor* q, const ::pkv_tensor* kv_cache,
                     const ::pkv_tensor* block_table, const ::pkv_tensor* seq_lens,
                     const ::pkv_tensor* sinks, int window, float scale, int page_size,
                     int num_kv_splits, const ::pkv_tensor* out, const ::pkv_tensor* lse,
                     cudaStream_t stream, GqaCall* call);

// Launch shape of a GQA decode call on scratch that holds max_items split
// partials and max_pairs (request, kv head) counters: the split cap (0 = the
// most that fit, at most 256), the grid (CTAs per SM x SMs, or fewer for
// small calls) and the kernel's target item count.  PKV_ERR_WORKSPACE when
// the call does not fit.  Every entry point launching the GQA kernel uses it.
struct GqaShape {
  int cap, grid, target_items;
  int cluster;    // > 1: cluster mode with this many splits per (request, kv head) at most
  int min_pages;  // fewest pages a split may hold
};
int gqa_launch_shape(int64_t pairs, int cap_req, int64_t max_items, int64_t max_pairs,
                     int num_sms, int max_blocks, int page_size, GqaShape* shape);
// Device address of the error word of pkv_paged_decode_attn_noalloc's static
// scratch on `device`, or null before that device's first such call.
int* noalloc_error_word(int device);
int abi_fail(int code, const char* message);
int abi_cuda_fail(cudaError_t e, const char* what);

// ---------------------------------------------------------------- MLA --
constexpr int kMlaHeads = 128;
constexpr int kMlaLk = 576;
constexpr int kMlaLv = 512;
constexpr int kMlaHalf = kMlaLv / 2;        // output dims per CTA
constexpr int kMlaTile = 32;                // keys per pipeline tile
constexpr int kMlaMinTiles = 128;           // a split holds at least 4096 keys
// CTA-pair launches split more coarsely (6144 keys) when the batch still has
// a unit for every CTA pair at that size: each unit costs ~8 us of start,
// query load and merge on top of its tiles, and on B = 32 qlen 4 batches
// (lengths U[512, 8192], four seeds, same process) 128 -> 192 measured
// 223.2 / 221.2 / 221.2 / 202.8 -> 200.7 / 210.9 / 200.7 / 184.3 us.
constexpr int kMlaMinTilesWide = 192;
constexpr int64_t kMlaPartialFloats = int64_t(kMlaHeads) * kMlaHalf + 2 * kMlaHeads;

struct MlaParams {
  const uint16_t* q;             // bf16 [B*qlen, 128, 576]
  int64_t q_sr, q_sh;
  const uint8_t* kv;             // latent cache base
  int64_t kv_stok, kv_spage;     // token / page strides in bytes
  const int32_t* bt;
  int64_t bt_sb;
  int max_blocks;
  int num_pages;
  const int32_t* seq_lens;
  const int32_t* real_seq_lens;  // or null
  const float* k_scale;          // device scalar or null (FP8 only)
  uint16_t* out;                 // bf16 [B*qlen, 128, 512]
  int64_t o_sr, o_sh;
  float* lse;                    // [B*qlen, 128]
  int64_t lse_sr, lse_sh;
  int B, qlen, cap, page_size;
  float scale;
  int pair_slots;                // CTA pairs that run at once (SMs / 2)
  float* partials;               // [slots][128*256 + 256]
  int64_t max_slots;
  int* counters;                 // [(b*qlen + t)*2 + half]
  int* plan;                     // [grid] unit of each CTA (written by the planning kernel)
  int* err;
  // native FP8 (e4m3 query): codes [B*qlen, 128, 576] and fp32 scales [B*qlen, 128]
  const uint8_t* q8;
  int64_t q8_sr, q8_sh;
  const float* q_scale;
  int64_t qs_sr, qs_sh;
};

// The planning kernel: writes p.plan[0, grid) (one CTA; programmatic dependent
// launch): one entry per verify CTA, or with `pair` one per CTA pair (a pair
// takes two consecutive verify tokens).
cudaError_t launch_mla_plan(const MlaParams& p, int grid, cudaStream_t stream, bool pair);
// bf16 latent cache, even qlen: the planning kernel, then the verify kernel on
// CTA pairs (grid CTAs, clusters of 2; v_map: the cache as (64 dims, token,
// 9 chunks, page) with a box of (64, 16, 2, 1), 128-byte swizzle).
cudaError_t launch_mla_verify_pair(const MlaParams& p, const CUtensorMap& q_map,
                                   const CUtensorMap& kv_map, const CUtensorMap& v_map, int grid,
                                   cudaStream_t stream);
cudaError_t launch_mla_verify(const MlaParams& p, const CUtensorMap& q_map,
                              const CUtensorMap& kv_map, bool fp8, int grid, cudaStream_t stream);
// Native FP8: planning kernel, then the verify kernel with S = Q8 K8^T on
// kind::f8f6f4 (kv_map: the e4m3 cache as (64 dims, token, 9 chunks, page) with
// a box of (64, 8, 9, 1) and 64-byte swizzle).
cudaError_t launch_mla_verify_native(const MlaParams& p, const CUtensorMap& kv_map, int grid,
                                     cudaStream_t stream);

// Per-(row, head) e4m3 quantisation of an MLA query: scale = absmax / 448,
// code = e4m3(q / scale) (round to nearest even, saturating).
struct QuantParams {
  const uint16_t* q;      // bf16 [R, H, 576]
  int64_t q_sr, q_sh;     // element strides
  uint8_t* q8;            // [R, H, 576], row stride q8_sr, head stride 576
  int64_t q8_sr;
  float* q_scale;         // [R, H], row stride qs_sr, head stride 1
  int64_t qs_sr;
  int R, H;
};
cudaError_t launch_mla_quantize_q(const QuantParams& p, cudaStream_t stream);

// ---------------------------------------------------------- KV append --
struct AppendParams {
  const uint16_t* k;     // GQA: k [B, Hkv, 128]; MLA: latent [B*qlen, 576]
  const uint16_t* v;     // GQA: v [B, Hkv, 128]; MLA: unused
  int64_t s_sb, s_sh;    // source strides (elements): GQA [b, h]; MLA [row, -]
  uint8_t* cache;        // cache base
  int64_t c_sblk, c_sh, c_stok;  // bytes: block/page, kv head (GQA), token
  int num_blocks;
  const int32_t* bt;
  int64_t bt_sb;
  int max_blocks;
  const int32_t* seq_lens;
  int B, Hkv, qlen, page_size;
  int fp8;               // MLA: e4m3 cache
  const float* k_scale;  // MLA FP8: device scalar or null
  int* err;
};
cudaError_t launch_gqa_kv_append(const AppendParams& p, cudaStream_t stream);
// one CTA whose bounded mbarrier wait runs out and raises DEVERR_WAIT_TIMEOUT in err
cudaError_t launch_wait_selftest(int* err, cudaStream_t stream);
cudaError_t launch_mla_kv_append(const AppendParams& p, cudaStream_t stream);

// ----------------------------------- decode with a window and first tokens --
constexpr int kPagedWarps = 4;      // of a CTA
constexpr int kPagedMaxGroup = 16;  // query heads per kv head
constexpr int kPagedMaxBatch = 2048;

// Decode over a bf16 cache, or an e4m3 cache with one fp32 scale for K and one
// for V per (page, kv head).  The token of a request of length L sees keys
// [0, first) and [L - window, L) (all of [0, L) when window <= 0).
struct PagedParams {
  const uint16_t* q;             // bf16 [B, Hq, D]
  int64_t q_sb, q_sh;
  const float* kv_scale;         // [num_blocks, Hkv, 2] (K, V), or null (bf16 cache)
  int64_t s_sblk, s_sh;          // its strides in floats
  const int32_t* bt;
  int64_t bt_sb;
  int max_blocks, num_blocks;
  const int32_t* seq_lens;
  const float* sinks;            // [Hq] or null
  uint16_t* out;                 // bf16 [B, Hq, D]
  int64_t o_sb, o_sh;
  float* lse;                    // [B, Hq] or null
  int64_t lse_sb, lse_sh;
  int B, Hkv, G, D, page_size;
  int window, first;
  float scale;
  int page_shift;                // log2(page_size)
  int grid;
  int cluster;                   // > 0: cluster mode, this many CTAs for each pair
  bool warps;                    // there are partials for shares of warps
  float* partials;               // two slots for each CTA (each warp in the warp mode)
  int* slot_counters;            // [2 * grid] arrival counters of merge groups
  int* pair_counters;            // [B * Hkv] arrival counters of the groups (of the warps)
  int* err;
};
struct PagedShape {
  int ctas_per_sm, part_floats;  // floats of one partial
  int chunks;                    // 128-byte pieces of a token's [K | V] row
};
PagedShape paged_attn_shape(int D, bool fp8, int G);
// kv_map: the cache as (128-byte piece's elements, token, piece, kv head, page),
// box (a piece, 16 tokens, all pieces, 1, 1), 128-byte swizzle.
cudaError_t launch_paged_attn(const PagedParams& p, const CUtensorMap& kv_map, cudaStream_t stream);
// A CTA's share of the work is counted in 16-token tiles plus a cost for each
// (request, kv head) pair, and is no smaller than kPagedMinCost.  64 requests of
// log-uniform lengths, e4m3: 80.5 us at a cost of 4, 54.4 at 8, 51.5 at 12, 52.0 at 16.
constexpr int kPagedPairCost = 12;
constexpr int kPagedMinCost = 16;
constexpr int kPagedMaxCluster = 8;
// Most tiles of a CTA in the cluster mode, but for full waves (bf16, a window of 1024 on 16 x 8 kv heads,
// 33 tiles each: 15.4 us in clusters, 17.2 without).
constexpr int kPagedClusterTiles = 48;
// Most tiles of a pair in the warp mode, in which one warp merges a pair's parts: 150 x 8
// kv heads of up to 2000 keys take 60.4 us in equal shares of CTAs, 57.1 in the warp mode,
// but a batch with one such request among very short ones gives it dozens of parts.
constexpr int kPagedWarpTiles = 64;

// ------------------------------------- decode of groups with shared tokens --
// Requests [cu_groups[g], cu_groups[g + 1]) share their first shared_lens[g] tokens.  One
// grid (prefix_attn.cu) attends to what is shared, once for all rows of a group, the next
// (paged_attn.cuh) to each request's own tokens; both leave 32-bit (O, m, l) parts, which
// the third (prefix_combine.cu) adds up.
constexpr int kPrefixRows = 256;     // query rows of a unit: two tiles of 128
constexpr int kPrefixTileKeys = 128; // keys of a step
// A CTA's share is counted in 16-key boxes plus a cost for each unit; it is a multiple of a
// tile's boxes, so that every CTA of a cut unit has a tile, and no smaller than kPrefixMinShare
// (64 requests behind 512 tokens take 20 us with 16, 22 with 24, 23 with 32; 4 requests 12.6,
// 13.4 and 14.4; 4 behind 8192 17.6, 16.4 and 18.3).  At a cost of 24, 64 requests behind 2048
// tokens take 27.7 us instead of 24.8, 33 e4m3 requests with heads of 64 34.8 instead of 34.1,
// but 128 requests behind 32768 126 instead of 128.
// Units (a group's blocks of kPrefixRows rows of a kv head) are laid end to end in the space of
// costs, and CTA c takes places [c share, (c + 1) share): whole tiles whose first box lies in
// them.
constexpr int kPrefixUnitCost = 40;
constexpr int kPrefixMinShare = 16;
struct PrefixParams {
  const int32_t* cu_groups;      // [groups + 1]
  const int32_t* shared_lens;    // [groups]
  int groups, grid;
  // per request: {first request of its group | row blocks of a kv head << 16, place of the
  // group's first unit, shared boxes (-1: padding), share of a CTA}
  int4* info;                    // [B]
  uint32_t* queue;               // the next share of the requests' own tokens; 0 between calls
  // of a request's own tokens; {m, l, reference of O, -}
  float4* own_o;                 // [Hkv][D / 4][B G]
  float4* own_ml;                // [Hkv][B G]
  // the part of a unit's first CTA: rows b G + h of each kv head
  float4* first_o;               // [Hkv][D / 4][B G]
  float2* first_ml;              // [Hkv][B G]
  // the part of a CTA whose range begins inside a unit
  float4* rest_o;                // [grid][D / 4][kPrefixRows]
  float2* rest_ml;               // [grid][kPrefixRows]
};
inline int64_t prefix_workspace_bytes(int64_t B, int64_t Hq, int64_t D, int64_t grid) {
  return B * 16 + B * Hq * (2 * D * 4 + 24) + grid * kPrefixRows * (D * 4 + 8);
}
// kv_map: the cache as (64 dims, token, piece, kv head, page), box (64, P, 1, 1, 1), 128-byte
// swizzle; e4m3: (D, token, K | V, kv head, page), box (D, P, 1, 1, 1), no swizzle.
cudaError_t launch_prefix_attn(const PagedParams& p, const PrefixParams& x, const CUtensorMap& kv_map,
                               cudaStream_t stream);
// The grids after it; kv_map as launch_paged_attn's.
cudaError_t launch_prefix_own(const PagedParams& p, const PrefixParams& x, const CUtensorMap& kv_map,
                              cudaStream_t stream);
cudaError_t launch_prefix_combine(const PagedParams& p, const PrefixParams& x, cudaStream_t stream);

// ------------------------------------------------ append to an e4m3 cache --
struct AppendFp8Params {
  const uint16_t *k, *v;         // bf16 [T, Hkv, D]
  int64_t s_st, s_sh;            // source strides (elements): token, head
  uint8_t* cache;                // e4m3 [num_blocks, Hkv, P, 2D]
  int64_t c_sblk, c_sh, c_stok;  // bytes
  float* scale;                  // [num_blocks, Hkv, 2]
  int64_t sc_sblk, sc_sh;        // floats
  const int32_t* bt;
  int64_t bt_sb;
  int max_blocks, num_blocks;
  const int32_t* seq_lens;
  const int32_t* cu;             // [B + 1] or null (T / B tokens each)
  int64_t T;
  int B, Hkv, D, page_size;
  int* err;
};
cudaError_t launch_gqa_kv_append_fp8(const AppendFp8Params& p, cudaStream_t stream);

// ---------------------------------------- head norms and rotation of q and k --
// cache != null: keys and values go into the paged cache, else keys go to k_out.
struct RopeParams {
  const uint16_t *q, *k, *v;     // bf16 [T, Hq, D], [T, Hkv, D]; v with the cache alone
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;  // strides (elements): token, head
  const void *qw, *kw;           // [D] weights of the norms, or null
  int qw_f32, kw_f32;            // fp32 (else bf16)
  float eps;
  const int32_t* positions;      // [T] or null (cache: a token's place in its request)
  const uint2* turns;            // [rot / 2]: turns per position, units of 2^-64
  float factor;                  // of cosines and sines
  int rot, interleaved;          // rot 0: no rotation
  uint16_t *q_out, *k_out;
  int64_t qo_st, qo_sh, ko_st, ko_sh;
  int64_t T;
  int Hq, Hkv, D;
  uint16_t* cache;               // bf16 [num_blocks, Hkv, P, 2D] or null
  int64_t c_sblk, c_sh, c_stok;  // elements
  const int32_t* bt;
  int64_t bt_sb;
  int max_blocks, num_blocks;
  const int32_t* seq_lens;
  const int32_t* cu;             // [B + 1] or null (T / B tokens each)
  int B, page_size;
  int* err;
};
cudaError_t launch_rope(const RopeParams& p, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------- cache pages --
constexpr int kPagesMaxRows = 8192;    // rows of a block table that a page call works on
constexpr int kPagesMaxTensors = 64;   // tensors of one pages_copy call

// A block table with its lengths and the pool's reference counts.
struct PageTables {
  int32_t* bt;
  int64_t bt_sb;
  int rows, max_blocks;
  int32_t* seq_lens;
  int32_t* refs;                 // [num_pages]: table entries that name the page
  int num_pages, page_size;
  int* err;
};
struct PagesCopyTensor {
  uint8_t* base;
  int64_t stride, bytes;         // of a page
  int num_pages;
};
struct PagesCopyParams {
  PagesCopyTensor t[kPagesMaxTensors];
  int num_tensors;
  const int32_t *src, *dst;      // [n], -1: nothing to copy
  int n;
  int* err;
};
cudaError_t launch_pages_copy(const PagesCopyParams& p, int num_sms, cudaStream_t stream);
// scratch of fork and reserve (n entries), and of compact, in ints
inline int64_t pages_scratch_ints(int64_t n, int64_t num_pages) { return 8 + 2 * n + num_pages; }
inline int64_t pages_compact_ints(int64_t num_pages) { return num_pages + num_pages / 4096 + 2; }
cudaError_t launch_pages_fork(const PageTables& t, const int32_t* parents, const int32_t* children,
                              int n, int32_t* copy_src, int32_t* copy_dst, int* scratch,
                              cudaStream_t stream);
cudaError_t launch_pages_release(const PageTables& t, const int32_t* rows, const int32_t* keep,
                                 int n, cudaStream_t stream);
// window > 0, first >= 0; t.rows > 0
cudaError_t launch_pages_trim(const PageTables& t, int window, int first, cudaStream_t stream);
cudaError_t launch_pages_reserve(const PageTables& t, const int32_t* rows, const int32_t* lens,
                                 int n, int* scratch, cudaStream_t stream);
cudaError_t launch_pages_compact(const PageTables& t, int32_t* copy_src, int32_t* copy_dst, int n,
                                 int32_t* num_moves, int* scratch, cudaStream_t stream);

// Large dynamic shared memory is an attribute of a kernel on the current
// device: set it the first time a kernel launches on each device.
template <typename Kernel>
inline cudaError_t set_smem_attr_once(Kernel* fn, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (uint64_t(1) << dev) : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// The counter region of the workspace holds 2^20 ints: the first half for
// (request, kv head) counters, the second half for split-group counters.
constexpr int64_t kTopCounters = int64_t(1) << 19;

}  // namespace pkv
