// prefix_attn.cu -- decode attention of groups of requests to the tokens they share,
// read once for all rows of a group, on tcgen05; a bf16 cache, or an e4m3 cache with one
// fp32 scale for K and one for V per (page, kv head).
//
// A group's rows for kv head k are the G query heads of each of its requests, one request
// after the other; all of them see the shared keys j < S (whole 16-key boxes, see
// prefix_common.cuh), so nothing is masked but what is left of the last tile:
//   x_j = scale ks(page of j) q . k_j,   m = max_j x_j
//   O = sum_j e^(x_j - m) vs(page of j) v_j,   l = sum_j e^(x_j - m)
// O, m and l go to the workspace in 32 bits; the grid after this one (paged_attn.cuh)
// attends to each request's own keys, the third (prefix_combine.cu) adds up all parts.
//
// With many rows (a key of 512 bytes is multiplied with 1024 rows, say) a step takes its slots 1770
// cycles, of which 1024 are products: bound by a slot's chain of scores, exponentials and weights,
// which two slots cover in part, and by power, which takes a tenth of the clock.  With few rows:
// latency, see below.
//
//  * A unit is (group, kv head, block of 256 rows); units are laid end to end, counted in
//    16-key boxes plus a cost for each, and CTA c takes an equal share of the whole, whose
//    cuts fall on 128-key tiles.  One CTA per SM, on as many SMs as the shares need.
//  * Two slots, each with a score tile S[128 x 128] and an accumulator O[128 x D] in
//    tensor memory and 128 softmax threads, one per row.  More than 128 rows: slot s has
//    rows 128 s .. and both go through all tiles.  Fewer: both slots have the same rows, slot
//    s tiles s, s + 2, .., and slot 0 adds up the two at the end (each of its threads reads
//    the other's row of tensor memory).  While one slot's threads are at their
//    exponentials, the tensor cores work for the other.
//  * Warps 0 and 3 ask for K and V of a tile by TMA, a lane for a page and a warp for half of
//    them, into a ring of operands; warps 1 and 2 issue S = Q K^T (M 128, N 128 keys, K D) and
//    O += P V (M 128, N D, K 128) of a slot each, P read from tensor memory, where it overlays
//    S.  (One warp for both took 1740 cycles a step of 1024 cycles of products, the rest its
//    waits and commits.)  e4m3 tiles land in a ring of their own, and four warps rewrite K as
//    fp16 and V as bf16 (both exact).
//  * The reference m of a row moves when a score passes it by more than 2^8, and O is
//    rescaled in tensor memory then; the scores of a step are there only after O of the
//    steps before is, so that needs no wait.  P, times its value's scale, is rounded once to
//    bf16, whose exponents are those of 32-bit values: up to 2^-8 of each weight, as in the
//    decode of a bf16 cache.  Also for e4m3, whose decode has tf32 weights: as two bf16 terms
//    (2^-16) they take half as many products again, and the samples below 202 us instead of
//    156, 33 requests with heads of 64 44.2 instead of 35.6.
//
// Measured (GB300, whole calls in a graph, 64 query and 8 kv heads of 128; the cuBLAS rate is 1929
// TFLOP/s, 1759 for seconds on end): 128 requests behind 131072 tokens 390 to 398 us = 1.4 PFLOP/s; on
// inputs that change from call to call, for seconds, 420 us = 1.31, at 1.37 kW and 1.88 GHz (of 2.07).
// 64 requests behind 8192 tokens and up to 2048 of their own 45.6 us, of which this grid has 25: a
// start of 6 us (three dependent reads), 1 us a step, parts written in 2.  58 forked e4m3 samples
// behind 500 to 32768 tokens (438 MB) 154 us; the same of bf16 (876 MB) 155 us = 84 % of the copy
// bandwidth.  e4m3 tiles of few rows wait for one another along the chain of copy, rewriting,
// products and exponentials; the rewriting's own work is 5 % (with 8 codes a thread at a time and 8
// reads under way 157 us then, with 16 and 4 164, with nothing rewritten 149), memory and the
// tensor pipe are each busy for a third of the time.
#include <algorithm>

#include "pkv_internal.h"
#include "prefix_common.cuh"
#include "prefix_ring.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

#include <cuda_fp16.h>

namespace pkv {
namespace {

constexpr int kTile = kPrefixTileKeys, kTileBoxes = kTile / 16;
constexpr int kSlotWarp0 = 4;  // softmax warps: 4..7 slot 0, 8..11 slot 1
constexpr int kSlotThreads = 128;
constexpr int kScaleTiles = 8;  // tiles whose scales are kept: more than keys are ahead of the weights
// Shares of at least so many tiles are read in turned order, see part_at.  128 requests behind
// 131072 tokens (shares of 216 tiles, 537 MB) take 390 us instead of 406 and, where power limits
// them, 430 instead of 459 (DRAM reads 0.80 GB instead of 2.15); behind 32768 (54 tiles) 127 and
// 128.  Shares of 8 to 16 tiles, whose keys L2 holds in any order, lose: e4m3 heads of 64 35.4 us
// instead of 34.0.
constexpr int kTurnTiles = 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;   // log2 units
// Instead of a unit of 0, which a masked score of -inf must not meet: it takes scores below 2^128 to
// less than 2^-21, and leaves units of normal size as they are.
constexpr float kLeast = 0x1p-149f;

// barriers
enum {
  kOpFull = 0, kOpEmpty = 8, kRawFull = 16, kRawEmpty = 22, kSFull = 28, kPReady = 30, kODone = 32,
  kQFull = 34, kQFree = 35, kPHalf = 36, kTurn = 38, kScaleFull = 40, kNumBars = kScaleFull + kScaleTiles,
};

template <int D_, bool kFp8_>
struct PrefixCfg {
  static constexpr int D = D_;
  static constexpr bool kFp8 = kFp8_;
  static constexpr int kThreads = kFp8 ? 512 : 384;  // e4m3: warps 12..15 convert
  static constexpr int kConverters = 128;
  static constexpr int kFewRegs = kFp8 ? 72 : 120, kManyRegs = kFp8 ? 184 : 192;
  static_assert((kThreads - 256) * kFewRegs + 256 * kManyRegs <= kThreads * (kFp8 ? 128 : 168),
                "registers of the launch");
  static constexpr int kChunks = D / 64;            // 128-byte pieces of an operand's row
  static constexpr int kChunkBytes = kTile * 128;   // 16 KB
  static constexpr int kOpBytes = kChunks * kChunkBytes;
  static constexpr int kRawBytes = kTile * D;       // an e4m3 operand
  static constexpr int kOps = D == 64 ? (kFp8 ? 6 : 8) : (kFp8 ? 3 : 4);
  // A unit of one query tile has an operand more, in the other tile's place, where there are
  // three: with three, the next step's keys wait for the products of this step's values.  Free
  // it is then: the three before it hold among them the last keys of a unit of two tiles, and
  // a unit's accumulators are done before the next one's queries are written.
  static constexpr bool kExtraOp = kOps == 3;
  static constexpr int kRaws = D == 64 ? 6 : 3;
  static constexpr int kOffOps = 2 * kOpBytes;  // behind two query tiles
  static constexpr int kOffRaw = kOffOps + kOps * kOpBytes;
  static constexpr int kOffScale = kOffRaw + (kFp8 ? kRaws * kRawBytes : 0);
  static constexpr int kOffMl = kOffScale + kScaleTiles * kTileBoxes * 8;
  static constexpr int kOffBars = kOffMl + kSlotThreads * 8;
  static constexpr int kOffMisc = kOffBars + kNumBars * 8;
  static constexpr int kOffPlaces = kOffMisc + 80;
  static constexpr int smem_bytes(int groups) { return kOffPlaces + (groups + 1) * 8 + 1024; }
  static_assert(smem_bytes(kPagedMaxBatch) <= 227 * 1024, "shared memory");
  static_assert(4 * (plan_ints(kPagedMaxBatch) + kPagedMaxBatch + 1) <= kOffScale, "room for the plan of the groups");
};

// A place of the ring in shared memory.
template <class C>
__device__ __forceinline__ uint32_t op_offset(int place) {
  return C::kExtraOp && place == C::kOps ? C::kOpBytes : C::kOffOps + place * C::kOpBytes;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {  // RNE, lo in bits 0..15
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A CTA's part of a unit.
template <bool kFp8>
struct Part {
  int first, lead;      // the group's first request, and its first that is not empty
  int rows;             // of the block
  int row0;             // of the block within the group
  int kvh;
  int boxes, t0, t1;    // shared boxes; tiles of this part
  int turn;             // its first step's tile is t0 + turn
  bool whole_start;     // it holds the first tile
  int next;             // place of the next unit
  __device__ __forceinline__ int tiles() const { return t1 - t0; }
  __device__ __forceinline__ bool dual() const { return rows > kSlotThreads; }
  // steps of the two slots together: step j is slot j & 1's
  __device__ __forceinline__ int steps() const { return dual() ? 2 * tiles() : tiles(); }
  __device__ __forceinline__ int tile(int j) const { return dual() ? j >> 1 : j; }
  // The tile of the unit that comes t-th: from t0 + turn on, then those before it.
  __device__ __forceinline__ int at(int t) const {
    t += turn;
    return t0 + (t < tiles() ? t : t - tiles());
  }
  __device__ __forceinline__ OperandOrder order() const { return {kFp8 || dual(), tiles()}; }
};

// The unit that holds place f < the CTA's end `to`.
template <bool kFp8>
__device__ __forceinline__ Part<kFp8> part_at(const PagedParams& p, const PrefixParams& x,
                                              const int* places, int f, int to, int share) {
  Part<kFp8> r;
  const int* at = places + x.groups + 1;
  int lo = 0, hi = x.groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (places[mid] <= f) lo = mid; else hi = mid - 1;
  }
  r.first = at[lo] & 0xffff;
  r.lead = at[lo] >> 16;
  const int rows = ((at[lo + 1] & 0xffff) - r.first) * p.G;
  const int blocks = (rows + kPrefixRows - 1) / kPrefixRows;
  const int per = (places[lo + 1] - places[lo]) / (p.Hkv * blocks);
  const int unit = (f - places[lo]) / per, begin = places[lo] + unit * per;
  r.boxes = per - kPrefixUnitCost;
  r.kvh = unit / blocks;
  r.row0 = unit % blocks * kPrefixRows;
  r.rows = min(rows - r.row0, kPrefixRows);
  r.next = begin + per;
  auto cut = [&](int y) {
    return y >= r.next ? (r.boxes + kTileBoxes - 1) / kTileBoxes
                       : max(y - begin - kPrefixUnitCost, 0) / kTileBoxes;
  };
  r.t0 = cut(f);
  r.t1 = cut(to);
  r.whole_start = r.t0 == 0;
  // CTAs begin with tiles a share apart, so that those with other rows of the same keys, whose
  // cuts fall elsewhere, read a tile at about the same time: once from DRAM, then from L2.
  const int period = share / kTileBoxes, start = (r.t0 + period - 1) / period * period;
  r.turn = period >= kTurnTiles && start < r.t1 ? start - r.t0 : 0;
  return r;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ PrefixParams x,
                       const __grid_constant__ CUtensorMap kv_map) {
  constexpr int D = C::D;
  constexpr bool kFp8 = C::kFp8;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base_u32 = (raw + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* places = reinterpret_cast<int*>(base + C::kOffPlaces);
  int* misc = reinterpret_cast<int*>(base + C::kOffMisc);
  auto bar = [&](int i) { return base_u32 + C::kOffBars + 8u * i; };

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const bool slot = (i & ~1) == kPReady || (i & ~1) == kPHalf;
      const bool both = i == kQFree || (i >= kOpEmpty && i < kRawFull);  // of the MMA issuers
      const bool op_full = i >= kOpFull && i < kOpEmpty;
      const bool asked = !kFp8 && op_full;  // of the TMA producers
      mbar_init(bar(i), slot           ? kSlotThreads
                        : i == kQFull   ? 2 * kSlotThreads
                        : both || asked ? 2
                                        : 1);
    }
    fence_barrier_init();
    tma_prefetch_desc(&kv_map);
  }
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(misc + 16), 512);
    tc::tmem_relinquish();
  }
  // The grid after this one reads ahead of its own wait, which is sound as every CTA of
  // this one has waited before it lets it start.
  griddep_wait();
  if (blockIdx.x == 0) {
    // it is 0, unless calls that shared the workspace ran at once
    if (tid == 0) {
      atomicExch(x.queue, 0u);
      __threadfence();
    }
    __syncthreads();
  }
  griddep_launch_dependents();

  // ---- places of the groups' units ----
  // what stays of the plan: places, and per group the first request and the first that is
  // not empty
  int* rows = places + x.groups + 1;
  int total, share;
  {
    int* lead = reinterpret_cast<int*>(base) + plan_ints(x.groups);
    const GroupPlan plan =
        plan_groups<C::kThreads, true>(p, x, reinterpret_cast<int*>(base), lead, blockIdx.x == 0);
    if (warp == 0) {
      int run = 0;
      for (int g0 = 0; g0 < plan.groups; g0 += 32) {
        const int g = g0 + lane;
        int cost = 0;
        if (g < plan.groups && plan.boxes[g] > 0)
          cost = p.Hkv * blocks_of(p, plan, g) * (plan.boxes[g] + kPrefixUnitCost);
        int incl = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        if (g < plan.groups) {
          places[g] = run + incl - cost;
          rows[g] = plan.cu[g] | min(lead[g], p.B - 1) << 16;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (lane == 0) {
        places[plan.groups] = run;
        rows[plan.groups] = plan.groups ? plan.cu[plan.groups] : 0;
      }
    }
    __syncthreads();
    total = places[plan.groups];
    // Whole tiles: a CTA with a little less would have as many at most, and the SMs that are
    // left are the next grid's (64 requests behind 512 tokens 25.3 -> 20.8 us).
    share = max((total + (int)gridDim.x - 1) / (int)gridDim.x, kPrefixMinShare);
    share = (share + kTileBoxes - 1) / kTileBoxes * kTileBoxes;
    if (blockIdx.x == gridDim.x - 1) {  // for prefix_combine.cu
      for (int b = tid; b < p.B; b += C::kThreads) {
        const int g = plan.groups ? plan.find(b) : -1;
        const bool in = b >= plan.first() && b < plan.end();
        int4 at = make_int4(0, 0, in ? 0 : -1, share);
        if (in && g >= 0)
          at = make_int4(plan.cu[g] | blocks_of(p, plan, g) << 16, places[g], plan.boxes[g], share);
        x.info[b] = at;
      }
    }
    fence_proxy_async_smem();  // the plan lies where tiles come
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc + 16);
  const int from = min((long long)blockIdx.x * share, (long long)total);
  const int to = min((long long)from + share, (long long)total);

  // Registers: the softmax warpgroups take what the others give back (at launch 512 x 128, or
  // 384 x 168).
  if (warp < kSlotWarp0 || warp >= kSlotWarp0 + 8) setmaxnreg_dec<C::kFewRegs>();
  if (warp == 0 || (warp == 3 && !kFp8)) {
    // ============================ TMA producers ============================
    // An operation takes its warp some 50 cycles to issue, whatever its size, so two warps ask
    // for half of each operand's pages.  Both go through all operands in order: a warp that
    // skipped some would take an old phase of a place's barrier for a new one.
    // (e4m3 operands are half as large, and come from one warp.)
    const int half = warp == 3;
    const int in_tile = 7 - p.page_shift;  // log2 of a tile's pages
    const int batch = 32 >> in_tile;       // tiles whose pages the lanes look up at once
    const int sub = lane & ((1 << in_tile) - 1);
    const bool asks = kFp8 || (in_tile == 0 ? half == 0 : sub >> (in_tile - 1) == half);
    const uint32_t bytes = kFp8 ? C::kRawBytes : C::kOpBytes >> (in_tile == 0 ? (half ? 31 : 0) : 1);
    int op = 0, tiles = 0;                 // operands and tiles of units before
    OpRing<C::kOps, C::kExtraOp> ring;
    for (int f = from; f < to;) {
      const auto u = part_at<kFp8>(p, x, places, f, to, share);
      f = u.next;
      if (u.tiles() <= 0) continue;
      const int32_t* table = p.bt + (int64_t)u.lead * p.bt_sb;
      const int end = min(u.boxes, u.t1 * kTileBoxes) * 16;  // tokens
      ring.begin(u.dual());
      auto page_of = [&](int t) {  // this lane's page of tiles t ..
        t += lane >> in_tile;
        const int page = (u.at(t) << in_tile) + sub;
        return t < u.tiles() && page << p.page_shift < end ? __ldg(table + min(page, p.max_blocks - 1)) : INT_MAX;
      };
      auto scale_of = [&](int page) {
        float2 s = make_float2(0.f, 0.f);
        if (kFp8 && half == 0 && page >= 0 && page < p.num_blocks)
          s = __ldg(reinterpret_cast<const float2*>(p.kv_scale + (int64_t)page * p.s_sblk +
                                                    u.kvh * p.s_sh));
        return s;
      };
      // Pages of an even and of an odd batch; those of the next one, and a tile later their
      // scales, are read ahead.
      int pages[2] = {page_of(0), 0};
      float2 scale = scale_of(pages[0]), next_scale = scale;
      for (int n = 0; n < 2 * u.tiles(); ++n, ++op) {
        const int t = u.order().tile_of(n), at = t & (batch - 1);
        const bool values = u.order().are_values(n), odd = t & batch;
        if (!values) {
          if (at == 0) {
            scale = next_scale;
            const int now = odd ? pages[1] : pages[0];
            if (half == 0 && now != INT_MAX && (now < 0 || now >= p.num_blocks))
              atomicOr(p.err, DEVERR_BAD_BLOCK);
          }
          // (the values of the batch before have been asked for)
          if (at == 1) {
            const int next = page_of(t - 1 + batch);
            if (odd) pages[0] = next; else pages[1] = next;
          }
          if (kFp8 && at == 2) next_scale = scale_of(odd ? pages[0] : pages[1]);
        }
        int page = odd ? pages[1] : pages[0];
        if (page < 0 || page >= p.num_blocks) page = p.num_blocks;  // past the cache: zeros
        const bool mine = lane >> in_tile == at;
        const int e = kFp8 ? op % C::kRaws : ring.place(n);
        const int full = (kFp8 ? kRawFull : kOpFull) + e;
        const uint32_t phase = kFp8 ? op / C::kRaws : ring.phase(n);
        mbar_wait(bar((kFp8 ? kRawEmpty : kOpEmpty) + e), (phase & 1) ^ 1u, p.err);
        if (lane == 0) mbar_arrive_expect_tx(bar(full), bytes);
        if (kFp8 && half == 0 && !values) {  // the scales' place is free: see kScaleTiles
          const int place = (tiles + t) % kScaleTiles;
          if (mine)
            for (int b = 0; b < 1 << (p.page_shift - 4); ++b)
              *reinterpret_cast<float2*>(base + C::kOffScale +
                                         (place * kTileBoxes + (sub << (p.page_shift - 4)) + b) * 8) = scale;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kScaleFull + place));
        }
        __syncwarp();
        if (mine && asks) {
          if constexpr (kFp8) {
            tma_load_5d(base_u32 + C::kOffRaw + e * C::kRawBytes + (sub << p.page_shift) * D, &kv_map,
                        bar(full), 0, 0, values, u.kvh, page);
          } else {
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_5d(base_u32 + op_offset<C>(e) + c * C::kChunkBytes + (sub << p.page_shift) * 128,
                          &kv_map, bar(full), 0, 0, (values ? C::kChunks : 0) + c, u.kvh, page);
          }
        }
      }
      tiles += u.tiles();
      ring.end(2 * u.tiles());
    }
  } else if (warp == 1 || warp == 2) {
    // ===================== MMA issuers, one for each slot =====================
    constexpr uint32_t kIdS = kFp8 ? tc::idesc_f16_f32(128, kTile) : tc::idesc_bf16_f32(128, kTile, false, false);
    constexpr uint32_t kIdPv = tc::idesc_bf16_f32(128, D, false, true);
    const int slot = warp - 1;
    const uint32_t tS = tmem + slot * kTile, tO = tmem + 2 * kTile + slot * D;
    // The slots take turns at the tensor cores, a step's products each: left to themselves they
    // fall into step, and the tensor cores stand still while both are at their exponentials.
    int units = 0, before = 0;      // the slot whose turn was the last
    uint32_t ready = 0, turns = 0;  // phases of P; of this slot's turns
    OpRing<C::kOps, C::kExtraOp> ring;
    for (int f = from; f < to;) {
      const auto u = part_at<kFp8>(p, x, places, f, to, share);
      f = u.next;
      if (u.tiles() <= 0) continue;
      const int steps = u.steps();
      const bool dual = u.dual();
      const uint32_t q = base_u32 + (dual ? slot : 0) * C::kOpBytes;
      ring.begin(dual);
      mbar_wait(bar(kQFull), units & 1, p.err);
      // an operand is free when both slots have read it, or one that reads it alone
      auto release = [&](int n) {
        const int e = ring.place(n);
        tc::commit_elect(bar(kOpEmpty + e));
        if (!dual) tc::commit_elect(bar(kOpEmpty + e));
      };
      auto wait_op = [&](int n) { mbar_wait(bar(kOpFull + ring.place(n)), ring.phase(n), p.err); };
      if (slot >= steps && lane == 0) mbar_arrive(bar(kQFree));  // a single step is slot 0's
      // A turn: the values of step j, the scores of step j + 2 (the first turn: of step `slot`).
      for (int j = slot - 2; j < steps; j += 2) {
        const bool first = j < 0, more = j + 2 < steps;
        if (first && !more) continue;
        const int kn = more ? u.order().keys(u.tile(j + 2)) : 0, vn = first ? 0 : u.order().values(u.tile(j));
        // All that can be waited for is, before the turn.  (The next e4m3 keys of a unit of one
        // query tile are rewritten behind the other slot's values, and so come late.)
        if (more && (!kFp8 || dual || first)) wait_op(kn);
        if (!first) {
          wait_op(vn);
          mbar_wait(bar(kPHalf + slot), ready & 1, p.err);
        }
        if (first ? slot == 1 || before == 1 : steps > 1) {
          mbar_wait(bar(kTurn + slot), turns & 1, p.err);
          ++turns;
        }
        tc::fence_after_sync();
        if (!first) {
          const uint32_t b = base_u32 + op_offset<C>(ring.place(vn));
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks) {
            if (ks == kTile / 32) {
              mbar_wait(bar(kPReady + slot), ready & 1, p.err);
              tc::fence_after_sync();
            }
            tc::mma_bf16_ts_elect(
                tO, tS + ks * 8,
                tc::smem_desc(b + ks * 2048, C::kChunkBytes, 1024, tc::kSwizzle128), kIdPv,
                j > 1 || ks > 0);
          }
          ++ready;
          release(vn);
          if (!more) tc::commit_elect(bar(kODone + slot));
          if (kFp8 && !dual && more) wait_op(kn);
        }
        if (more) {
          const uint32_t b = base_u32 + op_offset<C>(ring.place(kn));
          tc::fence_after_sync();
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc::mma_bf16_elect(
                  tS, tc::smem_desc(q + c * C::kChunkBytes + ks * 32, 16, 1024, tc::kSwizzle128),
                  tc::smem_desc(b + c * C::kChunkBytes + ks * 32, 16, 1024, tc::kSwizzle128), kIdS,
                  (c | ks) != 0);
        }
        // the other slot's turn: its first after this one's first, else if it has a step left;
        // the next unit begins with slot 0
        if ((slot == 1 || (first ? steps > 1 : j + 1 < steps)) && lane == 0)
          mbar_arrive(bar(kTurn + (slot ^ 1)));
        if (more) {
          tc::commit_elect(bar(kSFull + slot));
          release(kn);
          if (j + 4 >= steps) tc::commit_elect(bar(kQFree));
        }
      }
      before = (steps - 1) & 1;
      ring.end(2 * u.tiles());
      ++units;
    }
  } else if (warp >= kSlotWarp0 && warp < kSlotWarp0 + 8) {
    // ======================= softmax, one thread per row ===================
    setmaxnreg_inc<C::kManyRegs>();
    const int slot = (warp - kSlotWarp0) >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lanes + slot * kTile, tO = tmem + lanes + 2 * kTile + slot * D;
    const float scale2 = fabsf(p.scale) * kLog2e;
    float c2 = fmaxf(scale2, kLeast);  // log2 units of a score
    const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;  // of the query's signs
    float2* other_ml = reinterpret_cast<float2*>(base + C::kOffMl);  // at a unit's end
    float* row_scale = reinterpret_cast<float*>(other_ml);           // at its start
    int units = 0, tiles = 0;
    uint32_t got = 0, done[2] = {0, 0};  // phases of S; of O
    for (int f = from; f < to;) {
      const auto u = part_at<kFp8>(p, x, places, f, to, share);
      f = u.next;
      if (u.tiles() <= 0) continue;
      const int steps = u.steps();
      const bool dual = u.dual();
      // ---- query rows: 128 each, or half of one tile each; rows past the block are zero ----
      if (units > 0) mbar_wait(bar(kQFree), (units - 1) & 1, p.err);
      {
        // 16-byte units; a thread's are kStep rows apart, so its unit k and swizzle stay
        constexpr int kUnits = D / 8, kStep = kSlotThreads / kUnits, kMine = 128 / kStep;
        const int n = dual ? kMine : kMine / 2, tile = dual ? slot : 0;
        const int r0 = (dual ? 0 : 64 * slot) + row / kUnits, k = row % kUnits;
        int at = u.row0 + 128 * tile + r0, b = u.first + at / p.G, h = at % p.G;
        const int db = kStep / p.G, dh = kStep % p.G, end = u.row0 + u.rows;
        uint4 v[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          v[i] = make_uint4(0, 0, 0, 0);
          if (i < n && at < end)
            v[i] = __ldg(reinterpret_cast<const uint4*>(p.q + b * p.q_sb + (u.kvh * p.G + h) * p.q_sh) + k);
          at += kStep;
          b += db;
          h += dh;
          if (h >= p.G) h -= p.G, ++b;
        }
        uint8_t* dst = base + tile * C::kOpBytes + (k >> 3) * C::kChunkBytes + r0 * 128 +
                       (((k & 7) ^ (r0 & 7)) * 16);
        static_assert(kStep % 8 == 0, "the swizzle of a thread's rows");
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          if (i >= n) break;
          if constexpr (kFp8) {
            // To fp16, as the keys are: 2^up brings the row's largest element into [2^14,
            // 2^15); exact but for elements below 2^-29 of it.  0 and non-finite rows stay.
            uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, big = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              big = max(big, max((w[e] << 16) & 0x7fffffffu, w[e] & 0x7fff0000u));
#pragma unroll
            for (int o = kUnits / 2; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
            const int ex = (int)(big >> 23);
            const int up = ex == 0 || ex == 255 ? 0 : max(min(127 + 14 - ex, 126), -126);
            const float mul = __uint_as_float((uint32_t)(up + 127) << 23);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_f16(__uint_as_float(w[e] << 16) * mul, __uint_as_float(w[e] & 0xffff0000u) * mul);
            v[i] = make_uint4(w[0], w[1], w[2], w[3]);
            if (k == 0) row_scale[128 * tile + r0 + i * kStep] = __uint_as_float((uint32_t)(127 - up) << 23);
          }
          *reinterpret_cast<uint4*>(dst + i * kStep * 128) =
              make_uint4(v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(kQFull));
      if (kFp8) {  // each row's scale is another thread's
        named_bar_sync(1, 2 * kSlotThreads);
        c2 = scale2 * row_scale[(dual ? 128 * slot : 0) + row];
        // All have read before anyone writes there again: slot 1 its m and l, at once if the unit
        // has one step, or the next unit's scales (a place of their own does not fit beside 2048
        // groups).
        named_bar_sync(1, 2 * kSlotThreads);
      }
      const int mine = dual ? min(u.rows - 128 * slot, 128) : u.rows;  // rows of this slot
      const bool live = 32 * (warp & 3) < mine;  // of the warp: else it only keeps step
      float m = -INFINITY, l = 0.f;              // m in log2 units
      for (int j = slot; j < steps; j += 2) {
        mbar_wait(bar(kSFull + slot), got & 1, p.err);
        ++got;
        const int t = u.tile(j), at = tiles + t;
        if (kFp8) mbar_wait(bar(kScaleFull + at % kScaleTiles), (at / kScaleTiles) & 1, p.err);
        __syncwarp();
        tc::fence_after_sync();
        if (live) {
          const int valid = min(u.boxes - u.at(t) * kTileBoxes, kTileBoxes);  // boxes
          const float2* sc = reinterpret_cast<const float2*>(base + C::kOffScale) +
                             (at % kScaleTiles) * kTileBoxes;
          // log2 units of a score of box h, never 0
          auto unit = [&](int h) { return kFp8 ? __fmaf_rn(c2, sc[h].x, kLeast) : c2; };
          // Half of the row at a time in registers: two pieces of 32 keys, from piece c on.
          uint32_t s[2][32];
          auto load = [&](int c) {
            tc::ld_32x32b_x32(tS + 32 * c, s[0]);
            tc::ld_32x32b_x32(tS + 32 * c + 32, s[1]);
            tc::wait_ld();
            if (valid < 2 * c + 4) {
#pragma unroll
              for (int h = 0; h < 4; ++h)
                if (2 * c + h >= valid)
#pragma unroll
                  for (int i = 0; i < 16; ++i) s[h / 2][16 * (h & 1) + i] = 0xff800000u;  // -inf
            }
          };
          auto largest = [&](int c) {
            float a[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const uint32_t* y = s[h / 2] + 16 * (h & 1);
              a[h] = max3(__uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2]));
#pragma unroll
              for (int i = 3; i < 15; i += 2)
                a[h] = max3(a[h], __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
              a[h] = fmaxf(a[h], __uint_as_float(y[15]));
              if (kFp8) a[h] *= unit(2 * c + h);
            }
            const float top = fmaxf(max3(a[0], a[1], a[2]), a[3]);
            return kFp8 ? top : top * c2;
          };
          float2 sum[2] = {};
          auto weights = [&](int c, float ref, uint32_t (&w)[2][16]) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const float ks = unit(2 * c + h), vs = kFp8 ? sc[2 * c + h].y : 1.f;
              const float2 k2 = make_float2(ks, ks), r2 = make_float2(ref, ref);
              const uint32_t* x = s[h / 2] + 16 * (h & 1);
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const float2 y =
                    fma2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), k2, r2);
                float2 e = make_float2(ex2(y.x), ex2(y.y));
                sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], e);
                if (kFp8) e = mul2(e, make_float2(vs, vs));
                w[h / 2][8 * (h & 1) + i / 2] = pack_bf16(e.x, e.y);
              }
            }
          };
          // The first half's weights are taken with the reference as it stands, and again in the
          // rare case that a score of the row moves it.  One copy of the code for both halves.
          uint32_t w[2][16];
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            load(c);
            top = fmaxf(top, largest(c));
            if (c == 2) {
              const bool move = top > m + kSlack || (m == -INFINITY && top > m);
              if (__any_sync(0xffffffffu, move)) {
                const float mn = move ? top : m;
                const float keep = m == -INFINITY ? 0.f : ex2(m - mn);
                if (j > 1) {
#pragma unroll 1
                  for (int d = 0; d < D; d += 16) {
                    uint32_t o[16];
                    tc::ld_32x32b_x16(tO + d, o);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                    tc::st_32x32b_x16(tO + d, o);
                  }
                }
                l *= keep;
                m = mn;
                sum[0] = sum[1] = make_float2(0.f, 0.f);
                c = -2;
                continue;
              }
              tc::st_32x32b_x16(tS, w[0]);
              tc::st_32x32b_x16(tS + 16, w[1]);
              tc::wait_st();
              tc::fence_before_sync();
              mbar_arrive(bar(kPHalf + slot));  // the first half's product can begin
            }
            weights(c, m == -INFINITY ? 0.f : -m, w);
          }
          tc::st_32x32b_x16(tS + 32, w[0]);
          tc::st_32x32b_x16(tS + 48, w[1]);
          sum[0] = add2(sum[0], sum[1]);
          l += sum[0].x + sum[0].y;
          tc::wait_st();
        } else {
          mbar_arrive(bar(kPHalf + slot));
        }
        tc::fence_before_sync();
        mbar_arrive(bar(kPReady + slot));
      }

      // ---- the part of this row: O, m, l ----
      const bool both = steps > 1;
      float w0 = 1.f, w1 = 0.f;
      if (!dual) {  // slot 1's tiles of the same rows
        if (slot == 1) other_ml[row] = make_float2(m, l);
        named_bar_sync(1, 2 * kSlotThreads);
        if (slot == 0) {
          const float2 o = other_ml[row];
          const float mn = fmaxf(m, o.x);
          if (mn > -INFINITY) {
            w0 = m == -INFINITY ? 0.f : ex2(m - mn);
            w1 = o.x == -INFINITY ? 0.f : ex2(o.x - mn);
            // a NaN stays one
            l = l * w0 + o.y * w1;
            m = mn;
          } else {
            l += o.y;
          }
        }
      }
      if (slot == 0 || dual) mbar_wait(bar(kODone + slot), done[slot] & 1, p.err);
      if (!dual && slot == 0 && both) mbar_wait(bar(kODone + 1), done[1] & 1, p.err);
      ++done[0];
      done[1] += both;
      __syncwarp();
      tc::fence_after_sync();
      if (live && (slot == 0 || dual)) {
        const int at = u.row0 + 128 * slot + row;  // row of the group
        const int64_t rows = (int64_t)p.B * p.G, where = (int64_t)u.first * p.G + at;
        float4* dst;
        float2* ml;
        int64_t step;
        if (u.whole_start) {
          dst = x.first_o + u.kvh * (D / 4) * rows + where;
          ml = x.first_ml + u.kvh * rows + where;
          step = rows;
        } else {
          dst = x.rest_o + (int64_t)blockIdx.x * (D / 4) * kPrefixRows + 128 * slot + row;
          ml = x.rest_ml + (int64_t)blockIdx.x * kPrefixRows + 128 * slot + row;
          step = kPrefixRows;
        }
        const bool write = 128 * slot + row < u.rows;
        if (write) *ml = make_float2(m, l);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32], o1[32];
          tc::ld_32x32b_x32(tO + 32 * c, o);
          if (!dual && both) tc::ld_32x32b_x32(tO + D + 32 * c, o1);
          tc::wait_ld();
          if (!dual && both) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * w0 + __uint_as_float(o1[i]) * w1);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (write)
              dst[(8 * c + i) * step] =
                  make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                              __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
        }
      }
      tc::fence_before_sync();
      if (!dual) named_bar_sync(2, 2 * kSlotThreads);  // slot 1's accumulator has been read
      tiles += u.tiles();
      ++units;
    }
  } else if (kFp8 && warp >= kSlotWarp0 + 8) {
    // ============= e4m3 operand -> bf16 operand, swizzled for the MMA =============
    const int ct = tid - 32 * (kSlotWarp0 + 8);
    int op = 0;
    OpRing<C::kOps, C::kExtraOp> ring;
    for (int f = from; f < to;) {
      const auto u = part_at<kFp8>(p, x, places, f, to, share);
      f = u.next;
      if (u.tiles() <= 0) continue;
      ring.begin(u.dual());
      for (int i = 0; i < 2 * u.tiles(); ++i, ++op) {
        const int er = op % C::kRaws, eo = ring.place(i);
        mbar_wait(bar(kRawFull + er), (op / C::kRaws) & 1, p.err);
        const uint8_t* src = base + C::kOffRaw + er * C::kRawBytes;
        uint8_t* dst = base + op_offset<C>(eo);
        // 8 codes each, a 16-byte unit of the operand; a thread's are kStep rows apart, which keeps
        // the unit and the swizzle
        constexpr int kUnits = D / 8, kStep = C::kConverters / kUnits, kMine = kTile / kStep;
        static_assert(kStep % 8 == 0, "the swizzle of a thread's rows");
        const int r0 = ct / kUnits, q = ct % kUnits;
        dst += (q >> 3) * C::kChunkBytes + r0 * 128 + ((q & 7) ^ (r0 & 7)) * 16;
        constexpr int kBatch = 8;
        static_assert(kMine % kBatch == 0, "batches");
#pragma unroll 1
        for (int k0 = 0; k0 < kMine; k0 += kBatch) {
          uint2 w[kBatch];
          uint32_t o[kBatch][4];
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            w[k] = *reinterpret_cast<const uint2*>(src + (ct + (k0 + k) * C::kConverters) * 8);
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const uint32_t wv[2] = {w[k].x, w[k].y};
#pragma unroll
            for (int h = 0; h < 4; ++h)
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
                  : "=r"(o[k][h])
                  : "h"((uint16_t)(wv[h / 2] >> (16 * (h & 1)))));
          }
          if (i & 1) {  // values: to bf16, as P is
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const float2 fv = __half22float2(*reinterpret_cast<const __half2*>(&o[k][h]));
                o[k][h] = pack_bf16(fv.x, fv.y);
              }
          }
          // the first batch before the operand's place is free
          if (k0 == 0) mbar_wait(bar(kOpEmpty + eo), ring.phase(i) ^ 1u, p.err);
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            *reinterpret_cast<uint4*>(dst + (k0 + k) * kStep * 128) =
                make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
        }
        fence_proxy_async_smem();  // the MMA reads through the async proxy
        __syncwarp();
        named_bar_sync(3, C::kConverters);
        if (ct == 0) {
          mbar_arrive(bar(kRawEmpty + er));
          mbar_arrive(bar(kOpFull + eo));
        }
      }
      ring.end(2 * u.tiles());
    }
  }

  tc::fence_before_sync();
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <class C>
cudaError_t launch_prefix(const PagedParams& p, const PrefixParams& x, const CUtensorMap& map,
                          cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e =
      set_smem_attr_once(prefix_attn_kernel<C>, C::smem_bytes(kPagedMaxBatch), done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(x.grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::smem_bytes(x.groups);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_attn_kernel<C>, p, x, map);
}

}  // namespace

cudaError_t launch_prefix_attn(const PagedParams& p, const PrefixParams& x, const CUtensorMap& map,
                               cudaStream_t stream) {
  if (p.D == 64)
    return p.kv_scale ? launch_prefix<PrefixCfg<64, true>>(p, x, map, stream)
                      : launch_prefix<PrefixCfg<64, false>>(p, x, map, stream);
  return p.kv_scale ? launch_prefix<PrefixCfg<128, true>>(p, x, map, stream)
                    : launch_prefix<PrefixCfg<128, false>>(p, x, map, stream);
}

}  // namespace pkv
