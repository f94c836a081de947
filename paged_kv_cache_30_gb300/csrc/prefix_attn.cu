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
// Bound by the tensor cores and the exponentials of many rows (a key of 512 bytes is
// multiplied with 512 rows, say), by memory of few.
//
//  * A unit is (group, kv head, block of 256 rows); units are laid end to end, counted in
//    16-key boxes plus a cost for each, and CTA c takes an equal share of the whole, whose
//    cuts fall on 128-key tiles.  One CTA per SM.
//  * Two slots, each with a score tile S[128 x 128] and an accumulator O[128 x D] in
//    tensor memory and 128 softmax threads, one per row.  More than 128 rows: slot s has
//    rows 128 s .. and both go through all tiles.  Fewer: both slots have the same rows, slot
//    s tiles s, s + 2, .., and slot 0 adds up the two at the end (each of its threads reads
//    the other's row of tensor memory).  While one slot's threads are at their
//    exponentials, the tensor cores work for the other.
//  * warp 0 asks for K and V of a tile by TMA, lane l for 16-key box l, into a ring of
//    operands; warp 1 issues S = Q K^T (M 128, N 128 keys, K D) and O += P V (M 128, N D,
//    K 128), P read from tensor memory, where it overlays S.  e4m3 tiles land in a ring of
//    their own, and six warps rewrite them as bf16 (exact).
//  * The reference m of a row moves when a score passes it by more than 2^8, and O is
//    rescaled in tensor memory then; the scores of a step are there only after O of the
//    steps before is, so that needs no wait.  P, times its value's scale, is rounded once to
//    bf16, whose exponents are those of 32-bit values: 2^-9 of each weight, as in the decode
//    of a bf16 cache.
#include <algorithm>

#include "pkv_internal.h"
#include "prefix_common.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

#include <cuda_fp16.h>

namespace pkv {
namespace {

constexpr int kTile = kPrefixTileKeys, kTileBoxes = kTile / 16;
constexpr int kSlotWarp0 = 4;  // softmax warps: 4..7 slot 0, 8..11 slot 1
constexpr int kSlotThreads = 128;
constexpr int kScaleTiles = 8;  // tiles whose scales are kept
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;   // log2 units
constexpr float kTiny = 1e-37f;  // times any score that is finite: no change of its weight

// barriers
enum {
  kOpFull = 0, kOpEmpty = 8, kRawFull = 16, kRawEmpty = 22, kSFull = 28, kPReady = 30, kODone = 32,
  kQFull = 34, kQFree = 35, kPHalf = 36, kScaleFull = 38, kNumBars = kScaleFull + kScaleTiles,
};

template <int D_, bool kFp8_>
struct PrefixCfg {
  static constexpr int D = D_;
  static constexpr bool kFp8 = kFp8_;
  static constexpr int kThreads = kFp8 ? 512 : 384;  // e4m3: warps 2, 3, 12..15 convert
  static constexpr int kConverters = 192;
  static constexpr int kFewRegs = kFp8 ? 72 : 88, kManyRegs = kFp8 ? 184 : 208;
  static_assert((kThreads - 256) * kFewRegs + 256 * kManyRegs <= kThreads * (kFp8 ? 128 : 168),
                "registers of the launch");
  static constexpr int kChunks = D / 64;            // 128-byte pieces of an operand's row
  static constexpr int kChunkBytes = kTile * 128;   // 16 KB
  static constexpr int kOpBytes = kChunks * kChunkBytes;
  static constexpr int kRawBytes = kTile * D;       // an e4m3 operand
  static constexpr int kOps = D == 64 ? (kFp8 ? 6 : 8) : (kFp8 ? 3 : 4);
  static constexpr int kRaws = D == 64 ? 6 : 3;
  static constexpr int kOffOps = 2 * kOpBytes;  // behind two query tiles
  static constexpr int kOffRaw = kOffOps + kOps * kOpBytes;
  static constexpr int kOffScale = kOffRaw + (kFp8 ? kRaws * kRawBytes : 0);
  static constexpr int kOffMl = kOffScale + kScaleTiles * kTileBoxes * 8;
  static constexpr int kOffBars = kOffMl + kSlotThreads * 8;
  static constexpr int kOffMisc = kOffBars + kNumBars * 8;
  static constexpr int kOffPlaces = kOffMisc + 128;
  static constexpr int smem_bytes(int groups) { return kOffPlaces + (groups + 1) * 8 + 1024; }
  static_assert(smem_bytes(kPagedMaxBatch) <= 227 * 1024, "shared memory");
  static_assert(4 * 4 * (kPagedMaxBatch + 1) <= kOffScale, "room for the plan of the groups");
};

// A read that stays where it is: eight scales held over a step cost registers.
__device__ __forceinline__ float lds_f32(const void* at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(smem_u32(at)));
  return v;
}

// A CTA's part of a unit.
struct Part {
  int first, lead;      // the group's first request, and its first that is not empty
  int rows;             // of the block
  int row0;             // of the block within the group
  int kvh;
  int boxes, t0, t1;    // shared boxes; tiles of this part
  bool whole_start;     // it holds the first tile
  int next;             // place of the next unit
  __device__ __forceinline__ int tiles() const { return t1 - t0; }
  __device__ __forceinline__ bool dual() const { return rows > kSlotThreads; }
  // steps of the two slots together: step j is slot j & 1's
  __device__ __forceinline__ int steps() const { return dual() ? 2 * tiles() : tiles(); }
  __device__ __forceinline__ int tile(int j) const { return dual() ? j >> 1 : j; }
};

// The unit that holds place f < the CTA's end `to`.
__device__ __forceinline__ Part part_at(const PagedParams& p, const PrefixParams& x,
                                        const int* places, int f, int to) {
  Part r;
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
      mbar_init(bar(i), slot ? kSlotThreads : i == kQFull ? 2 * kSlotThreads : 1);
    }
    fence_barrier_init();
    tma_prefetch_desc(&kv_map);
  }
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(misc + 24), 512);
    tc::tmem_relinquish();
  }
  // The grid after this one reads ahead of its own wait, which is sound as every CTA of
  // this one has waited before it lets it start.
  griddep_wait();
  griddep_launch_dependents();

  // ---- places of the groups' units ----
  // what stays of the plan: places, and per group the first request and the first that is
  // not empty
  int* rows = places + x.groups + 1;
  int total, share;
  {
    int* mem = reinterpret_cast<int*>(base);
    int* lead = mem + plan_ints(x.groups);
    const GroupPlan plan =
        plan_groups<C::kThreads, true>(p, x, mem, lead, misc, blockIdx.x == 0);
    total = plan.groups ? plan.places[plan.groups] : 0;
    share = plan.share;
    for (int i = tid; i <= plan.groups; i += C::kThreads) {
      places[i] = plan.places[i];
      rows[i] = plan.cu[i] | (i < plan.groups ? min(lead[i], p.B - 1) : 0) << 16;
    }
    fence_proxy_async_smem();  // the plan lies where tiles come
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc + 24);
  const int from = min((long long)blockIdx.x * share, (long long)total);
  const int to = min(from + share, total);
  const uint32_t ops = base_u32 + C::kOffOps;

  // Registers: the softmax warpgroups take what the others give back (at launch 512 x 128, or
  // 384 x 168).
  if (warp < kSlotWarp0 || warp >= kSlotWarp0 + 8) setmaxnreg_dec<C::kFewRegs>();
  if (warp == 0) {
    // ============================ TMA producer ============================
    int op = 0, tiles = 0;  // operands and tiles asked for
    for (int f = from; f < to;) {
      const Part u = part_at(p, x, places, f, to);
      f = u.next;
      if (u.tiles() <= 0) continue;
      const int32_t* table = p.bt + (int64_t)u.lead * p.bt_sb;
      int blk = 0, off = 0;
      float2 scale = make_float2(0.f, 0.f);
      for (int t = u.t0; t < u.t1; ++t, ++tiles) {
        if (((t - u.t0) & 3) == 0) {  // the boxes of four tiles
          const int box = t * kTileBoxes + lane, tok = box * 16;
          blk = p.num_blocks;  // past the cache: reads as zeros
          off = tok & (p.page_size - 1);
          scale = make_float2(0.f, 0.f);
          if (box < u.boxes) {
            const int page = __ldg(table + min(tok >> p.page_shift, p.max_blocks - 1));
            if (page < 0 || page >= p.num_blocks) {
              if (box < u.t1 * kTileBoxes) atomicOr(p.err, DEVERR_BAD_BLOCK);
            } else {
              blk = page;
              if (kFp8)
                scale = __ldg(reinterpret_cast<const float2*>(
                    p.kv_scale + (int64_t)page * p.s_sblk + u.kvh * p.s_sh));
            }
          }
        }
        const bool mine = lane / kTileBoxes == ((t - u.t0) & 3);
        const int box = lane % kTileBoxes;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++op) {
          constexpr int kRing = kFp8 ? C::kRaws : C::kOps;
          const int e = op % kRing, full = (kFp8 ? kRawFull : kOpFull) + e;
          mbar_wait(bar((kFp8 ? kRawEmpty : kOpEmpty) + e), ((op / kRing) & 1) ^ 1u, p.err);
          if (lane == 0) mbar_arrive_expect_tx(bar(full), kFp8 ? C::kRawBytes : C::kOpBytes);
          if (kFp8 && kv == 0) {  // the scales' place is free: see kScaleTiles
            if (mine)
              *reinterpret_cast<float2*>(base + C::kOffScale +
                                         ((tiles % kScaleTiles) * kTileBoxes + box) * 8) = scale;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kScaleFull + tiles % kScaleTiles));
          }
          __syncwarp();
          if (mine) {
            if constexpr (kFp8) {
              tma_load_5d(base_u32 + C::kOffRaw + e * C::kRawBytes + box * 16 * D, &kv_map, bar(full),
                          0, off, kv, u.kvh, blk);
            } else {
#pragma unroll
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_5d(ops + e * C::kOpBytes + c * C::kChunkBytes + box * 2048, &kv_map, bar(full),
                            0, off, kv * C::kChunks + c, u.kvh, blk);
            }
          }
        }
      }
    }
  } else if (warp == 1) {
    // ============================= MMA issuer =============================
    constexpr uint32_t kIdS = tc::idesc_bf16_f32(128, kTile, false, false);
    constexpr uint32_t kIdPv = tc::idesc_bf16_f32(128, D, false, true);
    int op0 = 0, units = 0;
    uint32_t ready[2] = {0, 0};  // phases of P
    for (int f = from; f < to;) {
      const Part u = part_at(p, x, places, f, to);
      f = u.next;
      if (u.tiles() <= 0) continue;
      const int steps = u.steps();
      const bool dual = u.dual();
      mbar_wait(bar(kQFull), units & 1, p.err);
      auto scores = [&](int j) {
        const int slot = j & 1, op = op0 + 2 * u.tile(j), e = op % C::kOps;
        mbar_wait(bar(kOpFull + e), (op / C::kOps) & 1, p.err);
        tc::fence_after_sync();
        const uint32_t a = base_u32 + (dual ? slot : 0) * C::kOpBytes, b = ops + e * C::kOpBytes;
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_bf16_elect(
                tmem + slot * kTile,
                tc::smem_desc(a + c * C::kChunkBytes + ks * 32, 16, 1024, tc::kSwizzle128),
                tc::smem_desc(b + c * C::kChunkBytes + ks * 32, 16, 1024, tc::kSwizzle128), kIdS,
                (c | ks) != 0);
        tc::commit_elect(bar(kSFull + slot));
        if (!dual || slot == 1) tc::commit_elect(bar(kOpEmpty + e));
        if (j == steps - 1) tc::commit_elect(bar(kQFree));
      };
      auto values = [&](int j) {
        const int slot = j & 1, op = op0 + 2 * u.tile(j) + 1, e = op % C::kOps;
        mbar_wait(bar(kOpFull + e), (op / C::kOps) & 1, p.err);
        mbar_wait(bar(kPHalf + slot), ready[slot] & 1, p.err);
        tc::fence_after_sync();
        const uint32_t b = ops + e * C::kOpBytes;
#pragma unroll
        for (int ks = 0; ks < kTile / 16; ++ks) {
          if (ks == kTile / 32) {
            mbar_wait(bar(kPReady + slot), ready[slot] & 1, p.err);
            tc::fence_after_sync();
          }
          tc::mma_bf16_ts_elect(
              tmem + 2 * kTile + slot * D, tmem + slot * kTile + ks * 8,
              tc::smem_desc(b + ks * 2048, C::kChunkBytes, 1024, tc::kSwizzle128), kIdPv,
              j > 1 || ks > 0);
        }
        ++ready[slot];
        if (!dual || slot == 1) tc::commit_elect(bar(kOpEmpty + e));
        if (j + 2 >= steps) tc::commit_elect(bar(kODone + slot));
      };
      scores(0);
      if (steps > 1) scores(1);
      for (int j = 0; j < steps; ++j) {
        values(j);
        if (j + 2 < steps) scores(j + 2);
      }
      op0 += 2 * u.tiles();
      ++units;
    }
  } else if (warp >= kSlotWarp0 && warp < kSlotWarp0 + 8) {
    // ======================= softmax, one thread per row ===================
    setmaxnreg_inc<C::kManyRegs>();
    const int slot = (warp - kSlotWarp0) >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lanes + slot * kTile, tO = tmem + lanes + 2 * kTile + slot * D;
    const float c2 = fmaxf(fabsf(p.scale) * kLog2e, kTiny);
    const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;  // of the query's signs
    float2* other_ml = reinterpret_cast<float2*>(base + C::kOffMl);
    int units = 0, tiles = 0;
    uint32_t got = 0, done[2] = {0, 0};  // phases of S; of O
    for (int f = from; f < to;) {
      const Part u = part_at(p, x, places, f, to);
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
        for (int i = 0; i < kMine; ++i)
          if (i < n)
            *reinterpret_cast<uint4*>(dst + i * kStep * 128) =
                make_uint4(v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(kQFull));
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
          const int valid = min(u.boxes - (u.t0 + t) * kTileBoxes, kTileBoxes);  // boxes
          const float2* sc = reinterpret_cast<const float2*>(base + C::kOffScale) +
                             (at % kScaleTiles) * kTileBoxes;
          uint32_t s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::ld_32x32b_x32(tS + 32 * c, s[c]);
          // log2 units of a score of box h (never 0: no infinity times 0)
          auto unit = [&](int h) { return kFp8 ? fmaxf(c2 * lds_f32(sc + h), kTiny) : c2; };
          tc::wait_ld();
          if (valid < kTileBoxes) {
#pragma unroll
            for (int h = 0; h < kTileBoxes; ++h)
              if (h >= valid)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[h / 2][16 * (h & 1) + i] = 0xff800000u;  // -inf
          }
          float top = -INFINITY;
          {
            float a[kTileBoxes];
#pragma unroll
            for (int h = 0; h < kTileBoxes; ++h) {
              const uint32_t* y = s[h / 2] + 16 * (h & 1);
              a[h] = fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
#pragma unroll
              for (int i = 2; i < 16; i += 2)
                a[h] = fmaxf(fmaxf(a[h], __uint_as_float(y[i])), __uint_as_float(y[i + 1]));
              if (kFp8) a[h] *= unit(h);
            }
#pragma unroll
            for (int h = 0; h < kTileBoxes; h += 2) top = fmaxf(fmaxf(top, a[h]), a[h + 1]);
            if (!kFp8) top *= c2;
          }
          const bool move = top > m + kSlack || (m == -INFINITY && top > m);
          if (__any_sync(0xffffffffu, move)) {
            const float mn = move ? top : m;
            const float keep = m == -INFINITY ? 0.f : ex2(m - mn);
            if (j > 1) {
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tc::ld_32x32b_x16(tO + 16 * c, o);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                tc::st_32x32b_x16(tO + 16 * c, o);
              }
            }
            l *= keep;
            m = mn;
          }
          const float ref = m == -INFINITY ? 0.f : -m;
          float2 sum[2] = {};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int box = 2 * c + h;
              const float ks = unit(box), vs = kFp8 ? lds_f32(&sc[box].y) : 1.f;
              const float2 k2 = make_float2(ks, ks), r2 = make_float2(ref, ref);
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const float2 y = fma2(make_float2(__uint_as_float(s[c][16 * h + i]),
                                                  __uint_as_float(s[c][16 * h + i + 1])), k2, r2);
                float2 e = make_float2(ex2(y.x), ex2(y.y));
                sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], e);
                if (kFp8) e = mul2(e, make_float2(vs, vs));
                w[8 * h + i / 2] = pack_bf16(e.x, e.y);
              }
            }
            tc::st_32x32b_x16(tS + 16 * c, w);
            if (c == 1) {  // the first half's product can begin
              tc::wait_st();
              tc::fence_before_sync();
              mbar_arrive(bar(kPHalf + slot));
            }
          }
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
  } else if (kFp8) {
    // ============= e4m3 operand -> bf16 operand, swizzled for the MMA =============
    const int ct = warp < 4 ? tid - 64 : tid - 384 + 64;  // 0 .. 191
    int op = 0;
    for (int f = from; f < to;) {
      const Part u = part_at(p, x, places, f, to);
      f = u.next;
      for (int i = 0; i < 2 * max(u.tiles(), 0); ++i, ++op) {
        const int er = op % C::kRaws, eo = op % C::kOps;
        mbar_wait(bar(kRawFull + er), (op / C::kRaws) & 1, p.err);
        mbar_wait(bar(kOpEmpty + eo), ((op / C::kOps) & 1) ^ 1u, p.err);
        const uint8_t* src = base + C::kOffRaw + er * C::kRawBytes;
        uint8_t* dst = base + C::kOffOps + eo * C::kOpBytes;
        // 16 codes each; a thread's are kStep rows apart, which keeps the unit and the swizzle
        constexpr int kUnits = D / 16, kStep = C::kConverters / kUnits;
        constexpr int kMine = (kTile + kStep - 1) / kStep;
        static_assert(C::kConverters % kUnits == 0 && kStep % 8 == 0, "converters");
        const int r0 = ct / kUnits, q = ct % kUnits, odd = (q >> 2) & 1;
        // dims 16 q .. + 15: units 2 q' and 2 q' + 1 of piece q / 4, which begin with different
        // units, for the banks
        const uint32_t at = (q >> 2) * C::kChunkBytes + r0 * 128;
        const uint32_t a0 = at + ((2 * (q & 3) + odd) ^ (r0 & 7)) * 16;
        const uint32_t a1 = at + ((2 * (q & 3) + 1 - odd) ^ (r0 & 7)) * 16;
        uint4 w[kMine];
#pragma unroll
        for (int k = 0; k < kMine; ++k)
          if (r0 + k * kStep < kTile)
            w[k] = *reinterpret_cast<const uint4*>(src + (ct + k * C::kConverters) * 16);
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          if (r0 + k * kStep >= kTile) break;
          const uint32_t wv[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
          uint32_t o[8];
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            uint32_t f16x2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f16x2) : "h"((uint16_t)(wv[h / 2] >> (16 * (h & 1)))));
            const float2 fv = __half22float2(*reinterpret_cast<const __half2*>(&f16x2));
            o[h] = pack_bf16(fv.x, fv.y);
          }
          const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
          *reinterpret_cast<uint4*>(dst + a0 + k * kStep * 128) = odd ? hi : lo;
          *reinterpret_cast<uint4*>(dst + a1 + k * kStep * 128) = odd ? lo : hi;
        }
        fence_proxy_async_smem();  // the MMA reads through the async proxy
        __syncwarp();
        named_bar_sync(3, C::kConverters);
        if (ct == 0) {
          mbar_arrive(bar(kRawEmpty + er));
          mbar_arrive(bar(kOpFull + eo));
        }
      }
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
