// paged_attn.cu -- GQA decode attention over a paged cache in which a request
// sees a sliding window and its first tokens, for a bf16 cache and for an e4m3
// cache with one fp32 scale for K and one for V per (page, kv head).
//
// For every request b (length L) and query head h (kv head h / G):
//   x_j = scale * ks(page of j) * q . k_j          (ks = vs = 1 for bf16)
//   out = sum_j e^(x_j - m) vs(page of j) v_j / (sum_j e^(x_j - m) + e^(sink_h - m))
//   lse = m + log sum_j e^(x_j - m)                (keys alone; -inf without a key)
// over j in [0, first) and [max(L - window, 0), L), m = max_j x_j.
//
// Bound by memory: every visible key and value is read once, from DRAM.
//
//  * Work: the 16-token tiles that hold a visible key, laid end to end over
//    (request, kv head) pairs.  CTA c takes an equal share of all tiles plus
//    kPairCost for each pair (starting and ending a pair costs a CTA about as much
//    as that many tiles), so the CTAs end together whatever the lengths; a cut
//    within a few tiles of a pair's border moves to the border.  Each CTA finds its
//    cuts in a prefix sum of the requests' tile counts, in shared memory.
//  * Each of the four warps takes every fourth tile of the CTA's range through a
//    ring of its own: a lane asks for a tile with one TMA operation, the warp reads the
//    fragments of a landed tile into registers, and a lane asks for the next tile
//    into the same stage.  No warp waits for another, and a ring runs on
//    across the borders of requests.  Block-table entries (and scales) are read
//    32 tiles ahead, one lane each.
//  * S[rows x 16 tokens] = Q K^T and O^T[dims x rows] += V^T P^T on
//    mma.m16n8k16, rows = the G query heads (one or two blocks of 8); the second
//    on mma.m16n8k8 in tf32 for e4m3.  e4m3 keys become fp16 and values tf32
//    exactly; the query is scaled to fp16's range by a power of two for each row
//    (exact but for elements below 2^-29 of the row's largest).
//  * One pass with a running reference m near the maximum and the sum l in 32 bits.
//    With scales, the accumulator holds sum_j 2^(x_j + log2 vs_j - R) code_j under a
//    running maximum R of its own, so a page of large or small values keeps its
//    precision.  Each weight is rounded once, to tf32: by 2^-11 of itself, down to 2^-126
//    of the largest.  The largest may be a first token's, or of a page with large
//    values, and have next to nothing to add, so the others need their bits however small
//    they are beside it.  fp16 weights lose them below 2^-14 and all below 2^-25 of it (16
//    nats under a first token without a value, 6000 keys were off by half); they take
//    1 to 2 % less time for heads of 128, 10 to 15 % less for heads of 64 and for 16 rows.
//    For the bf16 cache the weights are rounded to bf16, as V is bf16.
//  * Cluster mode, for few and short requests (the rule is the caller's): a cluster of
//    CTAs takes one pair each, a CTA an equal part of its tiles, and the threads of all
//    merge the parts through distributed shared memory (a 1001-key window on 33 x 4 kv
//    heads 10.7 us; with fp16 weights 10.1, and 12.1 where the first CTA merged alone): no
//    scan of the lengths, no global partials (see launch_paged_attn's caller for what it
//    measured).
//  * Without clusters the kernel chooses by the lengths that it reads.  Warp mode, for
//    many short requests: the shares are the warps', which write a pair that they hold
//    whole from their accumulators, without a merge of warps or a barrier; of the warps
//    that share a pair the last to arrive merges the accumulators that all have
//    published, in order.  Whole pairs, an equal number for each CTA, where that ends no
//    later than equal shares with their merges.
//  * Otherwise, a request cut between CTAs: each publishes its 32-bit (O, m, l, R); the last
//    CTA of a group of up to kMergeGroup (an arrival counter) merges the group, the last
//    group merges the groups: each warp a fourth of the parts in order, then the warps'
//    results (one request of 16000 keys: 16.1 us; with fp16 weights 15.1, and 18.4 where one
//    thread per output went through all parts).  Results do not depend on timing.
//
// Measured (GB300, graph replays; the copy bandwidth is 6786 GB/s): e4m3, 8 requests
// of 131072 keys, 8 kv heads of 128: 314 us = 6.85 TB/s; 64 requests of up to 32768
// keys (272 MB): 51.4 us = 5.3 TB/s, of which 4 us pass before the first tile arrives
// (lengths, table, tile: three dependent reads) and the CTAs end over the last 10;
// bf16, a window of 4096 + 64 on 32 requests: 83 us = 6.4 TB/s; four short requests:
// 5.0 us.  1 GB of e4m3 heads of 128 reads at 96 % (up to 8 query heads per kv head)
// and 80 % (16), of 64 at 83 and 68 % (bound by the latency of a warp's instructions, 12
// warps an SM); bf16 at 97 to 100 %.  A tile's way through a warp is about 700 cycles
// (bf16; e4m3 1200 with fp16 weights), of which the 16 products of S take 150 to 250.
#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kWarps = kPagedWarps;
enum : int {
  kPagedShares,   // CTAs take equal shares of all tiles
  kPagedCluster,  // a cluster of CTAs takes a (request, kv head) pair
  kPagedWarp,     // warps take equal shares of all tiles
};
constexpr int kThreads = kWarps * 32;
// One request of 131072 keys and one kv head: 19.0 us at 16, 19.3 at 12, 20.9 at 8; of 16000
// keys and 8 kv heads: 16.0, 16.2, 15.7; 4 requests of up to 16000: 15.2, 14.4, 14.4.
constexpr int kMergeGroup = 12;
constexpr int kPairCost = kPagedPairCost;
// The same for a warp in the warp mode: 2000 requests of 1 to 64 keys take 14.1 us at
// 2, 15.0 at 3, 14.8 at 5; 1000 x 8 of up to 300 keys 51.9, 50.0, 51.0.
constexpr int kWarpPairCost = 3;
// What cuts inside pairs cost a CTA, in tiles: whole pairs (up to two a CTA) where the
// longest ones end no later.  Tables as wide as for 65536 keys, on / off: 48 x 8 kv heads
// of 800 to 1000 keys 22.3 / 24.2 us, 56 x 8 of 1500 32.2 / 36.9, 400 of 10 to 500 keys
// 12.9 / 14.3; 110 x 8 of 10 to 1000, which the rule leaves, 36.6 / 30.3.
constexpr uint32_t kEndCost = 24;
// A cut this near a pair's border moves there.  Wider costs more than the merges it
// saves: at 32, 33 requests of a 1001-key window take 13.5 us in equal shares, 13.0 at 8.
constexpr int kSnapTiles = 8;
constexpr int kWarpSnapTiles = 4;  // in the warp mode; 8: 45.2 us instead of 40.4 for 256 x 8 pairs
constexpr float kSlack = 8.f;      // log2 units: weights stay below 2^8
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D_, bool kFp8_, int NB_>
struct Cfg {
  static constexpr int D = D_, NB = NB_;
  static constexpr bool kFp8 = kFp8_;
  static constexpr int kRows = 8 * NB;
  // tiles of a step: two of 2 KB share a step's waits and checks (1 GB of e4m3 heads of
  // 64: 178 us, 185 with one), but for 16 rows (222 us, 216 with one)
  static constexpr int U = D == 64 && kFp8 && NB == 1 ? 2 : 1;
  static constexpr int kChunks = 2 * D * (kFp8 ? 1 : 2) / 128;  // 128-byte pieces of a [K | V] row
  static constexpr int kTileBytes = 16 * 128 * kChunks;
  // CTAs per SM, as many as the registers of the loop allow without spilling (four for
  // e4m3 heads of 64 spilled, with fp16 weights: 1 GB at 79 % of the copy bandwidth, not 91)
  static constexpr int kCtas = D == 128 ? (NB == 1 && kFp8 ? 3 : 2) : (NB == 1 && !kFp8 ? 4 : 3);
  static constexpr int kWbRow = D + 4;
  static constexpr int kWbFloats = kRows * kWbRow + 3 * kRows;  // O, m, l, R of one warp
  static constexpr int kPartFloats = kRows * D + 3 * kRows;
  // query rows of two pairs (of one where two do not fit beside two stages)
  static constexpr int kQSlots = D == 128 && NB == 2 && !kFp8 ? 1 : 2;
  static constexpr int kQBytes = kQSlots * kRows * D * 2;
  // Stages of a warp's ring: 96 to 128 KB asked for per SM.  More is not better: three
  // stages for e4m3 heads of 128 (144 KB) read 8 x 131072 keys in 332 us, two in 317 (fp16
  // weights); fewer than five for e4m3 heads of 64: 1 GB in 182 us (4), 180 (3), against 178.
  static constexpr int kStages = kTileBytes == 2048 ? 5 : kTileBytes == 4096 && kCtas == 2 ? 3 : 2;
  static constexpr int kOffWb = kWarps * kStages * kTileBytes;
  static constexpr int kOffQ = kOffWb + kWarps * kWbFloats * 4;
  static constexpr int kOffBars = kOffQ + kQBytes;
  static constexpr int kOffMisc = kOffBars + kWarps * kStages * 8;
  static constexpr int kOffPrefix = kOffMisc + 64;
  static constexpr int smem_bytes(int B) { return kOffPrefix + (B + 1) * 4 + 1024; }
  static_assert(kOffWb % 1024 == 0 && kOffQ % 16 == 0 && kOffBars % 8 == 0, "shared-memory offsets");
  static_assert(kStages <= 32, "a batch of look-ups covers the ring");
  static_assert(kWarps * 2 * kRows * D * 2 <= kWarps * kWbFloats * 4, "query rows of the warps");
  static_assert(kCtas * (smem_bytes(kPagedMaxBatch) + 1024) <= 228 * 1024, "CTAs per SM");
};

// The tiles that a request of length L needs: [0, head) and [head + gap, end).
struct Span {
  int L, start, first;  // visible: j < first, or start <= j < L
  int head, gap, tiles;
};

__device__ __forceinline__ Span span_of(const PagedParams& p, int raw) {
  Span s;
  s.L = min(max(raw, 0), p.max_blocks * p.page_size);
  s.start = (p.window > 0 && s.L > p.window) ? s.L - p.window : 0;
  s.first = min(p.first, s.start);
  const int end = (s.L + 15) >> 4, from = s.start >> 4;
  s.head = (s.first + 15) >> 4;
  if (s.head >= from) s.head = from;
  s.gap = from - s.head;
  s.tiles = end - s.gap;
  return s;
}

// Exclusive scan of one int per thread over the CTA; scratch: one int per warp.
__device__ __forceinline__ int block_scan(int v, int* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < kWarps - 1; ++w) before += w < warp ? scratch[w] : 0;
  return before + incl - v;
}

// Places count tiles of all pairs in order (or tiles and pair costs): below 2^31,
// which the host sees to.
struct Pair {
  int b, kvh, n;  // request, kv head, tiles
  int begin;      // place of its first tile
};

// The pair at place f when request b's pairs begin at place (prefix[b] + extra b) Hkv
// and are `extra` + its tiles long.  lo: the request.
template <int extra>
__device__ __forceinline__ Pair pair_of(const int* prefix, int Hkv, int f, int lo) {
  Pair r;
  r.b = lo;
  r.n = prefix[lo + 1] - prefix[lo];
  const int base = (prefix[lo] + extra * lo) * Hkv, len = r.n + extra;
  r.kvh = (int)((uint32_t)(f - base) / (uint32_t)len);
  r.begin = base + r.kvh * len;
  return r;
}

// For one lane: the last request that begins at or before f, by bisection.
template <int extra>
__device__ __forceinline__ Pair pair_at_lane(const int* prefix, int B, int Hkv, int f) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((prefix[mid] + extra * mid) * Hkv <= f) lo = mid; else hi = mid - 1;
  }
  return pair_of<extra>(prefix, Hkv, f, lo);
}

// For groups of kLanes lanes (a warp, or its halves) with one f each: kLanes
// requests at a time (2 steps for up to kLanes^2 requests).
template <int extra, int kLanes>
__device__ __forceinline__ Pair pair_at_group(const int* prefix, int B, int Hkv, int f) {
  const int lane = threadIdx.x & 31, sub = lane % kLanes, step = (B + kLanes - 1) / kLanes;
  const uint32_t group = kLanes == 32 ? 0xffffffffu : 0xffffu << (lane & 16);
  auto before = [&](int b) {  // how many of the group's requests begin at or before f
    const bool yes = b < B && (prefix[b] + extra * b) * Hkv <= f;
    return __popc(__ballot_sync(0xffffffffu, yes) & group);
  };
  int lo = before(min(sub * step, B)) - 1;
  if (step > 1) {
    const int base = lo * step, end = min(base + step, B);
    int cnt = 0;
    for (int i = 0; i < step; i += kLanes)
      cnt += before(base + i + sub < end ? base + i + sub : B);
    lo = base + cnt - 1;
  }
  return pair_of<extra>(prefix, Hkv, f, lo);
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {  // RNE, lo in bits 0..15
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 codes (bits 0..15) to fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16_hi(uint32_t w) {  // bits 16..31
  uint32_t r;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(r) : "r"(w));
  return r;
}

// 16 bytes to shared memory, `bytes` of them from src, the rest zero.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <bool kFp16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (kFp16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    mma_bf16_16816(d, a0, a1, a2, a3, b0, b1);
}

// The same with C = 0.
template <bool kFp16>
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (kFp16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// D += A B over 8 tokens in tf32: 11 significant bits and the exponents of 32-bit values.
__device__ __forceinline__ void mma_tf32(float (&d)[4], float a0, float a1, float a2, float a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)),
        "r"(__float_as_uint(a3)), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t to_tf32(float x) {  // to nearest
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float2 f16x2_f32(uint32_t w) {
  float2 f;
  asm("{.reg .f16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}"
      : "=f"(f.x), "=f"(f.y) : "r"(w));
  return f;
}

// This thread's part of the output: row er (a query head of the kv head), dims
// [ed, ed + N); sink in log2 units, -inf for none.
template <class C, int N>
__device__ __forceinline__ void finalize(const PagedParams& p, int b, int kvh, int er, int ed,
                                         float sink, const float (&o)[N], float m, float l, float R) {
  if (er >= p.G) return;
  const int head = kvh * p.G + er;
  float f = 0.f;
  if (l != 0.f) {
    const float den = l + ex2(sink - m);
    f = (C::kFp8 ? ex2(R - m) : 1.f) / den;
  }
  uint16_t* dst = p.out + b * p.o_sb + head * p.o_sh + ed;
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f),
                   pack_bf16(o[4] * f, o[5] * f), pack_bf16(o[6] * f, o[7] * f));
  else
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f));
  if (ed == 0 && p.lse)
    p.lse[b * p.lse_sb + head * p.lse_sh] = l != 0.f ? __fmaf_rn(m, kLn2, logf(l)) : -INFINITY;
}

// Weight of a partial with reference r under the common reference M.
__device__ __forceinline__ float weight(float r, float M) { return r == -INFINITY ? 0.f : ex2(r - M); }

template <class C>
__device__ __forceinline__ void store_partial(const PagedParams& p, int slot, int er, int ed,
                                              const float (&o)[C::D / 16], float m, float l, float R) {
  float* dst = p.partials + (int64_t)slot * C::kPartFloats + er * C::D + ed;
#pragma unroll
  for (int e = 0; e < C::D / 16; e += 4)
    *reinterpret_cast<float4*>(dst + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
  if (ed == 0) {
    float* st = p.partials + (int64_t)slot * C::kPartFloats + C::kRows * C::D + er;
    st[0] = m;
    st[C::kRows] = l;
    st[2 * C::kRows] = R;
  }
}

// The four warps' (O, m, l, R) in shared memory merged, for rows er and er + 8, dims
// [ed, ed + E).
template <class C>
__device__ __forceinline__ void combine_warps(const float* wbuf, int er, int ed,
                                              float (&o)[C::NB][C::D / 16], float (&mc)[C::NB],
                                              float (&lc)[C::NB], float (&Rc)[C::NB]) {
  constexpr int E = C::D / 16;
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb) {
    const float* st = wbuf + C::kRows * C::kWbRow + er + 8 * nb;
    mc[nb] = Rc[nb] = -INFINITY;
    lc[nb] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      mc[nb] = fmaxf(mc[nb], st[w * C::kWbFloats]);
      Rc[nb] = fmaxf(Rc[nb], st[w * C::kWbFloats + 2 * C::kRows]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) o[nb][e] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* sw = st + w * C::kWbFloats;
      lc[nb] = __fmaf_rn(weight(sw[0], mc[nb]), sw[C::kRows], lc[nb]);
      const float wt = weight(sw[2 * C::kRows], Rc[nb]);
      const float* ow = wbuf + w * C::kWbFloats + (er + 8 * nb) * C::kWbRow + ed;
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 a = *reinterpret_cast<const float4*>(ow + e);
        o[nb][e] = __fmaf_rn(wt, a.x, o[nb][e]);
        o[nb][e + 1] = __fmaf_rn(wt, a.y, o[nb][e + 1]);
        o[nb][e + 2] = __fmaf_rn(wt, a.z, o[nb][e + 2]);
        o[nb][e + 3] = __fmaf_rn(wt, a.w, o[nb][e + 3]);
      }
    }
  }
}

// Slot of a pair's part i, whose first part is CTA (warp) c0's.
__device__ __forceinline__ int part_slot(int c0, int i) { return 2 * (c0 + i) + (i == 0 ? 1 : 0); }

// The warp's part of merging a pair's parts first, first + step, .. before end: every
// fourth, in order, into its own (O, m, l, R) in shared memory.  A lane has floats
// 128 u + 4 lane .. + 3 of the partial, and the statistics of row `lane`.  A call, as its
// registers would cost the loop over tiles some of its own (e4m3 heads of 64 on 1 GB, with
// fp16 weights: 91 % of the copy bandwidth, 90 inlined).
template <class C>
__device__ __noinline__ void gather_partials(const float* partials, int c0, int first, int step,
                                             int end, float* wb) {
  constexpr int kUnits = C::kRows * C::D / 128;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float m = -INFINITY, l = 0.f, R = -INFINITY;
  float4 a[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) a[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = first + warp * step; i < end; i += kWarps * step) {
    const float* src = partials + (int64_t)part_slot(c0, i) * C::kPartFloats;
    const float* st = src + C::kRows * C::D + min(lane, C::kRows - 1);
    const float mk = __ldcg(st), lk = __ldcg(st + C::kRows), Rk = __ldcg(st + 2 * C::kRows);
    float4 v[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) v[u] = ldcg_f4(src + 128 * u + 4 * lane);
    const float mn = fmaxf(m, mk), Rn = fmaxf(R, Rk);
    l = __fmaf_rn(weight(m, mn), l, weight(mk, mn) * lk);
    const float keep = weight(R, Rn), add = weight(Rk, Rn);
    m = mn;
    R = Rn;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int row = (128 * u + 4 * lane) / C::D;
      const float x = __shfl_sync(0xffffffffu, keep, row), y = __shfl_sync(0xffffffffu, add, row);
      a[u].x = __fmaf_rn(x, a[u].x, y * v[u].x);
      a[u].y = __fmaf_rn(x, a[u].y, y * v[u].y);
      a[u].z = __fmaf_rn(x, a[u].z, y * v[u].z);
      a[u].w = __fmaf_rn(x, a[u].w, y * v[u].w);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int i = 128 * u + 4 * lane;
    *reinterpret_cast<float4*>(wb + i / C::D * C::kWbRow + i % C::D) = a[u];
  }
  if (lane < C::kRows) {
    float* st = wb + C::kRows * C::kWbRow + lane;
    st[0] = m;
    st[C::kRows] = l;
    st[2 * C::kRows] = R;
  }
}

// The same for a warp whose lanes hold the accumulators of the products: lane
// (g, t) = (lane / 4, lane % 4) has columns 2t and 2t + 1, which are the kv head's query
// rows 8 nb + 2t and 8 nb + 2t + 1, and the statistics of rows 8 nb + g.
template <class C>
__device__ __forceinline__ void warp_store_partial(const PagedParams& p, int slot,
                                                   const float (&acc)[C::NB][C::D / 16][4],
                                                   const float (&m)[C::NB], const float (&l)[C::NB],
                                                   const float (&R)[C::NB]) {
  const int lane = threadIdx.x & 31;
  float* dst = p.partials + (int64_t)slot * C::kPartFloats;
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb) {
#pragma unroll
    for (int c = 0; c < C::D / 16; ++c)
      *reinterpret_cast<float4*>(dst + ((nb * (C::D / 16) + c) * 32 + lane) * 4) =
          make_float4(acc[nb][c][0], acc[nb][c][1], acc[nb][c][2], acc[nb][c][3]);
    if ((lane & 3) == 0) {
      float* st = dst + C::kRows * C::D + 8 * nb + (lane >> 2);
      st[0] = m[nb];
      st[C::kRows] = l[nb];
      st[2 * C::kRows] = C::kFp8 ? R[nb] : m[nb];
    }
  }
}

template <class C>
__device__ __forceinline__ void warp_merge_partials(const PagedParams& p, int c0, int n,
                                                    float (&acc)[C::NB][C::D / 16][4],
                                                    float (&m)[C::NB], float (&l)[C::NB],
                                                    float (&R)[C::NB]) {
  const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb) {
    m[nb] = R[nb] = -INFINITY;
    l[nb] = 0.f;
#pragma unroll
    for (int c = 0; c < C::D / 16; ++c)
      acc[nb][c][0] = acc[nb][c][1] = acc[nb][c][2] = acc[nb][c][3] = 0.f;
    for (int k = 0; k < n; ++k) {
      const float* src = p.partials + (int64_t)part_slot(c0, k) * C::kPartFloats;
      const float* st = src + C::kRows * C::D + 8 * nb + (lane >> 2);
      const float mk = __ldcg(st), lk = __ldcg(st + C::kRows), Rk = __ldcg(st + 2 * C::kRows);
      float4 v[C::D / 16];
#pragma unroll
      for (int c = 0; c < C::D / 16; ++c)
        v[c] = ldcg_f4(src + ((nb * (C::D / 16) + c) * 32 + lane) * 4);
      const float mn = fmaxf(m[nb], mk), Rn = fmaxf(R[nb], Rk);
      l[nb] = __fmaf_rn(weight(m[nb], mn), l[nb], weight(mk, mn) * lk);
      const float a = weight(R[nb], Rn), w = weight(Rk, Rn);
      m[nb] = mn;
      R[nb] = Rn;
      const float a0 = __shfl_sync(0xffffffffu, a, 8 * t), a1 = __shfl_sync(0xffffffffu, a, 8 * t + 4);
      const float w0 = __shfl_sync(0xffffffffu, w, 8 * t), w1 = __shfl_sync(0xffffffffu, w, 8 * t + 4);
#pragma unroll
      for (int c = 0; c < C::D / 16; ++c) {
        acc[nb][c][0] = __fmaf_rn(a0, acc[nb][c][0], w0 * v[c].x);
        acc[nb][c][1] = __fmaf_rn(a1, acc[nb][c][1], w1 * v[c].y);
        acc[nb][c][2] = __fmaf_rn(a0, acc[nb][c][2], w0 * v[c].z);
        acc[nb][c][3] = __fmaf_rn(a1, acc[nb][c][3], w1 * v[c].w);
      }
    }
  }
}

template <class C>
__device__ __forceinline__ void warp_finalize(const PagedParams& p, int b, int kvh,
                                              const float (&sink)[C::NB],
                                              const float (&acc)[C::NB][C::D / 16][4],
                                              const float (&m)[C::NB], const float (&l)[C::NB],
                                              const float (&R)[C::NB]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint16_t* out = p.out + b * p.o_sb + (int64_t)(kvh * p.G) * p.o_sh;
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb) {
    const int row = 8 * nb + g, r0 = 8 * nb + 2 * t;
    float f = 0.f;
    if (l[nb] != 0.f)
      f = (C::kFp8 ? ex2(R[nb] - m[nb]) : 1.f) / (l[nb] + ex2(sink[nb] - m[nb]));
    if (t == 0 && p.lse && row < p.G)
      p.lse[b * p.lse_sb + (kvh * p.G + row) * p.lse_sh] =
          l[nb] != 0.f ? __fmaf_rn(m[nb], kLn2, logf(l[nb])) : -INFINITY;
    const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
    for (int c = 0; c < C::D / 16; ++c) {
      const float(&a)[4] = acc[nb][c];
      if constexpr (C::kFp8) {  // dims 16 c + 2g and the next of both rows
        uint16_t* dst = out + 16 * c + 2 * g;
        if (r0 < p.G)
          *reinterpret_cast<uint32_t*>(dst + r0 * p.o_sh) = pack_bf16(a[0] * f0, a[2] * f0);
        if (r0 + 1 < p.G)
          *reinterpret_cast<uint32_t*>(dst + (r0 + 1) * p.o_sh) = pack_bf16(a[1] * f1, a[3] * f1);
      } else {
        // dims 16 c + g and 16 c + 8 + g of both rows: lanes of an even g and the next
        // trade, so that each has two dims of one row to write
        const bool odd = g & 1;
        const float x = __shfl_xor_sync(0xffffffffu, odd ? a[0] * f0 : a[1] * f1, 4);
        const float y = __shfl_xor_sync(0xffffffffu, odd ? a[2] * f0 : a[3] * f1, 4);
        uint16_t* dst = out + (r0 + odd) * p.o_sh + 16 * c + (g & ~1);
        if (r0 + odd < p.G) {
          *reinterpret_cast<uint32_t*>(dst) =
              odd ? pack_bf16(x, a[1] * f1) : pack_bf16(a[0] * f0, x);
          *reinterpret_cast<uint32_t*>(dst + 8) =
              odd ? pack_bf16(y, a[3] * f1) : pack_bf16(a[2] * f0, y);
        }
      }
    }
  }
}

// The CTA's work, after the prologue below.  next: the pair in the cluster mode; whole:
// equal numbers of pairs for the CTAs instead of equal shares of tiles.
template <class C, int kMode>
__device__ __forceinline__ void attend(const PagedParams& p, const CUtensorMap& kv_map,
                                       uint8_t* base, uint32_t base_u32, Pair next, bool whole) {
  constexpr bool kCluster = kMode == kPagedCluster, kPerWarp = kMode == kPagedWarp;
  constexpr int D = C::D, NB = C::NB, U = C::U, kStages = C::kStages, E = D / 16;
  constexpr bool kFp8 = C::kFp8;
  constexpr int kCost = kPerWarp ? kWarpPairCost : kPairCost;
  float* wbuf = reinterpret_cast<float*>(base + C::kOffWb);
  int* misc = reinterpret_cast<int*>(base + C::kOffMisc);
  const int* prefix = reinterpret_cast<const int*>(base + C::kOffPrefix);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = base_u32 + warp * kStages * C::kTileBytes;
  const uint32_t bars = base_u32 + C::kOffBars + warp * kStages * 8;
  const int B = p.B, Hkv = p.Hkv;

  // This CTA's tiles (the warp's in the warp mode) are [f0, f1) of all pairs' (of one
  // pair's in the cluster mode).
  int f0, f1, chunk = 0, snap = 0;
  const int part = kCluster ? (int)blockIdx.x % p.cluster : 0;
  if constexpr (kCluster) {
    f0 = (int)((long long)next.n * part / p.cluster);
    f1 = (int)((long long)next.n * (part + 1) / p.cluster);
  } else if (whole) {
    auto place = [&](uint32_t cta) {  // of the first tile of its first pair
      const int i = (int)((long long)B * Hkv * cta / gridDim.x), b = i / Hkv;
      return b == B ? prefix[B] * Hkv
                    : prefix[b] * Hkv + i % Hkv * (prefix[b + 1] - prefix[b]);
    };
    f0 = place(blockIdx.x);
    f1 = place(blockIdx.x + 1);
  } else {
    // cuts are placed in the space of costs and turned into places of tiles
    const int tiles = prefix[B] * Hkv, total = tiles + kCost * B * Hkv;
    const uint32_t shares = kPerWarp ? gridDim.x * kWarps : gridDim.x;
    const uint32_t share = kPerWarp ? blockIdx.x * kWarps + warp : blockIdx.x;
    chunk = max((int)(((uint32_t)total + shares - 1) / shares), kPerWarp ? 1 : kPagedMinCost);
    snap = min(kPerWarp ? kWarpSnapTiles : kSnapTiles, chunk / 2);
    // lanes 0..15 place this share's cut, lanes 16..31 the next one's
    const long long x = ((long long)share + (lane >> 4)) * chunk;
    const int y = (int)min(x, (long long)total - 1);
    const Pair r = pair_at_group<kCost, 16>(prefix, B, Hkv, y);
    const int at = y - r.begin - kCost;  // the pair's tiles before the cut
    int f = prefix[r.b] * Hkv + r.kvh * r.n + (at <= snap ? 0 : r.n - at <= snap ? r.n : at);
    if (x >= total) f = tiles;
    f0 = __shfl_sync(0xffffffffu, f, 0);
    f1 = __shfl_sync(0xffffffffu, f, 16);
  }
  // this warp's n-th tile is at place w0 + kStep n
  constexpr int kStep = kPerWarp ? 1 : kWarps;
  const int w0 = kPerWarp ? f0 : f0 + warp;
  const int count = f1 > w0 ? (f1 - w0 + kStep - 1) / kStep : 0;

  // ---- the loader ----
  const int pshift = p.page_shift;
  int l_blk = 0, l_pos = 0;     // lane's tile of the batch of 32: page; kv head, tile in the page
  int n_blk = 0, n_pos = 0;     // the same of the next batch
  float2 sc0 = make_float2(0.f, 0.f), sc1 = sc0;  // (ks, vs) of an even, an odd batch
  auto look_up = [&](int n) {
    n_blk = n_pos = 0;
    if (n >= count) return;
    const int f = w0 + kStep * n;
    const Pair r = kCluster || (f >= next.begin && f < next.begin + next.n)
                       ? next : pair_at_lane<0>(prefix, B, Hkv, f);
    const Span s = span_of(p, __ldg(p.seq_lens + r.b));
    int tau = f - r.begin;
    if (tau >= s.head) tau += s.gap;
    const int page = min(tau >> (pshift - 4), p.max_blocks - 1);  // whatever the lengths do meanwhile
    n_pos = (r.kvh << 3) | (tau & ((1 << (pshift - 4)) - 1));
    n_blk = __ldg(p.bt + r.b * p.bt_sb + page);
  };
  // batch `at` becomes the current one
  auto turn = [&](int at) {
    l_blk = n_blk;
    l_pos = n_pos;
    const bool in = 32 * at + lane < count, good = l_blk >= 0 && l_blk < p.num_blocks;
    if (in && !good) atomicOr(p.err, DEVERR_BAD_BLOCK);  // reads as zeros
    if (kFp8) {
      const float2* at_scale = reinterpret_cast<const float2*>(
          p.kv_scale + (int64_t)l_blk * p.s_sblk + (l_pos >> 3) * p.s_sh);
      // no use of the loaded value here: nothing waits for it
      if (at & 1) {
        sc1 = make_float2(0.f, 0.f);
        if (in && good) sc1 = __ldg(at_scale);
      } else {
        sc0 = make_float2(0.f, 0.f);
        if (in && good) sc0 = __ldg(at_scale);
      }
    }
  };
  auto issue = [&](int n, int s) {  // tile n < count into stage s = n % kStages
    if ((n & 15) == 0) {
      if (n & 16) look_up((n & ~31) + 32 + lane);  // the next batch
      else turn(n >> 5);
    }
    if (lane == (n & 31)) {  // the lane that looked the tile up
      mbar_arrive_expect_tx(bars + 8 * s, C::kTileBytes);
      tma_load_5d(ring + s * C::kTileBytes, &kv_map, bars + 8 * s, 0, (l_pos & 7) * 16, 0,
                  l_pos >> 3, l_blk);
    }
  };
  // The 8 (16) query rows of a pair, 16 bytes a thread, rows past the group zero.  A
  // warp that has pairs of its own keeps their rows where others merge.
  constexpr int kQSlots = kPerWarp ? 2 : C::kQSlots;
  uint16_t* qbuf = kPerWarp ? reinterpret_cast<uint16_t*>(wbuf) + warp * 2 * C::kRows * D
                            : reinterpret_cast<uint16_t*>(base + C::kOffQ);
  auto load_q = [&](const Pair& r, int slot) {
#pragma unroll
    for (int i = kPerWarp ? lane : tid; i < C::kRows * D / 8; i += kPerWarp ? 32 : kThreads) {
      const int row = i / (D / 8), d = i % (D / 8) * 8;
      const bool in = row < p.G;
      cp_async_16(smem_u32(qbuf + (slot * C::kRows + row) * D + d),
                  p.q + r.b * p.q_sb + (r.kvh * p.G + (in ? row : 0)) * p.q_sh + d, in ? 16 : 0);
    }
  };
  int slot = 0;
  if (f0 < f1) {
    if (!kCluster) next = pair_at_group<0, 32>(prefix, B, Hkv, f0);
    load_q(next, 0);
  }
  __syncwarp();  // the ring's barriers are lane 0's
  look_up(lane);
  int issued = 0;
  for (; issued < min(count, kStages); ++issued) issue(issued, issued);

  // ---- fragment addresses ----
  // ldmatrix: matrix mi = lane / 8 takes its 8 rows from lanes 8 mi .. 8 mi + 7.
  // K: matrices (tokens 0..7, unit u), (0..7, u + 1), (8..15, u), (8..15, u + 1).
  // V (transposed): (tokens 0..7, unit u), (8..15, u), (0..7, u + 1), (8..15, u + 1).
  // The 128-byte swizzle XORs a 16-byte unit's index with its token modulo 8.
  const int g = lane >> 2, t = lane & 3, mi = lane >> 3, r8 = lane & 7;
  // A row's unit u = 8 c + v is unit v of 128-byte piece c: 2048 c bytes on, and, with
  // the lane's own bit of v and its row's swizzle in the base, v's other bits by XOR.
  const uint32_t k_base = (uint32_t)(r8 + 8 * (mi >> 1)) * 128u + (uint32_t)((mi & 1) ^ r8) * 16u;
  const uint32_t v_base = (uint32_t)(r8 + 8 * (mi & 1)) * 128u + (uint32_t)((mi >> 1) ^ r8) * 16u;
  auto at_unit = [](uint32_t row_base, int unit) {  // unit even
    return (row_base ^ (uint32_t)(unit & 7) * 16u) + (uint32_t)(unit >> 3) * 2048u;
  };
  constexpr int kUnits = D * (kFp8 ? 1 : 2) / 16;  // 16-byte units of a K (or V) row

  const int er = tid >> 4, ed = (tid & 15) * E;  // this thread's part of an output
  const int sr = kPerWarp ? g : er;  // the row whose sink this thread needs
  float* my_wb = wbuf + warp * C::kWbFloats;
  bool ok = true;
  int n = 0, stage = 0;  // the warp's next tile and its stage
  uint32_t parity = 0;

  for (int f = f0; f < f1;) {
    const Pair pr = next;
    cp_async_wait_all();
    if (kPerWarp) __syncwarp(); else __syncthreads();  // the query rows are in; wbuf and misc are free
    const int seg_end = min(pr.begin + pr.n, f1);
    const Span sp = span_of(p, __ldg(p.seq_lens + pr.b));

    // ---- the query rows as the A operand; the next pair's rows are asked for ----
    const uint16_t* q_rows = qbuf + slot * C::kRows * D;
    if (!kCluster && seg_end < f1) {
      next = pair_at_group<0, 32>(prefix, B, Hkv, seg_end);
      if (kQSlots == 2) load_q(next, slot ^ 1);
    }
    float sink[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      sink[nb] = p.sinks && sr + 8 * nb < p.G
                     ? __ldg(p.sinks + pr.kvh * p.G + sr + 8 * nb) * kLog2e : -INFINITY;
    uint32_t qa[D / 16][2 * NB];
    float row_scale[NB];  // logits of row g (g + 8) in log2 units per unit of S
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const uint16_t* q = q_rows + (g + 8 * nb) * D;
      row_scale[nb] = p.scale * kLog2e;
      if constexpr (kFp8) {
        // k-step c, columns 2t, 2t + 1, 2t + 8, 2t + 9 <- dims 16 c + 4 t .. + 3
        uint2 w[D / 16];
        uint32_t big = 0;  // largest magnitude, as bits
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          w[c] = *reinterpret_cast<const uint2*>(q + 16 * c + 4 * t);
          big = max(max(big, max((w[c].x << 16) & 0x7fffffffu, w[c].x & 0x7fff0000u)),
                    max((w[c].y << 16) & 0x7fffffffu, w[c].y & 0x7fff0000u));
        }
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^up brings the largest element into [2^14, 2^15); 0 and non-finite rows stay
        const int ex = (int)(big >> 23);
        const int up = ex == 0 || ex == 255 ? 0 : max(min(127 + 14 - ex, 126), -126);
        const float mul = __uint_as_float((uint32_t)(up + 127) << 23);
        row_scale[nb] *= __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          qa[c][nb] = pack_f16(__uint_as_float(w[c].x << 16) * mul,
                               __uint_as_float(w[c].x & 0xffff0000u) * mul);
          qa[c][NB + nb] = pack_f16(__uint_as_float(w[c].y << 16) * mul,
                                    __uint_as_float(w[c].y & 0xffff0000u) * mul);
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          qa[c][nb] = *reinterpret_cast<const uint32_t*>(q + 16 * c + 2 * t);
          qa[c][NB + nb] = *reinterpret_cast<const uint32_t*>(q + 16 * c + 8 + 2 * t);
        }
      }
    }

    if (!kCluster && kQSlots == 1 && seg_end < f1) {
      __syncthreads();  // every warp has its rows
      load_q(next, 0);
    }

    float acc[NB][E][4];
    float m[NB], l[NB], R[NB], m_ref[NB], R_ref[NB];  // m_ref: m, or 0 before a key was seen
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb] = R[nb] = -INFINITY;
      m_ref[nb] = R_ref[nb] = 0.f;
      l[nb] = 0.f;
#pragma unroll
      for (int c = 0; c < E; ++c) acc[nb][c][0] = acc[nb][c][1] = acc[nb][c][2] = acc[nb][c][3] = 0.f;
    }

    const int seg_n = (seg_end - w0 + kStep - 1) / kStep;  // this warp's tiles end here
    for (int took; ok && n < seg_n; n += took) {
      took = min(U, seg_n - n);
      int at[U];  // stages; an absent second tile reads the first again and counts for nothing
      uint32_t par[U];
      at[0] = stage;
      par[0] = parity;
      if (++stage == kStages) stage = 0, parity ^= 1;
      if (U == 2) {
        at[U - 1] = took == 2 ? stage : at[0];
        par[U - 1] = took == 2 ? parity : par[0];
        if (took == 2 && ++stage == kStages) stage = 0, parity ^= 1;
      }
      // the scales of the tiles, before their batch's registers can be turned over
      float ks[U], lv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        ks[u] = 1.f;
        lv[u] = 0.f;
        if (kFp8) {
          const int k = U == 2 && u >= took ? n : n + u;
          const bool odd = k & 32;
          ks[u] = __shfl_sync(0xffffffffu, odd ? sc1.x : sc0.x, k & 31);
          lv[u] = lg2(__shfl_sync(0xffffffffu, odd ? sc1.y : sc0.y, k & 31));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) ok = mbar_wait(bars + 8 * at[u], par[u], p.err) && ok;
      if (!ok) break;
      uint32_t kf[U][kUnits / 2][4], vf[U][kUnits / 2][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t tile = ring + at[u] * C::kTileBytes;
#pragma unroll
        for (int i = 0; i < kUnits / 2; ++i)
          ldsm_x4(at_unit(tile + k_base, 2 * i), kf[u][i][0], kf[u][i][1], kf[u][i][2], kf[u][i][3]);
#pragma unroll
        for (int i = 0; i < kUnits / 2; ++i)
          ldsm_x4_trans(at_unit(tile + v_base, kUnits + 2 * i), vf[u][i][0], vf[u][i][1],
                        vf[u][i][2], vf[u][i][3]);
      }
      // ---- S = Q K^T: tokens 0..7 (sa) and 8..15 (sb), kChains sums each ----
      constexpr int kChains = D == 128 ? 2 : 1;
      float sa[U][kChains][4], sb[U][kChains][4];
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const uint32_t a0 = qa[c][0], a1 = NB == 2 ? qa[c][1] : 0u;
        const uint32_t a2 = qa[c][NB], a3 = NB == 2 ? qa[c][NB + 1] : 0u;
        const int ch = c % kChains;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t x0, x1, y0, y1;
          if constexpr (kFp8) {
            const uint32_t x = kf[u][c / 2][c & 1], y = kf[u][c / 2][2 + (c & 1)];
            x0 = e4m3x2_f16(x); x1 = e4m3x2_f16_hi(x);
            y0 = e4m3x2_f16(y); y1 = e4m3x2_f16_hi(y);
          } else {
            x0 = kf[u][c][0]; x1 = kf[u][c][1];
            y0 = kf[u][c][2]; y1 = kf[u][c][3];
          }
          if (c < kChains) {
            mma0<kFp8>(sa[u][ch], a0, a1, a2, a3, x0, x1);
            mma0<kFp8>(sb[u][ch], a0, a1, a2, a3, y0, y1);
          } else {
            mma<kFp8>(sa[u][ch], a0, a1, a2, a3, x0, x1);
            mma<kFp8>(sb[u][ch], a0, a1, a2, a3, y0, y1);
          }
        }
      }
      // The fragments are in registers: the stages are free.  Asking for their next
      // tiles takes the issuing lane some 150 cycles, which the products above cover.
      fence_proxy_async_smem();
      __syncwarp();
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < took && issued < count) issue(issued++, at[u]);

      // logits in log2 units: tokens 2t, 2t + 1, 2t + 8, 2t + 9
      float x[NB][U][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float c2 = kFp8 ? row_scale[nb] * ks[u] : row_scale[nb];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float(&sx)[kChains][4] = i < 2 ? sa[u] : sb[u];
            const int e = 2 * nb + (i & 1);
            x[nb][u][i] = (kChains == 2 ? sx[0][e] + sx[kChains - 1][e] : sx[0][e]) * c2;
          }
        }

      // ---- visibility ----
#pragma unroll
      for (int u = 0; u < U; ++u) {
        int tau = w0 - pr.begin + kStep * (n + u);
        if (tau >= sp.head) tau += sp.gap;
        const int tok = tau * 16;
        if (u < took && tok + 16 <= sp.L && (tok >= sp.start || tok + 16 <= sp.first)) continue;
        bool see[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = tok + 2 * t + (i & 1) + 8 * (i >> 1);
          see[i] = u < took && j < sp.L && (j >= sp.start || j < sp.first);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            if (!see[i]) x[nb][u][i] = -INFINITY;
        }
        // values that nobody sees may be anything: zero them, as 0 * NaN is NaN
        const uint32_t mlo = (see[0] ? 0xffffu : 0u) | (see[1] ? 0xffff0000u : 0u);
        const uint32_t mhi = (see[2] ? 0xffffu : 0u) | (see[3] ? 0xffff0000u : 0u);
#pragma unroll
        for (int i = 0; i < kUnits / 2; ++i) {
          vf[u][i][0] &= mlo; vf[u][i][1] &= mhi; vf[u][i][2] &= mlo; vf[u][i][3] &= mhi;
        }
      }

      // ---- online softmax: the references m (of l) and R (of the accumulator) move only
      // when a logit passes them by more than kSlack, so that most tiles need no
      // reduction over the row's lanes; any reference gives the same result ----
      bool pass = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float(&y)[4] = x[nb][u];
          const float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
          pass |= top > m[nb] + kSlack;
          if (kFp8) pass |= top + lv[u] > R[nb] + kSlack;
        }
      if (__any_sync(0xffffffffu, pass)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float mx = -INFINITY, mu = -INFINITY;  // largest logit; largest with its value's scale
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float(&y)[4] = x[nb][u];
            float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            mx = fmaxf(mx, top);
            mu = fmaxf(mu, top + lv[u]);
          }
          const float mn = fmaxf(m[nb], mx);
          m_ref[nb] = mn == -INFINITY ? 0.f : mn;
          const float alpha = ex2(m[nb] - m_ref[nb]);
          l[nb] *= alpha;
          m[nb] = mn;
          float beta = alpha;
          if (kFp8) {
            const float Rn = fmaxf(R[nb], mu);
            R_ref[nb] = Rn == -INFINITY ? 0.f : Rn;
            beta = ex2(R[nb] - R_ref[nb]);
            R[nb] = Rn;
          }
          // rows 2t, 2t + 1 are the accumulator's columns; their factors are on lanes 8t, 8t + 4
          const float b0 = __shfl_sync(0xffffffffu, beta, 8 * t);
          const float b1 = __shfl_sync(0xffffffffu, beta, 8 * t + 4);
#pragma unroll
          for (int c = 0; c < E; ++c) {
            acc[nb][c][0] *= b0; acc[nb][c][1] *= b1; acc[nb][c][2] *= b0; acc[nb][c][3] *= b1;
          }
        }
      }
      uint32_t pb[NB][U][kFp8 ? 4 : 2];  // tf32; bf16 pairs
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float(&y)[4] = x[nb][u];
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = ex2(y[i] - m_ref[nb]);
          l[nb] += (e[0] + e[1]) + (e[2] + e[3]);
          if constexpr (kFp8) {
            const float d = lv[u] - R_ref[nb];
#pragma unroll
            for (int i = 0; i < 4; ++i) pb[nb][u][i] = to_tf32(ex2(y[i] + d));
          } else {
            pb[nb][u][0] = pack_bf16(e[0], e[1]);
            pb[nb][u][1] = pack_bf16(e[2], e[3]);
          }
        }

      // ---- O^T += V^T P^T ----
      if constexpr (kFp8) {
        // A register of codes holds (token 2t: dims 2g, 2g + 1; token 2t + 1: the same), the
        // next one tokens 2t + 8 and 2t + 9: as k = t and t + 4 of two products, which are
        // E apart as the second adds to the first.
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < E; ++c) {
              const uint32_t w = __byte_perm(vf[u][c / 2][2 * (c & 1) + h], 0, 0x3120);
              const float2 r0 = f16x2_f32(e4m3x2_f16(w)), r1 = f16x2_f32(e4m3x2_f16_hi(w));
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma_tf32(acc[nb][c], r0.x, r1.x, r0.y, r1.y, pb[nb][u][2 * h], pb[nb][u][2 * h + 1]);
            }
      } else {
        // units 2c and 2c + 1 of V: dims 16c + g and 16c + 8 + g
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int c = 0; c < E; ++c)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma<false>(acc[nb][c], vf[u][c][0], vf[u][c][2], vf[u][c][1], vf[u][c][3],
                         pb[nb][u][0], pb[nb][u][1]);
      }
    }

#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      l[nb] += __shfl_xor_sync(0xffffffffu, l[nb], 1);
      l[nb] += __shfl_xor_sync(0xffffffffu, l[nb], 2);
    }
    if constexpr (kPerWarp) {
      bool last = true;
      if (f != pr.begin || seg_end != pr.begin + pr.n) {
        // Contributors and slots as below, of warps.
        const int x0 = pr.begin + (pr.b * Hkv + pr.kvh + 1) * kCost;
        const int c0 = (x0 + snap) / chunk, c1 = (x0 + pr.n - snap - 1) / chunk;
        const int me = (int)blockIdx.x * kWarps + warp - c0;
        warp_store_partial<C>(p, part_slot(c0, me), acc, m, l, R);
        __syncwarp();
        int* cnt = p.pair_counters + pr.b * Hkv + pr.kvh;
        int arrived = 0;
        if (lane == 0) arrived = atomic_add_acq_rel_gpu(cnt, 1);
        last = __shfl_sync(0xffffffffu, arrived, 0) == c1 - c0;
        __syncwarp();
        if (last) {
          if (lane == 0) store_relaxed_gpu(cnt, 0);
          warp_merge_partials<C>(p, c0, c1 - c0 + 1, acc, m, l, R);
        }
      }
      if (last) warp_finalize<C>(p, pr.b, pr.kvh, sink, acc, m, l, R);
    } else {
      // ---- merge the warps ----
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float* r0 = my_wb + (8 * nb + 2 * t) * C::kWbRow;
        float* r1 = r0 + C::kWbRow;
#pragma unroll
        for (int c = 0; c < E; ++c) {
          // rows of the accumulator: dims 16c + 2g and 16c + 2g + 1 (e4m3), 16c + g and + 8 (bf16)
          const int d0 = 16 * c + (kFp8 ? 2 * g : g), d1 = d0 + (kFp8 ? 1 : 8);
          r0[d0] = acc[nb][c][0]; r1[d0] = acc[nb][c][1];
          r0[d1] = acc[nb][c][2]; r1[d1] = acc[nb][c][3];
        }
        if (t == 0) {
          float* st = my_wb + C::kRows * C::kWbRow + 8 * nb + g;
          st[0] = m[nb];
          st[C::kRows] = l[nb];
          st[2 * C::kRows] = kFp8 ? R[nb] : m[nb];
        }
      }
      __syncthreads();
      float o[NB][E], mc[NB], lc[NB], Rc[NB];
      combine_warps<C>(wbuf, er, ed, o, mc, lc, Rc);

      if (kCluster && p.cluster > 1) {
        // this part's result, where the cluster's other CTAs find it
        __syncthreads();  // every warp has read wbuf
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float* dst = wbuf + (er + 8 * nb) * D + ed;
#pragma unroll
          for (int e = 0; e < E; ++e) dst[e] = o[nb][e];
          if (ed == 0) {
            float* st = wbuf + C::kRows * D + er + 8 * nb;
            st[0] = mc[nb];
            st[C::kRows] = lc[nb];
            st[2 * C::kRows] = Rc[nb];
          }
        }
      } else if (kCluster || (f == pr.begin && seg_end == pr.begin + pr.n)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          finalize<C>(p, pr.b, pr.kvh, er + 8 * nb, ed, sink[nb], o[nb], mc[nb], lc[nb], Rc[nb]);
      } else if constexpr (!kCluster) {
        // Contributors: the CTA whose range holds the first tile (slot 2 c + 1) and the
        // ones whose cuts lie inside (slot 2 c), more than snap tiles from either border.
        const int x0 = pr.begin + (pr.b * Hkv + pr.kvh + 1) * kPairCost;
        const int c0 = (x0 + snap) / chunk, c1 = (x0 + pr.n - snap - 1) / chunk;
        const int parts = c1 - c0 + 1, me = (int)blockIdx.x - c0;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          store_partial<C>(p, part_slot(c0, me), er + 8 * nb, ed, o[nb], mc[nb], lc[nb], Rc[nb]);
        const int gi = me / kMergeGroup, gfirst = gi * kMergeGroup;
        const int gsize = min(kMergeGroup, parts - gfirst);
        const int groups = (parts + kMergeGroup - 1) / kMergeGroup;
        int* gcnt = p.slot_counters + part_slot(c0, gfirst);
        int* tcnt = p.pair_counters + pr.b * Hkv + pr.kvh;
        __syncthreads();
        if (tid == 0) misc[8] = atomic_add_acq_rel_gpu(gcnt, 1);
        __syncthreads();
        if (misc[8] == gsize - 1) {
          if (tid == 0) store_relaxed_gpu(gcnt, 0);
          gather_partials<C>(p.partials, c0, gfirst, 1, gfirst + gsize, my_wb);
          __syncthreads();
          combine_warps<C>(wbuf, er, ed, o, mc, lc, Rc);
          bool whole = groups == 1;
          if (!whole) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              store_partial<C>(p, part_slot(c0, gfirst), er + 8 * nb, ed, o[nb], mc[nb], lc[nb], Rc[nb]);
            __syncthreads();
            if (tid == 0) misc[9] = atomic_add_acq_rel_gpu(tcnt, 1);
            __syncthreads();
            if (misc[9] == groups - 1) {
              if (tid == 0) store_relaxed_gpu(tcnt, 0);
              gather_partials<C>(p.partials, c0, 0, kMergeGroup, parts, my_wb);
              __syncthreads();
              combine_warps<C>(wbuf, er, ed, o, mc, lc, Rc);
              whole = true;
            }
          }
          if (whole) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              finalize<C>(p, pr.b, pr.kvh, er + 8 * nb, ed, sink[nb], o[nb], mc[nb], lc[nb], Rc[nb]);
          }
        }
      }
    }
    f = seg_end;
    slot ^= kQSlots - 1;
  }

  // A wait that gave up leaves copies in flight: wait for them (again with a
  // limit) before the shared memory goes to another CTA.
  if (!ok)
    for (; n < issued; ++n) mbar_wait(bars + 8 * (n % kStages), (n / kStages) & 1, p.err);

  if constexpr (kCluster) {
    if (next.n == 0 && part == 0) {  // no key
      for (int i = tid; i < p.G * (D / 8); i += kThreads) {
        const int h = next.kvh * p.G + i / (D / 8);
        *reinterpret_cast<uint4*>(p.out + next.b * p.o_sb + h * p.o_sh + (i % (D / 8)) * 8) =
            make_uint4(0, 0, 0, 0);
        if (i % (D / 8) == 0 && p.lse) p.lse[next.b * p.lse_sb + h * p.lse_sh] = -INFINITY;
      }
    }
    if (p.cluster > 1) {
      __syncwarp();
      cluster_sync();  // every part's result is visible
      // Four dims of a row for each thread of the cluster; all reads are in flight at
      // once, and the parts are added in order.
      const uint32_t wb = smem_u32(wbuf);
      for (int i = part * kThreads + tid; next.n > 0 && i < p.G * (D / 4); i += p.cluster * kThreads) {
        const int row = i / (D / 4), d = i % (D / 4) * 4;
        float ms[kPagedMaxCluster], ls[kPagedMaxCluster], Rs[kPagedMaxCluster];
        float4 v[kPagedMaxCluster];
        // a part without a tile left nothing
        auto has = [&](int r) {
          return r < p.cluster && (int)((long long)next.n * r / p.cluster) <
                                      (int)((long long)next.n * (r + 1) / p.cluster);
        };
#pragma unroll
        for (int r = 0; r < kPagedMaxCluster; ++r) {
          ms[r] = Rs[r] = -INFINITY;
          if (!has(r)) continue;
          const uint32_t at = map_shared_rank(wb, r), st = at + 4u * (C::kRows * D + row);
          ms[r] = ld_cluster_f32(st);
          ls[r] = ld_cluster_f32(st + 4u * C::kRows);
          Rs[r] = ld_cluster_f32(st + 4u * 2 * C::kRows);
          v[r] = ld_cluster_f4(at + 4u * (row * D + d));
        }
        float m = -INFINITY, l = 0.f, R = m, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < kPagedMaxCluster; ++r) {
          m = fmaxf(m, ms[r]);
          R = fmaxf(R, Rs[r]);
        }
#pragma unroll
        for (int r = 0; r < kPagedMaxCluster; ++r) {
          if (!has(r)) continue;
          l = __fmaf_rn(weight(ms[r], m), ls[r], l);
          const float w = weight(Rs[r], R);
          o[0] = __fmaf_rn(w, v[r].x, o[0]);
          o[1] = __fmaf_rn(w, v[r].y, o[1]);
          o[2] = __fmaf_rn(w, v[r].z, o[2]);
          o[3] = __fmaf_rn(w, v[r].w, o[3]);
        }
        const float sink = p.sinks ? __ldg(p.sinks + next.kvh * p.G + row) * kLog2e : -INFINITY;
        finalize<C>(p, next.b, next.kvh, row, d, sink, o, m, l, R);
      }
      __syncwarp();
      cluster_sync();  // the parts stay until they have been read
    }
  }
}

template <class C, bool kCluster>
__global__ void __launch_bounds__(kThreads, C::kCtas)
    paged_attn_kernel(const __grid_constant__ PagedParams p,
                      const __grid_constant__ CUtensorMap kv_map) {
  constexpr int D = C::D;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base_u32 = (raw + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.B, Hkv = p.Hkv;

  if (lane == 0) {
    const uint32_t bars = base_u32 + C::kOffBars + warp * C::kStages * 8;
    for (int s = 0; s < C::kStages; ++s) mbar_init(bars + 8 * s, 1);
    fence_barrier_init();
  }
  if (tid == 0) tma_prefetch_desc(&kv_map);
  griddep_wait();  // nothing of the caller's is read before

  if constexpr (kCluster) {
    Pair pair = {};
    pair.b = (int)blockIdx.x / p.cluster / Hkv;
    pair.kvh = (int)blockIdx.x / p.cluster % Hkv;
    const int len = __ldg(p.seq_lens + pair.b);
    if (blockIdx.x % p.cluster == 0 && pair.kvh == 0 && len > p.max_blocks * p.page_size)
      atomicOr(p.err, DEVERR_SEQ_TOO_LONG);
    pair.n = span_of(p, len).tiles;
    griddep_launch_dependents();
    attend<C, kPagedCluster>(p, kv_map, base, base_u32, pair, false);
  } else {
    int* misc = reinterpret_cast<int*>(base + C::kOffMisc);
    int* prefix = reinterpret_cast<int*>(base + C::kOffPrefix);
    // ---- prefix[b]: tiles per kv head before request b; the most of a request ----
    int most = 0;
    {
      const int per = (B + kThreads - 1) / kThreads, b0 = tid * per;
      int mine = 0;
      for (int b = b0; b < min(b0 + per, B); ++b) {
        const int len = __ldg(p.seq_lens + b);
        if (blockIdx.x == 0 && len > p.max_blocks * p.page_size) atomicOr(p.err, DEVERR_SEQ_TOO_LONG);
        const int tiles = span_of(p, len).tiles;
        mine += tiles;
        most = max(most, tiles);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) misc[kWarps + warp] = most;
      int run = block_scan(mine, misc);
      for (int b = b0; b < min(b0 + per, B); ++b) {
        prefix[b] = run;
        run += span_of(p, __ldg(p.seq_lens + b)).tiles;
        if (b == B - 1) prefix[B] = run;
      }
    }
    __syncthreads();
    griddep_launch_dependents();

    // requests without a key
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
      if (prefix[b + 1] != prefix[b]) continue;
      for (int i = tid; i < Hkv * p.G * (D / 8); i += kThreads) {
        const int h = i / (D / 8);
        *reinterpret_cast<uint4*>(p.out + b * p.o_sb + h * p.o_sh + (i % (D / 8)) * 8) =
            make_uint4(0, 0, 0, 0);
        if (i % (D / 8) == 0 && p.lse) p.lse[b * p.lse_sb + h * p.lse_sh] = -INFINITY;
      }
    }

    // ---- how the work is cut, by what the lengths turn out to be ----
    // Whole pairs save a CTA the merges at its two ends, which cost about kEndCost.
#pragma unroll
    for (int w = 0; w < kWarps; ++w) most = max(most, misc[kWarps + w]);
    const uint32_t pairs = B * Hkv, waves = (pairs + gridDim.x - 1) / gridDim.x;
    // Warp mode: what the merge of a CTA's warps costs a short pair is saved, where there
    // are pairs enough for the warps.  On / off, e4m3: 2000 x 8 kv heads of 30 to 60 keys
    // 60.1 / 119.4 us, 1000 x 8 of up to 300 keys, heads of 64, 50.0 / 75.8, 256 x 8 of 10
    // to 700 keys 40.4 / 47.2, of 700 to 768 keys 69.9 / 76.2; a bf16 window of 128 on
    // 512 x 8 kv heads 58.3 / 63.9.  64 x 8 of up to 32768 keys lose, 63.5 / 51.5.
    if (p.warps && waves > 2 && most <= kPagedWarpTiles) {
      attend<C, kPagedWarp>(p, kv_map, base, base_u32, Pair{}, false);
    } else {
      const uint32_t share = max(((uint32_t)prefix[B] * Hkv + kPairCost * pairs) / gridDim.x,
                                 (uint32_t)kPagedMinCost);
      attend<C, kPagedShares>(p, kv_map, base, base_u32, Pair{},
                              waves <= 2 && waves * (most + kPairCost) <= share + kEndCost);
    }
  }
}

template <class C, bool kCluster>
cudaError_t launch_mode(const PagedParams& p, const CUtensorMap& map, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e =
      set_smem_attr_once(paged_attn_kernel<C, kCluster>, C::smem_bytes(kPagedMaxBatch), done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::smem_bytes(kCluster ? 0 : p.B);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster ? p.cluster : 1;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster && p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, paged_attn_kernel<C, kCluster>, p, map);
}

template <class C>
cudaError_t launch_t(const PagedParams& p, const CUtensorMap& map, cudaStream_t stream) {
  return p.cluster ? launch_mode<C, true>(p, map, stream) : launch_mode<C, false>(p, map, stream);
}

template <typename F>
auto with_cfg(int D, bool fp8, int G, F f) {
  if (D == 64) {
    if (fp8) return G <= 8 ? f(Cfg<64, true, 1>()) : f(Cfg<64, true, 2>());
    return G <= 8 ? f(Cfg<64, false, 1>()) : f(Cfg<64, false, 2>());
  }
  if (fp8) return G <= 8 ? f(Cfg<128, true, 1>()) : f(Cfg<128, true, 2>());
  return G <= 8 ? f(Cfg<128, false, 1>()) : f(Cfg<128, false, 2>());
}

}  // namespace

PagedShape paged_attn_shape(int D, bool fp8, int G) {
  return with_cfg(D, fp8, G, [](auto c) {
    using C = decltype(c);
    return PagedShape{C::kCtas, C::kPartFloats, C::kChunks};
  });
}

cudaError_t launch_paged_attn(const PagedParams& p, const CUtensorMap& map, cudaStream_t stream) {
  return with_cfg(p.D, p.kv_scale != nullptr, p.G,
                  [&](auto c) { return launch_t<decltype(c)>(p, map, stream); });
}

}  // namespace pkv
