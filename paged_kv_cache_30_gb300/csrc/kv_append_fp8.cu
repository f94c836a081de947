// kv_append_fp8.cu -- writes new tokens into a paged e4m3 cache that keeps one
// fp32 scale for K and one for V per (page, kv head).
//
// For each page that receives tokens, each kv head, and K and V apart:
//   a     = max |x| over the page's new values that are finite
//   need  = 0 if a = 0, else the smallest power of two s >= 2^-100 with a <= 448 s
//   s_old = the page's scale, or 0 when the page holds no token before the new ones
//   s     = max(s_old, need)
//   code  = e4m3(x / s) for the new tokens, e4m3(code * (s_old / s)) for the held
//           ones when s > s_old (round to nearest even, saturating at +-448)
// Scales that grow are powers of two, so re-encoding the held tokens is exact
// but for codes that leave e4m3's normal range (below 2^-6 of the new scale).
//
// Bound by memory for prompts (bf16 read once, codes written once), by latency
// for single tokens.  A team of warps (1, 2 or 4, so that a page's rows are 16 to
// 32 loads a lane) takes one kv head of `slab` consecutive rows (1 when there are
// few, a page's when there are many): it finds the first row's request with a
// 32-way search of cu_tokens and walks the pages that begin in its rows, loading
// the rows of a page to shared memory at once (up to 32 16-byte copies a lane)
// before it reduces, and encoding them from there.
//
// Measured (GB300, 8 kv heads of 128, graph replays): 64 single tokens 2.9 us, 1024
// of them 7.6 us; 12.5 k tokens of ragged prompts (77 MB) 16.3 us = 4.7 TB/s, 32 k
// tokens 31.6 us = 6.4 TB/s (94 % of the measured copy bandwidth; pages of 32 and 128
// tokens 88 and 82 %).  What is left is the chain of dependent reads that a warp
// begins with (request, length, page, rows): about 4 us, hidden only by other warps.
#include <algorithm>

#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;  // of a CTA at most
// Single warps with more than this many rows of a page are CTAs of their own, so that a
// place is free again when one warp is done (16 k tokens, pages of 32, heads of 128: 14.6
// us, 15.9 in CTAs of two, 17.5 of four); with fewer the launch of so many CTAs costs more
// (1024 single tokens, 8 kv heads: 8.4 us, 7.7 in CTAs of four).
constexpr int kAlone = 8;
// Single rows a warp until there are this many.  16 requests of up to 2000 tokens, 2 kv
// heads: 6.6 us, 8.2 at 4096 and 8.9 at 8192 (pages of 32, heads of 128); 100 of up to 160,
// 4 kv heads, pages of 128: 9.9 us, 12.2 at 2048.
constexpr int kFullWarps = 3200;
constexpr int kMaxHeld = 32;
constexpr float kMinScale = 7.888609052210118e-31f;  // 2^-100

// Smallest power of two s >= 2^-100 with a <= 448 s (448 = 1.75 * 2^8); 0 for a = 0.
__device__ __forceinline__ float pow2_scale(float a) {
  if (a == 0.f) return 0.f;
  const uint32_t u = __float_as_uint(a);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -100 ? kMinScale : __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;  // NaN and infinities set no scale
}

// 8 bf16 values (one 16-byte unit) -> floats
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Largest magnitudes of two interleaved lists of bf16 values, as bit patterns.
__device__ __forceinline__ uint32_t max_abs(uint32_t big, const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("max.u16x2 %0, %0, %1;" : "+r"(big) : "r"(w[i] & 0x7fff7fffu));
  return big;
}

__device__ __forceinline__ uint2 encode8(const float (&f)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = (uint32_t)e4m3x2(f[4 * i], f[4 * i + 1]) |
           ((uint32_t)e4m3x2(f[4 * i + 2], f[4 * i + 3]) << 16);
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void decode8(const uint2& u, float (&f)[8]) {
  const uint32_t w[2] = {u.x, u.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[i / 2] >> (16 * (i & 1)))));
    asm("{.reg .f16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}"
        : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
        : "r"(h2));
  }
}

// A request's rows [r0, r1) of the new ones and its length.
struct Request {
  int r0, r1, len;
};
__device__ __forceinline__ Request request_at(const AppendFp8Params& p, int b) {
  return {__ldg(p.cu + b), __ldg(p.cu + b + 1), __ldg(p.seq_lens + b)};
}

// The last request that begins at or before row r (-1: none), 32 requests at a time.
// The last step reads all that is asked of a request, so that nothing waits for a read
// after it.
__device__ __forceinline__ int request_of(const AppendFp8Params& p, long long r, Request& q) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = p.B;  // among requests [lo, lo + len); an earlier one begins before r
  int found = -1;
  bool all = true;  // q holds all of request `found`
  while (len > 0) {
    const int step = (len + 31) >> 5, at = lo + lane * step;
    const bool in = lane * step < len;
    const Request mine = !in ? Request{} : step == 1 ? request_at(p, at) : Request{__ldg(p.cu + at)};
    const bool yes = in && mine.r0 <= r;
    const int cnt = __popc(__ballot_sync(0xffffffffu, yes));
    if (cnt == 0) break;
    all = step == 1;
    q.r0 = __shfl_sync(0xffffffffu, mine.r0, cnt - 1);
    q.r1 = __shfl_sync(0xffffffffu, mine.r1, cnt - 1);
    q.len = __shfl_sync(0xffffffffu, mine.len, cnt - 1);
    found = lo + (cnt - 1) * step;
    len = min(step - 1, lo + len - found - 1);
    lo = found + 1;
  }
  if (!all) q = request_at(p, found);
  return found;
}

__device__ __forceinline__ void cp_async_16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// A row [K | V] of 2D values takes 2D/8 lanes of 8 values; a warp covers
// RPW = 32 / (2D/8) rows at once, a team of kTeam warps kTeam times as many.  `hold`
// keeps the first `held` 16-byte units of each lane in shared memory
// (hold[32 i + lane] is read by the lane that asked for it); later ones are read
// twice.  exchange: 2 x 2 floats per warp, turn: pages of the team so far.  False: the
// page is not in the cache.
template <int D, int kTeam>
__device__ __forceinline__ bool append_page(const AppendFp8Params& p, int h, long long r, int n,
                                            int blk, int slot0, uint4* hold, int held,
                                            float* exchange, int& turn) {
  constexpr int LPR = 2 * D / 8, RPW = 32 / LPR, RPT = RPW * kTeam;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, unit = lane % LPR;
  const int sub = warp % kTeam * RPW + lane / LPR;  // this lane's rows: sub, sub + RPT, ...
  const bool is_v = unit >= LPR / 2;
  const uint16_t* src =
      (is_v ? p.v : p.k) + (r + sub) * p.s_st + h * p.s_sh + (unit % (LPR / 2)) * 8;
  const int64_t step = RPT * p.s_st;
  const int mine = n > sub ? (n - sub + RPT - 1) / RPT : 0;  // this lane's units
  const int first = min(mine, held);
  hold += lane;
  for (int i = 0; i < first; ++i) cp_async_16(hold + 32 * i, src + i * step);
  auto load = [&](int i) { return __ldg(reinterpret_cast<const uint4*>(src + i * step)); };

  // the page is needed from here on
  const bool good = blk >= 0 && blk < p.num_blocks;
  uint8_t* dst = p.cache + (good ? blk : 0) * p.c_sblk + h * p.c_sh + sub * p.c_stok + unit * 8;
  float* scale = p.scale + (good ? blk : 0) * p.sc_sblk + h * p.sc_sh + (is_v ? 1 : 0);
  const float s_old = good && slot0 > 0 ? *scale : 0.f;
  uint32_t big = 0;  // magnitudes are compared as bf16 bit patterns, two at a time
  for (int i = first; i < mine; ++i) big = max_abs(big, load(i));
  cp_async_wait_all();
  if (!good) return false;
#pragma unroll 4
  for (int i = 0; i < first; ++i) big = max_abs(big, hold[32 * i]);
  float a = __uint_as_float(max(big << 16, big & 0xffff0000u));
  __syncwarp();
  if (__any_sync(0xffffffffu, !(a < INFINITY))) {  // NaN and infinities set no scale
    a = 0.f;
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      float f[8];
      unpack8(load(i), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) a = fmaxf(a, finite_abs(f[e]));
    }
    __syncwarp();
  }
#pragma unroll
  for (int o = 1; o < LPR / 2; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if (RPW > 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16));
  if (kTeam > 1) {
    // two buffers: a warp may begin the team's next page while another still reads this one's
    float* team_max = exchange + (turn++ & 1) * 2 * kWarps;
    if (lane % LPR % (LPR / 2) == 0) team_max[2 * warp + is_v] = a;
    named_bar_sync(1 + warp / kTeam, 32 * kTeam);
#pragma unroll
    for (int w = 0; w < kTeam; ++w) a = fmaxf(a, team_max[2 * (warp / kTeam * kTeam + w) + is_v]);
  }

  const float s = fmaxf(s_old, pow2_scale(a));
  __syncwarp();  // every lane (before the barrier: of every warp) has read the old scale
  if (sub == 0 && unit % (LPR / 2) == 0) *scale = s;
  if (s > s_old && slot0 > 0) {
    const float f0 = __fdiv_rn(s_old, s);
#pragma unroll 4
    for (int i = 0; sub + i < slot0; i += RPT) {
      uint2* at = reinterpret_cast<uint2*>(dst + i * p.c_stok);
      float f[8];
      decode8(*at, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= f0;
      *at = encode8(f);
    }
  }
  const float div = s > 0.f ? s : 1.f;
  dst += slot0 * p.c_stok;
  const int64_t dst_step = RPT * p.c_stok;
  if ((__float_as_uint(div) & 0x7fffffu) == 0) {
    // s is a power of two (a grown scale is one): x / s is the product with 1 / s
    const float inv = 1.f / div;
    auto put = [&](const uint4& u, int i) {
      float f[8];
      unpack8(u, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= inv;
      *reinterpret_cast<uint2*>(dst + i * dst_step) = encode8(f);
    };
#pragma unroll 4
    for (int i = 0; i < first; ++i) put(hold[32 * i], i);
    for (int i = first; i < mine; ++i) put(load(i), i);
  } else {
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      float f[8];
      unpack8(load(i), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __fdiv_rn(f[e], div);
      *reinterpret_cast<uint2*>(dst + i * dst_step) = encode8(f);
    }
  }
  return true;
}

template <int D, int kTeam>
__global__ void __launch_bounds__(kWarps * 32, 7)
    append_kernel(const AppendFp8Params p, int slab, int held) {
  extern __shared__ uint4 hold[];
  __shared__ float exchange[2 * 2 * kWarps];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, P = p.page_size;
  const long long team = ((long long)blockIdx.x * (blockDim.x >> 5) + warp) / kTeam;
  const int h = (int)(team % p.Hkv);
  long long r = team / p.Hkv * slab;
  const long long end = min(r + slab, (long long)p.T);
  if (r >= end) return;
  int turn = 0;

  const int each = p.cu ? 0 : (int)(p.T / p.B);
  Request q;
  int b;
  if (p.cu) {
    b = request_of(p, r, q);
    if (b < 0) {  // rows before the first request are padding
      b = 0;
      q = request_at(p, 0);
      r = q.r0;
    }
  } else {
    b = (int)(r / each);
    q = {b * each, (b + 1) * each, __ldg(p.seq_lens + b)};
  }
  for (;;) {
    const long long r0 = q.r0, r1 = min((long long)q.r1, (long long)p.T);
    if (r0 < 0) return;
    if (r < r1) {  // else an empty request, or padding behind the last one
      const long long first = (long long)q.len - r1;  // position of row i: first + i
      r = min(max(r, -first), r1);  // tokens at negative positions are dropped
      while (r < end && r < r1) {
        const long long pos = first + r;
        const int slot0 = (int)(pos % P);
        const int n = (int)min((long long)(P - slot0), r1 - r);
        // a page belongs to the warp of its first new row
        if (r == r0 || r == -first || slot0 == 0) {
          const long long pg = pos / P;
          const int blk = pg < p.max_blocks ? __ldg(p.bt + b * p.bt_sb + pg) : -1;
          if (!append_page<D, kTeam>(p, h, r, n, blk, slot0, hold + warp * 32 * held, held,
                                     exchange, turn) &&
              lane == 0)
            atomicOr(p.err, pg < p.max_blocks ? DEVERR_BAD_BLOCK : DEVERR_SEQ_TOO_LONG);
        }
        r += n;
      }
      if (r < r1) return;
    }
    if (r >= end || ++b >= p.B) return;
    q = p.cu ? request_at(p, b) : Request{q.r1, q.r1 + each, __ldg(p.seq_lens + b)};
  }
}

}  // namespace

template <int D, int kTeam>
static cudaError_t launch_t(const AppendFp8Params& p, int most, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e =
      set_smem_attr_once(append_kernel<D, kTeam>, kWarps * 32 * 16 * kMaxHeld, done);
  if (e != cudaSuccess) return e;
  // rows a team walks: up to a page's once single rows give every SM warps enough
  int slab = 1;
  while (slab < most && p.T * p.Hkv * kTeam / slab > kFullWarps) slab *= 2;
  const long long warps = (p.T + slab - 1) / slab * p.Hkv * kTeam;
  // 16-byte units a lane holds
  const int rows = 32 / (2 * D / 8) * kTeam;
  const int held = std::min((most + rows - 1) / rows, kMaxHeld);
  cudaLaunchConfig_t cfg = {};
  const int cta = kTeam == 1 && most > kAlone ? 1 : kWarps;
  cfg.gridDim = dim3((unsigned)((warps + cta - 1) / cta));
  cfg.blockDim = dim3(cta * 32);
  cfg.dynamicSmemBytes = cta * 32 * 16 * held;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_kernel<D, kTeam>, p, slab, held);
}

cudaError_t launch_gqa_kv_append_fp8(const AppendFp8Params& p, cudaStream_t stream) {
  // rows that a page receives on average, and a team for 16 to 32 loads a lane of them
  // (two warps for 32 rows of 2 x 128 took 18.1 us for 16 k tokens, one takes 14.6)
  const int most = (int)std::min<int64_t>(p.page_size, (p.T + p.B - 1) / p.B);
  if (p.D == 64)
    return most <= 32   ? launch_t<64, 1>(p, most, stream)
           : most <= 64 ? launch_t<64, 2>(p, most, stream)
                        : launch_t<64, 4>(p, most, stream);
  return most <= 32 ? launch_t<128, 1>(p, most, stream) : launch_t<128, 4>(p, most, stream);
}

}  // namespace pkv
