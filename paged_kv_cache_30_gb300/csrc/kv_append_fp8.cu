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
// One warp per (token, kv head); the warp of a page's first new token (its
// leader) does the page's work, the others leave.
#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 8;
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

// A row [K | V] of 2D values takes 2D/8 lanes of 8 values; a warp covers
// 32 / (2D/8) rows at once.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const AppendFp8Params p) {
  constexpr int LPR = 2 * D / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (w >= p.T * p.Hkv) return;
  const long long r = w / p.Hkv;
  const int h = (int)(w % p.Hkv), P = p.page_size;

  // request b of row r, its first row r0 and the row after its last one
  int b;
  long long r0, r1;
  if (p.cu) {
    int lo = 0, hi = p.B;  // the number of requests that begin at or before r
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu + mid) <= r) lo = mid + 1; else hi = mid;
    }
    b = lo - 1;
    if (b < 0) return;
    r0 = __ldg(p.cu + b);
    r1 = min((long long)__ldg(p.cu + b + 1), (long long)p.T);
    if (r0 < 0 || r >= r1) return;  // rows outside every request are left alone
  } else {
    const long long n = p.T / p.B;
    b = (int)(r / n);
    r0 = b * n;
    r1 = r0 + n;
  }
  const long long pos = (long long)__ldg(p.seq_lens + b) - (r1 - r);
  if (pos < 0 || (r != r0 && pos % P != 0)) return;  // not the page's first new token
  const long long pg = pos / P;
  const int slot0 = (int)(pos % P);
  const int n = (int)min((long long)(P - slot0), r1 - r);
  if (pg >= p.max_blocks) {
    if (lane == 0) atomicOr(p.err, DEVERR_SEQ_TOO_LONG);
    return;
  }
  const int blk = __ldg(p.bt + b * p.bt_sb + pg);
  if (blk < 0 || blk >= p.num_blocks) {
    if (lane == 0) atomicOr(p.err, DEVERR_BAD_BLOCK);
    return;
  }
  const int sub = lane / LPR, unit = lane % LPR;
  const bool is_v = unit >= LPR / 2;
  const uint16_t* src = (is_v ? p.v : p.k) + h * p.s_sh + (unit % (LPR / 2)) * 8;
  uint8_t* dst = p.cache + blk * p.c_sblk + h * p.c_sh + unit * 8;
  float* scale = p.scale + blk * p.sc_sblk + h * p.sc_sh + (is_v ? 1 : 0);

  float a = 0.f;
  for (int i = sub; i < n; i += RPW) {
    float f[8];
    unpack8(*reinterpret_cast<const uint4*>(src + (r + i) * p.s_st), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) a = fmaxf(a, finite_abs(f[e]));
  }
#pragma unroll
  for (int o = 1; o < LPR / 2; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if (RPW > 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16));

  const float s_old = slot0 > 0 ? *scale : 0.f;
  const float s = fmaxf(s_old, pow2_scale(a));
  __syncwarp();  // every lane has read the old scale
  if (sub == 0 && unit % (LPR / 2) == 0) *scale = s;
  if (s > s_old && slot0 > 0) {
    const float f0 = __fdiv_rn(s_old, s);
    for (int i = sub; i < slot0; i += RPW) {
      uint2* at = reinterpret_cast<uint2*>(dst + i * p.c_stok);
      float f[8];
      decode8(*at, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= f0;
      *at = encode8(f);
    }
  }
  const float div = s > 0.f ? s : 1.f;
  for (int i = sub; i < n; i += RPW) {
    float f[8];
    unpack8(*reinterpret_cast<const uint4*>(src + (r + i) * p.s_st), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __fdiv_rn(f[e], div);
    *reinterpret_cast<uint2*>(dst + (slot0 + i) * p.c_stok) = encode8(f);
  }
}

}  // namespace

cudaError_t launch_gqa_kv_append_fp8(const AppendFp8Params& p, cudaStream_t stream) {
  const long long warps = p.T * p.Hkv;
  const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps);
  if (p.D == 64)
    append_kernel<64><<<grid, kWarps * 32, 0, stream>>>(p);
  else
    append_kernel<128><<<grid, kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pkv
