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
// One warp per (request, query head): lane l holds dims [l D/32, (l + 1) D/32)
// of q and of the output; one pass over the keys with the running maximum and
// sum in 32 bits.
#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float e4m3_to_f32(uint8_t c) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)c));
  float f;
  asm("{.reg .f16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, l;}" : "=f"(f) : "r"(h2));
  return f;
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kWarps * 32) paged_attn_kernel(const PagedParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int Hq = p.Hkv * p.G;
  if (w >= (long long)p.B * Hq) return;
  const int b = (int)(w / Hq), h = (int)(w % Hq), kvh = h / p.G, P = p.page_size;
  int L = __ldg(p.seq_lens + b);
  if (L > p.max_blocks * P) {
    if (lane == 0) atomicOr(p.err, DEVERR_SEQ_TOO_LONG);
    L = p.max_blocks * P;
  }
  const int start = (p.window > 0 && L > p.window) ? L - p.window : 0;
  const int first = min(p.first, start);
  float q[E], o[E];
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float((uint32_t)p.q[b * p.q_sb + h * p.q_sh + lane * E + e] << 16);
    o[e] = 0.f;
  }
  const float c2 = p.scale * kLog2e;
  float m = -INFINITY, l = 0.f;
  for (int j = first > 0 ? 0 : start; j < L; j = (j + 1 == first) ? start : j + 1) {
    const int blk = __ldg(p.bt + b * p.bt_sb + j / P);
    float k[E], v[E], ks = 1.f, vs = 1.f;
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0) atomicOr(p.err, DEVERR_BAD_BLOCK);
      for (int e = 0; e < E; ++e) k[e] = v[e] = 0.f;  // reads as zeros
    } else {
      const uint8_t* row = p.kv + blk * p.kv_sblk + kvh * p.kv_sh + (j % P) * p.kv_stok;
      for (int e = 0; e < E; ++e) {
        const int d = lane * E + e;
        if (kFp8) {
          k[e] = e4m3_to_f32(row[d]);
          v[e] = e4m3_to_f32(row[D + d]);
        } else {
          k[e] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[d] << 16);
          v[e] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[D + d] << 16);
        }
      }
      if (kFp8) {
        const float* sc = p.kv_scale + blk * p.s_sblk + kvh * p.s_sh;
        ks = sc[0];
        vs = sc[1];
      }
    }
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = __fmaf_rn(q[e], k[e], s);
    for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    const float x = s * ks * c2;
    const float mn = fmaxf(m, x);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float alpha = ex2(m - ref), pr = ex2(x - ref);
    l = __fmaf_rn(l, alpha, pr);
    for (int e = 0; e < E; ++e) o[e] = __fmaf_rn(o[e], alpha, pr * vs * v[e]);
    m = mn;
  }
  float inv = 0.f;
  if (l != 0.f) inv = 1.f / (l + (p.sinks ? ex2(__ldg(p.sinks + h) * kLog2e - m) : 0.f));
  for (int e = 0; e < E; ++e)
    p.out[b * p.o_sb + h * p.o_sh + lane * E + e] = (uint16_t)pack_bf16(o[e] * inv, 0.f);
  if (lane == 0 && p.lse)
    p.lse[b * p.lse_sb + h * p.lse_sh] = l != 0.f ? m * kLn2 + logf(l) : -INFINITY;
}

template <int D, bool kFp8>
cudaError_t launch_t(const PagedParams& p, cudaStream_t stream) {
  const long long warps = (long long)p.B * p.Hkv * p.G;
  paged_attn_kernel<D, kFp8>
      <<<(unsigned)((warps + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attn(const PagedParams& p, cudaStream_t stream) {
  if (p.D == 64) return p.kv_scale ? launch_t<64, true>(p, stream) : launch_t<64, false>(p, stream);
  return p.kv_scale ? launch_t<128, true>(p, stream) : launch_t<128, false>(p, stream);
}

}  // namespace pkv
