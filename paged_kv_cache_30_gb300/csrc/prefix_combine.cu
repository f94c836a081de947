// prefix_combine.cu -- adds up the parts of a decode call with shared tokens: for each row
// (request, query head) that of the request's own tokens (paged_attn.cuh) and those of the
// shared ones (prefix_attn.cu), in order, and writes out and lse:
//   m = max_i m_i,  l = sum_i l_i 2^(m_i - m),  out = sum_i O_i 2^(R_i - m) / (l + 2^(sink - m))
// with R_i the reference of O_i (m_i but for an e4m3 cache's own tokens), all in log2 units.
//
// Latency: a read of the row's place, then all of its parts at once.  A CTA has 8
// neighbouring rows of a kv head, whose 16-byte quads of 4 elements lie side by side; a
// thread one row and every 16th quad.  The grid before does not wait for the parts of the
// first, as it would if it added them: 64 requests behind 8192 tokens took 71.5 us so.
#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kRows = 8, kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float weight(float r, float M) { return r == -INFINITY ? 0.f : ex2(r - M); }

template <int D>
__global__ void __launch_bounds__(kThreads)
    prefix_combine_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ PrefixParams x) {
  constexpr int kQuads = D / 4 / (kThreads / kRows);  // of a thread
  constexpr int kAtOnce = 16 / kQuads;                // parts whose reads are under way
  const int64_t rows = (int64_t)p.B * p.G;
  const int64_t row = (int64_t)blockIdx.x * kRows + (threadIdx.x & (kRows - 1));
  const int q0 = threadIdx.x / kRows, kvh = blockIdx.y;
  griddep_wait();
  griddep_launch_dependents();
  if (row >= rows) return;
  const int b = (int)(row / p.G), h = (int)(row % p.G), head = kvh * p.G + h;
  const int4 at = __ldcg(x.info + b);
  const int len = __ldg(p.seq_lens + b);
  const float sink = p.sinks ? __ldg(p.sinks + head) * kLog2e : -INFINITY;
  // asked for with them; what was not written is not used
  const float4 ml = __ldcg(x.own_ml + kvh * rows + row);
  float4 o[kQuads];
#pragma unroll
  for (int k = 0; k < kQuads; ++k)
    o[k] = __ldcg(x.own_o + (kvh * (D / 4) + q0 + 16 * k) * rows + row);
  if (at.z < 0) return;  // padding
  uint16_t* out = p.out + b * p.o_sb + head * p.o_sh;
  float* lse = p.lse ? p.lse + b * p.lse_sb + head * p.lse_sh : nullptr;
  if (len <= 0) {
#pragma unroll
    for (int k = 0; k < kQuads; ++k)
      *reinterpret_cast<uint2*>(out + 4 * (q0 + 16 * k)) = make_uint2(0, 0);
    if (lse && q0 == 0) *lse = -INFINITY;
    return;
  }
  float m = ml.x, l = ml.y, R = ml.z;

  // The shared tokens' parts: of the CTAs from the one that holds the end of the unit's first
  // tile to the one that holds the unit's end.
  int n = 0, c0 = 0, in_block = 0;
  if (at.z > 0) {
    const int blocks = at.x >> 16;
    const int in_group = (b - (at.x & 0xffff)) * p.G + h;
    const int begin = at.y + kPrefixUnitCost +
                      (kvh * blocks + in_group / kPrefixRows) * (kPrefixUnitCost + at.z);
    c0 = (begin + min(at.z, kPrefixTileKeys / 16) - 1) / at.w;
    n = (begin + at.z - 1) / at.w - c0 + 1;
    in_block = in_group % kPrefixRows;
  }
  for (int i0 = 0; i0 < n; i0 += kAtOnce) {
    float2 pm[kAtOnce];
    float4 v[kAtOnce][kQuads];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      pm[i] = make_float2(-INFINITY, 0.f);
      if (i0 + i >= n) continue;
      const int64_t cta = c0 + i0 + i;
      const bool first = i0 + i == 0;
      pm[i] = __ldcg(first ? x.first_ml + kvh * rows + row : x.rest_ml + cta * kPrefixRows + in_block);
#pragma unroll
      for (int k = 0; k < kQuads; ++k)
        v[i][k] = __ldcg(first ? x.first_o + (kvh * (D / 4) + q0 + 16 * k) * rows + row
                               : x.rest_o + (cta * (D / 4) + q0 + 16 * k) * kPrefixRows + in_block);
    }
    float mn = m;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) mn = fmaxf(mn, pm[i].x);
    const float Rn = fmaxf(R, mn), keep = weight(R, Rn);
    l *= weight(m, mn);
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      o[k].x *= keep; o[k].y *= keep; o[k].z *= keep; o[k].w *= keep;
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (i0 + i >= n) continue;
      l = __fmaf_rn(weight(pm[i].x, mn), pm[i].y, l);
      const float w = weight(pm[i].x, Rn);
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        o[k].x = __fmaf_rn(w, v[i][k].x, o[k].x);
        o[k].y = __fmaf_rn(w, v[i][k].y, o[k].y);
        o[k].z = __fmaf_rn(w, v[i][k].z, o[k].z);
        o[k].w = __fmaf_rn(w, v[i][k].w, o[k].w);
      }
    }
    m = mn;
    R = Rn;
  }
  const float f = l != 0.f ? ex2(R - m) / (l + ex2(sink - m)) : 0.f;
#pragma unroll
  for (int k = 0; k < kQuads; ++k)
    *reinterpret_cast<uint2*>(out + 4 * (q0 + 16 * k)) =
        make_uint2(pack_bf16(o[k].x * f, o[k].y * f), pack_bf16(o[k].z * f, o[k].w * f));
  if (lse && q0 == 0) *lse = l != 0.f ? __fmaf_rn(m, kLn2, logf(l)) : -INFINITY;
}

}  // namespace

cudaError_t launch_prefix_combine(const PagedParams& p, const PrefixParams& x, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)p.B * p.G + kRows - 1) / kRows), p.Hkv);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.D == 64 ? cudaLaunchKernelEx(&cfg, prefix_combine_kernel<64>, p, x)
                   : cudaLaunchKernelEx(&cfg, prefix_combine_kernel<128>, p, x);
}

}  // namespace pkv
