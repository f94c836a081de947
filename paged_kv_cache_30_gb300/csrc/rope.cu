// rope.cu -- queries and keys of new tokens: an RMS norm for each head and the
// rotation by their positions, written to q_out and k_out, or with the values into
// a paged bf16 cache.
//
// For every token t (position n) and head, in 32 bits, rounded once to bf16:
//   y        = x w / sqrt(mean x^2 + eps)                       (y = x without weights)
//   (a, b)   = c (y_i cos - y_j sin), c (y_j cos + y_i sin),    angle = 2 pi n turns_p
// for pair p = (i, j) of the first rot dims: (p, p + rot / 2), or (2p, 2p + 1).
//
// The angle is exact at any position: turns_p is a fraction of a turn in units of
// 2^-64, its product with n wraps at whole turns, and the upper half of what is left
// goes to sincospi.  A 32-bit product of position and frequency is off by 0.06 at
// position 10^6.
//
// Bound by memory for many tokens (each element read and written once), by latency
// for few.  A lane has 8 neighbouring elements of a row (one 16-byte load), D / 8
// lanes a row; partners of the half layout are rot / 16 lanes apart.  A CTA takes 1
// to 8 tokens: its threads fill a table of their sines and cosines, and each warp
// stays with one token, whose part of the table it keeps in registers over that
// token's heads.  Few tokens are split among CTAs by heads.
#include <algorithm>

#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kMaxTokens = 8;  // of a CTA
constexpr int kUnroll = 4;     // rows a lane has under way

enum : int { kNone, kHalf, kInterleaved };

// The last of n requests that begins at or before row t (-1: none), for a whole warp.
__device__ __forceinline__ int request_of(const int32_t* cu, int n, long long t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  for (;;) {
    const int step = (len + 31) / 32;
    const bool yes = lane * step < len && __ldg(cu + lo + lane * step) <= t;
    const int before = __popc(__ballot_sync(0xffffffffu, yes));
    if (before == 0) return lo - 1;
    lo += (before - 1) * step;
    len = min(step, len - (before - 1) * step);
    if (step == 1) return lo;
  }
}

// Where a token goes: its rotary position (negative: nothing of it is written) and the
// element of the cache at which its kv head 0 begins (negative: not into the cache).
struct Place {
  int pos;
  long long at;
};

template <bool kAppend>
__device__ __forceinline__ Place place_of(const RopeParams& p, long long t) {
  Place r = {-1, -1};
  if (p.positions) r.pos = __ldg(p.positions + t);
  else if (!kAppend) r.pos = 0;  // norms alone
  if constexpr (kAppend) {
    int b, left;  // request; its new tokens from this one on
    if (p.cu) {
      b = request_of(p.cu, p.B, t);
      left = b < 0 ? 0 : (int)min(__ldg(p.cu + b + 1) - t, 1ll << 30);
    } else {
      const long long each = p.T / p.B;
      b = (int)(t / each);
      left = (int)(each - t % each);
    }
    if (left <= 0) return {-1, -1};  // behind the last request
    const int pos = __ldg(p.seq_lens + b) - left;
    if (pos < 0) return {-1, -1};
    if (!p.positions) r.pos = pos;
    const int page = pos / p.page_size;
    if (r.pos < 0) return r;
    if (page >= p.max_blocks) {
      if ((threadIdx.x & 31) == 0) atomicOr(p.err, DEVERR_SEQ_TOO_LONG);
      return r;
    }
    const int blk = __ldg(p.bt + b * p.bt_sb + page);
    if (blk < 0 || blk >= p.num_blocks) {
      if ((threadIdx.x & 31) == 0) atomicOr(p.err, DEVERR_BAD_BLOCK);
      return r;
    }
    r.at = (long long)blk * p.c_sblk + (long long)(pos % p.page_size) * p.c_stok;
  }
  return r;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// 8 weights of a norm from element d on.
__device__ __forceinline__ void load_weights(const void* w, bool f32, int d, float (&f)[8]) {
  if (!w) return;
  if (f32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __ldg(static_cast<const float*>(w) + d + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(w) + d + i) << 16);
  }
}

template <int D, bool kAppend, int kPairs>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const __grid_constant__ RopeParams p, int tokens) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows of a warp
  __shared__ float2 table[kMaxTokens * D / 2];        // (cos, sin) times the factor
  __shared__ Place places[kMaxTokens];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int mine = warp % tokens;  // this warp's token of the CTA's
  const long long t0 = (long long)blockIdx.x * tokens, t = t0 + mine;
  const int d = lane % kLanes * 8;
  griddep_wait();
  griddep_launch_dependents();

  // Rows of a token: query heads, key heads, and on the way into the cache value heads.
  const int heads = p.Hq + p.Hkv * (kAppend ? 2 : 1);
  const int subs = kWarps / tokens * (int)gridDim.y, sub = warp / tokens + kWarps / tokens * blockIdx.y;
  const int step = subs * kRows;  // from a lane's row to its next
  int row = sub * kRows + lane / kLanes;
  auto source = [&](int r) {
    const uint16_t* s = r < p.Hq ? p.q + t * p.q_st + r * p.q_sh
                        : r < p.Hq + p.Hkv ? p.k + t * p.k_st + (r - p.Hq) * p.k_sh
                                           : p.v + t * p.v_st + (r - p.Hq - p.Hkv) * p.v_sh;
    return reinterpret_cast<const uint4*>(s + d);
  };
  uint4 x[kUnroll];
  auto load = [&](int r) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      x[u] = make_uint4(0, 0, 0, 0);
      if (t < p.T && r + u * step < heads) x[u] = *source(r + u * step);
    }
  };
  load(row);  // under way while the token's place is found

  float qw[8], kw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) qw[i] = kw[i] = 1.f;
  load_weights(p.qw, p.qw_f32, d, qw);
  load_weights(p.kw, p.kw_f32, d, kw);

  if (warp < tokens && t < p.T) {
    const Place r = place_of<kAppend>(p, t);
    if (lane == 0) places[warp] = r;
  }
  __syncthreads();
  if constexpr (kPairs != kNone) {
    const int half = p.rot / 2;
    for (int i = tid; i < tokens * half; i += kThreads) {
      const int tok = i / half;
      if (t0 + tok >= p.T) break;
      const uint2 f = __ldg(p.turns + i % half);
      const uint64_t turns = ((uint64_t)f.y << 32 | f.x) * (uint64_t)(uint32_t)places[tok].pos;
      float s, c;
      sincospif((float)(int)(turns >> 32) * 0x1p-31f, &s, &c);
      table[tok * (D / 2) + i % half] = make_float2(c * p.factor, s * p.factor);
    }
    __syncthreads();
  }
  if (t >= p.T) return;
  const Place place = places[mine];
  if (place.pos < 0) return;

  // This lane's pairs: 8 of the half layout (as first or as second element), 4 interleaved.
  const int half = p.rot / 2;
  const bool rotates = d < p.rot, second = kPairs == kHalf && d >= half;
  float2 cs[kPairs == kInterleaved ? 4 : 8];
  if constexpr (kPairs != kNone) {
    const int at = kPairs == kHalf ? (second ? d - half : d) : d / 2;
#pragma unroll
    for (int i = 0; i < (kPairs == kInterleaved ? 4 : 8); ++i)
      cs[i] = rotates ? table[mine * (D / 2) + at + i] : make_float2(1.f, 0.f);
    if (kPairs == kHalf && !second)  // y_i cos - y_j sin
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i].y = -cs[i].y;
  }
  const int partner = kPairs == kHalf && rotates ? (second ? lane - half / 8 : lane + half / 8) : lane;

  // All lanes go the same number of steps: partners trade elements.
  for (int first = sub * kRows; first < heads; first += kUnroll * step, row += kUnroll * step) {
    uint4 now[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) now[u] = x[u];
    if (first + kUnroll * step < heads) load(row + kUnroll * step);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = row + u * step;
      if (first + u * step >= heads) break;  // the same for the warp
      const bool is_q = r < p.Hq, is_v = kAppend && r >= p.Hq + p.Hkv;
      float y[8];
      unpack8(now[u], y);
      if (p.qw || p.kw) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __fmaf_rn(y[i], y[i], ss);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss * (1.f / D) + p.eps);
        if (is_q ? p.qw != nullptr : p.kw != nullptr) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = y[i] * inv * (is_q ? qw[i] : kw[i]);
        }
      }
      float z[8];
      if constexpr (kPairs == kHalf) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float other = __shfl_sync(0xffffffffu, y[i], partner);
          z[i] = rotates ? __fmaf_rn(y[i], cs[i].x, other * cs[i].y) : y[i];
        }
      } else if constexpr (kPairs == kInterleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = y[2 * i], b = y[2 * i + 1];
          z[2 * i] = rotates ? __fmaf_rn(a, cs[i].x, -(b * cs[i].y)) : a;
          z[2 * i + 1] = rotates ? __fmaf_rn(b, cs[i].x, a * cs[i].y) : b;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = y[i];
      }
      if (r >= heads) continue;
      uint4 out = make_uint4(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]), pack_bf16(z[4], z[5]),
                             pack_bf16(z[6], z[7]));
      if (is_v) out = now[u];
      uint16_t* dst;
      if (is_q) {
        dst = p.q_out + t * p.qo_st + r * p.qo_sh + d;
      } else if constexpr (kAppend) {
        if (place.at < 0) continue;
        const int h = is_v ? r - p.Hq - p.Hkv : r - p.Hq;
        dst = p.cache + place.at + h * p.c_sh + (is_v ? D : 0) + d;
      } else {
        dst = p.k_out + t * p.ko_st + (r - p.Hq) * p.ko_sh + d;
      }
      *reinterpret_cast<uint4*>(dst) = out;
    }
  }
}

template <int D, bool kAppend, int kPairs>
cudaError_t launch_t(const RopeParams& p, int num_sms, cudaStream_t stream) {
  const int heads = p.Hq + p.Hkv * (kAppend ? 2 : 1), rows = 32 / (D / 8);
  int tokens = 1;
  while (tokens < 4 && p.T / (2 * tokens) >= 4 * num_sms) tokens *= 2;
  const int64_t ctas = (p.T + tokens - 1) / tokens;
  // a CTA for each SM and a row a warp, if there are rows
  const int most = std::max(1, (heads + rows * kWarps / tokens - 1) / (rows * kWarps / tokens));
  const int parts = (int)std::max<int64_t>(1, std::min<int64_t>(most, 2 * num_sms / ctas));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)parts);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<D, kAppend, kPairs>, p, tokens);
}

template <int D, bool kAppend>
cudaError_t launch_d(const RopeParams& p, int num_sms, cudaStream_t stream) {
  if (p.rot == 0) return launch_t<D, kAppend, kNone>(p, num_sms, stream);
  return p.interleaved ? launch_t<D, kAppend, kInterleaved>(p, num_sms, stream)
                       : launch_t<D, kAppend, kHalf>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int num_sms, cudaStream_t stream) {
  if (p.cache)
    return p.D == 64 ? launch_d<64, true>(p, num_sms, stream)
                     : launch_d<128, true>(p, num_sms, stream);
  return p.D == 64 ? launch_d<64, false>(p, num_sms, stream)
                   : launch_d<128, false>(p, num_sms, stream);
}

}  // namespace pkv
