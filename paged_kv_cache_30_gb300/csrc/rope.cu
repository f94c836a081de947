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
// for few.  A warp has one token, or some of its heads where tokens are few: it finds
// the token's place, and each lane the sines and cosines of its own pairs, once for
// all heads.  A lane has 8 elements of a row, D / 8 lanes a row: both quads of four
// pairs (half layout: quads p / 4 and (p + rot / 2) / 4; else neighbours), so a
// rotation needs no other lane, and the norm's weights are folded into its sines and
// cosines.  Rows of the next batch are asked for before those of this one are used.
//
// Measured (GB300; the copy bandwidth is 6680 GB/s): 16384 tokens of 36 heads of 128 with norms
// 54.2 us = 5.6 TB/s; 17.6 k prompt tokens of 80 heads into the cache 118 us = 6.4 TB/s; 64 tokens
// of 72 heads 2.2 us, of 80 heads into the cache 3.7.
#include <algorithm>

#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
// Rows a lane has under way, and CTAs of an SM.  16384 tokens of 36 heads of 128 with norms:
// 54.2 us, 59.4 without the limit of registers, 61.5 with 2 rows and without it.  On data that
// L2 does not hold: 5001 of 27 heads of 64 with norms 12.1 us, 14.3 with 4 rows (with or without
// the limit 12.1, 12.4 with 8 CTAs); 8191 of 48 heads of 64 without norms into the cache 19.1
// us, 20.3 with 2 rows, 21.3 without the limit.
template <int D, bool kNorm>
constexpr int kBatch = D == 128 || !kNorm ? 4 : 2;
constexpr int kCtas = 6;

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
      left = b < 0 ? 0 : (int)max(__ldg(p.cu + b + 1) - t, 0ll);
    } else {
      const long long each = p.T / p.B;
      b = (int)(t / each);
      left = (int)(each - t % each);
    }
    if (left <= 0) return {-1, -1};  // behind the last request
    const int len = __ldg(p.seq_lens + b);
    if (len < left) return {-1, -1};  // (their difference need not be an int)
    const int pos = len - left;
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

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 4 weights of a norm from element d on.
__device__ __forceinline__ void load_weights(const void* w, bool f32, int d, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = !w    ? 1.f
           : f32 ? __ldg(static_cast<const float*>(w) + d + i)
                 : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(w) + d + i) << 16);
}

template <int D, bool kAppend, int kPairs, bool kNorm>
__global__ void __launch_bounds__(kThreads, kCtas)
    rope_kernel(const __grid_constant__ RopeParams p, int groups) {
  constexpr int kBatch = pkv::kBatch<D, kNorm>;
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows of a warp
  const int lane = threadIdx.x & 31, col = lane % kLanes;
  const long long t = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  // this warp's groups of kRows rows, of the token's query, key and value heads in turn
  const int g0 = (int)blockIdx.y * groups, g1 = g0 + groups;
  // this lane's two quads of elements
  const int half = p.rot / 2;
  const bool rotates = kPairs == kHalf ? col < p.rot / 8 : kPairs == kInterleaved && 8 * col < p.rot;
  const int da = kPairs == kHalf ? (rotates ? 4 * col : p.rot + 8 * (col - p.rot / 8)) : 8 * col;
  const int db = kPairs == kHalf && rotates ? da + half : da + 4;
  griddep_wait();
  griddep_launch_dependents();
  if (t >= p.T) return;

  struct Rows {  // of a kind of heads: where they are, and where they go (null: not there)
    const uint16_t* src;
    uint16_t* dst;
    int64_t from, to;  // strides
    int heads, first;  // first group
  };
  uint4 x[kBatch];
  auto load = [&](const Rows& r, int g, int end) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = (g + u - r.first) * kRows + lane / kLanes;
      if (g + u >= end || h >= r.heads) continue;
      const uint16_t* s = r.src + h * r.from;
      if constexpr (kPairs == kHalf) {
        const uint2 a = *reinterpret_cast<const uint2*>(s + da), b = *reinterpret_cast<const uint2*>(s + db);
        x[u] = make_uint4(a.x, a.y, b.x, b.y);
      } else {
        x[u] = *reinterpret_cast<const uint4*>(s + da);
      }
    }
  };
  const int q_groups = (p.Hq + kRows - 1) / kRows, k_groups = (p.Hkv + kRows - 1) / kRows;
  Rows rows = {p.q + t * p.q_st, p.q_out + t * p.qo_st, p.q_sh, p.qo_sh, p.Hq, 0};
  if (g0 >= q_groups)
    rows = {p.k + t * p.k_st, nullptr, p.k_sh, 0, p.Hkv, q_groups};
  int end = min(g1, g0 >= q_groups ? q_groups + k_groups : q_groups);
  load(rows, g0, end);  // under way while the token's place is found

  const Place place = place_of<kAppend>(p, t);
  if (place.pos < 0) return;
  float cs[4], sn[4];  // of this lane's pairs
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
    if (kPairs != kNone && rotates) {
      const uint2 f = __ldg(p.turns + 4 * col + i);
      const uint64_t turns = ((uint64_t)f.y << 32 | f.x) * (uint64_t)(uint32_t)place.pos;
      sincospif((float)(int)(turns >> 32) * 0x1p-31f, &sn[i], &cs[i]);
      cs[i] *= p.factor;
      sn[i] *= p.factor;
    }
  }

  int g = g0;
#pragma unroll 1
  for (int kind = g0 >= q_groups; kind < 2; ++kind) {
    // ---- query heads, key heads ----
    if (kind == 1) {
      if (g1 <= q_groups || p.Hkv == 0) return;
      if (g0 < q_groups) {
        rows = {p.k + t * p.k_st, nullptr, p.k_sh, 0, p.Hkv, q_groups};
        end = min(g1, q_groups + k_groups);
        g = q_groups;
        load(rows, g, end);
      }
      if constexpr (kAppend) {
        if (place.at >= 0) rows.dst = p.cache + place.at, rows.to = p.c_sh;
      } else {
        rows.dst = p.k_out + t * p.ko_st;
        rows.to = p.ko_sh;
      }
    }
    const void* weights = kind ? p.kw : p.qw;
    const bool norm = kNorm && weights;
    // with the weights: (a, b) -> (a ac + b bs, b bc + a as)
    float2 ac[2], bs[2], bc[2], as[2];
    {
      float wa[4], wb[4];
      load_weights(norm ? weights : nullptr, kind ? p.kw_f32 : p.qw_f32, da, wa);
      load_weights(norm ? weights : nullptr, kind ? p.kw_f32 : p.qw_f32, db, wb);
      if (kPairs == kInterleaved) {  // a: even elements, b: odd ones
        const float v[8] = {wa[0], wa[1], wa[2], wa[3], wb[0], wb[1], wb[2], wb[3]};
#pragma unroll
        for (int i = 0; i < 4; ++i) wa[i] = v[2 * i], wb[i] = v[2 * i + 1];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ac[i] = make_float2(wa[2 * i] * cs[2 * i], wa[2 * i + 1] * cs[2 * i + 1]);
        bs[i] = make_float2(-wb[2 * i] * sn[2 * i], -wb[2 * i + 1] * sn[2 * i + 1]);
        bc[i] = make_float2(wb[2 * i] * cs[2 * i], wb[2 * i + 1] * cs[2 * i + 1]);
        as[i] = make_float2(wa[2 * i] * sn[2 * i], wa[2 * i + 1] * sn[2 * i + 1]);
      }
    }
#pragma unroll 1
    for (; g < end; g += kBatch) {
      uint4 now[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) now[u] = x[u];
      load(rows, g + kBatch, end);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (g + u >= end) break;  // the same for the warp
        const int h = (g + u - rows.first) * kRows + lane / kLanes;
        float2 a[2], b[2];
        if constexpr (kPairs == kInterleaved) {
          a[0] = make_float2(lo_f32(now[u].x), lo_f32(now[u].y));
          a[1] = make_float2(lo_f32(now[u].z), lo_f32(now[u].w));
          b[0] = make_float2(hi_f32(now[u].x), hi_f32(now[u].y));
          b[1] = make_float2(hi_f32(now[u].z), hi_f32(now[u].w));
        } else {
          a[0] = make_float2(lo_f32(now[u].x), hi_f32(now[u].x));
          a[1] = make_float2(lo_f32(now[u].y), hi_f32(now[u].y));
          b[0] = make_float2(lo_f32(now[u].z), hi_f32(now[u].z));
          b[1] = make_float2(lo_f32(now[u].w), hi_f32(now[u].w));
        }
        if (norm) {
          float2 ss = mul2(a[0], a[0]);
          ss = fma2(a[1], a[1], ss);
          ss = fma2(b[0], b[0], ss);
          ss = fma2(b[1], b[1], ss);
          float s = ss.x + ss.y;
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          const float r = rsqrtf(__fmaf_rn(s, 1.f / D, p.eps));
          const float2 inv = make_float2(r, r);
          // Before the weights: an element near the end of the range times its weight would be
          // an infinity, which times the 0 of a head whose squares overflow is no 0.
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            a[i] = mul2(a[i], inv);
            b[i] = mul2(b[i], inv);
          }
        }
        float2 ya[2], yb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ya[i] = mul2(a[i], ac[i]);
          yb[i] = mul2(b[i], bc[i]);
          if (rotates) {  // other elements stay apart: an infinity times 0 is none of theirs
            ya[i] = fma2(b[i], bs[i], ya[i]);
            yb[i] = fma2(a[i], as[i], yb[i]);
          }
        }
        if (h >= rows.heads || !rows.dst) continue;
        uint16_t* d = rows.dst + h * rows.to;
        if constexpr (kPairs == kInterleaved) {
          *reinterpret_cast<uint4*>(d + da) =
              make_uint4(pack_bf16(ya[0].x, yb[0].x), pack_bf16(ya[0].y, yb[0].y),
                         pack_bf16(ya[1].x, yb[1].x), pack_bf16(ya[1].y, yb[1].y));
        } else if constexpr (kPairs == kHalf) {
          *reinterpret_cast<uint2*>(d + da) =
              make_uint2(pack_bf16(ya[0].x, ya[0].y), pack_bf16(ya[1].x, ya[1].y));
          *reinterpret_cast<uint2*>(d + db) =
              make_uint2(pack_bf16(yb[0].x, yb[0].y), pack_bf16(yb[1].x, yb[1].y));
        } else {
          *reinterpret_cast<uint4*>(d + da) =
              make_uint4(pack_bf16(ya[0].x, ya[0].y), pack_bf16(ya[1].x, ya[1].y),
                         pack_bf16(yb[0].x, yb[0].y), pack_bf16(yb[1].x, yb[1].y));
        }
      }
    }
  }
  if constexpr (kAppend) {  // ---- value heads: copied ----
    if (place.at < 0) return;
    const int v1 = min(g1, q_groups + 2 * k_groups);
#pragma unroll 1
    for (int v = max(g0, q_groups + k_groups); v < v1; v += kBatch) {
      uint4 y[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int h = (v + u - q_groups - k_groups) * kRows + lane / kLanes;
        if (v + u < v1 && h < p.Hkv)
          y[u] = *reinterpret_cast<const uint4*>(p.v + t * p.v_st + h * p.v_sh + 8 * col);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int h = (v + u - q_groups - k_groups) * kRows + lane / kLanes;
        if (v + u < v1 && h < p.Hkv)
          *reinterpret_cast<uint4*>(p.cache + place.at + h * p.c_sh + D + 8 * col) = y[u];
      }
    }
  }
}

template <int D, bool kAppend, int kPairs, bool kNorm>
cudaError_t launch_t(const RopeParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kRows = 32 / (D / 8);
  const int k_groups = (p.Hkv + kRows - 1) / kRows;
  const int all = (p.Hq + kRows - 1) / kRows + k_groups * (kAppend ? 2 : 1);
  // A token to a warp, or to several where that leaves an SM fewer than 8 warps (16 on the way
  // into the cache, where a warp first looks its page up).  64 tokens of 72 heads 2.2 us, 3.0
  // with 16; of 80 heads into the cache 3.7 us, 4.6 with 8.
  const int64_t parts =
      std::min<int64_t>(all, std::max<int64_t>(1, (kAppend ? 16 : 8) * num_sms / p.T));
  const int groups = (int)((all + parts - 1) / parts);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.T + kWarps - 1) / kWarps), (unsigned)((all + groups - 1) / groups));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<D, kAppend, kPairs, kNorm>, p, groups);
}

template <int D, bool kAppend, bool kNorm>
cudaError_t launch_n(const RopeParams& p, int num_sms, cudaStream_t stream) {
  if (p.rot == 0) return launch_t<D, kAppend, kNone, kNorm>(p, num_sms, stream);
  return p.interleaved ? launch_t<D, kAppend, kInterleaved, kNorm>(p, num_sms, stream)
                       : launch_t<D, kAppend, kHalf, kNorm>(p, num_sms, stream);
}

template <int D, bool kAppend>
cudaError_t launch_d(const RopeParams& p, int num_sms, cudaStream_t stream) {
  return p.qw || p.kw ? launch_n<D, kAppend, true>(p, num_sms, stream)
                      : launch_n<D, kAppend, false>(p, num_sms, stream);
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
