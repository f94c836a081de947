// prefix_ring.h -- the order in which a unit's operands (K and V of its tiles) go through
// prefix_attn.cu's ring, and the places and phases that they have there.  Plain C++, so that the
// model of the ring's barriers in the tests goes through the same code.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define PKV_RING __host__ __device__ __forceinline__
#else
#define PKV_RING inline
#endif

namespace pkv {

// Operands come in the order in which the steps use them: K0 V0 K1 V1 .. for two query tiles,
// K0 K1 V0 K2 V1 .. for one, whose steps j and j + 1 are at work together.  (Of an e4m3 cache
// always as for two, which has less to work out.)
struct OperandOrder {
  bool by_tile;
  int tiles;

  PKV_RING int keys(int t) const { return by_tile ? 2 * t : t > 0 ? 2 * t - 1 : 0; }
  PKV_RING int values(int t) const { return by_tile || t == tiles - 1 ? 2 * t + 1 : 2 * t + 2; }
  PKV_RING bool are_values(int n) const {  // operand n
    return by_tile ? n & 1 : n == 2 * tiles - 1 || (n > 0 && !(n & 1));
  }
  PKV_RING int tile_of(int n) const {
    return by_tile             ? n >> 1
           : n == 2 * tiles - 1 ? tiles - 1
           : n & 1             ? (n + 1) >> 1
           : n > 1             ? (n >> 1) - 1
                               : 0;
  }
};

// Operands of a unit in a ring of kOps places, for one of the roles that go through them: operand
// n's place, and the phase of its barriers.  With kExtraOp a unit of one query tile has a place
// more, number kOps.
template <int kOps, bool kExtraOp>
struct OpRing {
  uint32_t base = 0;  // phases of the places at the unit's start
  int mod = kOps;

  PKV_RING void begin(bool dual) {
    if (kExtraOp) mod = dual ? kOps : kOps + 1;
  }
  PKV_RING int uses(int n) const {  // n / mod
    return !kExtraOp ? n / kOps : mod == kOps ? n / kOps : n / (kOps + 1);
  }
  PKV_RING int place(int n) const { return n - uses(n) * mod; }
  PKV_RING uint32_t phase(int n) const { return ((base >> place(n)) ^ (uint32_t)uses(n)) & 1u; }
  PKV_RING void end(int n) {  // of a unit of n operands
    const int all = uses(n), left = place(n);
    // places below `left` were used once more
    const uint32_t low = (1u << left) - 1u, places = (1u << mod) - 1u;
    base ^= all & 1 ? places & ~low : low;
  }
};

}  // namespace pkv
