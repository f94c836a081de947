// paged_attn.cu -- the launches of paged_attn.cuh's kernels without shared tokens.
#include "paged_attn.cuh"

namespace pkv {

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
