// prefix_own.cu -- the launch of paged_attn.cuh's kernel for requests' own tokens behind
// shared ones: the grid after prefix_attn.cu's.
#include "paged_attn.cuh"

namespace pkv {

cudaError_t launch_prefix_own(const PagedParams& p, const PrefixParams& x, const CUtensorMap& kv_map,
                              cudaStream_t stream) {
  return with_cfg(p.D, p.kv_scale != nullptr, p.G, [&](auto c) {
    using C = decltype(c);
    constexpr int kMost = C::smem_bytes(kPagedMaxBatch) + plan_ints(kPagedMaxBatch) * 4;
    static_assert(kMost <= 227 * 1024, "shared memory");
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        set_smem_attr_once(paged_own_kernel<C>, kMost, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::smem_bytes(p.B) + plan_ints(x.groups) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_own_kernel<C>, p, kv_map, x);
  });
}

}  // namespace pkv
