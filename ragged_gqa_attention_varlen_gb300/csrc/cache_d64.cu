// cache_d64.cu -- instances of the paged cache's tile kernels at head dimension 64.
#include "cache_fwd.cuh"
#include "cache_weights.cuh"

namespace attn {
namespace kv {
template cudaError_t launch_fwd_d<64>(const CacheParams&, const FwdWs&, const CUtensorMap&,
                                      const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
template cudaError_t launch_weights_d<64>(const CacheParams&, const WeightsWs&, const CUtensorMap&,
                                          const CUtensorMap&, int, cudaStream_t);
}  // namespace kv
}  // namespace attn
