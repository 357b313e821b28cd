// cache_fwd_d64.cu -- instances of the cache attention kernel at head dimension 64.
#include "cache_fwd.cuh"

namespace attn {
namespace kv {
template cudaError_t launch_fwd_d<64>(const CacheParams&, const FwdWs&, const CUtensorMap&,
                                      const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
}  // namespace kv
}  // namespace attn
