// cache8_d128.cu -- instances of the 8-bit cache's tile kernel at head dimension 128.
#include "cache8_fwd.cuh"

namespace attn {
namespace kv {
template cudaError_t launch_fwd8_d<128>(const Cache8Params&, const FwdWs&, const CUtensorMap&,
                                       const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
}  // namespace kv
}  // namespace attn
