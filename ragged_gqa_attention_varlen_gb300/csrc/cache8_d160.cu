// cache8_d160.cu -- instances of the 8-bit cache's tile kernel at head dimension 160.
#include "cache8_fwd.cuh"

namespace attn {
namespace kv {
template cudaError_t launch_fwd8_d<160>(const Cache8Params&, const FwdWs&, const CUtensorMap&,
                                       const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
}  // namespace kv
}  // namespace attn
