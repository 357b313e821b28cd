// cache8_few_d160.cu -- instances of the 8-bit cache's kernel for few rows at head dimension 160.
#include "cache8_few.cuh"

namespace attn {
namespace kv {
template cudaError_t launch_few_d<160>(const Cache8Params&, const FwdWs&, const CUtensorMap&, const CUtensorMap&,
                                       const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
}  // namespace kv
}  // namespace attn
