// cache8_few_d64.cu -- instances of the 8-bit cache's kernel for few rows at head dimension 64.
#include "cache8_few.cuh"

namespace attn {
namespace kv {
template cudaError_t launch_few_d<64>(const Cache8Params&, const FwdWs&, const CUtensorMap&, const CUtensorMap&,
                                       const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
}  // namespace kv
}  // namespace attn
