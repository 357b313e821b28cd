// cache_weights.cu -- key weights over the paged cache: the sums of cut key
// tiles and the launches.
#include <cstring>

#include "cache_weights.cuh"

namespace attn {
namespace kv {

// the tile kernel's instances, in translation units of their own
extern template cudaError_t launch_weights_d<160>(const CacheParams&, const WeightsWs&,
                                                  const CUtensorMap&, const CUtensorMap&, int,
                                                  cudaStream_t);
extern template cudaError_t launch_weights_d<128>(const CacheParams&, const WeightsWs&,
                                                  const CUtensorMap&, const CUtensorMap&, int,
                                                  cudaStream_t);
extern template cudaError_t launch_weights_d<64>(const CacheParams&, const WeightsWs&,
                                                 const CUtensorMap&, const CUtensorMap&, int,
                                                 cudaStream_t);

namespace {

// Block c: the key tile whose row tiles are cut from CTA c on; its parts are
// added in the order of the row tiles.
__global__ void __launch_bounds__(128)
    join_weights_kernel(const __grid_constant__ CacheParams p, const __grid_constant__ WeightsWs w) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const WeightsCut c = reinterpret_cast<const WeightsCut*>(p.ws + w.cuts)[blockIdx.x];
  const float* parts = reinterpret_cast<const float*>(p.ws + w.sums);
  const int r = threadIdx.x, key = c.kt * kKeys + r;
  if (c.parts == 0 || key >= c.len) return;
  float sum = parts[(2 * blockIdx.x + 1) * 128 + r];
#pragma unroll 4
  for (int i = 1; i < c.parts; ++i) sum += parts[2 * (blockIdx.x + i) * 128 + r];
  const float* in = p.w_in[c.own];
  const float before = in ? in[c.row * p.wi_rs[c.own] + c.g * p.wi_hs[c.own] + key] : 0.f;
  p.w_out[c.own][c.row * p.wo_rs[c.own] + c.g * p.wo_hs[c.own] + key] = before + sum;
}

}  // namespace

size_t weights_workspace() { return weights_ws().total; }

cudaError_t launch_weights(const CacheParams& call, cudaStream_t s) {
  CacheParams p = call;
  p.tile_cost = 2;
  const int grid = device_ctas();
  if (grid < 1 || !encode_fn()) return cudaErrorInitializationError;
  const WeightsWs w = weights_ws();
  CUtensorMap tk, tkt;
  std::memset(&tkt, 0, sizeof tkt);
  if (!encode_pages(&tk, p, p.k, false) || (p.d == 160 && !encode_pages(&tkt, p, p.k, true)))
    return cudaErrorInvalidValue;
  cudaError_t e = p.d == 160   ? launch_weights_d<160>(p, w, tk, tkt, grid, s)
                  : p.d == 128 ? launch_weights_d<128>(p, w, tk, tkt, grid, s)
                               : launch_weights_d<64>(p, w, tk, tkt, grid, s);
  // with at most one row tile no key tile is cut
  if (e != cudaSuccess || p.total_q * p.R <= kRows) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_weights_kernel, p, w);
}

}  // namespace kv
}  // namespace attn
