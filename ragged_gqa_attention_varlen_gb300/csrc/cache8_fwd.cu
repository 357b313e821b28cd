// cache8_fwd.cu -- attention over the paged cache held in 8 bits: the tensor maps
// and the launches.
#include <cstring>

#include "cache_piece.cuh"

namespace attn {
namespace kv {

// the tile kernel's instances, in translation units of their own
template <int HD>
cudaError_t launch_fwd8_d(const Cache8Params&, const FwdWs&, const CUtensorMap&, const CUtensorMap&,
                          const CUtensorMap&, int, cudaStream_t);
extern template cudaError_t launch_fwd8_d<160>(const Cache8Params&, const FwdWs&, const CUtensorMap&,
                                               const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
extern template cudaError_t launch_fwd8_d<128>(const Cache8Params&, const FwdWs&, const CUtensorMap&,
                                               const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
extern template cudaError_t launch_fwd8_d<64>(const Cache8Params&, const FwdWs&, const CUtensorMap&,
                                              const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);

namespace {

// Boxes of `width` features of min(page_size, 128) rows of a page.
bool encode_bytes(CUtensorMap* m, const CacheParams& p, const Pages& pg, int width, CUtensorMapSwizzle swizzle) {
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.d), static_cast<cuuint64_t>(p.Hkv),
                        static_cast<cuuint64_t>(p.page_size), static_cast<cuuint64_t>(p.num_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(pg.head), static_cast<cuuint64_t>(pg.slot),
                           static_cast<cuuint64_t>(pg.page)};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(width), 1,
                       static_cast<cuuint32_t>(p.page_size < kKeys ? p.page_size : kKeys), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(pg.base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_fwd8(const Cache8Params& call, cudaStream_t s) {
  Cache8Params p = call;
  // what a piece's start costs in steps, as in cache_fwd.cu
  p.c.tile_cost = p.c.softcap > 0.f ? 4 : 2;
  const int grid = device_ctas();
  if (grid < 1 || !encode_fn()) return cudaErrorInitializationError;
  const FwdWs w = fwd_ws(p.c.B, p.c.P, p.c.Hq, p.c.Hkv, p.c.d, p.c.total_q);
  CUtensorMap tk, tkt, tv;
  std::memset(&tkt, 0, sizeof tkt);
  const int d = p.c.d;
  if (!encode_bytes(&tk, p.c, p.c.k, d == 64 ? 64 : 128, d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B) ||
      (d == 160 && !encode_bytes(&tkt, p.c, p.c.k, 32, CU_TENSOR_MAP_SWIZZLE_32B)) ||
      !encode_bytes(&tv, p.c, p.c.v, d, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const cudaError_t e = d == 160   ? launch_fwd8_d<160>(p, w, tk, tkt, tv, grid, s)
                        : d == 128 ? launch_fwd8_d<128>(p, w, tk, tkt, tv, grid, s)
                                   : launch_fwd8_d<64>(p, w, tk, tkt, tv, grid, s);
  return e != cudaSuccess ? e : launch_join(p.c, w, s);
}

}  // namespace kv
}  // namespace attn
