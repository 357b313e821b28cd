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

template <int HD>
cudaError_t launch_few_d(const Cache8Params&, const FwdWs&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                         const CUtensorMap&, int, cudaStream_t);
extern template cudaError_t launch_few_d<160>(const Cache8Params&, const FwdWs&, const CUtensorMap&, const CUtensorMap&,
                                              const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
extern template cudaError_t launch_few_d<128>(const Cache8Params&, const FwdWs&, const CUtensorMap&, const CUtensorMap&,
                                              const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
extern template cudaError_t launch_few_d<64>(const Cache8Params&, const FwdWs&, const CUtensorMap&, const CUtensorMap&,
                                             const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);

namespace {

// Boxes of `width` features of min(page_size, rows) rows of a page.  Lines of 128
// bytes: a row of one head is no longer, and with 256 the neighbouring head's bytes
// came along and were gone when they were wanted (96 sequences of 8 heads: 697 MB
// read for 490, 120 us instead of 104).
bool encode_bytes(CUtensorMap* m, const CacheParams& p, const Pages& pg, int width, int rows, CUtensorMapSwizzle swizzle) {
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.d), static_cast<cuuint64_t>(p.Hkv),
                        static_cast<cuuint64_t>(p.page_size), static_cast<cuuint64_t>(p.num_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(pg.head), static_cast<cuuint64_t>(pg.slot),
                           static_cast<cuuint64_t>(pg.page)};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(width), 1,
                       static_cast<cuuint32_t>(p.page_size < rows ? p.page_size : rows), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(pg.base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Few rows a key: a sequence's tokens have at most kFewMost rows in a K/V head.  (The
// kernel for few rows is right for any number; it takes 8 rows at a time and reads the
// keys once for each 8.)  96 sequences over 425000 keys of 8 heads, d = 128, its time and
// that of the tiles of 128 rows: 4 rows 167 and 409 us, 8 rows 175 and 409, 16 rows 328
// and 411 (capped 355 and 440), 24 rows 482 and 411; 16 rows of one head of 160: 76 and
// 78.  Prefixes bring the rows of many sequences together and stay with the tiles.
//
// What the host knows is the average.  Where it is above kFewMost, or with prefixes, the
// tiles take all.  With one token a sequence (total_q = B) the kernel for few rows
// takes all: idle tiles behind it would cost 96 single tokens 9 us of 156 (the same
// number of tokens in a few of the sequences is right all the same, and slower).
// Otherwise both are launched and each takes its sequences by their own rows: one
// prompt among single tokens would re-read its keys for every 8 of its rows.  255
// single tokens over 500 to 8000 keys and one prompt of 769, 32 heads over 8 of 128, both
// kernels, the few-rows one alone, the tiles alone: a prompt behind nothing 442, 1053 and
// 1188 us, behind 60000 keys 1804, 7270 and 2527; one sequence of 200 tokens over 16000
// keys in a table of 256: 131, 541 and 126.  It costs batches that have few rows
// everywhere the launch of idle tiles: 96 sequences of 2 tokens 173, 166 and 434 us.
enum class Takes { tiles, few, both };
Takes who_takes(int B, int P, int R, int64_t total_q) {
  if (P > 0 || (total_q + B - 1) / B * R > kFewMost) return Takes::tiles;
  return total_q == B ? Takes::few : Takes::both;
}

// The workspace of a call; where both kernels work, the partial results of the one for few
// rows lie behind the other's (of 8 rows at most).
struct Fwd8Ws {
  FwdWs tiles, few;
  size_t total;
};
Fwd8Ws fwd8_ws(int B, int P, int Hq, int Hkv, int d, int64_t total_q) {
  Fwd8Ws w;
  w.tiles = w.few = fwd_ws(B, P, Hq, Hkv, d, total_q);
  w.total = w.tiles.total;
  if (B > 0 && who_takes(B, P, Hq / Hkv, total_q) == Takes::both) {
    constexpr size_t kRowsFew = 2 * kMaxCtas * 8;
    w.few.cut_rows = 8;
    w.few.stats = w.total;
    w.few.rows = w.few.stats + kRowsFew * sizeof(float4);
    w.total = w.few.rows + kRowsFew * d * sizeof(float);
  }
  return w;
}

}  // namespace

size_t fwd8_workspace(int B, int P, int Hq, int Hkv, int d, int64_t total_q) {
  return fwd8_ws(B, P, Hq, Hkv, d, total_q).total;
}

cudaError_t launch_fwd8(const Cache8Params& call, cudaStream_t s) {
  Cache8Params p = call;
  const int grid = device_ctas();
  if (grid < 1 || !encode_fn()) return cudaErrorInitializationError;
  const Fwd8Ws w = fwd8_ws(p.c.B, p.c.P, p.c.Hq, p.c.Hkv, p.c.d, p.c.total_q);
  const Takes takes = who_takes(p.c.B, p.c.P, p.c.R, p.c.total_q);
  CUtensorMap tk, tkt, tv, tvt;
  std::memset(&tkt, 0, sizeof tkt);
  std::memset(&tvt, 0, sizeof tvt);
  const int d = p.c.d, wide = d == 64 ? 64 : 128;
  const CUtensorMapSwizzle swizzle = d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (takes != Takes::tiles) {
    p.c.tile_cost = 2;  // the joins of a piece's warps and its first loads
    p.c.most_rows = takes == Takes::both ? kFewMost : 0;
    constexpr int kRowsBox = 64;
    if (!encode_bytes(&tk, p.c, p.c.k, wide, kRowsBox, swizzle) || !encode_bytes(&tv, p.c, p.c.v, wide, kRowsBox, swizzle) ||
        (d == 160 && (!encode_bytes(&tkt, p.c, p.c.k, 32, kRowsBox, CU_TENSOR_MAP_SWIZZLE_32B) ||
                      !encode_bytes(&tvt, p.c, p.c.v, 32, kRowsBox, CU_TENSOR_MAP_SWIZZLE_32B))))
      return cudaErrorInvalidValue;
    const cudaError_t e = d == 160   ? launch_few_d<160>(p, w.few, tk, tkt, tv, tvt, grid, s)
                          : d == 128 ? launch_few_d<128>(p, w.few, tk, tkt, tv, tvt, grid, s)
                                     : launch_few_d<64>(p, w.few, tk, tkt, tv, tvt, grid, s);
    if (e != cudaSuccess) return e;
    if (takes == Takes::few) return launch_join(p.c, w.few, 8, s);
    p.c.least_rows = kFewMost + 1;
    p.c.most_rows = INT32_MAX;
  }
  // what a piece's start costs in steps, as in cache_fwd.cu
  p.c.tile_cost = p.c.softcap > 0.f ? 4 : 2;
  if (!encode_bytes(&tk, p.c, p.c.k, wide, kKeys, swizzle) ||
      (d == 160 && !encode_bytes(&tkt, p.c, p.c.k, 32, kKeys, CU_TENSOR_MAP_SWIZZLE_32B)) ||
      !encode_bytes(&tv, p.c, p.c.v, d, kKeys, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const cudaError_t e = d == 160   ? launch_fwd8_d<160>(p, w.tiles, tk, tkt, tv, grid, s)
                        : d == 128 ? launch_fwd8_d<128>(p, w.tiles, tk, tkt, tv, grid, s)
                                   : launch_fwd8_d<64>(p, w.tiles, tk, tkt, tv, grid, s);
  if (e != cudaSuccess) return e;
  return takes == Takes::both ? launch_join(p.c, w.tiles, 0, s, &w.few) : launch_join(p.c, w.tiles, kRows, s);
}

}  // namespace kv
}  // namespace attn
