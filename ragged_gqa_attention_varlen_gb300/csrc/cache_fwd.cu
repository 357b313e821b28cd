// cache_fwd.cu -- attention over the paged cache: the merge of cut rows, the
// tensor maps and the launches.
#include <cstring>

#include "cache_fwd.cuh"

namespace attn {
namespace kv {

// the tile kernel's instances, in translation units of their own
extern template cudaError_t launch_fwd_d<160>(const CacheParams&, const FwdWs&, const CUtensorMap&,
                                              const CUtensorMap&, const CUtensorMap&, int,
                                              cudaStream_t);
extern template cudaError_t launch_fwd_d<128>(const CacheParams&, const FwdWs&, const CUtensorMap&,
                                              const CUtensorMap&, const CUtensorMap&, int,
                                              cudaStream_t);
extern template cudaError_t launch_fwd_d<64>(const CacheParams&, const FwdWs&, const CUtensorMap&,
                                             const CUtensorMap&, const CUtensorMap&, int,
                                             cudaStream_t);

namespace {

constexpr int kWarpsJ = 4;
constexpr int kHeadsJ = 8;  // rows (heads of a token) of a block

// Joins the partial results of a row.  Its own slots were computed in one
// part or several, and so was its prefix; part i has reference m_i, sums l_i (of
// its weights) and lr_i (of the rounded ones) and O_i (m_i in two terms, of
// which the parts of a segment share one: far rows' parts are weighed by the other
// without its roundings), and with factors 2^(m_i - max m) the row is sum O_i / sum lr_i, its lse from sum l_i.  Parts are
// added in the order of the keys, prefix last, so the result does not depend on
// which CTA finished first.  Rows that one part covers were
// written by the tile kernel already; rows without any key are written here.
// Eight heads of a token per block, eight lanes to the 128-byte line that holds
// four features of each, the features over four lanes and four warps.  A chain
// of dependent loads bounds it (sequence, plan, first part, parts); what does
// not depend on the tile kernel is read before the wait for it.
template <bool BF16, int HD>
__global__ void __launch_bounds__(kWarpsJ * 32)
    join_kernel(const __grid_constant__ CacheParams p, const __grid_constant__ FwdWs w) {
  constexpr int kUnits = HD / 4;                            // float4 of a row
  constexpr int kPer = (kUnits + 4 * kWarpsJ - 1) / (4 * kWarpsJ);  // of a thread
  const int tok = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y * kHeadsJ + (lane & 7);
  const int f0 = (lane >> 3) + 4 * warp;
  // Every block waits for the tile kernel before it ends, also those without
  // rows: what follows on the stream must not overlap it.
  if (h >= p.Hq) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int g = h / p.R, hr = h - g * p.R;
  const int2* meta = reinterpret_cast<const int2*>(p.ws + w.meta);
  const float4* stats = reinterpret_cast<const float4*>(p.ws + w.stats);
  const float4* part = reinterpret_cast<const float4*>(p.ws + w.rows);
  const int64_t row = static_cast<int64_t>(tok) * p.Hq + h;
  // The row's sequence; with one token each it is the token's own number, so
  // its lengths are read along with the test of that.
  int b = min(tok, p.B - 1);
  const int end = __ldg(p.cu_q + p.B);
  int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1), len = seg_len(p, true, b);
  if (tok >= end) {  // behind the last sequence
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  if (c0 > tok || c1 <= tok) {
    b = seq_of(p.cu_q, 0, p.B, tok);
    c0 = __ldg(p.cu_q + b);
    c1 = __ldg(p.cu_q + b + 1);
    len = seg_len(p, true, b);
  }
  // whether the row's own slots and its prefix have any step, and the row's
  // place in their row tiles
  bool has_own, has_prefix = false;
  int ro, rp = 0;
  {
    Seg own;
    own.own = 1;
    own.klo = 0;
    own.tok0 = c0;
    own.ntok = c1 - c0;
    own.len = len;
    const uint32_t x = static_cast<uint32_t>(tok - c0) * p.R + hr;
    int lo, hi;
    tile_keys(p, own, x / kRows, lo, hi);
    has_own = hi > lo;
    ro = x % kRows;
  }
  if (p.P) {
    const int pfx = prefix_of(p, b);
    if (pfx >= 0) {
      const int n = seg_len(p, false, pfx);
      has_prefix = prefix_klo(p, pfx, n) < n;
      const int tok0 = __ldg(p.cu_q + max(__ldg(p.cu_prefix + pfx), 0));
      rp = (static_cast<uint32_t>(tok - tok0) * p.R + hr) % kRows;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (first CTA, parts) of the two segments
  const int ok = reinterpret_cast<const FwdHead*>(p.ws)->ok;
  int2 mo = meta[row], mp = p.P ? meta[p.total_q * p.Hq + row] : make_int2(0, 0);
  if (!has_own) mo = make_int2(0, 0);
  if (!has_prefix) mp = make_int2(0, 0);
  if (!ok || (mo.y == 1 && mp.y == 0)) return;
  const int parts = mo.y + mp.y;
  auto row_of = [&](int i) -> int64_t {
    if (i < mo.y)
      return mo.y > 1 ? cut_row(w, mo.x + i, i == 0, ro) : whole_row(w, p.total_q, p.Hq, true, tok, h);
    i -= mo.y;
    return mp.y > 1 ? cut_row(w, mp.x + i, i == 0, rp) : whole_row(w, p.total_q, p.Hq, false, tok, h);
  };
  // Four parts at a time, all their loads first; the reference follows the
  // largest met so far.
  float top = -INFINITY, top0 = 0.f, l = 0.f, lr = 0.f;  // the reference: top + top0
  float4 acc[kPer] = {};
  for (int i0 = 0; i0 < parts; i0 += 4) {
    float4 s[4];
    float4 v[4][kPer];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = make_float4(-INFINITY, 0.f, 0.f, 0.f);  // m, l, lr, m0
      if (i0 + i < parts) {
        const int64_t pr = row_of(i0 + i);
        s[i] = stats[pr];
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (f0 + 4 * kWarpsJ * k < kUnits) v[i][k] = part[part_at<HD>(pr, f0 + 4 * kWarpsJ * k)];
      }
    }
    float up = top, up0 = top0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (s[i].y > 0.f && (s[i].x - up) + (s[i].w - up0) > 0.f) up = s[i].x, up0 = s[i].w;
    if (up != top || up0 != top0) {
      const float a = ex2_approx((top - up) + (top0 - up0));
      top = up;
      top0 = up0;
      l *= a;
      lr *= a;
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        acc[k] = make_float4(acc[k].x * a, acc[k].y * a, acc[k].z * a, acc[k].w * a);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!(s[i].y > 0.f)) continue;  // (a part without any weight may hold anything)
      const float a = ex2_approx((s[i].x - top) + (s[i].w - top0));
      l = fmaf(a, s[i].y, l);
      lr = fmaf(a, s[i].z, lr);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        acc[k].x = fmaf(a, v[i][k].x, acc[k].x);
        acc[k].y = fmaf(a, v[i][k].y, acc[k].y);
        acc[k].z = fmaf(a, v[i][k].z, acc[k].z);
        acc[k].w = fmaf(a, v[i][k].w, acc[k].w);
      }
    }
  }
  const float inv = lr > 0.f ? 1.f / lr : 0.f;
  uint16_t* out = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(tok) * p.out_ts +
                  static_cast<int64_t>(h) * p.out_hs;
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (f0 + 4 * kWarpsJ * k < kUnits)
      *reinterpret_cast<uint2*>(out + (f0 + 4 * kWarpsJ * k) * 4) =
          make_uint2(Pack<BF16>::two(acc[k].x * inv, acc[k].y * inv),
                     Pack<BF16>::two(acc[k].z * inv, acc[k].w * inv));
  if (f0 == 0)
    p.lse[row] = l > 0.f ? (top + log2f(l) + top0) * kLn2 : -INFINITY;
}

template <int HD>
auto join_for(const CacheParams& p) {
  return p.dtype == 1 ? join_kernel<true, HD> : join_kernel<false, HD>;
}

}  // namespace

bool encode_pages(CUtensorMap* m, const CacheParams& p, const Pages& pg, bool tail) {
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.d), static_cast<cuuint64_t>(p.Hkv),
                        static_cast<cuuint64_t>(p.page_size), static_cast<cuuint64_t>(p.num_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(pg.head) * 2, static_cast<cuuint64_t>(pg.slot) * 2,
                           static_cast<cuuint64_t>(pg.page) * 2};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(tail ? kHeadDim - 2 * kChunk : kChunk), 1,
                       static_cast<cuuint32_t>(p.page_size < kKeys ? p.page_size : kKeys), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode_fn()(m, p.dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                     4, const_cast<void*>(pg.base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE,
                     tail ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int device_ctas() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n < kMaxCtas ? n : kMaxCtas;
}

size_t fwd_workspace(int B, int P, int Hq, int Hkv, int d, int64_t total_q) {
  return fwd_ws(B, P, Hq, Hkv, d, total_q).total;
}

cudaError_t launch_fwd(const CacheParams& call, cudaStream_t s) {
  CacheParams p = call;
  // a piece's start takes about 7000 clk where a step takes 3600 (shared
  // prefix without a cap), and 11000 where a step takes 3000 and the first
  // tile is passed over twice (drafts with a cap of 3)
  p.tile_cost = fixed_reference(p) ? 4 : 2;
  const int grid = device_ctas();
  if (grid < 1 || !encode_fn()) return cudaErrorInitializationError;
  const FwdWs w = fwd_ws(p.B, p.P, p.Hq, p.Hkv, p.d, p.total_q);
  CUtensorMap tk, tkt, tv;
  std::memset(&tkt, 0, sizeof tkt);
  if (!encode_pages(&tk, p, p.k, false) || !encode_pages(&tv, p, p.v, false) ||
      (p.d == 160 && !encode_pages(&tkt, p, p.k, true)))
    return cudaErrorInvalidValue;
  cudaError_t e = p.d == 160   ? launch_fwd_d<160>(p, w, tk, tkt, tv, grid, s)
                  : p.d == 128 ? launch_fwd_d<128>(p, w, tk, tkt, tv, grid, s)
                               : launch_fwd_d<64>(p, w, tk, tkt, tv, grid, s);
  if (e != cudaSuccess) return e;
  // a programmatic dependent of the tile kernel: its blocks are placed early
  // and wait for the results
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.total_q), (p.Hq + kHeadsJ - 1) / kHeadsJ);
  cfg.blockDim = dim3(kWarpsJ * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto k = p.d == 160 ? join_for<160>(p) : (p.d == 128 ? join_for<128>(p) : join_for<64>(p));
  return cudaLaunchKernelEx(&cfg, k, p, w);
}

}  // namespace kv
}  // namespace attn
