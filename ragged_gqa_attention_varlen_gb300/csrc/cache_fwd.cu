// cache_fwd.cu -- attention over the paged cache: the merge of cut rows, the
// tensor maps and the launches.
#include <cstring>

#include "cache_fwd.cuh"

namespace attn {
namespace kv {

// the tile kernel's instances, in translation units of their own
extern template cudaError_t launch_fwd_d<160>(const CacheParams&, const CUtensorMap&,
                                              const CUtensorMap&, const CUtensorMap&, int,
                                              cudaStream_t);
extern template cudaError_t launch_fwd_d<128>(const CacheParams&, const CUtensorMap&,
                                              const CUtensorMap&, const CUtensorMap&, int,
                                              cudaStream_t);
extern template cudaError_t launch_fwd_d<64>(const CacheParams&, const CUtensorMap&,
                                             const CUtensorMap&, const CUtensorMap&, int,
                                             cudaStream_t);

namespace {

constexpr int kThreadsJ = 128;
constexpr int kRowsJ = 16;  // rows of one token a block joins

// Joins the partial results of a row.  Its own slots were computed in one
// part or several, and so was its prefix; part i has reference m_i, sums l_i
// and lr_i and O_i, and with weights 2^(m_i - max m) the row is sum O_i / sum
// lr_i.  Parts are added in the order of the keys, prefix last, so the result
// does not depend on which CTA finished first.  Rows that one part covers were
// written by the tile kernel already; rows without any key are written here.
template <bool BF16>
__global__ void __launch_bounds__(kThreadsJ) join_kernel(const __grid_constant__ CacheParams p) {
  const int tok = blockIdx.x / p.Hkv, g = blockIdx.x - tok * p.Hkv;
  const FwdWs w = fwd_ws(p.B, p.P, p.Hq, p.Hkv, p.d, p.total_q);
  const int2* info = reinterpret_cast<const int2*>(p.ws + w.info);
  const int2* meta = reinterpret_cast<const int2*>(p.ws + w.meta);
  const float4* stats = reinterpret_cast<const float4*>(p.ws + w.stats);
  const float4* part = reinterpret_cast<const float4*>(p.ws + w.rows);
  if (tok >= __ldg(p.cu_q + p.B)) return;  // behind the last sequence
  const int b = seq_of(p.cu_q, 0, p.B, tok);
  const int pfx = p.P ? prefix_of(p, b) : -1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!reinterpret_cast<const FwdHead*>(p.ws)->ok) return;
  const Seg own = seg_load(p, p.P + b);
  const int2 io = info[p.P + b];
  const int2 ip = pfx >= 0 ? info[pfx] : make_int2(0, 0);
  const int h0 = blockIdx.y * kRowsJ, nr = min(kRowsJ, p.R - h0), units = p.d / 4;
  for (int u = threadIdx.x; u < nr * units; u += kThreadsJ) {
    const int hr = h0 + u / units, f = u - (hr - h0) * units;
    const int h = g * p.R + hr;
    const int64_t xo = static_cast<int64_t>(tok - own.tok0) * p.R + hr;
    const int to = static_cast<int>(xo / kRows), ro = static_cast<int>(xo - static_cast<int64_t>(to) * kRows);
    int no = io.y;
    if (no < 0) {
      int lo, hi;
      tile_keys(p, own, to, lo, hi);
      no = tile_steps(lo, hi);
    }
    int2 mo = make_int2(0, 0), mp = mo;  // (first CTA, parts) of the two segments
    int rp = 0;
    if (no > 0) mo = meta[io.x + g * seg_tiles(p, own) + to];
    if (ip.y > 0) {
      const Seg pre = seg_load(p, pfx);
      const int64_t xp = static_cast<int64_t>(tok - pre.tok0) * p.R + hr;
      const int tp = static_cast<int>(xp / kRows);
      rp = static_cast<int>(xp - static_cast<int64_t>(tp) * kRows);
      mp = meta[ip.x + g * seg_tiles(p, pre) + tp];
    }
    if (mo.y == 1 && mp.y == 0) continue;
    const int parts = mo.y + mp.y;
    auto row_of = [&](int i) -> int64_t {
      if (i < mo.y)
        return mo.y > 1 ? cut_row(w, mo.x + i, i == 0, ro) : whole_row(w, p.total_q, p.Hq, true, tok, h);
      i -= mo.y;
      return mp.y > 1 ? cut_row(w, mp.x + i, i == 0, rp) : whole_row(w, p.total_q, p.Hq, false, tok, h);
    };
    float top = -INFINITY;
    for (int i = 0; i < parts; ++i) {
      const float4 s = stats[row_of(i)];
      if (s.y > 0.f) top = fmaxf(top, s.x);
    }
    float l = 0.f, lr = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int i = 0; i < parts; ++i) {
      const int64_t r = row_of(i);
      const float4 s = stats[r], v = part[r * units + f];
      if (!(s.y > 0.f)) continue;
      const float a = ex2_approx(s.x - top);
      l = fmaf(a, s.y, l);
      lr = fmaf(a, s.z, lr);
      o.x = fmaf(a, v.x, o.x);
      o.y = fmaf(a, v.y, o.y);
      o.z = fmaf(a, v.z, o.z);
      o.w = fmaf(a, v.w, o.w);
    }
    const float inv = lr > 0.f ? 1.f / lr : 0.f;
    uint16_t* out = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(tok) * p.out_ts +
                    static_cast<int64_t>(h) * p.out_hs + f * 4;
    *reinterpret_cast<uint2*>(out) =
        make_uint2(Pack<BF16>::two(o.x * inv, o.y * inv), Pack<BF16>::two(o.z * inv, o.w * inv));
    if (f == 0)
      p.lse[static_cast<int64_t>(tok) * p.Hq + h] = l > 0.f ? (top + log2f(l)) * kLn2 : -INFINITY;
  }
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

cudaError_t launch_fwd(const CacheParams& p, cudaStream_t s) {
  const int grid = device_ctas();
  if (grid < 1 || !encode_fn()) return cudaErrorInitializationError;
  CUtensorMap tk, tkt, tv;
  std::memset(&tkt, 0, sizeof tkt);
  if (!encode_pages(&tk, p, p.k, false) || !encode_pages(&tv, p, p.v, false) ||
      (p.d == 160 && !encode_pages(&tkt, p, p.k, true)))
    return cudaErrorInvalidValue;
  cudaError_t e = p.d == 160   ? launch_fwd_d<160>(p, tk, tkt, tv, grid, s)
                  : p.d == 128 ? launch_fwd_d<128>(p, tk, tkt, tv, grid, s)
                               : launch_fwd_d<64>(p, tk, tkt, tv, grid, s);
  if (e != cudaSuccess) return e;
  // a programmatic dependent of the tile kernel: its blocks are placed early
  // and wait for the results
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.total_q * p.Hkv), (p.R + kRowsJ - 1) / kRowsJ);
  cfg.blockDim = dim3(kThreadsJ);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.dtype == 1 ? join_kernel<true> : join_kernel<false>, p);
}

}  // namespace kv
}  // namespace attn
