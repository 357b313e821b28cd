// cache_args.h -- checks of arguments that the C entry points of the generation
// calls share.
#pragma once
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <initializer_list>
#include <utility>

#include "../../include/attn_varlen.h"
#include "cache.cuh"

namespace attn {
namespace kv {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Base alignment and strides of the tensors a call reads or writes (`unit` elements
// are 16 bytes).  Rows that are only read may be expanded (a stride of 0).
struct Strided {
  const void* base;
  std::initializer_list<int64_t> strides;
};
inline bool strided_from(int64_t least, std::initializer_list<Strided> ts, int unit = 8) {
  for (const Strided& t : ts) {
    if (!aligned16(t.base)) return false;
    for (int64_t s : t.strides)
      if (s < least || s % unit) return false;
  }
  return true;
}
inline bool strided_ok(std::initializer_list<Strided> ts) { return strided_from(8, ts); }
inline bool readable(std::initializer_list<Strided> ts) { return strided_from(0, ts); }

// Whether the rows of `row` elements that a call writes share none (an expanded
// or overlapping output would hold whatever was written last).  Axes of one
// may have any stride.
struct Axis {
  int64_t n, stride;
};
inline bool distinct(int64_t row, std::initializer_list<Axis> axes) {
  Axis a[3];
  int k = 0;
  for (const Axis& x : axes) {  // in order of the strides
    if (x.n <= 1) continue;
    int i = k++;
    for (; i > 0 && a[i - 1].stride > x.stride; --i) a[i] = a[i - 1];
    a[i] = x;
  }
  __int128 extent = row;
  for (int i = 0; i < k; ++i) {
    if (a[i].stride < extent) return false;
    extent += static_cast<__int128>(a[i].n - 1) * a[i].stride;
  }
  return true;
}
// In place means the same elements.
inline bool in_place_ok(const void* in, const void* out, const Axis& in0, const Axis& in1, int64_t out0,
                 int64_t out1) {
  return in != out ||
         ((in0.n <= 1 || in0.stride == out0) && (in1.n <= 1 || in1.stride == out1));
}

// Elements of an array in memory: runs of `run` bytes on up to two axes (strides in
// bytes; negative ones are refused elsewhere).
struct Area {
  const void* base;
  __int128 run;
  Axis outer, inner;
  Area(const void* p, __int128 bytes, Axis a = {1, 0}, Axis b = {1, 0}) : base(p), run(bytes), outer(a), inner(b) {
    if (inner.stride > outer.stride && inner.n > 1) std::swap(outer, inner);
    for (Axis* x : {&outer, &inner})
      if (x->n <= 1 || x->stride <= 0) *x = {x->n < 1 ? 0 : 1, 0};
  }
  bool empty() const { return !base || run < 1 || outer.n < 1 || inner.n < 1; }
  __int128 at() const { return reinterpret_cast<uintptr_t>(base); }
  __int128 length() const { return (outer.n - 1) * static_cast<__int128>(outer.stride) + row(); }
  __int128 row() const { return (inner.n - 1) * static_cast<__int128>(inner.stride) + run; }
};
// Which of n pieces of `piece` bytes, `stride` apart, may meet [lo, hi) (relative to the first).
inline bool pieces_that_meet(const Axis& x, __int128 piece, __int128 lo, __int128 hi, __int128& from, __int128& to) {
  if (hi <= 0 || lo >= (x.n - 1) * static_cast<__int128>(x.stride) + piece) return false;
  from = x.stride && lo >= piece ? (lo - piece) / x.stride + 1 : 0;
  to = x.stride ? (hi - 1) / x.stride : 0;
  if (to > x.n - 1) to = x.n - 1;
  return from <= to;
}
inline bool meets(const Area& a, __int128 lo, __int128 hi) {
  __int128 i0, i1, j0, j1;
  if (!pieces_that_meet(a.outer, a.row(), lo, hi, i0, i1)) return false;
  for (__int128 i = i0; i <= i1; ++i)
    if (pieces_that_meet(a.inner, a.run, lo - i * a.outer.stride, hi - i * a.outer.stride, j0, j1)) return true;
  return false;
}
// Whether two arrays share a byte.  Runs of the one with fewer are looked for in the
// other, but only where the ranges that the arrays span meet at all.
inline bool share_memory(const Area& x, const Area& y) {
  if (x.empty() || y.empty() || x.at() >= y.at() + y.length() || y.at() >= x.at() + x.length()) return false;
  const bool swap = x.outer.n * x.inner.n > y.outer.n * y.inner.n;
  const Area &a = swap ? y : x, &b = swap ? x : y;
  for (int64_t i = 0; i < a.outer.n; ++i)
    for (int64_t j = 0; j < a.inner.n; ++j) {
      const __int128 lo = a.at() + i * static_cast<__int128>(a.outer.stride) + j * static_cast<__int128>(a.inner.stride) - b.at();
      if (meets(b, lo, lo + a.run)) return true;
    }
  return false;
}

inline bool dim_ok(int d) { return d == 160 || d == 128 || d == 64; }
inline bool page_ok(int ps) { return ps >= 16 && ps <= 1024 && (ps & (ps - 1)) == 0; }
inline int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

inline attn_status rotary_args(const int32_t* positions, int axes, const double* inv_freq, int pairs,
                        int head_dim, int64_t total) {
  if (axes < 1 || pairs < 1 || 2 * pairs > head_dim) return ATTN_ERR_INVALID;
  if (total > 0 && (!positions || !inv_freq)) return ATTN_ERR_INVALID;
  return ATTN_OK;
}

inline attn_status done(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

inline bool table_readable(int rows, const int32_t* table, int64_t rs, int width, const int32_t* lens) {
  return rows == 0 || (table && lens && width >= 1 && (rs >= 0 || rows == 1));
}
// The table of a call that writes to its pages: its rows are apart.
inline bool table_ok(int rows, const int32_t* table, int64_t rs, int width, const int32_t* lens) {
  return table_readable(rows, table, rs, width, lens) && (rs >= width || rows <= 1);
}

// Whether what an append writes beside the pages is apart from what its other blocks
// of threads still read, and from one another.
inline bool append_outputs_apart(int B, int Hkv, int64_t total, int page_size, const int32_t* table, int64_t table_rs,
                                 int width, const int32_t* lens, const int32_t* cu_new, const int32_t* positions,
                                 int64_t axis_stride, int axes, const double* inv_freq, const int32_t* pair_axis,
                                 int pairs, const int32_t* key_pos, int64_t kp_rs, int64_t kp_hs, const float* scores,
                                 int64_t sc_rs, int64_t sc_hs, const int32_t* lens_out) {
  const int64_t slots = static_cast<int64_t>(width) * page_size;
  const bool turned = inv_freq != nullptr;
  const Area in[] = {{lens, 4 * static_cast<__int128>(B)},
                     {cu_new, 4 * (static_cast<__int128>(B) + 1)},
                     {table, 4 * static_cast<__int128>(width), {B, 4 * table_rs}},
                     {positions, 4 * static_cast<__int128>(total), {turned ? axes : 1, 4 * axis_stride}},
                     {inv_freq, 8 * static_cast<__int128>(turned ? pairs : 0)},
                     {pair_axis, 4 * static_cast<__int128>(turned ? pairs : 0)}};
  const Area out[] = {{lens_out, 4 * static_cast<__int128>(B)},
                      {key_pos, 4 * static_cast<__int128>(slots), {B, 4 * kp_rs}, {Hkv, 4 * kp_hs}},
                      {scores, 4 * static_cast<__int128>(slots), {B, 4 * sc_rs}, {Hkv, 4 * sc_hs}}};
  for (const Area& o : out) {
    for (const Area& i : in)
      if (share_memory(o, i)) return false;
    for (const Area& x : out)
      if (&x != &o && share_memory(o, x)) return false;
  }
  return true;
}

// What attention and the key weights share.  `unit`: the pages' elements in 16
// bytes.
inline attn_status read_args(CacheParams& p, attn_dtype dtype, int B, int P, int Hq, int Hkv, int head_dim,
                      int64_t total_q, const void* q, int64_t q_ts, int64_t q_hs, Pages k, Pages v,
                      bool with_v, int num_pages, int page_size, const Table& own,
                      const Table& prefix, const int32_t* cu_prefix, const int32_t* cu_q,
                      const int32_t* q_pos, const float* slopes, int64_t slopes_bs, int causal,
                      int wl, int wr, float softcap, float scale_multiplier, float* lse,
                      int32_t* status, int unit = 8) {
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_INVALID;
  if (B < 0 || P < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || total_q < 0) return ATTN_ERR_INVALID;
  if (!dim_ok(head_dim)) return ATTN_ERR_UNSUPPORTED;
  if (B > ATTN_MAX_BATCH || P > ATTN_MAX_BATCH) return ATTN_ERR_UNSUPPORTED;
  if (total_q * Hq > INT32_MAX || Hq > 65536) return ATTN_ERR_UNSUPPORTED;
  if (!std::isfinite(softcap) || !std::isfinite(scale_multiplier)) return ATTN_ERR_INVALID;
  if ((B == 0 && total_q > 0) || (B == 0 && P > 0)) return ATTN_ERR_INVALID;
  if (B == 0) return ATTN_OK;
  if (!page_ok(page_size) || num_pages < 1) return ATTN_ERR_UNSUPPORTED;
  if (!cu_q || !table_readable(B, own.pages, own.rs, own.width, own.lens)) return ATTN_ERR_INVALID;
  if (P > 0 && (!cu_prefix || !table_readable(P, prefix.pages, prefix.rs, prefix.width, prefix.lens)))
    return ATTN_ERR_INVALID;
  if (static_cast<int64_t>(own.width) * page_size > INT32_MAX / 2 ||
      static_cast<int64_t>(prefix.width) * page_size > INT32_MAX / 2)
    return ATTN_ERR_UNSUPPORTED;
  if (total_q > 0 && (own.pos || (P > 0 && prefix.pos)) && !q_pos) return ATTN_ERR_INVALID;
  if (slopes && B > 1 && slopes_bs != 0 && slopes_bs < Hq) return ATTN_ERR_INVALID;
  if (!k.base || (with_v && !v.base) || (total_q > 0 && (!q || !lse))) return ATTN_ERR_INVALID;
  if (total_q > 0 && !readable({{q, {q_ts, q_hs}}})) return ATTN_ERR_ALIGNMENT;
  if (!strided_from(unit, {{k.base, {k.page, k.slot, k.head}}}, unit)) return ATTN_ERR_ALIGNMENT;
  if (with_v && !strided_from(unit, {{v.base, {v.page, v.slot, v.head}}}, unit)) return ATTN_ERR_ALIGNMENT;
  p.dtype = dtype;
  p.B = B;
  p.P = P;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.d = head_dim;
  p.R = Hq / Hkv;
  p.inv_R = 1.f / static_cast<float>(p.R);
  p.total_q = total_q;
  p.q = q;
  p.q_ts = q_ts;
  p.q_hs = q_hs;
  p.k = k;
  p.v = v;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.page_log2 = log2_of(page_size);
  p.own = own;
  p.prefix = prefix;
  p.cu_prefix = cu_prefix;
  p.cu_q = cu_q;
  p.q_pos = q_pos;
  p.slopes = slopes;
  p.slopes_bs = slopes_bs;
  // positions lie in [0, 2^30): a wider window changes nothing
  const int far = 1 << 30;
  const int right = causal ? 0 : wr;
  p.wl = wl < 0 ? -1 : (wl > far ? far : wl);
  p.wr = right < 0 ? -1 : (right > far ? far : right);
  p.softcap = softcap;
  p.sigma = static_cast<float>(static_cast<double>(scale_multiplier) /
                               std::sqrt(static_cast<double>(head_dim)));
  p.lse = lse;
  p.status = status;
  return ATTN_OK;
}

inline bool workspace_ok(const void* ws, size_t have, size_t need) {
  return ws && have >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

}  // namespace kv
}  // namespace attn
