// cache_more_host.cu -- the C ABI of norms with rotation, of the cache held in 8
// bits and of the calls that move pages: argument validation and the launches.
#include <vector>

#include "cache_args.h"

using namespace attn;
using namespace attn::kv;

namespace {

attn_status norm_args(NormParams& p, attn_dtype dtype, int64_t total, int Hq, int Hkv, int head_dim, float eps,
                      const int32_t* positions, int64_t axis_stride, int axes, const double* inv_freq,
                      const int32_t* pair_axis, int pairs, int interleaved, int inverse) {
  std::memset(&p, 0, sizeof p);
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_INVALID;
  if (total < 0 || total > INT32_MAX || Hq < 1 || Hkv < 0) return ATTN_ERR_INVALID;
  if (!dim_ok(head_dim) || Hq + static_cast<int64_t>(Hkv) > 65535) return ATTN_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return ATTN_ERR_INVALID;
  if (inv_freq) {
    const attn_status st = rotary_args(positions, axes, inv_freq, pairs, head_dim, total);
    if (st != ATTN_OK) return st;
  }
  p.dtype = dtype;
  p.d = head_dim;
  p.T = total;
  p.eps = eps;
  p.r = {inv_freq, pair_axis, positions, axis_stride, axes, inv_freq ? pairs : 0, interleaved != 0, inverse};
  return ATTN_OK;
}

// One tensor's rows: [total, H, d] read at x (and dy), written at out.
attn_status norm_rows(int64_t total, int H, int d, const void* x, int64_t ts, int64_t hs, const void* dy, int64_t dts,
                      int64_t dhs, bool backward, void* out, int64_t ots, int64_t ohs) {
  if (!x || !out || (backward && !dy)) return ATTN_ERR_INVALID;
  if (!readable({{x, {ts, hs}}}) || (backward && !readable({{dy, {dts, dhs}}})) || !strided_ok({{out, {ots, ohs}}}))
    return ATTN_ERR_ALIGNMENT;
  if (!distinct(d, {{total, ots}, {H, ohs}}) || !in_place_ok(x, out, {total, ts}, {H, hs}, ots, ohs) ||
      (backward && !in_place_ok(dy, out, {total, dts}, {H, dhs}, ots, ohs)))
    return ATTN_ERR_INVALID;
  return ATTN_OK;
}

bool block_ok(int block, int page_size) { return block >= 16 && block <= 128 && (block & (block - 1)) == 0 && block <= page_size; }
bool scale_strides(const Scales& s) { return s.page >= 0 && s.block >= 0 && s.head >= 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Entries of an int32 array, and a table's.
struct Span {
  const void* base;
  __int128 n;
};
Span span(const void* p, int64_t n) { return {p, n}; }
Span span(const void* p, int rows, int64_t stride, int width) {
  return {p, rows > 0 ? static_cast<__int128>(rows - 1) * stride + width : 0};
}
bool meet(const Span& a, const Span& b) {
  if (!a.base || !b.base || a.n < 1 || b.n < 1) return false;
  const __int128 x = reinterpret_cast<uintptr_t>(a.base), y = reinterpret_cast<uintptr_t>(b.base);
  return x < y + 4 * b.n && y < x + 4 * a.n;
}
// Whether the outputs are apart from one another and from the inputs; the first `own`
// of them may be the inputs at their places instead.
bool outputs_apart(std::initializer_list<Span> in, std::initializer_list<Span> out, int own) {
  for (size_t i = 0; i < out.size(); ++i) {
    const Span& o = out.begin()[i];
    for (size_t j = 0; j < in.size(); ++j) {
      const Span& x = in.begin()[j];
      const bool same = i == j && static_cast<int>(i) < own && o.base == x.base;
      if (!same && meet(o, x)) return false;
    }
    for (size_t j = 0; j < i; ++j)
      if (meet(o, out.begin()[j])) return false;
  }
  return true;
}

// The pools that a call moves, as its kernels see them.
attn_status moved_pools(const attn_pool* src, const attn_pool* dst, int n, int page_size, int src_pages, int dst_pages,
                        std::vector<MovedPool>& out) {
  if (n < 0 || (n > 0 && (!src || !dst))) return ATTN_ERR_INVALID;
  if (n > 4096) return ATTN_ERR_UNSUPPORTED;
  out.resize(n);
  for (int i = 0; i < n; ++i) {
    const attn_pool &a = src[i], &b = dst[i];
    if (!a.base || !b.base || a.rows < 1 || a.pieces < 1 || a.bytes < 1) return ATTN_ERR_INVALID;
    if (a.rows != b.rows || a.pieces != b.pieces || a.bytes != b.bytes) return ATTN_ERR_INVALID;
    if (a.rows > page_size || page_size % a.rows) return ATTN_ERR_INVALID;
    if (static_cast<int64_t>(a.rows) * a.pieces * a.bytes > INT32_MAX / 2) return ATTN_ERR_UNSUPPORTED;
    int64_t bits = a.bytes;
    for (const attn_pool* q : {&a, &b})
      bits |= static_cast<int64_t>(reinterpret_cast<uintptr_t>(q->base)) | q->page_stride | q->row_stride | q->piece_stride;
    if (bits & 3) return ATTN_ERR_ALIGNMENT;
    for (const attn_pool* q : {&a, &b})
      if (q->page_stride < 0 || q->row_stride < 0 || q->piece_stride < 0) return ATTN_ERR_ALIGNMENT;
    if (!distinct(b.bytes, {{dst_pages, b.page_stride}, {b.rows, b.row_stride}, {b.pieces, b.piece_stride}}) ||
        (a.base == b.base && (a.page_stride != b.page_stride || a.row_stride != b.row_stride || a.piece_stride != b.piece_stride)))
      return ATTN_ERR_INVALID;
    MovedPool& m = out[i];
    m.src = a.base;
    m.dst = b.base;
    m.src_page = a.page_stride;
    m.src_row = a.row_stride;
    m.src_piece = a.piece_stride;
    m.dst_page = b.page_stride;
    m.dst_row = b.row_stride;
    m.dst_piece = b.piece_stride;
    m.rows = a.rows;
    m.pieces = a.pieces;
    m.bytes = a.bytes;
    m.flat = 1;
    for (const attn_pool* q : {&a, &b}) {
      if (q->pieces > 1 && q->piece_stride != q->bytes) m.flat = 0;
      if (q->rows > 1 && q->row_stride != static_cast<int64_t>(q->pieces) * q->bytes) m.flat = 0;
    }
    m.wide = (bits & 15) == 0;
    if (m.flat && !m.wide && (static_cast<int64_t>(a.pieces) * a.bytes) % 16 == 0) {
      // pieces of few bytes in rows of whole units
      int64_t outer = static_cast<int64_t>(a.pieces) * a.bytes;
      for (const attn_pool* q : {&a, &b}) outer |= static_cast<int64_t>(reinterpret_cast<uintptr_t>(q->base)) | q->page_stride;
      if ((outer & 15) == 0) {
        m.wide = 1;
        m.bytes = a.pieces * a.bytes;
        m.pieces = 1;
      }
    }
  }
  return ATTN_OK;
}

}  // namespace

extern "C" attn_status attn_varlen_norm_rotary(
    attn_dtype dtype, int64_t total, int Hq, int Hkv, int head_dim, const void* q, int64_t q_ts, int64_t q_hs,
    const void* k, int64_t k_ts, int64_t k_hs, const float* q_weight, const float* k_weight, float eps,
    const int32_t* positions, int64_t axis_stride, int axes, const double* inv_freq, const int32_t* pair_axis,
    int pairs, int interleaved, void* q_out, int64_t qo_ts, int64_t qo_hs, void* k_out, int64_t ko_ts, int64_t ko_hs,
    void* stream) {
  NormParams p;
  attn_status st = norm_args(p, dtype, total, Hq, Hkv, head_dim, eps, positions, axis_stride, axes, inv_freq,
                             pair_axis, pairs, interleaved, 0);
  if (st != ATTN_OK || total == 0) return st;
  st = norm_rows(total, Hq, head_dim, q, q_ts, q_hs, nullptr, 0, 0, false, q_out, qo_ts, qo_hs);
  if (st == ATTN_OK && Hkv > 0) st = norm_rows(total, Hkv, head_dim, k, k_ts, k_hs, nullptr, 0, 0, false, k_out, ko_ts, ko_hs);
  if (st != ATTN_OK) return st;
  if (!aligned4(q_weight) || !aligned4(k_weight)) return ATTN_ERR_ALIGNMENT;
  p.t[0] = {q, q_ts, q_hs, nullptr, 0, 0, q_weight, q_out, qo_ts, qo_hs, nullptr, Hq};
  p.t[1] = {k, k_ts, k_hs, nullptr, 0, 0, k_weight, k_out, ko_ts, ko_hs, nullptr, Hkv};
  return done(launch_norm(p, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t attn_varlen_norm_rotary_bwd_workspace_size(int64_t total, int Hq, int Hkv, int head_dim) {
  if (total < 0 || total > INT32_MAX || Hq < 1 || Hkv < 0 || !dim_ok(head_dim)) return 0;
  return norm_bwd_workspace(total, Hq, Hkv, head_dim);
}

extern "C" attn_status attn_varlen_norm_rotary_bwd(
    attn_dtype dtype, int64_t total, int Hq, int Hkv, int head_dim, const void* dq_out, int64_t dqo_ts, int64_t dqo_hs,
    const void* dk_out, int64_t dko_ts, int64_t dko_hs, const void* q, int64_t q_ts, int64_t q_hs, const void* k,
    int64_t k_ts, int64_t k_hs, const float* q_weight, const float* k_weight, float eps, const int32_t* positions,
    int64_t axis_stride, int axes, const double* inv_freq, const int32_t* pair_axis, int pairs, int interleaved,
    void* dq, int64_t dq_ts, int64_t dq_hs, void* dk, int64_t dk_ts, int64_t dk_hs, float* dq_weight, float* dk_weight,
    void* workspace, size_t workspace_bytes, void* stream) {
  NormParams p;
  attn_status st = norm_args(p, dtype, total, Hq, Hkv, head_dim, eps, positions, axis_stride, axes, inv_freq,
                             pair_axis, pairs, interleaved, 1);
  if (st != ATTN_OK) return st;
  if (Hkv == 0 && dk_weight) return ATTN_ERR_INVALID;
  if (dq_weight && dq_weight == dk_weight) return ATTN_ERR_INVALID;
  if (total == 0 && !dq_weight && !dk_weight) return ATTN_OK;
  if (total > 0) {
    st = norm_rows(total, Hq, head_dim, q, q_ts, q_hs, dq_out, dqo_ts, dqo_hs, true, dq, dq_ts, dq_hs);
    if (st == ATTN_OK && Hkv > 0)
      st = norm_rows(total, Hkv, head_dim, k, k_ts, k_hs, dk_out, dko_ts, dko_hs, true, dk, dk_ts, dk_hs);
    if (st != ATTN_OK) return st;
  }
  if (!aligned4(q_weight) || !aligned4(k_weight) || !aligned4(dq_weight) || !aligned4(dk_weight)) return ATTN_ERR_ALIGNMENT;
  if ((dq_weight || dk_weight) && !workspace_ok(workspace, workspace_bytes, norm_bwd_workspace(total, Hq, Hkv, head_dim)))
    return ATTN_ERR_WORKSPACE;
  p.t[0] = {q, q_ts, q_hs, dq_out, dqo_ts, dqo_hs, q_weight, dq, dq_ts, dq_hs, dq_weight, Hq};
  p.t[1] = {k, k_ts, k_hs, dk_out, dko_ts, dko_hs, k_weight, dk, dk_ts, dk_hs, dk_weight, Hkv};
  p.partial = static_cast<float*>(workspace);
  return done(launch_norm_bwd(p, static_cast<cudaStream_t>(stream)));
}

extern "C" attn_status attn_varlen_cache8_append(
    attn_dtype dtype, int B, int Hkv, int head_dim, int64_t total, const void* k, int64_t k_ts, int64_t k_hs,
    const void* v, int64_t v_ts, int64_t v_hs, void* k_cache, int64_t kc_ps, int64_t kc_ss, int64_t kc_hs,
    void* v_cache, int64_t vc_ps, int64_t vc_ss, int64_t vc_hs, float* k_scale, int64_t ks_ps, int64_t ks_bs,
    int64_t ks_hs, float* v_scale, int64_t vs_ps, int64_t vs_bs, int64_t vs_hs, int num_pages, int page_size,
    int scale_block, const int32_t* table, int64_t table_rs, int table_width, const int32_t* lens,
    const int32_t* cu_new, const int32_t* positions, int64_t axis_stride, int axes, const double* inv_freq,
    const int32_t* pair_axis, int pairs, int interleaved, int norm, const float* k_weight, float eps, int32_t* key_pos,
    int64_t kp_rs, int64_t kp_hs, int32_t* lens_out, int32_t* device_status, void* stream) {
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_INVALID;
  if (B < 0 || Hkv < 1 || total < 0 || total > INT32_MAX) return ATTN_ERR_INVALID;
  if (!dim_ok(head_dim) || B > ATTN_MAX_BATCH || Hkv > 4096) return ATTN_ERR_UNSUPPORTED;
  if (B == 0) return total == 0 ? ATTN_OK : ATTN_ERR_INVALID;
  if (!page_ok(page_size) || num_pages < 1 || !block_ok(scale_block, page_size)) return ATTN_ERR_UNSUPPORTED;
  if (!cu_new || !table_ok(B, table, table_rs, table_width, lens) || lens_out == lens) return ATTN_ERR_INVALID;
  if (static_cast<int64_t>(table_width) * page_size > INT32_MAX / 2) return ATTN_ERR_UNSUPPORTED;
  if (inv_freq) {
    const attn_status st = rotary_args(positions, axes, inv_freq, pairs, head_dim, total);
    if (st != ATTN_OK) return st;
  }
  if (!append_outputs_apart(B, Hkv, total, page_size, table, table_rs, table_width, lens, cu_new, positions, axis_stride, axes,
                            inv_freq, pair_axis, pairs, key_pos, kp_rs, kp_hs, nullptr, 0, 0, lens_out))
    return ATTN_ERR_INVALID;
  if (norm && (!(eps >= 0.f) || !std::isfinite(eps))) return ATTN_ERR_INVALID;
  if (!k_cache || !v_cache || !k_scale || !v_scale || (total > 0 && (!k || !v))) return ATTN_ERR_INVALID;
  if (!strided_from(16, {{k_cache, {kc_ps, kc_ss, kc_hs}}, {v_cache, {vc_ps, vc_ss, vc_hs}}}, 16)) return ATTN_ERR_ALIGNMENT;
  if (total > 0 && !readable({{k, {k_ts, k_hs}}, {v, {v_ts, v_hs}}})) return ATTN_ERR_ALIGNMENT;
  const Scales ks = {k_scale, ks_ps, ks_bs, ks_hs}, vs = {v_scale, vs_ps, vs_bs, vs_hs};
  if (!aligned4(k_scale) || !aligned4(v_scale) || !aligned4(k_weight) || !scale_strides(ks) || !scale_strides(vs))
    return ATTN_ERR_ALIGNMENT;
  const int64_t slots = static_cast<int64_t>(table_width) * page_size;
  const int64_t blocks = page_size / scale_block;
  if (!distinct(head_dim, {{num_pages, kc_ps}, {page_size, kc_ss}, {Hkv, kc_hs}}) ||
      !distinct(head_dim, {{num_pages, vc_ps}, {page_size, vc_ss}, {Hkv, vc_hs}}) ||
      !distinct(1, {{num_pages, ks_ps}, {blocks, ks_bs}, {Hkv, ks_hs}}) ||
      !distinct(1, {{num_pages, vs_ps}, {blocks, vs_bs}, {Hkv, vs_hs}}) || k_cache == v_cache || k_scale == v_scale ||
      (key_pos && !distinct(slots, {{B, kp_rs}, {Hkv, kp_hs}})))
    return ATTN_ERR_INVALID;
  Append8Params p;
  std::memset(&p, 0, sizeof p);
  AppendParams& a = p.a;
  a.dtype = dtype;
  a.B = B;
  a.Hkv = Hkv;
  a.d = head_dim;
  a.T = total;
  a.kx = k;
  a.vx = v;
  a.k_ts = k_ts;
  a.k_hs = k_hs;
  a.v_ts = v_ts;
  a.v_hs = v_hs;
  a.k = {k_cache, kc_ps, kc_ss, kc_hs};
  a.v = {v_cache, vc_ps, vc_ss, vc_hs};
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.page_log2 = log2_of(page_size);
  a.table = table;
  a.table_rs = table_rs;
  a.width = table_width;
  a.lens = lens;
  a.cu_new = cu_new;
  a.r = {inv_freq, pair_axis, positions, axis_stride, axes, pairs, interleaved != 0, 0};
  a.key_pos = key_pos;
  a.kp_rs = kp_rs;
  a.kp_hs = kp_hs;
  a.lens_out = lens_out;
  a.status = device_status;
  p.ks = ks;
  p.vs = vs;
  p.block = scale_block;
  p.block_log2 = log2_of(scale_block);
  p.k_weight = k_weight;
  p.norm = norm != 0;
  p.eps = eps;
  return done(launch_append8(p, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t attn_varlen_cache8_fwd_workspace_size(int B, int P, int Hq, int Hkv, int head_dim, int64_t total_q) {
  if (B < 0 || P < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || total_q < 0 || !dim_ok(head_dim)) return 0;
  return fwd8_workspace(B, P, Hq, Hkv, head_dim, total_q);
}

extern "C" attn_status attn_varlen_cache8_fwd(
    attn_dtype dtype, int B, int P, int Hq, int Hkv, int head_dim, int64_t total_q, const void* q, int64_t q_ts,
    int64_t q_hs, const void* k_cache, int64_t kc_ps, int64_t kc_ss, int64_t kc_hs, const void* v_cache, int64_t vc_ps,
    int64_t vc_ss, int64_t vc_hs, const float* k_scale, int64_t ks_ps, int64_t ks_bs, int64_t ks_hs,
    const float* v_scale, int64_t vs_ps, int64_t vs_bs, int64_t vs_hs, int num_pages, int page_size, int scale_block,
    const int32_t* table, int64_t table_rs, int table_width, const int32_t* lens, const int32_t* prefix_table,
    int64_t prefix_rs, int prefix_width, const int32_t* prefix_lens, const int32_t* cu_prefix, const int32_t* cu_q,
    const int32_t* q_pos, const int32_t* key_pos, int64_t kp_rs, int64_t kp_hs, const int32_t* prefix_key_pos,
    int64_t pkp_rs, int64_t pkp_hs, const float* alibi_slopes, int64_t slopes_bs, int causal, int window_left,
    int window_right, float softcap, float scale_multiplier, void* out, int64_t out_ts, int64_t out_hs, float* lse,
    void* workspace, size_t workspace_bytes, int32_t* device_status, void* stream) {
  Cache8Params p8;
  std::memset(&p8, 0, sizeof p8);
  CacheParams& p = p8.c;
  const attn_status st = read_args(
      p, dtype, B, P, Hq, Hkv, head_dim, total_q, q, q_ts, q_hs, {k_cache, kc_ps, kc_ss, kc_hs},
      {v_cache, vc_ps, vc_ss, vc_hs}, true, num_pages, page_size,
      {table, table_rs, table_width, lens, key_pos, kp_rs, kp_hs},
      {prefix_table, prefix_rs, prefix_width, prefix_lens, prefix_key_pos, pkp_rs, pkp_hs}, cu_prefix, cu_q, q_pos,
      alibi_slopes, slopes_bs, causal, window_left, window_right, softcap, scale_multiplier, lse, device_status, 16);
  if (st != ATTN_OK) return st;
  if (B == 0) return ATTN_OK;
  if (!block_ok(scale_block, page_size)) return ATTN_ERR_UNSUPPORTED;
  if (!k_scale || !v_scale) return ATTN_ERR_INVALID;
  p8.ks = {const_cast<float*>(k_scale), ks_ps, ks_bs, ks_hs};
  p8.vs = {const_cast<float*>(v_scale), vs_ps, vs_bs, vs_hs};
  if (!aligned4(k_scale) || !aligned4(v_scale) || !scale_strides(p8.ks) || !scale_strides(p8.vs)) return ATTN_ERR_ALIGNMENT;
  if (total_q == 0) return ATTN_OK;
  if (!out) return ATTN_ERR_INVALID;
  if (!strided_ok({{out, {out_ts, out_hs}}})) return ATTN_ERR_ALIGNMENT;
  if (!distinct(head_dim, {{total_q, out_ts}, {Hq, out_hs}})) return ATTN_ERR_INVALID;
  if (!workspace_ok(workspace, workspace_bytes, fwd8_workspace(B, P, Hq, Hkv, head_dim, total_q)))
    return ATTN_ERR_WORKSPACE;
  p.out = out;
  p.out_ts = out_ts;
  p.out_hs = out_hs;
  p.ws = static_cast<uint8_t*>(workspace);
  p8.block_log2 = log2_of(scale_block);
  return done(launch_fwd8(p8, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t attn_varlen_cache_fork_workspace_size(int rows, int table_width, int num_pages) {
  if (rows < 0 || rows > ATTN_MAX_BATCH || table_width < 1 || num_pages < 1 ||
      static_cast<int64_t>(rows) * table_width > (1 << 28) || num_pages > (1 << 28))
    return 0;
  return fork_workspace(rows, table_width, num_pages);
}

extern "C" attn_status attn_varlen_cache_fork(
    int rows, int num_pages, int page_size, const attn_pool* pools, int npools, const int32_t* table, int64_t table_rs,
    int table_width, const int32_t* lens, const int32_t* held, const int32_t* refs, const int32_t* parents,
    const int32_t* room, int32_t* table_out, int64_t table_out_rs, int32_t* lens_out, int32_t* held_out,
    int32_t* refs_out, void* workspace, size_t workspace_bytes, int32_t* device_status, void* stream) {
  if (rows < 0 || num_pages < 1 || table_width < 1) return ATTN_ERR_INVALID;
  if (rows > ATTN_MAX_BATCH || !page_ok(page_size) || static_cast<int64_t>(rows) * table_width > (1 << 28) ||
      num_pages > (1 << 28) || static_cast<int64_t>(table_width) * page_size > INT32_MAX / 2)
    return ATTN_ERR_UNSUPPORTED;
  if (!refs || !refs_out) return ATTN_ERR_INVALID;
  if (rows > 0 && (!table || !lens || !held || !parents || !table_out || !lens_out || !held_out)) return ATTN_ERR_INVALID;
  if (rows > 1 && (table_rs < table_width || table_out_rs < table_width)) return ATTN_ERR_INVALID;
  if (rows > 1 && table_out == table && table_out_rs != table_rs) return ATTN_ERR_INVALID;
  if (!outputs_apart({span(table, rows, table_rs, table_width), span(lens, rows), span(held, rows), span(refs, num_pages),
                      span(parents, rows), span(room, rows)},
                     {span(table_out, rows, table_out_rs, table_width), span(lens_out, rows), span(held_out, rows),
                      span(refs_out, num_pages)},
                     4))
    return ATTN_ERR_INVALID;
  std::vector<MovedPool> m;
  attn_status st;
  try {
    st = moved_pools(pools, pools, npools, page_size, num_pages, num_pages, m);
  } catch (...) {  // (no host memory for the list)
    return ATTN_ERR_CUDA;
  }
  if (st != ATTN_OK) return st;
  if (!workspace_ok(workspace, workspace_bytes, fork_workspace(rows, table_width, num_pages))) return ATTN_ERR_WORKSPACE;
  const ForkParams p = {rows, table_width, num_pages, log2_of(page_size), table, table_rs, lens, held, refs, parents, room,
                        table_out, table_out_rs, lens_out, held_out, refs_out, static_cast<uint8_t*>(workspace), device_status};
  return done(launch_fork(p, m.data(), npools, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t attn_varlen_cache_compact_workspace_size(int num_pages) {
  return num_pages < 1 || num_pages > (1 << 28) ? 0 : compact_workspace(num_pages);
}

extern "C" attn_status attn_varlen_cache_compact(
    int num_pages, int page_size, const attn_pool* pools, int npools, int rows, const int32_t* table, int64_t table_rs,
    int table_width, const int32_t* held, int32_t* table_out, int64_t table_out_rs, int prefix_rows,
    const int32_t* prefix_table, int64_t prefix_rs, int prefix_width, const int32_t* prefix_held,
    int32_t* prefix_table_out, int64_t prefix_out_rs, const int32_t* refs, int32_t* refs_out, int32_t* live,
    void* workspace, size_t workspace_bytes, int32_t* device_status, void* stream) {
  if (rows < 0 || prefix_rows < 0 || num_pages < 1) return ATTN_ERR_INVALID;
  if (rows > ATTN_MAX_BATCH || prefix_rows > ATTN_MAX_BATCH || !page_ok(page_size) || num_pages > (1 << 28))
    return ATTN_ERR_UNSUPPORTED;
  if (!refs || !refs_out || !live) return ATTN_ERR_INVALID;
  CompactParams p;
  std::memset(&p, 0, sizeof p);
  p.t[0] = {rows, table_width, table, table_rs, held, table_out, table_out_rs};
  p.t[1] = {prefix_rows, prefix_width, prefix_table, prefix_rs, prefix_held, prefix_table_out, prefix_out_rs};
  for (const CompactTable& t : p.t) {
    if (t.R == 0) continue;
    if (t.W < 1 || !t.table || !t.held || !t.out) return ATTN_ERR_INVALID;
    if (static_cast<int64_t>(t.R) * t.W > (1 << 28)) return ATTN_ERR_UNSUPPORTED;
    if (t.R > 1 && (t.rs < t.W || t.out_rs < t.W || (t.out == t.table && t.out_rs != t.rs))) return ATTN_ERR_INVALID;
  }
  const CompactTable &s = p.t[0], &f = p.t[1];
  if (!outputs_apart({span(s.table, s.R, s.rs, s.W), span(f.table, f.R, f.rs, f.W), span(refs, num_pages), span(s.held, s.R),
                      span(f.held, f.R)},
                     {span(s.out, s.R, s.out_rs, s.W), span(f.out, f.R, f.out_rs, f.W), span(refs_out, num_pages), span(live, 1)}, 3))
    return ATTN_ERR_INVALID;
  std::vector<MovedPool> m;
  attn_status st;
  try {
    st = moved_pools(pools, pools, npools, page_size, num_pages, num_pages, m);
  } catch (...) {
    return ATTN_ERR_CUDA;
  }
  if (st != ATTN_OK) return st;
  if (!workspace_ok(workspace, workspace_bytes, compact_workspace(num_pages))) return ATTN_ERR_WORKSPACE;
  p.N = num_pages;
  p.page_log2 = log2_of(page_size);
  p.refs = refs;
  p.refs_out = refs_out;
  p.live = live;
  p.ws = static_cast<uint8_t*>(workspace);
  p.status = device_status;
  return done(launch_compact(p, m.data(), npools, static_cast<cudaStream_t>(stream)));
}

extern "C" attn_status attn_varlen_cache_copy(int count, const int32_t* src_pages, const int32_t* dst_pages,
                                              int num_src_pages, int num_dst_pages, int page_size,
                                              const attn_pool* src_pools, const attn_pool* dst_pools, int npools,
                                              int32_t* device_status, void* stream) {
  if (count < 0 || num_src_pages < 1 || num_dst_pages < 1) return ATTN_ERR_INVALID;
  if (!page_ok(page_size) || num_src_pages > (1 << 28) || num_dst_pages > (1 << 28)) return ATTN_ERR_UNSUPPORTED;
  if (count > 0 && (!src_pages || !dst_pages)) return ATTN_ERR_INVALID;
  std::vector<MovedPool> m;
  attn_status st;
  try {
    st = moved_pools(src_pools, dst_pools, npools, page_size, num_src_pages, num_dst_pages, m);
  } catch (...) {
    return ATTN_ERR_CUDA;
  }
  if (st != ATTN_OK || count == 0 || npools == 0) return st;
  return done(launch_copy_pages(src_pages, dst_pages, count, num_src_pages, num_dst_pages, m.data(), npools, device_status,
                                static_cast<cudaStream_t>(stream)));
}
