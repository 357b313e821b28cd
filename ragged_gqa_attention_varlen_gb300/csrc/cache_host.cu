// cache_host.cu -- the C ABI of the generation calls: argument validation and
// the launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <initializer_list>

#include "../../include/attn_varlen.h"
#include "cache.cuh"

using namespace attn;
using namespace attn::kv;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Base alignment and strides of the 16-bit tensors a call reads or writes.  Rows
// that are only read may be expanded (a stride of 0).
struct Strided {
  const void* base;
  std::initializer_list<int64_t> strides;
};
bool strided_from(int64_t least, std::initializer_list<Strided> ts) {
  for (const Strided& t : ts) {
    if (!aligned16(t.base)) return false;
    for (int64_t s : t.strides)
      if (s < least || s % 8) return false;
  }
  return true;
}
bool strided_ok(std::initializer_list<Strided> ts) { return strided_from(8, ts); }
bool readable(std::initializer_list<Strided> ts) { return strided_from(0, ts); }

// Whether the rows of `row` elements that a call writes share none (an expanded
// or overlapping output would hold whatever was written last).  Axes of one
// may have any stride.
struct Axis {
  int64_t n, stride;
};
bool distinct(int64_t row, std::initializer_list<Axis> axes) {
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
bool in_place_ok(const void* in, const void* out, const Axis& in0, const Axis& in1, int64_t out0,
                 int64_t out1) {
  return in != out ||
         ((in0.n <= 1 || in0.stride == out0) && (in1.n <= 1 || in1.stride == out1));
}

bool dim_ok(int d) { return d == 160 || d == 128 || d == 64; }
bool page_ok(int ps) { return ps >= 16 && ps <= 1024 && (ps & (ps - 1)) == 0; }
int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

attn_status rotary_args(const int32_t* positions, int axes, const double* inv_freq, int pairs,
                        int head_dim, int64_t total) {
  if (axes < 1 || pairs < 1 || 2 * pairs > head_dim) return ATTN_ERR_INVALID;
  if (total > 0 && (!positions || !inv_freq)) return ATTN_ERR_INVALID;
  return ATTN_OK;
}

attn_status done(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

bool table_readable(int rows, const int32_t* table, int64_t rs, int width, const int32_t* lens) {
  return rows == 0 || (table && lens && width >= 1 && (rs >= 0 || rows == 1));
}
// The table of a call that writes to its pages: its rows are apart.
bool table_ok(int rows, const int32_t* table, int64_t rs, int width, const int32_t* lens) {
  return table_readable(rows, table, rs, width, lens) && (rs >= width || rows <= 1);
}

// What attention and the key weights share.
attn_status read_args(CacheParams& p, attn_dtype dtype, int B, int P, int Hq, int Hkv, int head_dim,
                      int64_t total_q, const void* q, int64_t q_ts, int64_t q_hs, Pages k, Pages v,
                      bool with_v, int num_pages, int page_size, const Table& own,
                      const Table& prefix, const int32_t* cu_prefix, const int32_t* cu_q,
                      const int32_t* q_pos, const float* slopes, int64_t slopes_bs, int causal,
                      int wl, int wr, float softcap, float scale_multiplier, float* lse,
                      int32_t* status) {
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
  if (!strided_ok({{k.base, {k.page, k.slot, k.head}}})) return ATTN_ERR_ALIGNMENT;
  if (with_v && !strided_ok({{v.base, {v.page, v.slot, v.head}}})) return ATTN_ERR_ALIGNMENT;
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

bool workspace_ok(const void* ws, size_t have, size_t need) {
  return ws && have >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

}  // namespace

extern "C" attn_status attn_varlen_rotary(
    attn_dtype dtype, int64_t total, int Hq, int Hkv, int head_dim, const void* q, int64_t q_ts,
    int64_t q_hs, const void* k, int64_t k_ts, int64_t k_hs, const int32_t* positions,
    int64_t axis_stride, int axes, const double* inv_freq, const int32_t* pair_axis, int pairs,
    int interleaved, int inverse, void* q_out, int64_t qo_ts, int64_t qo_hs, void* k_out,
    int64_t ko_ts, int64_t ko_hs, void* stream) {
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_INVALID;
  if (total < 0 || total > INT32_MAX || Hq < 1 || Hkv < 0) return ATTN_ERR_INVALID;
  if (!dim_ok(head_dim)) return ATTN_ERR_UNSUPPORTED;
  if (Hq + static_cast<int64_t>(Hkv) > 65535) return ATTN_ERR_UNSUPPORTED;
  const attn_status st = rotary_args(positions, axes, inv_freq, pairs, head_dim, total);
  if (st != ATTN_OK) return st;
  if (total == 0) return ATTN_OK;
  if (!q || !q_out || (Hkv > 0 && (!k || !k_out))) return ATTN_ERR_INVALID;
  if (!readable({{q, {q_ts, q_hs}}}) || !strided_ok({{q_out, {qo_ts, qo_hs}}}))
    return ATTN_ERR_ALIGNMENT;
  if (Hkv > 0 && (!readable({{k, {k_ts, k_hs}}}) || !strided_ok({{k_out, {ko_ts, ko_hs}}})))
    return ATTN_ERR_ALIGNMENT;
  if (!distinct(head_dim, {{total, qo_ts}, {Hq, qo_hs}}) ||
      (Hkv > 0 && !distinct(head_dim, {{total, ko_ts}, {Hkv, ko_hs}})) ||
      !in_place_ok(q, q_out, {total, q_ts}, {Hq, q_hs}, qo_ts, qo_hs) ||
      !in_place_ok(k, k_out, {Hkv > 0 ? total : 0, k_ts}, {Hkv, k_hs}, ko_ts, ko_hs))
    return ATTN_ERR_INVALID;
  RotaryParams p;
  std::memset(&p, 0, sizeof p);
  p.dtype = dtype;
  p.d = head_dim;
  p.T = total;
  p.r = {inv_freq, pair_axis, positions, axis_stride, axes, pairs, interleaved != 0, inverse != 0};
  p.t[0] = {q, q_ts, q_hs, q_out, qo_ts, qo_hs, Hq};
  p.t[1] = {k, k_ts, k_hs, k_out, ko_ts, ko_hs, Hkv};
  return done(launch_rotary(p, static_cast<cudaStream_t>(stream)));
}

extern "C" attn_status attn_varlen_cache_append(
    attn_dtype dtype, int B, int Hkv, int head_dim, int64_t total, const void* k, int64_t k_ts,
    int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs, void* k_cache, int64_t kc_ps,
    int64_t kc_ss, int64_t kc_hs, void* v_cache, int64_t vc_ps, int64_t vc_ss, int64_t vc_hs,
    int num_pages, int page_size, const int32_t* table, int64_t table_rs, int table_width,
    const int32_t* lens, const int32_t* cu_new, const int32_t* positions, int64_t axis_stride,
    int axes, const double* inv_freq, const int32_t* pair_axis, int pairs, int interleaved,
    int32_t* key_pos, int64_t kp_rs, int64_t kp_hs, float* scores, int64_t sc_rs, int64_t sc_hs,
    int32_t* lens_out, int32_t* device_status, void* stream) {
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_INVALID;
  if (B < 0 || Hkv < 1 || total < 0 || total > INT32_MAX) return ATTN_ERR_INVALID;
  if (!dim_ok(head_dim) || B > ATTN_MAX_BATCH || Hkv > 4096) return ATTN_ERR_UNSUPPORTED;
  if (B == 0) return total == 0 ? ATTN_OK : ATTN_ERR_INVALID;
  if (!page_ok(page_size) || num_pages < 1) return ATTN_ERR_UNSUPPORTED;
  if (!cu_new || !table_ok(B, table, table_rs, table_width, lens) || lens_out == lens)
    return ATTN_ERR_INVALID;
  if (static_cast<int64_t>(table_width) * page_size > INT32_MAX / 2) return ATTN_ERR_UNSUPPORTED;
  if (inv_freq) {
    const attn_status st = rotary_args(positions, axes, inv_freq, pairs, head_dim, total);
    if (st != ATTN_OK) return st;
  }
  if (!k_cache || !v_cache || (total > 0 && (!k || !v))) return ATTN_ERR_INVALID;
  if (!strided_ok({{k_cache, {kc_ps, kc_ss, kc_hs}}, {v_cache, {vc_ps, vc_ss, vc_hs}}}))
    return ATTN_ERR_ALIGNMENT;
  if (total > 0 && !readable({{k, {k_ts, k_hs}}, {v, {v_ts, v_hs}}})) return ATTN_ERR_ALIGNMENT;
  const int64_t slots = static_cast<int64_t>(table_width) * page_size;
  if (!distinct(head_dim, {{num_pages, kc_ps}, {page_size, kc_ss}, {Hkv, kc_hs}}) ||
      !distinct(head_dim, {{num_pages, vc_ps}, {page_size, vc_ss}, {Hkv, vc_hs}}) ||
      (key_pos && !distinct(slots, {{B, kp_rs}, {Hkv, kp_hs}})) ||
      (scores && !distinct(slots, {{B, sc_rs}, {Hkv, sc_hs}})))
    return ATTN_ERR_INVALID;
  AppendParams p;
  std::memset(&p, 0, sizeof p);
  p.dtype = dtype;
  p.B = B;
  p.Hkv = Hkv;
  p.d = head_dim;
  p.T = total;
  p.kx = k;
  p.vx = v;
  p.k_ts = k_ts;
  p.k_hs = k_hs;
  p.v_ts = v_ts;
  p.v_hs = v_hs;
  p.k = {k_cache, kc_ps, kc_ss, kc_hs};
  p.v = {v_cache, vc_ps, vc_ss, vc_hs};
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.page_log2 = log2_of(page_size);
  p.table = table;
  p.table_rs = table_rs;
  p.width = table_width;
  p.lens = lens;
  p.cu_new = cu_new;
  p.r = {inv_freq, pair_axis, positions, axis_stride, axes, pairs, interleaved != 0, 0};
  p.key_pos = key_pos;
  p.kp_rs = kp_rs;
  p.kp_hs = kp_hs;
  p.scores = scores;
  p.sc_rs = sc_rs;
  p.sc_hs = sc_hs;
  p.lens_out = lens_out;
  p.status = device_status;
  return done(launch_append(p, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t attn_varlen_cache_fwd_workspace_size(int B, int P, int Hq, int Hkv, int head_dim,
                                                       int64_t total_q) {
  if (B < 0 || P < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || total_q < 0 || !dim_ok(head_dim)) return 0;
  return fwd_workspace(B, P, Hq, Hkv, head_dim, total_q);
}

extern "C" attn_status attn_varlen_cache_fwd(
    attn_dtype dtype, int B, int P, int Hq, int Hkv, int head_dim, int64_t total_q, const void* q,
    int64_t q_ts, int64_t q_hs, const void* k_cache, int64_t kc_ps, int64_t kc_ss, int64_t kc_hs,
    const void* v_cache, int64_t vc_ps, int64_t vc_ss, int64_t vc_hs, int num_pages,
    int page_size, const int32_t* table, int64_t table_rs, int table_width, const int32_t* lens,
    const int32_t* prefix_table, int64_t prefix_rs, int prefix_width, const int32_t* prefix_lens,
    const int32_t* cu_prefix, const int32_t* cu_q, const int32_t* q_pos, const int32_t* key_pos,
    int64_t kp_rs, int64_t kp_hs, const int32_t* prefix_key_pos, int64_t pkp_rs, int64_t pkp_hs,
    const float* alibi_slopes, int64_t slopes_bs, int causal, int window_left, int window_right,
    float softcap, float scale_multiplier, void* out, int64_t out_ts, int64_t out_hs, float* lse,
    void* workspace, size_t workspace_bytes, int32_t* device_status, void* stream) {
  CacheParams p;
  std::memset(&p, 0, sizeof p);
  const attn_status st = read_args(
      p, dtype, B, P, Hq, Hkv, head_dim, total_q, q, q_ts, q_hs, {k_cache, kc_ps, kc_ss, kc_hs},
      {v_cache, vc_ps, vc_ss, vc_hs}, true, num_pages, page_size,
      {table, table_rs, table_width, lens, key_pos, kp_rs, kp_hs},
      {prefix_table, prefix_rs, prefix_width, prefix_lens, prefix_key_pos, pkp_rs, pkp_hs},
      cu_prefix, cu_q, q_pos, alibi_slopes, slopes_bs, causal, window_left, window_right, softcap,
      scale_multiplier, lse, device_status);
  if (st != ATTN_OK || total_q == 0) return st;
  if (!out) return ATTN_ERR_INVALID;
  if (!strided_ok({{out, {out_ts, out_hs}}})) return ATTN_ERR_ALIGNMENT;
  if (!distinct(head_dim, {{total_q, out_ts}, {Hq, out_hs}})) return ATTN_ERR_INVALID;
  if (!workspace_ok(workspace, workspace_bytes, fwd_workspace(B, P, Hq, Hkv, head_dim, total_q)))
    return ATTN_ERR_WORKSPACE;
  p.out = out;
  p.out_ts = out_ts;
  p.out_hs = out_hs;
  p.ws = static_cast<uint8_t*>(workspace);
  return done(kv::launch_fwd(p, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t attn_varlen_cache_weights_workspace_size(void) { return weights_workspace(); }

extern "C" attn_status attn_varlen_cache_weights(
    attn_dtype dtype, int B, int P, int Hq, int Hkv, int head_dim, int64_t total_q, const void* q,
    int64_t q_ts, int64_t q_hs, const void* k_cache, int64_t kc_ps, int64_t kc_ss, int64_t kc_hs,
    int num_pages, int page_size, const int32_t* table, int64_t table_rs, int table_width,
    const int32_t* lens, const int32_t* prefix_table, int64_t prefix_rs, int prefix_width,
    const int32_t* prefix_lens, const int32_t* cu_prefix, const int32_t* cu_q,
    const int32_t* q_pos, const int32_t* key_pos, int64_t kp_rs, int64_t kp_hs,
    const int32_t* prefix_key_pos, int64_t pkp_rs, int64_t pkp_hs, const float* alibi_slopes,
    int64_t slopes_bs, int causal, int window_left, int window_right, float softcap,
    float scale_multiplier, const float* lse, const float* scores_in, int64_t si_rs,
    int64_t si_hs, float* scores_out, int64_t so_rs, int64_t so_hs, const float* prefix_scores_in,
    int64_t psi_rs, int64_t psi_hs, float* prefix_scores_out, int64_t pso_rs, int64_t pso_hs,
    void* workspace, size_t workspace_bytes, int32_t* device_status, void* stream) {
  CacheParams p;
  std::memset(&p, 0, sizeof p);
  const attn_status st = read_args(
      p, dtype, B, P, Hq, Hkv, head_dim, total_q, q, q_ts, q_hs, {k_cache, kc_ps, kc_ss, kc_hs},
      {nullptr, 0, 0, 0}, false, num_pages, page_size,
      {table, table_rs, table_width, lens, key_pos, kp_rs, kp_hs},
      {prefix_table, prefix_rs, prefix_width, prefix_lens, prefix_key_pos, pkp_rs, pkp_hs},
      cu_prefix, cu_q, q_pos, alibi_slopes, slopes_bs, causal, window_left, window_right, softcap,
      scale_multiplier, const_cast<float*>(lse), device_status);
  if (st != ATTN_OK || B == 0) return st;
  const int64_t slots = static_cast<int64_t>(table_width) * page_size;
  const int64_t prefix_slots = static_cast<int64_t>(prefix_width) * page_size;
  if (!scores_out || !distinct(slots, {{B, so_rs}, {Hkv, so_hs}}) ||
      !in_place_ok(scores_in, scores_out, {B, si_rs}, {Hkv, si_hs}, so_rs, so_hs))
    return ATTN_ERR_INVALID;
  if (P > 0 && prefix_scores_out &&
      (!distinct(prefix_slots, {{P, pso_rs}, {Hkv, pso_hs}}) ||
       !in_place_ok(prefix_scores_in, prefix_scores_out, {P, psi_rs}, {Hkv, psi_hs}, pso_rs, pso_hs)))
    return ATTN_ERR_INVALID;
  p.w_in[1] = scores_in;
  p.wi_rs[1] = si_rs;
  p.wi_hs[1] = si_hs;
  p.w_out[1] = scores_out;
  p.wo_rs[1] = so_rs;
  p.wo_hs[1] = so_hs;
  if (P > 0) {
    p.w_in[0] = prefix_scores_in;
    p.wi_rs[0] = psi_rs;
    p.wi_hs[0] = psi_hs;
    p.w_out[0] = prefix_scores_out;
    p.wo_rs[0] = pso_rs;
    p.wo_hs[0] = pso_hs;
  }
  if (!workspace_ok(workspace, workspace_bytes, weights_workspace())) return ATTN_ERR_WORKSPACE;
  p.ws = static_cast<uint8_t*>(workspace);
  return done(launch_weights(p, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t attn_varlen_cache_evict_workspace_size(int S, int Hkv, int table_width,
                                                         int page_size, int budget) {
  if (S < 0 || Hkv < 1 || table_width < 1 || !page_ok(page_size) || budget < 1) return 0;
  return evict_workspace(S, Hkv, static_cast<int64_t>(table_width) * page_size, budget);
}

extern "C" attn_status attn_varlen_cache_evict(
    int S, int Hkv, int head_dim, void* k_cache, int64_t kc_ps, int64_t kc_ss, int64_t kc_hs,
    void* v_cache, int64_t vc_ps, int64_t vc_ss, int64_t vc_hs, int num_pages, int page_size,
    const int32_t* table, int64_t table_rs, int table_width, const int32_t* lens,
    const float* scores, int64_t sc_rs, int64_t sc_hs, const int32_t* key_pos, int64_t kp_rs,
    int64_t kp_hs, const int32_t* next_pos, int budget, int recent, float* scores_out,
    int64_t so_rs, int64_t so_hs, int32_t* key_pos_out, int64_t po_rs, int64_t po_hs,
    int32_t* lens_out, void* workspace, size_t workspace_bytes, int32_t* device_status,
    void* stream) {
  if (S < 0 || Hkv < 1 || budget < 1 || recent < 0 || recent > budget) return ATTN_ERR_INVALID;
  if (!dim_ok(head_dim) || S > ATTN_MAX_BATCH ||
      static_cast<int64_t>(S) * Hkv > INT32_MAX / 2)
    return ATTN_ERR_UNSUPPORTED;
  if (S == 0) return ATTN_OK;
  if (!page_ok(page_size) || num_pages < 1) return ATTN_ERR_UNSUPPORTED;
  if (!table_ok(S, table, table_rs, table_width, lens)) return ATTN_ERR_INVALID;
  const int64_t slots = static_cast<int64_t>(table_width) * page_size;
  if (slots > INT32_MAX / 2) return ATTN_ERR_UNSUPPORTED;
  if (!k_cache || !v_cache || !scores || !key_pos || !next_pos || !scores_out || !key_pos_out ||
      !lens_out)
    return ATTN_ERR_INVALID;
  if ((scores_out == scores && (so_rs != sc_rs || so_hs != sc_hs)) ||
      (key_pos_out == key_pos && (po_rs != kp_rs || po_hs != kp_hs)))
    return ATTN_ERR_INVALID;
  if (!strided_ok({{k_cache, {kc_ps, kc_ss, kc_hs}}, {v_cache, {vc_ps, vc_ss, vc_hs}}}))
    return ATTN_ERR_ALIGNMENT;
  if (!distinct(head_dim, {{num_pages, kc_ps}, {page_size, kc_ss}, {Hkv, kc_hs}}) ||
      !distinct(head_dim, {{num_pages, vc_ps}, {page_size, vc_ss}, {Hkv, vc_hs}}) ||
      !distinct(slots, {{S, so_rs}, {Hkv, so_hs}}) ||
      !distinct(slots, {{S, po_rs}, {Hkv, po_hs}}))
    return ATTN_ERR_INVALID;
  if (!workspace_ok(workspace, workspace_bytes, evict_workspace(S, Hkv, slots, budget)))
    return ATTN_ERR_WORKSPACE;
  EvictParams p;
  std::memset(&p, 0, sizeof p);
  p.S = S;
  p.Hkv = Hkv;
  p.d = head_dim;
  p.k = {k_cache, kc_ps, kc_ss, kc_hs};
  p.v = {v_cache, vc_ps, vc_ss, vc_hs};
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.page_log2 = log2_of(page_size);
  p.table = table;
  p.table_rs = table_rs;
  p.width = table_width;
  p.lens = lens;
  p.scores = scores;
  p.sc_rs = sc_rs;
  p.sc_hs = sc_hs;
  p.key_pos = key_pos;
  p.kp_rs = kp_rs;
  p.kp_hs = kp_hs;
  p.next_pos = next_pos;
  p.budget = budget;
  p.recent = recent;
  p.scores_out = scores_out;
  p.so_rs = so_rs;
  p.so_hs = so_hs;
  p.pos_out = key_pos_out;
  p.po_rs = po_rs;
  p.po_hs = po_hs;
  p.lens_out = lens_out;
  p.ws = static_cast<uint8_t*>(workspace);
  p.status = device_status;
  return done(launch_evict(p, static_cast<cudaStream_t>(stream)));
}
