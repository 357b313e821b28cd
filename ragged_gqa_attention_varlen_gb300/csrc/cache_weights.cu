// cache_weights.cu -- the attention weight that each cached key receives.
#include "../../include/attn_varlen.h"
#include "cache.cuh"

namespace attn {
namespace kv {
namespace {

constexpr int kThreadsA = 128;
constexpr int kPerLane = kHeadDim / 32;

struct Row {
  int b, g, qpos, prefix, prefix_len, own_len;
};

// What packed row (token, head) reads; false: the token is behind the last
// sequence, or the call's lengths are inconsistent.
__device__ bool find_row(const CacheParams& p, int tok, int h, Row& r) {
  if (p.B == 0 || tok >= __ldg(p.cu_q + p.B)) return false;
  r.b = seq_of(p.cu_q, 0, p.B, tok);
  const int c0 = __ldg(p.cu_q + r.b), c1 = __ldg(p.cu_q + r.b + 1);
  r.own_len = __ldg(p.own.lens + r.b);
  r.prefix = p.P ? prefix_of(p, r.b) : -1;
  r.prefix_len = r.prefix >= 0 ? __ldg(p.prefix.lens + r.prefix) : 0;
  if (c0 > tok || c1 <= tok || c1 > p.total_q) {
    report(p.status, ATTN_DEV_BAD_CU);
    return false;
  }
  if (r.own_len < 0 || r.own_len > (static_cast<int64_t>(p.own.width) << p.page_log2) ||
      r.prefix_len < 0 ||
      (r.prefix >= 0 && r.prefix_len > (static_cast<int64_t>(p.prefix.width) << p.page_log2))) {
    report(p.status, ATTN_DEV_BAD_CACHE);
    return false;
  }
  r.g = h / p.R;
  r.qpos = p.q_pos ? __ldg(p.q_pos + tok) : r.prefix_len + r.own_len - (c1 - c0) + (tok - c0);
  return true;
}

template <bool BF16>
__device__ __forceinline__ void load_lane(const uint16_t* row, int d, float (&x)[kPerLane]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) x[i] = i * 32 + lane < d ? to_float<BF16>(row[i * 32 + lane]) : 0.f;
}

__device__ __forceinline__ float dot(const float (&a)[kPerLane], const float (&b)[kPerLane]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// The logit of an admissible (query, key) pair, or -inf.
__device__ __forceinline__ float logit(const CacheParams& p, float qk, int qpos, int kpos, float slope) {
  if (kpos < pos_lo(p, qpos) || kpos > pos_hi(p, qpos)) return -INFINITY;
  float x = qk * p.sigma;
  if (p.softcap > 0.f) x = p.softcap * tanhf(x / p.softcap);
  return x - slope * static_cast<float>(abs(qpos - kpos));
}

__device__ __forceinline__ int key_position(const Table& t, int row, int g, int j, int base) {
  return t.pos ? __ldg(t.pos + row * t.pos_rs + g * t.pos_hs + j) : base + j;
}

// One warp per (segment, K/V head, slot): gridDim.y = segment * Hkv + head.
template <bool BF16>
__global__ void __launch_bounds__(kThreadsA) weights_rows_kernel(const __grid_constant__ CacheParams p) {
  const int seg = blockIdx.y / p.Hkv, g = blockIdx.y - seg * p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = seg >= p.P, row = part ? seg - p.P : seg;
  if (!p.w_out[part]) return;
  const Table& t = part ? p.own : p.prefix;
  const int len = __ldg(t.lens + row);
  if (len < 0 || len > (static_cast<int64_t>(t.width) << p.page_log2)) {
    report(p.status, ATTN_DEV_BAD_CACHE);
    return;
  }
  const int b0 = part ? row : __ldg(p.cu_prefix + row), b1 = part ? row + 1 : __ldg(p.cu_prefix + row + 1);
  const int t0 = __ldg(p.cu_q + b0), t1 = __ldg(p.cu_q + b1);
  if (t0 < 0 || t1 < t0 || t1 > p.total_q) {
    report(p.status, ATTN_DEV_BAD_CU);
    return;
  }
  for (int j = blockIdx.x * 4 + warp; j < len; j += gridDim.x * 4) {
    const int64_t ko = slot_row(p, p.k, t.pages + row * t.rs, j);
    float k[kPerLane] = {}, w = 0.f;
    if (ko >= 0)
      load_lane<BF16>(static_cast<const uint16_t*>(p.k.base) + ko + g * p.k.head, p.d, k);
    else if (lane == 0)
      report(p.status, ATTN_DEV_BAD_CACHE);
    for (int tok = t0; tok < t1; ++tok) {
      Row r;
      if (!find_row(p, tok, g * p.R, r)) continue;
      const int kpos = key_position(t, row, g, j, part ? r.prefix_len : 0);
      for (int i = 0; i < p.R; ++i) {
        const int h = g * p.R + i;
        float q[kPerLane];
        load_lane<BF16>(static_cast<const uint16_t*>(p.q) + tok * p.q_ts + h * p.q_hs, p.d, q);
        const float z = logit(p, dot(q, k), r.qpos, kpos,
                              p.slopes ? __ldg(p.slopes + r.b * p.slopes_bs + h) : 0.f);
        const float e = __ldg(p.lse + static_cast<int64_t>(tok) * p.Hq + h);
        if (z != -INFINITY && e != -INFINITY) w += expf(z - e);
      }
    }
    if (lane == 0) {
      const float in = p.w_in[part] ? p.w_in[part][row * p.wi_rs[part] + g * p.wi_hs[part] + j] : 0.f;
      p.w_out[part][row * p.wo_rs[part] + g * p.wo_hs[part] + j] = in + w;
    }
  }
}

}  // namespace

size_t weights_workspace(int, int, int, int64_t, int64_t) { return 256; }

cudaError_t launch_weights(const CacheParams& p, cudaStream_t s) {
  const dim3 grid(256, static_cast<unsigned>((p.P + p.B) * p.Hkv));
  (p.dtype == 1 ? weights_rows_kernel<true> : weights_rows_kernel<false>)<<<grid, kThreadsA, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace kv
}  // namespace attn
