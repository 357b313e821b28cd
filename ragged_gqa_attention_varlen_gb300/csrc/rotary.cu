// rotary.cu -- rotary positions with several axes, on packed q and k and on
// new K rows on their way into the paged cache.
//
// Pair i of a row is features (i, i + n) (halves) or (2i, 2i + 1)
// (interleaved) of the first 2n features; it is turned by the angle
// t = positions[axis(i)][token] * inv_freq[i]:
//   a' = a cos t - b sin t,   b' = b cos t + a sin t.
// The map is orthogonal, so its vector-Jacobian product is the turn by -t.
//
// The angle is reduced exactly: inv_freq / 2 pi (in 64 bits) is taken modulo
// one turn and scaled to a 64-bit fraction F, and position * F modulo 2^64 is
// the fraction of a turn with an error below |position| * 2^-53 / 2 pi * |t /
// position| (the rounding of inv_freq / 2 pi).  In fp32, a position of 10^6
// would leave the angle 0.06 wrong.  Its top 32 bits, as a signed fraction,
// go to sincospif.
//
// Bound by memory: every row is read and written once.  A block takes a few
// tokens, so that one pair's sine serves all heads.
#include "../../include/attn_varlen.h"
#include "cache.cuh"

namespace attn {
namespace kv {
namespace {

constexpr int kThreadsR = 256;
constexpr int kItemsR = 1024;      // 16-byte units (pairs of them for halves) a block takes, about
constexpr int kMaxTokensR = 32;
constexpr int kMaxPairs = kHeadDim / 2;

// Fraction of a turn per position, as a 64-bit binary fraction.
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
  const double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  const double f = t - floor(t);                       // [0, 1]
  return f < 1.0 ? static_cast<uint64_t>(f * 18446744073709551616.0) : 0ull;
}

// cos and sin of pairs [0, pairs) for ntok tokens from tok0 on.
__device__ __forceinline__ void fill_turns(const RotaryTable& r, int64_t tok0, int ntok,
                                           float2 (*cs)[kMaxPairs]) {
  for (int u = threadIdx.x; u < ntok * r.pairs; u += blockDim.x) {
    const int t = u / r.pairs, i = u - t * r.pairs;
    int ax = r.pair_axis ? __ldg(r.pair_axis + i) : 0;
    ax = min(max(ax, 0), r.axes - 1);
    const int64_t pos = __ldg(r.positions + ax * r.axis_stride + tok0 + t);
    const uint64_t turns = static_cast<uint64_t>(pos) * turn_fraction(__ldg(r.inv_freq + i));
    // the top 32 bits as a signed fraction of a turn, in half turns
    const float h = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
    float sn, cn;
    sincospif(h, &sn, &cn);
    cs[t][i] = make_float2(cn, r.inverse ? -sn : sn);
  }
}

template <bool BF16>
__device__ __forceinline__ void turn2(float2 c, float& a, float& b) {
  const float x = a;
  a = x * c.x - b * c.y;
  b = b * c.x + x * c.y;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t f = Pack<BF16>::unpack(w[i]);
    v[2 * i] = f2_lo(f);
    v[2 * i + 1] = f2_hi(f);
  }
}

// 16-byte units of a row: with VEC, `rot_units` items that turn (a pair of
// units for halves, one for interleaved) and then units that are copied.
// Without (pairs not a multiple of 8, or 4 interleaved) an item is one pair
// or one copied feature.
struct RowItems {
  int turning, total;
};
template <bool VEC>
__host__ __device__ __forceinline__ RowItems row_items(int d, int pairs, bool interleaved) {
  RowItems it;
  it.turning = VEC ? (interleaved ? pairs / 4 : pairs / 8) : pairs;
  it.total = it.turning + (VEC ? (d - 2 * pairs) / 8 : d - 2 * pairs);
  return it;
}

// Item u of one row.
template <bool BF16, bool VEC>
__device__ __forceinline__ void row_item(const uint16_t* x, uint16_t* y, int u, int turning,
                                         int pairs, bool interleaved, const float2* cs) {
  if (VEC) {
    if (u >= turning) {
      const int f = 2 * pairs + (u - turning) * 8;
      *reinterpret_cast<uint4*>(y + f) = *reinterpret_cast<const uint4*>(x + f);
    } else if (interleaved) {
      float v[8];
      unpack8<BF16>(*reinterpret_cast<const uint4*>(x + u * 8), v);
#pragma unroll
      for (int i = 0; i < 4; ++i) turn2<BF16>(cs[u * 4 + i], v[2 * i], v[2 * i + 1]);
      *reinterpret_cast<uint4*>(y + u * 8) = pack8<BF16>(v);
    } else {
      float a[8], b[8];
      const uint4 ua = *reinterpret_cast<const uint4*>(x + u * 8);
      const uint4 ub = *reinterpret_cast<const uint4*>(x + pairs + u * 8);
      unpack8<BF16>(ua, a);
      unpack8<BF16>(ub, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) turn2<BF16>(cs[u * 8 + i], a[i], b[i]);
      *reinterpret_cast<uint4*>(y + u * 8) = pack8<BF16>(a);
      *reinterpret_cast<uint4*>(y + pairs + u * 8) = pack8<BF16>(b);
    }
  } else {
    if (u >= turning) {
      y[2 * pairs + u - turning] = x[2 * pairs + u - turning];
    } else {
      const int fa = interleaved ? 2 * u : u, fb = interleaved ? 2 * u + 1 : u + pairs;
      float a = to_float<BF16>(x[fa]), b = to_float<BF16>(x[fb]);
      turn2<BF16>(cs[u], a, b);
      y[fa] = from_float<BF16>(a);
      y[fb] = from_float<BF16>(b);
    }
  }
}

// gridDim.x: runs of `ntok` tokens; gridDim.y: runs of `heads` heads over
// both tensors.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreadsR)
    rotary_kernel(const __grid_constant__ RotaryParams p, int ntok, int heads) {
  __shared__ float2 cs[kMaxTokensR][kMaxPairs];
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * ntok;
  ntok = static_cast<int>(min(static_cast<int64_t>(ntok), p.T - tok0));
  const int h0 = blockIdx.y * heads;
  const int nh = min(heads, p.t[0].H + p.t[1].H - h0);
  fill_turns(p.r, tok0, ntok, cs);
  __syncthreads();
  const RowItems it = row_items<VEC>(p.d, p.r.pairs, p.r.interleaved);
  for (int u = threadIdx.x; u < ntok * nh * it.total; u += kThreadsR) {
    const int row = u / it.total, t = row / nh;
    const int h = h0 + row - t * nh;
    const RotaryTensor& x = p.t[h >= p.t[0].H];
    const int hh = h >= p.t[0].H ? h - p.t[0].H : h;
    row_item<BF16, VEC>(static_cast<const uint16_t*>(x.x) + (tok0 + t) * x.ts + hh * x.hs,
                        static_cast<uint16_t*>(x.out) + (tok0 + t) * x.ots + hh * x.ohs,
                        u - row * it.total, it.turning, p.r.pairs, p.r.interleaved, cs[t]);
  }
}

// New tokens into their pages: K rows turned (when the call has rotary
// positions), V rows copied.  A token whose slot has no valid page is skipped
// and reported.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreadsR)
    append_kernel(const __grid_constant__ AppendParams p, int ntok) {
  __shared__ float2 cs[kMaxTokensR][kMaxPairs];
  __shared__ int64_t row_k[kMaxTokensR], row_v[kMaxTokensR];  // first element, or -1
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * ntok;
  ntok = static_cast<int>(min(static_cast<int64_t>(ntok), p.T - tok0));
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < p.B; b += kThreadsR) {
      const int c0 = __ldg(p.cu_new + b), c1 = __ldg(p.cu_new + b + 1);
      if (c0 < 0 || c1 < c0 || c1 > p.T || (b == 0 && c0 != 0)) report(p.status, ATTN_DEV_BAD_CU);
      if (p.lens_out) p.lens_out[b] = __ldg(p.lens + b) + c1 - c0;
    }
  }
  for (int t = threadIdx.x; t < ntok; t += kThreadsR) {
    const int tok = static_cast<int>(tok0) + t;
    int64_t rk = -1, rv = -1;
    if (tok < __ldg(p.cu_new + p.B)) {  // tokens behind the last sequence are left out
      const int b = seq_of(p.cu_new, 0, p.B, tok);
      const int64_t slot = static_cast<int64_t>(__ldg(p.lens + b)) + tok - __ldg(p.cu_new + b);
      int page = -1;
      if (slot >= 0 && (slot >> p.page_log2) < p.width)
        page = __ldg(p.table + b * p.table_rs + (slot >> p.page_log2));
      if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) {
        const int in = static_cast<int>(slot) & (p.page_size - 1);
        rk = page * p.k.page + in * p.k.slot;
        rv = page * p.v.page + in * p.v.slot;
        for (int g = 0; g < p.Hkv; ++g) {
          if (p.key_pos)
            p.key_pos[b * p.kp_rs + g * p.kp_hs + slot] =
                p.r.positions ? __ldg(p.r.positions + tok) : static_cast<int32_t>(slot);
          if (p.scores) p.scores[b * p.sc_rs + g * p.sc_hs + slot] = 0.f;
        }
      } else {
        report(p.status, ATTN_DEV_BAD_CACHE);
      }
    }
    row_k[t] = rk;
    row_v[t] = rv;
  }
  if (p.r.inv_freq) fill_turns(p.r, tok0, ntok, cs);
  __syncthreads();
  const int pairs = p.r.inv_freq ? p.r.pairs : 0;
  const RowItems it = row_items<VEC>(p.d, pairs, p.r.interleaved);
  const RowItems iv = row_items<true>(p.d, 0, false);
  const int per = p.Hkv * (it.total + iv.total);
  for (int u = threadIdx.x; u < ntok * per; u += kThreadsR) {
    const int t = u / per;
    int w = u - t * per;
    if (row_k[t] < 0) continue;
    if (w < p.Hkv * it.total) {
      const int g = w / it.total;
      row_item<BF16, VEC>(
          static_cast<const uint16_t*>(p.kx) + (tok0 + t) * p.k_ts + g * p.k_hs,
          static_cast<uint16_t*>(const_cast<void*>(p.k.base)) + row_k[t] + g * p.k.head,
          w - g * it.total, it.turning, pairs, p.r.interleaved, cs[t]);
    } else {
      w -= p.Hkv * it.total;
      const int g = w / iv.total;
      row_item<BF16, true>(
          static_cast<const uint16_t*>(p.vx) + (tok0 + t) * p.v_ts + g * p.v_hs,
          static_cast<uint16_t*>(const_cast<void*>(p.v.base)) + row_v[t] + g * p.v.head,
          w - g * iv.total, 0, 0, false, nullptr);
    }
  }
}

bool vector_pairs(int pairs, bool interleaved) { return pairs % (interleaved ? 4 : 8) == 0; }

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t s) {
  const bool vec = vector_pairs(p.r.pairs, p.r.interleaved);
  const int H = p.t[0].H + p.t[1].H;
  const RowItems it = vec ? row_items<true>(p.d, p.r.pairs, p.r.interleaved)
                          : row_items<false>(p.d, p.r.pairs, p.r.interleaved);
  int ntok = kItemsR / (H * it.total);
  ntok = ntok < 1 ? 1 : (ntok > kMaxTokensR ? kMaxTokensR : ntok);
  int heads = H;
  if (ntok == 1 && H * it.total > 2 * kItemsR) heads = (kItemsR + it.total - 1) / it.total;
  const dim3 grid(static_cast<unsigned>((p.T + ntok - 1) / ntok), (H + heads - 1) / heads);
  auto k = p.dtype == 1 ? (vec ? rotary_kernel<true, true> : rotary_kernel<true, false>)
                        : (vec ? rotary_kernel<false, true> : rotary_kernel<false, false>);
  k<<<grid, kThreadsR, 0, s>>>(p, ntok, heads);
  return cudaGetLastError();
}

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
  const int pairs = p.r.inv_freq ? p.r.pairs : 0;
  const bool vec = vector_pairs(pairs, p.r.interleaved);
  const int per = p.Hkv * 2 * (p.d / 8);
  int ntok = kItemsR / per;
  ntok = ntok < 1 ? 1 : (ntok > kMaxTokensR ? kMaxTokensR : ntok);
  const unsigned grid = p.T > 0 ? static_cast<unsigned>((p.T + ntok - 1) / ntok) : 1u;
  auto k = p.dtype == 1 ? (vec ? append_kernel<true, true> : append_kernel<true, false>)
                        : (vec ? append_kernel<false, true> : append_kernel<false, false>);
  k<<<grid, kThreadsR, 0, s>>>(p, ntok);
  return cudaGetLastError();
}

}  // namespace kv
}  // namespace attn
