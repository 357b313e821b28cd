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
// would leave the angle 0.06 wrong.  Its top 32 bits, as a signed fraction in
// [-pi, pi), go to the fast sine and cosine, good to 2^-21.2 there: 2^-9 of a
// rounding of the 16-bit results.
//
// Bound by memory: every row is read and written once.  A block takes a few
// tokens, so that one pair's sine serves all heads.  16000 tokens of 96 + 1 heads
// of 160 features take 174 us (5.7 TB/s, 85 % of a copy's rate); 17000 tokens of
// one head appended 14 us, where the lookups and sines before the copies count.
#include <type_traits>

#include "../../include/attn_varlen.h"
#include "rowfrag.cuh"

namespace attn {
namespace kv {
namespace {

constexpr int kThreadsR = 256;
constexpr int kItemsR = 4096;   // 16-byte units (pairs of them for halves) a block turns, at most
constexpr int kItemsA = 2048;   // ... and appends
static_assert(kMaxTokensR <= kThreadsR, "a thread looks one token up");

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

// Item u of a row: loaded first, turned and stored later, so that a thread has
// the loads of several items in flight.  Rows are read and written once:
// streaming accesses, which leave the caches to others.
template <bool BF16>
struct VecItem {
  uint4 a, b;
  __device__ __forceinline__ void load(const uint16_t* x, int u, int turning, int pairs,
                                       bool interleaved) {
    const int f = u < turning ? u * 8 : 2 * pairs + (u - turning) * 8;
    a = __ldcs(reinterpret_cast<const uint4*>(x + f));
    if (u < turning && !interleaved) b = __ldcs(reinterpret_cast<const uint4*>(x + pairs + f));
  }
  __device__ __forceinline__ void store(uint16_t* y, int u, int turning, int pairs,
                                        bool interleaved, const float2* cs) {
    if (u >= turning) {
      __stcs(reinterpret_cast<uint4*>(y + 2 * pairs + (u - turning) * 8), a);
      return;
    }
    float va[8], vb[8];
    unpack8<BF16>(a, va);
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) turn2<BF16>(cs[u * 4 + i], va[2 * i], va[2 * i + 1]);
    } else {
      unpack8<BF16>(b, vb);
#pragma unroll
      for (int i = 0; i < 8; ++i) turn2<BF16>(cs[u * 8 + i], va[i], vb[i]);
      __stcs(reinterpret_cast<uint4*>(y + pairs + u * 8), pack8<BF16>(vb));
    }
    __stcs(reinterpret_cast<uint4*>(y + u * 8), pack8<BF16>(va));
  }
};
template <bool BF16>
struct ScalarItem {
  uint16_t a, b;
  __device__ __forceinline__ void load(const uint16_t* x, int u, int turning, int pairs,
                                       bool interleaved) {
    if (u >= turning) {
      a = x[2 * pairs + u - turning];
    } else {
      a = x[interleaved ? 2 * u : u];
      b = x[interleaved ? 2 * u + 1 : u + pairs];
    }
  }
  __device__ __forceinline__ void store(uint16_t* y, int u, int turning, int pairs,
                                        bool interleaved, const float2* cs) {
    if (u >= turning) {
      y[2 * pairs + u - turning] = a;
      return;
    }
    float va = to_float<BF16>(a), vb = to_float<BF16>(b);
    turn2<BF16>(cs[u], va, vb);
    y[interleaved ? 2 * u : u] = from_float<BF16>(va);
    y[interleaved ? 2 * u + 1 : u + pairs] = from_float<BF16>(vb);
  }
};
template <bool BF16, bool VEC>
using Item = typename std::conditional<VEC, VecItem<BF16>, ScalarItem<BF16>>::type;

// gridDim.x: runs of `ntok` tokens; gridDim.y: runs of `heads` heads over
// both tensors.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreadsR)
    rotary_kernel(const __grid_constant__ RotaryParams p, int ntok, int heads) {
  __shared__ Turns turns;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * ntok;
  ntok = static_cast<int>(min(static_cast<int64_t>(ntok), p.T - tok0));
  const int h0 = blockIdx.y * heads;
  const int nh = min(heads, p.t[0].H + p.t[1].H - h0);
  fill_turns(p.r, tok0, ntok, turns);
  __syncthreads();
  const RowItems it = row_items<VEC>(p.d, p.r.pairs, p.r.interleaved);
  const float inv_total = 1.f / it.total, inv_nh = 1.f / nh;
  const int all = ntok * nh * it.total;
  constexpr int kBatch = 4;
  for (int u0 = threadIdx.x; u0 < all; u0 += kThreadsR * kBatch) {
    Item<BF16, VEC> item[kBatch];
    uint16_t* out[kBatch];
    int at[kBatch], tok[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int u = u0 + k * kThreadsR;
      if (u < all) {
        const int row = quotient(u, inv_total), t = quotient(row, inv_nh);
        const int h = h0 + row - t * nh;
        const RotaryTensor& x = p.t[h >= p.t[0].H];
        const int64_t hh = h >= p.t[0].H ? h - p.t[0].H : h;
        tok[k] = t;
        at[k] = u - row * it.total;
        out[k] = static_cast<uint16_t*>(x.out) + (tok0 + t) * x.ots + hh * x.ohs;
        item[k].load(static_cast<const uint16_t*>(x.x) + (tok0 + t) * x.ts + hh * x.hs, at[k],
                     it.turning, p.r.pairs, p.r.interleaved);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (u0 + k * kThreadsR < all)
        item[k].store(out[k], at[k], it.turning, p.r.pairs, p.r.interleaved, turns.cs[tok[k]]);
  }
}

// New tokens into their pages: K rows turned (when the call has rotary
// positions), V rows copied.  Every block checks the whole of cu_new (along
// with its lookups): a call whose runs of tokens contradict one another writes
// nothing.  A sequence that does not fit its table is left out, and so is a token
// whose page is out of the pool.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreadsR)
    append_kernel(const __grid_constant__ AppendParams p, int ntok) {
  __shared__ Turns turns;
  __shared__ int64_t row_k[kMaxTokensR], row_v[kMaxTokensR];  // first element, or -1
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * ntok;
  ntok = static_cast<int>(min(static_cast<int64_t>(ntok), p.T - tok0));
  int bad = 0;
  for (int b = threadIdx.x; b < p.B; b += kThreadsR) {
    const int c0 = __ldg(p.cu_new + b), c1 = __ldg(p.cu_new + b + 1);
    bad |= c0 < 0 || c1 < c0 || c1 > p.T || (b == 0 && c0 != 0);
  }
  // kMaxTokensR <= kThreadsR: a token is one thread's
  int seq = -1, slot = 0;  // of this thread's token, if it is taken
  if (static_cast<int>(threadIdx.x) < ntok) {
    const int t = threadIdx.x, tok = static_cast<int>(tok0) + t;
    int64_t rk = -1, rv = -1;
    if (tok < __ldg(p.cu_new + p.B)) {  // tokens behind the last sequence are left out
      const int b = seq_of(p.cu_new, 0, p.B, tok);
      const int c0 = __ldg(p.cu_new + b), c1 = __ldg(p.cu_new + b + 1);
      int page = -1;
      // (cu_new may be anything still: only a token of its own run is looked up)
      const int at = c0 >= 0 && c0 <= tok && tok < c1 ? append_at(p, b, c1 - c0) : -1;
      if (at >= 0) {
        slot = at + tok - c0;
        page = __ldg(p.table + b * p.table_rs + (slot >> p.page_log2));
      }
      if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) {
        const int in = slot & (p.page_size - 1);
        rk = page * p.k.page + in * p.k.slot;
        rv = page * p.v.page + in * p.v.slot;
        seq = b;
      } else {
        seq = -2;
      }
    }
    row_k[t] = rk;
    row_v[t] = rv;
  }
  // few tokens: the turns along with the lookups; many: after the V rows
  const bool early = p.r.inv_freq && ntok * p.r.pairs <= kThreadsR;
  if (early) fill_turns(p.r, tok0, ntok, turns);
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0) {
    if (bad && threadIdx.x == 0) report(p.status, ATTN_DEV_BAD_CU);
    for (int b = threadIdx.x; b < p.B && (p.lens_out || !bad); b += kThreadsR) {
      const int n = bad ? 0 : __ldg(p.cu_new + b + 1) - __ldg(p.cu_new + b);
      const int at = append_at(p, b, n);
      if (!bad && at < 0) report(p.status, ATTN_DEV_BAD_CACHE);
      if (p.lens_out) p.lens_out[b] = at < 0 ? __ldg(p.lens + b) : at + n;
    }
  }
  if (bad) return;
  if (seq >= 0) {
    const int tok = static_cast<int>(tok0) + threadIdx.x;
    for (int g = 0; g < p.Hkv; ++g) {
      if (p.key_pos)
        p.key_pos[seq * p.kp_rs + g * p.kp_hs + slot] = p.r.positions ? __ldg(p.r.positions + tok) : slot;
      if (p.scores) p.scores[seq * p.sc_rs + g * p.sc_hs + slot] = 0.f;
    }
  } else if (seq == -2) {
    report(p.status, ATTN_DEV_BAD_CACHE);
  }
  // V rows and K rows: each thread's loads of four (two) units go out together.
  // Of few tokens, the upper half of the threads takes V and the lower K.
  const int step = early ? kThreadsR / 2 : kThreadsR;
  const bool upper = static_cast<int>(threadIdx.x) >= step;
  if (!early || upper) {
    const int units = p.d / 8, per = p.Hkv * units, all = ntok * per;
    const float inv_per = 1.f / per, inv_units = 1.f / units;
    for (int u0 = threadIdx.x - (upper ? step : 0); u0 < all; u0 += 4 * step) {
      uint4 v[4];
      uint16_t* out[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int u = u0 + k * step, t = quotient(u, inv_per), w = u - t * per;
        const int64_t g = quotient(w, inv_units);
        const int f = (w - static_cast<int>(g) * units) * 8;
        out[k] = nullptr;
        if (u < all && row_v[t] >= 0) {
          out[k] = static_cast<uint16_t*>(const_cast<void*>(p.v.base)) + row_v[t] + g * p.v.head + f;
          v[k] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.vx) +
                                                       (tok0 + t) * p.v_ts + g * p.v_hs + f));
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (out[k]) *reinterpret_cast<uint4*>(out[k]) = v[k];
    }
  }
  if (p.r.inv_freq && !early) {
    fill_turns(p.r, tok0, ntok, turns);
    __syncthreads();
  }
  if (early && upper) return;
  const int pairs = p.r.inv_freq ? p.r.pairs : 0;
  const RowItems it = row_items<VEC>(p.d, pairs, p.r.interleaved);
  const int per = p.Hkv * it.total, all = ntok * per;
  const float inv_per = 1.f / per, inv_total = 1.f / it.total;
  for (int u0 = threadIdx.x; u0 < all; u0 += 2 * step) {
    Item<BF16, VEC> item[2];
    uint16_t* out[2];
    int at[2], tok[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int u = u0 + k * step, t = quotient(u, inv_per), w = u - t * per;
      const int64_t g = quotient(w, inv_total);
      out[k] = nullptr;
      tok[k] = t;
      at[k] = w - static_cast<int>(g) * it.total;
      if (u < all && row_k[t] >= 0) {
        out[k] = static_cast<uint16_t*>(const_cast<void*>(p.k.base)) + row_k[t] + g * p.k.head;
        item[k].load(static_cast<const uint16_t*>(p.kx) + (tok0 + t) * p.k_ts + g * p.k_hs, at[k],
                     it.turning, pairs, p.r.interleaved);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (out[k]) item[k].store(out[k], at[k], it.turning, pairs, p.r.interleaved, turns.cs[tok[k]]);
  }
}

// Tokens of a block: as many as `most` items hold, but enough blocks for four
// rounds of the SMs (a single round of few blocks is a chain of latencies).
int block_tokens(int64_t T, int64_t items_per_token, int most) {
  int64_t n = most / items_per_token;
  const int64_t spread = T / (4 * 152);
  n = n < spread ? n : spread;
  return static_cast<int>(n < 1 ? 1 : (n > kMaxTokensR ? kMaxTokensR : n));
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t s) {
  const bool vec = vector_pairs(p.r.pairs, p.r.interleaved);
  const int H = p.t[0].H + p.t[1].H;
  const RowItems it = vec ? row_items<true>(p.d, p.r.pairs, p.r.interleaved)
                          : row_items<false>(p.d, p.r.pairs, p.r.interleaved);
  const int ntok = block_tokens(p.T, static_cast<int64_t>(H) * it.total, kItemsR);
  int heads = H;
  // few tokens of many heads: the heads over several blocks
  if (ntok == 1 && H * it.total > 1024) heads = (512 + it.total - 1) / it.total;
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
  const int ntok = block_tokens(p.T, per, kItemsA);
  const unsigned grid = p.T > 0 ? static_cast<unsigned>((p.T + ntok - 1) / ntok) : 1u;
  auto k = p.dtype == 1 ? (vec ? append_kernel<true, true> : append_kernel<true, false>)
                        : (vec ? append_kernel<false, true> : append_kernel<false, false>);
  k<<<grid, kThreadsR, 0, s>>>(p, ntok);
  return cudaGetLastError();
}

}  // namespace kv
}  // namespace attn
