// rotary.cuh -- what the kernels that turn rows by rotary positions share: the
// turns of a block's tokens and the arithmetic of a pair (rotary.cu has the
// definition).
#pragma once
#include "cache.cuh"

namespace attn {
namespace kv {

constexpr int kMaxTokensR = 32;  // tokens whose turns a block holds
constexpr int kMaxPairs = kHeadDim / 2;

// Fraction of a turn per position, as a 64-bit binary fraction.
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
  const double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  const double f = t - floor(t);                       // [0, 1]
  return f < 1.0 ? static_cast<uint64_t>(f * 18446744073709551616.0) : 0ull;
}

// x / n for 0 <= x < 2^20, as in head_div (n is fixed for a launch).
__device__ __forceinline__ int quotient(int x, float inv_n) {
  return static_cast<int>((static_cast<float>(x) + 0.5f) * inv_n);
}

// (cos, sin) of `pos` times a turn fraction: its top 32 bits as a signed
// fraction of a turn, times 2 pi.
__device__ __forceinline__ float2 turn_of(int64_t pos, uint64_t per_pos) {
  const uint64_t turns = static_cast<uint64_t>(pos) * per_pos;
  const float h = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 1.4629180792671596e-9f;
  float sn, cn;
  __sincosf(h, &sn, &cn);
  return make_float2(cn, sn);
}

struct Turns {
  alignas(16) float2 cs[kMaxTokensR][kMaxPairs];  // cos, sin
  uint64_t per_pos[kMaxPairs];        // turn_fraction of each pair
  int64_t row[kMaxPairs];             // its axis' row of the positions
};

// Where a token's row of `cs` holds pair i when a lane reads its eight pairs as
// four 16-byte units: unit c of lane l at c ^ (l / 2) % 4 of the lane's four, so
// the eight lanes of a shared memory pass meet every bank once (in order they
// met two groups of four banks, and a load took four times its passes).
__device__ __forceinline__ int spread_pair(int i) { return i ^ (((i >> 4) & 3) << 1); }

// cos and sin of every pair for ntok tokens from tok0 on, SPREAD: at spread_pair
// (whole block; the caller synchronises).  The 64-bit arithmetic is done once per pair and
// block: it runs at 1/50 of the fp32 rate here, and once per (pair, token) it
// took most of the time of calls with one head.
template <bool SPREAD = false>
__device__ __forceinline__ void fill_turns(const RotaryTable& r, int64_t tok0, int ntok, Turns& s) {
  const bool once = ntok * r.pairs <= static_cast<int>(blockDim.x);  // no pair is met twice
  for (int i = threadIdx.x; i < r.pairs && !once; i += blockDim.x) {
    int ax = r.pair_axis ? __ldg(r.pair_axis + i) : 0;
    ax = min(max(ax, 0), r.axes - 1);
    s.per_pos[i] = turn_fraction(__ldg(r.inv_freq + i));
    s.row[i] = ax * r.axis_stride;
  }
  const float inv_pairs = 1.f / r.pairs;
  auto turn = [&](int t, int i, int64_t pos, uint64_t per_pos) {
    const float2 c = turn_of(pos, per_pos);
    s.cs[t][SPREAD ? spread_pair(i) : i] = make_float2(c.x, r.inverse ? -c.y : c.y);
  };
  const int all = ntok * r.pairs;
  if (once) {
    const int u = threadIdx.x, t = quotient(u, inv_pairs), i = u - t * r.pairs;
    if (u < all) {
      const int ax = r.pair_axis ? __ldg(r.pair_axis + i) : 0;
      const int64_t row = min(max(ax, 0), r.axes - 1) * r.axis_stride;
      turn(t, i, __ldg(r.positions + row + tok0 + t), turn_fraction(__ldg(r.inv_freq + i)));
    }
    return;
  }
  __syncthreads();
  for (int u0 = threadIdx.x; u0 < all; u0 += 4 * blockDim.x) {
    int pos[4];  // four positions in flight
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = u0 + k * blockDim.x, t = quotient(u, inv_pairs);
      if (u < all) pos[k] = __ldg(r.positions + s.row[u - t * r.pairs] + tok0 + t);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = u0 + k * blockDim.x, t = quotient(u, inv_pairs), i = u - t * r.pairs;
      if (u < all) turn(t, i, pos[k], s.per_pos[i]);
    }
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

// The slots that sequence b's tokens take start here, or -1 when its length is
// negative or they do not all fit its table: none of them is taken then.
__device__ __forceinline__ int append_at(const AppendParams& p, int b, int n) {
  const int len = __ldg(p.lens + b);
  const int64_t slots = static_cast<int64_t>(p.width) << p.page_log2;
  return len >= 0 && static_cast<int64_t>(len) + n <= slots ? len : -1;
}

}  // namespace kv
}  // namespace attn
