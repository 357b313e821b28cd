// rowfrag.cuh -- a row of d features held by a few lanes, for kernels that need
// a whole row at once (its mean square, its largest value) and turn it.
//
// The row is cut into d / 16 items of two 16-byte units; lane j of the row's 4, 8
// or 10 lanes holds item j (two items a lane took twice the registers, and so
// half the loads in flight).  When the pairs allow it (VEC: pairs a multiple
// of 8 in halves, of 4 interleaved) an item is made so that a turn stays inside
// it: units i and i + pairs / 8 in halves, two neighbouring units interleaved.
// Other pair counts go through a row of shared memory.
#pragma once
#include "rotary.cuh"

namespace attn {
namespace kv {

template <int D>
struct RowShape {
  static constexpr int kItems = D / 16;
  static constexpr int kLanes = kItems;          // lanes of a row: an item each
  static constexpr int kRowsWarp = 32 / kLanes;  // rows of a warp (160: two lanes idle)
};

// First features of the two units of item i.
struct Units {
  int a, b;
};
template <bool VEC>
__device__ __forceinline__ Units item_units(int i, int pairs, bool interleaved) {
  Units u;
  const int turning = VEC && !interleaved ? pairs / 8 : 0;
  if (i < turning) {
    u.a = i * 8;
    u.b = pairs + i * 8;
  } else {
    u.a = i * 16;  // (2 * turning + 2 (i - turning) units)
    u.b = u.a + 8;
  }
  return u;
}

// A sum or maximum over the lanes of a row, the same bits in each of them.
template <int D, class Op>
__device__ __forceinline__ float row_all(float v, Op op) {
  constexpr int G = RowShape<D>::kLanes;
  v = op(v, __shfl_xor_sync(0xffffffffu, v, 1));
  if (G == 10) {  // five pairs
    const int lane = threadIdx.x & 31, base = lane - lane % G;
    float s = __shfl_sync(0xffffffffu, v, base);
#pragma unroll
    for (int j = 2; j < G; j += 2) s = op(s, __shfl_sync(0xffffffffu, v, (base + j) & 31));
    return s;
  }
  v = op(v, __shfl_xor_sync(0xffffffffu, v, 2));
  return G == 8 ? op(v, __shfl_xor_sync(0xffffffffu, v, 4)) : v;
}
template <int D>
__device__ __forceinline__ float row_sum(float v) {
  return row_all<D>(v, [](float a, float b) { return a + b; });
}
template <int D>
__device__ __forceinline__ float row_max(float v) {
  return row_all<D>(v, [](float a, float b) { return fmaxf(a, b); });
}

// Turn the two units of item i; turn(pair, a, b) gives (cos, sin) of a pair, which
// is an even one, and of the next.
template <class Turn>
__device__ __forceinline__ void turn_item(float (&a)[8], float (&b)[8], int i, int pairs,
                                          bool interleaved, Turn turn) {
  float2 c0, c1;
  if (!interleaved) {
    if (i < pairs / 8) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        turn(i * 8 + e, c0, c1);
        turn2<true>(c0, a[e], b[e]);
        turn2<true>(c1, a[e + 1], b[e + 1]);
      }
    }
    return;
  }
  if (2 * i < pairs / 4) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      turn(i * 8 + e, c0, c1);
      turn2<true>(c0, a[2 * e], a[2 * e + 1]);
      turn2<true>(c1, a[2 * e + 2], a[2 * e + 3]);
    }
  }
  if (2 * i + 1 < pairs / 4) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      turn(i * 8 + 4 + e, c0, c1);
      turn2<true>(c0, b[2 * e], b[2 * e + 1]);
      turn2<true>(c1, b[2 * e + 2], b[2 * e + 3]);
    }
  }
}

// The same for any number of pairs: `v` holds the lane's two units of the row
// (neighbouring ones), `row` is the row's buffer in shared memory.
// Warp-collective.
template <class Turn>
__device__ __forceinline__ void turn_row(float (&v)[2][8], float* row, int j, int pairs,
                                         bool interleaved, Turn turn) {
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) row[j * 16 + u * 8 + e] = v[u][e];
  __syncwarp();
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int f = j * 16 + u * 8 + e;
      if (f >= 2 * pairs) continue;
      const bool second = interleaved ? f & 1 : f >= pairs;
      const int pair = interleaved ? f >> 1 : (second ? f - pairs : f);
      const float other = row[interleaved ? f ^ 1 : (second ? f - pairs : f + pairs)];
      const float2 c = turn(pair);
      v[u][e] = second ? v[u][e] * c.x + other * c.y : v[u][e] * c.x - other * c.y;
    }
  __syncwarp();
}

inline bool vector_pairs(int pairs, bool interleaved) { return pairs % (interleaved ? 4 : 8) == 0; }

}  // namespace kv
}  // namespace attn
