// cache_share.h -- the part of a tile that falls into a CTA's share of the work
// (cache_sched.cuh); plain C++, so that the host can run it too.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define ATTN_SHARE __host__ __device__ __forceinline__
#else
#define ATTN_SHARE inline
#endif

namespace attn {
namespace kv {

struct Steps {
  int from, to;  // steps [from, to) of the tile; none: from >= to
};

// Of a tile whose n steps are the units [at, at + n), those inside [begin, end).
// Shares are compared in 64 bits before they are cut to the tile: a K/V head of a
// million-token prompt has more than 2^31 units, and a share may begin that far
// behind a tile.
ATTN_SHARE Steps share_steps(int64_t begin, int64_t end, int64_t at, int n) {
  const int64_t b = begin - at, e = end - at;
  Steps s;
  s.from = static_cast<int>(b < 0 ? 0 : (b > n ? n : b));
  s.to = static_cast<int>(e < 0 ? 0 : (e > n ? n : e));
  return s;
}

}  // namespace kv
}  // namespace attn
