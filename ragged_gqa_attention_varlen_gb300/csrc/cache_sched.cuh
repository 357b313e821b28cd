// cache_sched.cuh -- how attention over the paged cache is cut into pieces.
//
// A row tile is 128 (TR) consecutive packed rows of one segment and K/V head: row x
// is token x / R of the segment's tokens and head x % R of the group (R query
// heads per K/V head).  It visits the 128-key tiles that hold a key some row
// of it may attend to.  A tile of n steps costs n + tile_cost units (its
// Q rows, the first step's latency and its results cost as much as two to four
// steps); all
// tiles of a call, segment by segment, form one line of W units, and the CTA c
// of G takes units [c * per, (c + 1) * per), per = ceil(W / G): however uneven
// the lengths, every CTA does the same work in one go, and a long sequence of
// a small batch spreads over the whole GPU.  A row tile cut by such a border
// leaves one partial result per CTA, which the join kernel adds up.  Every CTA
// derives its share from the lengths itself, so nothing is launched before.
#pragma once
#include "cache.cuh"
#include "cache_share.h"

namespace attn {
namespace kv {

constexpr int kRows = 128;
constexpr int kMaxCtas = 160;  // CTAs of the attention and weights kernels, at most

struct Seg {
  int row;         // row of its table
  int tok0, ntok;  // its query tokens
  int len;         // its keys
  int klo;         // keys below are outside of every row's window
  int own;
};

// Masks cut the key range of each row tile of the segment differently.
__device__ __forceinline__ bool seg_varies(const CacheParams& p, const Seg& s) {
  return s.own && s.ntok > 1 && !p.q_pos && (p.wl >= 0 || p.wr >= 0);
}

// Keys [lo, hi) of which some row of row tile t may attend to one: exact
// bounds for own slots at default positions, where slot j stands at prefix_len
// + j and query i at prefix_len + len - ntok + i.
template <int TR = kRows>
__device__ __forceinline__ void tile_keys(const CacheParams& p, const Seg& s, int t, int& lo,
                                          int& hi) {
  lo = s.klo;
  hi = s.len;
  if (s.own && !p.q_pos) {
    const uint32_t x0 = static_cast<uint32_t>(t) * TR, R = p.R;
    const int i0 = static_cast<int>(x0 / R);
    const int i1 = min(s.ntok - 1, static_cast<int>((x0 + TR - 1) / R));
    const int64_t k0 = static_cast<int64_t>(s.len) - s.ntok;
    if (p.wl >= 0) lo = static_cast<int>(min(static_cast<int64_t>(s.len), max(static_cast<int64_t>(0), k0 + i0 - p.wl)));
    if (p.wr >= 0) hi = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(s.len), k0 + i1 + p.wr + 1)));
  }
  if (lo >= hi) lo = hi = 0;
}
__device__ __forceinline__ int tile_steps(int lo, int hi) {
  return hi > lo ? (hi + kKeys - 1) / kKeys - lo / kKeys : 0;
}

template <int TR = kRows>
__device__ __forceinline__ int seg_tiles(const CacheParams& p, const Seg& s) {
  return static_cast<int>((static_cast<int64_t>(s.ntok) * p.R + TR - 1) / TR);
}


// Keys of row `row` of the prefixes' table or the sequences' own.  A length that
// does not fit the table counts as 0 (seg_check reports it).
__device__ __forceinline__ int seg_len(const CacheParams& p, bool own, int row) {
  const Table& t = own ? p.own : p.prefix;
  const int n = __ldg(t.lens + row);
  return static_cast<unsigned>(n) <= static_cast<unsigned>(t.width) << p.page_log2 ? n : 0;
}

// The first slot of prefix pfx that some sequence's window reaches: at default
// positions query 0 of sequence b stands at prefix_len + own_len - Lq.
__device__ __forceinline__ int prefix_klo(const CacheParams& p, int pfx, int len) {
  if (p.wl < 0 || p.q_pos) return 0;
  // (cut to the batch: the arrays may not have been checked yet)
  const int b0 = max(__ldg(p.cu_prefix + pfx), 0), b1 = min(__ldg(p.cu_prefix + pfx + 1), p.B);
  int64_t lo = len;
  for (int b = b0; b < b1 && lo > 0; ++b) {
    const int nq = __ldg(p.cu_q + b + 1) - __ldg(p.cu_q + b);
    if (nq > 0) lo = min(lo, static_cast<int64_t>(len) + seg_len(p, true, b) - nq - p.wl);
  }
  return static_cast<int>(max(lo, static_cast<int64_t>(0)));
}

// Segment s (0 .. P+B-1).
__device__ __forceinline__ Seg seg_load(const CacheParams& p, int s) {
  Seg g;
  g.own = s >= p.P;
  g.row = g.own ? s - p.P : s;
  const int b0 = g.own ? g.row : __ldg(p.cu_prefix + g.row);
  const int b1 = g.own ? g.row + 1 : __ldg(p.cu_prefix + g.row + 1);
  g.tok0 = __ldg(p.cu_q + b0);
  g.ntok = __ldg(p.cu_q + b1) - g.tok0;
  g.len = seg_len(p, g.own, g.row);
  g.klo = g.own ? 0 : prefix_klo(p, g.row, g.len);
  return g;
}

// What a planner needs of a segment.
struct SegPlan {
  Seg s;
  int plen;    // keys of the prefix that it follows, or its own for a prefix
  int waits;   // its rows have results of another segment to be joined with
  int tiles;   // row tiles of a K/V head
  int each;    // steps of each row tile, -1: they differ
  int lo, hi;  // keys of the row tiles when they are all the same
};

template <int TR = kRows>
__device__ __forceinline__ SegPlan seg_plan(const CacheParams& p, int s) {
  SegPlan g;
  g.s = seg_load(p, s);
  if (p.most_rows) {
    const int64_t rows = static_cast<int64_t>(g.s.ntok) * p.R;
    if (rows < p.least_rows || rows > p.most_rows) g.s.ntok = 0;
  }
  g.plen = g.s.own ? 0 : g.s.len;
  g.waits = !g.s.own;
  if (g.s.own && p.P) {
    const int pfx = prefix_of(p, g.s.row);
    if (pfx >= 0) {
      g.plen = seg_len(p, false, pfx);
      g.waits = prefix_klo(p, pfx, g.plen) < g.plen;
    }
  }
  g.tiles = seg_tiles<TR>(p, g.s);
  g.each = seg_varies(p, g.s) ? -1 : 0;
  g.lo = g.hi = 0;
  if (g.each == 0 && g.tiles > 0) {
    tile_keys<TR>(p, g.s, 0, g.lo, g.hi);
    g.each = tile_steps(g.lo, g.hi);
  }
  return g;
}

// Cost of a tile of n steps.
__device__ __forceinline__ int tile_cost(const CacheParams& p, int n) {
  return n > 0 ? n + p.tile_cost : 0;
}

// Cost of one K/V head's row tiles (when they differ: one by one).
template <int TR = kRows>
__device__ __forceinline__ int64_t seg_cost(const CacheParams& p, const SegPlan& g) {
  if (g.each >= 0) return static_cast<int64_t>(g.tiles) * tile_cost(p, g.each);
  int64_t n = 0;
  for (int t = 0; t < g.tiles; ++t) {
    int lo, hi;
    tile_keys<TR>(p, g.s, t, lo, hi);
    n += tile_cost(p, tile_steps(lo, hi));
  }
  return n;
}

// x / R for 0 <= x < 2^20: the quotient's distance from an integer border is
// at least 1 / (2R), far above the error of the fp32 product.
__device__ __forceinline__ int head_div(const CacheParams& p, int x) {
  return static_cast<int>((static_cast<float>(x) + 0.5f) * p.inv_R);
}

// What is wrong with segment s's metadata, as status bits: with ATTN_DEV_BAD_CU
// the call does nothing, a bad length leaves out its segment's keys.
__device__ __forceinline__ int seg_check(const CacheParams& p, int s) {
  int bad = 0;
  if (s >= p.P) {
    const int b = s - p.P, c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1);
    if ((b == 0 && c0 != 0) || c0 < 0 || c1 < c0 || c1 > p.total_q) bad |= ATTN_DEV_BAD_CU;
    const int n = __ldg(p.own.lens + b);
    if (n < 0 || n > (static_cast<int64_t>(p.own.width) << p.page_log2)) bad |= ATTN_DEV_BAD_CACHE;
  } else {
    const int c0 = __ldg(p.cu_prefix + s), c1 = __ldg(p.cu_prefix + s + 1);
    if (c0 < 0 || c1 < c0 || c1 > p.B) bad |= ATTN_DEV_BAD_CU;
    const int n = __ldg(p.prefix.lens + s);
    if (n < 0 || n > (static_cast<int64_t>(p.prefix.width) << p.page_log2))
      bad |= ATTN_DEV_BAD_CACHE;
  }
  return bad;
}

// Quotient of non-negative values, by 32-bit division where they fit.
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Inclusive sums over a block of which the first `warps` warps hold values.
__device__ __forceinline__ int64_t block_scan(int64_t a, int warps, int64_t* tmp, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp < warps) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, a, o);
      if (lane >= o) a += x;
    }
    if (lane == 31) tmp[warp] = a;
  }
  __syncthreads();
  int64_t before = 0;
  total = 0;
  for (int w = 0; w < warps; ++w) {
    if (w == warp) before = total;
    total += tmp[w];
  }
  return a + before;
}

// Results of the plan, in shared memory.
struct Plan {
  int64_t per, begin, end;  // this CTA's units
  int64_t seg_begin;        // the first unit of that segment
  int seg;                  // the segment that holds unit `begin`
  int window;               // segments [seg, seg + window) of this array are filled
  int bad, pad;             // whether the cu arrays are inconsistent
  SegPlan segs[32];
  int64_t tmp[2][32];
};

// Whole block: this CTA's share of the work.  plan_of(s) plans segment s and
// cost_of(plan) is the cost of its tiles.  Returns false, for every thread,
// when there is nothing to do.  With as many threads as segments or more,
// every segment is read once, in one round of loads.
template <class PlanOf, class CostOf>
__device__ bool make_plan(const CacheParams& p, Plan* pl, PlanOf plan_of, CostOf cost_of) {
  const int nseg = p.P + p.B, tid = threadIdx.x, nt = blockDim.x;
  const bool one = nseg <= nt;
  SegPlan g = SegPlan();
  int bad = 0;
  if (one) {
    if (tid < nseg) {
      bad = seg_check(p, tid);
      if (!(bad & ATTN_DEV_BAD_CU)) g = plan_of(tid);
    }
  } else {
    for (int s = tid; s < nseg; s += nt) bad |= seg_check(p, s);
  }
  if (bad && blockIdx.x == 0) report(p.status, bad);
  if (tid == 0) {
    pl->bad = 0;
    pl->window = 0;
  }
  if (__syncthreads_or(bad & ATTN_DEV_BAD_CU)) {
    if (tid == 0) pl->bad = 1;
    __syncthreads();
    return false;
  }
  int64_t total = 0;
  int turn = 0;
  for (int pass = one ? 1 : 0; pass < 2; ++pass) {  // pass 0: the total of many segments
    int64_t before = 0;
    for (int s0 = 0; s0 < nseg; s0 += nt, turn ^= 1) {
      const int s = s0 + tid;
      int64_t mine = 0, sum;
      if (s < nseg) {
        if (!one) g = plan_of(s);
        mine = cost_of(g);
      }
      const int64_t upto = block_scan(mine, (min(nseg - s0, nt) + 31) / 32, pl->tmp[turn], sum);
      if (pass == 1) {
        if (one) total = sum;
        const int64_t per = div64(total + gridDim.x - 1, gridDim.x);
        const int64_t begin = per * blockIdx.x, first = before + upto - mine;
        if (s < nseg && mine > 0 && begin >= first && begin < first + mine) {
          pl->seg = s;
          pl->seg_begin = first;
        }
        if (s0 == 0 && tid == 0) {
          pl->per = per;
          pl->begin = begin;
          pl->end = min(total, begin + per);
        }
        if (one) {
          __syncthreads();
          const int at = s - pl->seg;
          if (pl->begin < pl->end && at >= 0 && at < 32 && s < nseg) pl->segs[at] = g;
          if (tid == 0) pl->window = 32;
        }
      }
      before += sum;
    }
    if (pass == 0) total = before;
  }
  __syncthreads();
  return pl->begin < pl->end;
}

}  // namespace kv
}  // namespace attn
