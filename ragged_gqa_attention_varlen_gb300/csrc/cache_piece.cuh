// cache_piece.cuh -- pieces of the work of attention over the paged cache: what
// the planning warp of a CTA hands to its other warps, and the places of partial
// results in the workspace.
#pragma once
#include "../../include/attn_varlen.h"
#include "cache_tile.cuh"

namespace attn {
namespace kv {

// Partial results of the forward in its workspace: byte offsets.
struct FwdWs {
  size_t meta, stats, rows, total;
  int64_t cut_rows;  // rows of one CTA's border piece
};
struct FwdHead {  // at offset 0
  int ok;
};
inline FwdWs fwd_ws(int B, int P, int Hq, int Hkv, int d, int64_t total_q) {
  FwdWs w;
  const int64_t x = total_q * (Hq / Hkv), all = total_q * Hq * (P ? 2 : 1);
  w.cut_rows = ((x < kRows ? x : kRows) + 7) / 8 * 8;
  const int64_t rows = (2 * kMaxCtas * w.cut_rows + (P ? all : 0) + 7) / 8 * 8;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  w.meta = 256;
  w.stats = w.meta + up(static_cast<size_t>(all) * sizeof(int2));
  w.rows = w.stats + up(static_cast<size_t>(rows) * sizeof(float4));
  w.total = w.rows + up(static_cast<size_t>(rows) * d * sizeof(float));
  (void)B;
  return w;
}
// meta: of every (own or prefix segment, token, head) whose row tile has steps,
// the CTA of the tile's first part and the number of parts.
// Partial row indices: CTA c's pieces of row tiles that continue from an
// earlier CTA (2c) or into a later one (2c + 1), then whole row tiles that
// wait for another segment's, by (own or prefix, token, head).
__device__ __forceinline__ int64_t cut_row(const FwdWs& w, int cta, bool first_part, int r) {
  return (2 * static_cast<int64_t>(cta) + (first_part ? 1 : 0)) * w.cut_rows + r;
}
__device__ __forceinline__ int64_t whole_row(const FwdWs& w, int64_t total_q, int Hq, bool own,
                                             int64_t tok, int h) {
  return 2 * kMaxCtas * w.cut_rows + ((own ? total_q : 0) + tok) * Hq + h;
}
// Place of features [4f, 4f + 4) of partial row `row`, in float4: eight rows'
// equal features share a 128-byte line.  The tile kernel holds a row per lane,
// so a warp's store then covers whole lines; row by row, each of its lanes
// would touch a line of its own (a 128-row tile took 11000 clk to store).
template <int HD>
__device__ __forceinline__ int64_t part_at(int64_t row, int f) {
  return ((row >> 3) * (HD / 4) + f) * 8 + (row & 7);
}

struct Piece {
  int row;  // of the segment's table; -1: the end
  int own, g;
  int tok, head;    // of the tile's first row: packed token, head in the group
  int rows;         // rows of the tile
  int tok0, ntok;   // the segment's tokens
  int len, plen;    // the segment's keys; the prefix's (position of own slot 0)
  int kt0, kt1;     // key tiles
  int klo, khi;     // keys that some row of the tile may attend to
  int mode;         // 0: writes out and lse; 1: partial of a cut tile; 2: partial of a whole tile
  int first;        // the tile's first part
  int parts;        // its parts
  int pad[3];
};

struct PieceRing {
  Piece piece[4];
  uint64_t full[4], empty[4];
};

__device__ __forceinline__ bool piece_take(PieceRing* r, uint32_t& k, Piece* out,
                                           volatile int* abort) {
  const int s = k & 3;
  if (!mbar_wait(&r->full[s], (k >> 2) & 1, abort)) return false;
  *out = r->piece[s];
  ++k;
  return true;
}
__device__ __forceinline__ void piece_done(PieceRing* r, uint32_t k_taken) {
  mbar_arrive(&r->empty[(k_taken - 1) & 3]);
}

// Sequences with at most this many rows of a K/V head are the kernel for few rows' where
// a call launches both (cache8_fwd.cu).
constexpr int kFewMost = 16;

// Joins the partial results behind the tile kernel (cache_fwd.cu).  tile_rows: rows of
// its tiles, 128 or 8; 0: 8 for sequences with few rows, whose results lie at `few`, else
// 128.
cudaError_t launch_join(const CacheParams& p, const FwdWs& w, int tile_rows, cudaStream_t s, const FwdWs* few = nullptr);

// One warp: this CTA's share as pieces, in the order of the segments.
template <int TR = kRows>
__device__ __forceinline__ void plan_pieces(const CacheParams& p, Plan* pl, PieceRing* ring,
                                            volatile int* s_abort) {
  const int lane = threadIdx.x & 31;
  uint32_t npub = 0;
  bool ok = true;
  // the next piece for the whole CTA
  auto publish = [&](const Piece& pc) -> bool {
    const int slot = npub & 3;
    if (npub >= 4 && !mbar_wait_warp(&ring->empty[slot], ((npub >> 2) - 1) & 1, s_abort))
      return false;
    if (lane == 0) {
      ring->piece[slot] = pc;
      mbar_arrive(&ring->full[slot]);
    }
    __syncwarp();
    ++npub;
    return true;
  };
  const int64_t per = pl->per, begin = pl->begin, end = pl->end;
  int64_t first = pl->seg_begin;
  const int s0 = pl->seg, known = pl->window;
  for (int s = s0; ok && first < end && s < p.P + p.B; ++s) {
    if (s - s0 >= known && ((s - s0) & 31) == 0) {  // the next 32 segments
      __syncwarp();
      if (s + lane < p.P + p.B) pl->segs[lane] = seg_plan<TR>(p, s + lane);
      __syncwarp();
    }
    const SegPlan g = pl->segs[(s - s0) & 31];
    const int nt = g.tiles;
    const bool varies = g.each < 0;
    int lo = g.lo, hi = g.hi;
    int64_t a = first;  // first unit of the row tile
    int gi = 0, t = 0;
    if (varies && begin > a) {  // skip whole K/V heads before this CTA's share
      int64_t sum = 0;
      for (int i = lane; i < nt; i += 32) {
        tile_keys<TR>(p, g.s, i, lo, hi);
        sum += tile_cost(p, tile_steps(lo, hi));
      }
      const int64_t cost = warp_sum64(sum);
      if (cost > 0) {
        gi = static_cast<int>(min(div64(begin - a, cost), static_cast<int64_t>(p.Hkv)));
        a += gi * cost;
      } else {
        gi = p.Hkv;
      }
    }
    if (!varies) {
      if (g.each > 0 && begin > a) {  // skip whole row tiles before this CTA's share
        const int cost = tile_cost(p, g.each);
        const int64_t skip = min(div64(begin - a, cost), static_cast<int64_t>(nt) * p.Hkv);
        a += skip * cost;
        gi = static_cast<int>(div64(skip, nt));
        t = static_cast<int>(skip - static_cast<int64_t>(gi) * nt);
      }
      if (g.each == 0) gi = p.Hkv;
    }
    for (; ok && gi < p.Hkv && a < end; ++gi, t = 0) {
      int64_t x0 = static_cast<int64_t>(t) * TR;  // the tile's first row
      int i0 = static_cast<int>(static_cast<uint32_t>(x0) / static_cast<uint32_t>(p.R));
      int h0 = static_cast<int>(x0 - static_cast<int64_t>(i0) * p.R);
      for (; ok && t < nt && a < end; ++t) {
        if (varies) tile_keys<TR>(p, g.s, t, lo, hi);
        const int n = varies ? tile_steps(lo, hi) : g.each;
        // units [a, a + tile_cost) carry no step
        const int64_t at = a + p.tile_cost;  // of step 0
        const Steps mine = share_steps(begin, end, at, n);
        const int f0 = mine.from, f1 = mine.to;
        if (f0 < f1) {
          Piece pc;
          pc.row = g.s.row;
          pc.own = g.s.own;
          pc.g = gi;
          pc.tok = g.s.tok0 + i0;
          pc.head = h0;
          pc.rows = static_cast<int>(min(static_cast<int64_t>(TR), static_cast<int64_t>(g.s.ntok) * p.R - x0));
          pc.tok0 = g.s.tok0;
          pc.ntok = g.s.ntok;
          pc.len = g.s.len;
          pc.plen = g.plen;
          pc.klo = lo;
          pc.khi = hi;
          pc.kt0 = lo / kKeys + f0;
          pc.kt1 = lo / kKeys + f1;
          pc.first = f0 == 0;
          pc.mode = f0 > 0 || f1 < n ? 1 : (g.waits ? 2 : 0);  // parts elsewhere; another segment
          pc.parts = f1 < n ? static_cast<int>(div64(at + n - 1, per)) - static_cast<int>(blockIdx.x) + 1 : 1;
          {  // the loads will soon ask for these
            const int32_t* row = (pc.own ? p.own.pages + pc.row * p.own.rs : p.prefix.pages + pc.row * p.prefix.rs);
            const int at = (min(pc.kt1 * kKeys, pc.len) - 1 >> p.page_log2) - lane;
            if (at >= pc.kt0 * kKeys >> p.page_log2) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + at));
          }
          ok = publish(pc);
        }
        a += tile_cost(p, n);
        x0 += TR;
        h0 += TR;
        if (p.R < 2 * TR) {
          const int dt = head_div(p, h0);
          i0 += dt;
          h0 -= dt * p.R;
        } else if (h0 >= p.R) {
          ++i0;
          h0 -= p.R;
        }
      }
    }
    if (varies && a >= end) break;
    first = varies ? a : first + static_cast<int64_t>(tile_cost(p, g.each)) * nt * p.Hkv;
  }
  Piece last = {};
  last.row = -1;
  if (ok) publish(last);
}

}  // namespace kv
}  // namespace attn
