// cache_weights.cuh -- the attention weight that each cached key receives: sum
// over the query rows that read it of 2^(z - lse), z the base-2 logit.
//
// Keys lie in the TMEM lanes: S^T = K Q^T (128 keys x up to 128 query rows),
// so a key's sum is a sum along one thread's columns and needs neither atomics
// nor exchange.  Two ways to walk, by the number of 128-row tiles of a
// segment's queries (as in cache_sched.cuh, which also cuts the work):
//   one row tile (single tokens, a few drafts): Q stays, key tiles stream by;
//     every step finishes its 128 keys.  Reading K once bounds it.
//   several: a key tile stays, Q tiles stream by.  When the row tiles of a key
//     tile are cut between CTAs, partial sums are added up by the join kernel.
//     No pipe bounds it (XU 22 %, ALU 21 %, tensor 10 % busy at 64 features): the
//     latency of one 16-column pass after another on the four warps of a step.
//
// Measured: one step over 64 caches (255000 keys, 64 heads, cap and ALiBi) 33 us
// (2.5 TB/s); five prompts of up to 1500 tokens behind 1000 keys, 32 heads over 8
// of 64 features, 83 us (216 TFLOP/s); 4300 tokens of prompts, 96 heads over one
// of 160 features, 627 us (328 TFLOP/s), with cap and ALiBi 992 us.
//
// Sums, logits and lse are fp32; ex2.approx (2^-22) and the tanh below (3e-7) are
// as good as an fp32 logit of their sizes: 2.5e-7 of the sums against 64 bits.
//
// Warps (512 threads): 0 loads K by TMA, 1 issues the products into four TMEM
// buffers, 2 plans, 4-11 sum (two groups of four, taking steps in turn, so
// that each key's sum stays in one thread), 12-15 gather Q rows with cp.async,
// with each row's lse, slope and position.
#pragma once
#include "../../include/attn_varlen.h"
#include "cache_tile.cuh"

namespace attn {
namespace kv {

// Workspace: the cut key tile that starts in each CTA, and partial sums.
struct WeightsCut {
  int parts;  // 0: none
  int own, row, g, kt, len;
};
struct WeightsWs {
  size_t cuts, sums, total;
};
inline WeightsWs weights_ws() {
  WeightsWs w;
  w.cuts = 0;
  w.sums = (kMaxCtas * sizeof(WeightsCut) + 255) / 256 * 256;
  w.total = w.sums + 2 * kMaxCtas * 128 * sizeof(float);
  return w;
}

struct WPiece {
  int row;  // of the segment's table; -1: the end
  int own, g, tok0, ntok, len, plen;
  int rows;      // query rows of a K/V head
  int kt0, kt1;  // key tiles to write
  int a0, a1;    // of these, those that some row reads
  int t0, t1;    // row tiles
  int cut;       // 0: whole; 1: partial sums, 2: those of the first part
  int pad;
};
struct WPieceRing {
  WPiece piece[4];
  uint64_t full[4], empty[4];
};

struct RowInfo {  // of a Q tile
  float nlse[128];    // -lse in base 2 (-inf: the row counts for nothing)
  float nslope[128];  // -slope in base 2
  int pos[128];
  float fpos[128];
  int least[4], most[4];  // positions of the valid rows, per loading warp
};

constexpr int kThreadsW = 512;

template <int HD>
struct WShape {
  static constexpr uint32_t kT = HD == 160 ? 40960 : HD * 256;  // a K-major tile
  static constexpr int kChunksK = (HD + 63) / 64;
  static constexpr int kKS = HD == 64 ? 6 : 3;
  static constexpr int kQS = HD == 160 ? 2 : (HD == 128 ? 3 : 4);
  static constexpr uint32_t kOffQ = kKS * kT;
  static constexpr int kIS = 8;  // row infos: Q's place is free after the product, theirs after the sums
  static constexpr uint32_t kOffInfo = kOffQ + kQS * kT;
  static constexpr uint32_t kOffSum = kOffInfo + kIS * sizeof(RowInfo);  // [2 pieces][128]
  static constexpr uint32_t kOffBar = (kOffSum + 2 * 128 * 4 + 15) / 16 * 16;
};

struct WBars {
  uint64_t k_full[6], k_empty[6], q_full[4], q_empty[4], info_full[8], info_read[8];
  uint64_t s_full[4], s_read[4], pair[4], drain;
  WPieceRing ring;
  Plan plan;
  uint32_t tmem;
  int abort;
};

// Row tiles [t0, t1) with a query that may attend to a key of tile kt.
__device__ __forceinline__ void key_tile_rows(const CacheParams& p, const SegPlan& g, int nt, int kt,
                                              int& t0, int& t1) {
  t0 = 0;
  t1 = nt;
  const int64_t ja = static_cast<int64_t>(kt) * kKeys;
  const int64_t jb = min(ja + kKeys, static_cast<int64_t>(g.s.len)) - 1;
  if (jb < g.s.klo) {
    t1 = 0;
  } else if (g.s.own && !p.q_pos) {
    const int64_t k0 = static_cast<int64_t>(g.s.len) - g.s.ntok;
    int64_t i0 = 0, i1 = g.s.ntok - 1;
    if (p.wr >= 0) i0 = max(i0, ja - p.wr - k0);
    if (p.wl >= 0) i1 = min(i1, jb + p.wl - k0);
    if (i0 > i1) {
      t1 = 0;
    } else {
      t0 = static_cast<int>(static_cast<uint32_t>(i0 * p.R) / kRows);
      t1 = static_cast<int>(static_cast<uint32_t>(i1 * p.R + p.R - 1) / kRows) + 1;
    }
  }
}

// A segment as this kernel walks it: waits = row tiles; with one row tile or
// none, tiles = 1 and each = key tiles; else tiles = key tiles and each = row
// tiles (-1: they differ).  lo, hi: the keys that a single row tile reads.
__device__ __forceinline__ SegPlan weights_plan(const CacheParams& p, int s) {
  SegPlan g = seg_plan(p, s);
  const int nt = g.tiles, kt = (g.s.len + kKeys - 1) / kKeys;
  g.waits = nt;
  if (!p.w_out[g.s.own] || kt == 0) {
    g.tiles = g.each = 0;
  } else if (nt <= 1) {
    g.tiles = 1;
    if (nt == 1 && seg_varies(p, g.s)) tile_keys(p, g.s, 0, g.lo, g.hi);
    g.each = kt;
  } else {
    const bool varies = seg_varies(p, g.s) || g.s.klo > 0;
    g.tiles = kt;
    g.each = varies ? -1 : nt;
  }
  return g;
}
__device__ __forceinline__ int64_t weights_cost(const CacheParams& p, const SegPlan& g) {
  if (g.each >= 0) return static_cast<int64_t>(g.tiles) * (g.each + p.tile_cost);
  int64_t n = 0;
  for (int kt = 0; kt < g.tiles; ++kt) {
    int t0, t1;
    key_tile_rows(p, g, g.waits, kt, t0, t1);
    n += t1 - t0 + p.tile_cost;
  }
  return n;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}

__device__ __forceinline__ bool wpiece_take(WPieceRing* r, uint32_t& k, WPiece* out,
                                            volatile int* abort) {
  const int s = k & 3;
  if (!mbar_wait(&r->full[s], (k >> 2) & 1, abort)) return false;
  *out = r->piece[s];
  ++k;
  return true;
}

template <bool BF16, int HD, bool CAP, bool POS>
__global__ void __launch_bounds__(kThreadsW, 1)
    cache_weights_kernel(const __grid_constant__ CacheParams p, const __grid_constant__ WeightsWs w,
                         const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tkt) {
  using S = WShape<HD>;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t* sK = sm;
  uint8_t* sQ = sm + S::kOffQ;
  RowInfo* sInfo = reinterpret_cast<RowInfo*>(sm + S::kOffInfo);
  float* sSum = reinterpret_cast<float*>(sm + S::kOffSum);
  WBars* bars = reinterpret_cast<WBars*>(sm + S::kOffBar);
  volatile int* s_abort = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  WeightsCut* cuts = reinterpret_cast<WeightsCut*>(p.ws + w.cuts);
  float* parts = reinterpret_cast<float*>(p.ws + w.sums);
  if (tid == 0) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    cuts[blockIdx.x].parts = 0;
  }

  Plan* pl = &bars->plan;
  bool busy = make_plan(
      p, pl, [&](int s) { return weights_plan(p, s); },
      [&](const SegPlan& g) -> int64_t { return weights_cost(p, g) * p.Hkv; });
  if (blockIdx.x == 0 && tid == 0) {
    if (smem_addr(sm) & 1023u) report(p.status, ATTN_DEV_SMEM_ALIGN);
  }
  if (!busy || (smem_addr(sm) & 1023u)) return;  // uniform

  if (tid == 0) {
    for (int b = 0; b < S::kKS; ++b) {
      mbar_init(&bars->k_full[b], 1);
      mbar_init(&bars->k_empty[b], 1);
    }
    for (int b = 0; b < S::kQS; ++b) {
      mbar_init(&bars->q_full[b], 4);
      mbar_init(&bars->q_empty[b], 1);
    }
    for (int b = 0; b < S::kIS; ++b) {
      mbar_init(&bars->info_full[b], 4);
      mbar_init(&bars->info_read[b], 8);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->s_read[b], 4);
      mbar_init(&bars->pair[b], 2);
      mbar_init(&bars->ring.full[b], 1);
      mbar_init(&bars->ring.empty[b], 14);  // K loads, products, 8 summing and 4 loading warps
    }
    mbar_init(&bars->drain, 1);
    fence_barrier_init();
    bars->abort = 0;
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;

  // one arrival per warp: the piece has been copied
  auto take = [&](uint32_t& k, WPiece& pc) -> bool {
    if (!__all_sync(0xffffffffu, wpiece_take(&bars->ring, k, &pc, s_abort))) return false;
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->ring.empty[(k - 1) & 3]);
    return pc.row >= 0;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ K loads
    if (lane == 0) {
      prefetch_tensormap(&tk);
      if (HD == 160) prefetch_tensormap(&tkt);
    }
    const int box = min(p.page_size, kKeys), pieces = kKeys / box;
    uint32_t nt = 0, st = 0, ph = 0, loaded = 0;
    WPiece pc;
    bool ok = true;
    while (ok && take(nt, pc)) {
      const Table& t = pc.own ? p.own : p.prefix;
      const int32_t* row = t.pages + pc.row * t.rs;
      const int ch = lane / pieces, pi = lane - ch * pieces;  // box: (chunk, row block)
      for (int kt = pc.a0; kt < pc.a1; ++kt) {
        const int key0 = kt * kKeys;
        const int have = min(pieces, (pc.len - key0 + box - 1) / box);
        const bool mine = ch < S::kChunksK && pi < have;
        const int page = mine ? tile_page(p, row, key0 + pi * box) : 0;
        if (loaded >= S::kKS && !(ok = mbar_wait_warp(&bars->k_empty[st], ph ^ 1, s_abort))) break;
        if (lane == 0) mbar_arrive_expect_tx(&bars->k_full[st], S::kT / pieces * have);
        __syncwarp();
        if (mine) {
          uint8_t* dst = sK + st * S::kT;
          const int slot = p.page_size > kKeys ? key0 & (p.page_size - 1) : 0;
          if (HD == 160 && ch == 2)
            tma_load_4d(dst + 2 * 16384 + pi * box * 64, &tkt, &bars->k_full[st], 128, pc.g, slot, page);
          else
            tma_load_4d(dst + ch * 16384 + pi * box * 128, &tk, &bars->k_full[st], ch * kChunk, pc.g,
                        slot, page);
        }
        ++loaded;
        if (++st == S::kKS) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (*s_abort && lane == 0) {  // let every load land before the CTA exits
      const uint32_t n = min(loaded, static_cast<uint32_t>(S::kKS));
      for (uint32_t f = loaded - n; f < loaded; ++f)
        wait_drain(&bars->k_full[f % S::kKS], (f / S::kKS) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ S^T = K Q^T
    uint32_t nt = 0, step = 0, ks = 0, kph = 0, qs = 0, qph = 0;
    WPiece pc;
    bool ok = true;
    while (ok && take(nt, pc)) {
      const bool many = pc.t1 - pc.t0 > 1;  // a Q tile per step
      for (int kt = pc.a0; ok && kt < pc.a1; ++kt) {
        for (int t = pc.t0; t < pc.t1; ++t, ++step) {
          if (t == pc.t0 && !(ok = mbar_wait_warp(&bars->k_full[ks], kph, s_abort))) break;
          if ((many || kt == pc.a0) && !(ok = mbar_wait_warp(&bars->q_full[qs], qph, s_abort))) break;
          if (step >= 4 && !(ok = mbar_wait_warp(&bars->s_read[step & 3], ((step - 4) >> 2) & 1, s_abort)))
            break;
          const bool last_q = many || kt == pc.a1 - 1, last_k = t == pc.t1 - 1;
          if (lane == 0) {
            tc_fence_after();
            const uint32_t kb = smem_addr(sK + ks * S::kT), qb = smem_addr(sQ + qs * S::kT);
            const int cols = (min(kRows, pc.rows - t * kRows) + 15) / 16 * 16;
            const uint32_t id = idesc_f16(128, cols, BF16, false, false);
#pragma unroll
            for (int k = 0; k < HD / 16; ++k)
              umma_ss(tmem + (step & 3) * 128, kmajor_desc(kb, k), kmajor_desc(qb, k), id, k > 0);
            umma_commit(&bars->s_full[step & 3]);
            if (last_q) umma_commit(&bars->q_empty[qs]);
            if (last_k) umma_commit(&bars->k_empty[ks]);
          }
          __syncwarp();
          if (last_q && ++qs == S::kQS) {
            qs = 0;
            qph ^= 1;
          }
          if (last_k && ++ks == S::kKS) {
            ks = 0;
            kph ^= 1;
          }
        }
      }
    }
    if (lane == 0) {
      umma_commit(&bars->drain);
      wait_drain(&bars->drain, 0);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ plan
    uint32_t npub = 0;
    bool ok = true;
    auto publish = [&](const WPiece& pc) -> bool {
      const int slot = npub & 3;
      if (npub >= 4 && !mbar_wait_warp(&bars->ring.empty[slot], ((npub >> 2) - 1) & 1, s_abort))
        return false;
      if (lane == 0) {
        bars->ring.piece[slot] = pc;
        mbar_arrive(&bars->ring.full[slot]);
      }
      __syncwarp();
      ++npub;
      return true;
    };
    const int64_t per = pl->per, begin = pl->begin, end = pl->end;
    int64_t a = pl->seg_begin;  // first unit of the tile
    const int s0 = pl->seg, known = pl->window;
    for (int s = s0; ok && a < end && s < p.P + p.B; ++s) {
      if (s - s0 >= known && ((s - s0) & 31) == 0) {  // the next 32 segments
        __syncwarp();
        if (s + lane < p.P + p.B) pl->segs[lane] = weights_plan(p, s + lane);
        __syncwarp();
      }
      const SegPlan g = pl->segs[(s - s0) & 31];
      const int nt = g.waits;
      // skip whole K/V heads, and whole tiles of the same cost, before this CTA's share
      int g0 = 0, tile = 0;
      if (begin > a && g.tiles > 0) {
        int64_t cost = 0;  // of a K/V head
        if (g.each >= 0) {
          cost = static_cast<int64_t>(g.tiles) * (g.each + p.tile_cost);
        } else {
          int64_t sum = 0;
          for (int kt = lane; kt < g.tiles; kt += 32) {
            int t0, t1;
            key_tile_rows(p, g, nt, kt, t0, t1);
            sum += t1 - t0 + p.tile_cost;
          }
          cost = warp_sum64(sum);
        }
        g0 = static_cast<int>(min(div64(begin - a, cost), static_cast<int64_t>(p.Hkv)));
        a += g0 * cost;
        if (g.each >= 0 && g0 < p.Hkv) {
          tile = static_cast<int>(div64(begin - a, g.each + p.tile_cost));
          a += static_cast<int64_t>(tile) * (g.each + p.tile_cost);
        }
      }
      for (int gi = g0; ok && gi < p.Hkv && a < end; ++gi, tile = 0) {
        for (int t = tile; ok && t < g.tiles && a < end; ++t) {
          WPiece pc;
          pc.row = g.s.row;
          pc.own = g.s.own;
          pc.g = gi;
          pc.tok0 = g.s.tok0;
          pc.ntok = g.s.ntok;
          pc.len = g.s.len;
          pc.plen = g.plen;
          pc.rows = g.s.ntok * p.R;
          pc.cut = 0;
          pc.t0 = 0;
          pc.t1 = nt;
          int n = g.each;
          if (nt > 1) {
            if (g.each < 0) {
              key_tile_rows(p, g, nt, t, pc.t0, pc.t1);
              n = pc.t1 - pc.t0;
            }
          }
          // units [a, a + p.tile_cost) carry no step; a tile without any step
          // belongs to the CTA of its first unit
          const int64_t at = a + p.tile_cost;
          const Steps mine = share_steps(begin, end, at, n);
          const int f0 = mine.from, f1 = mine.to;
          if (f0 < f1 || (n == 0 && a >= begin)) {
            if (nt <= 1) {
              pc.kt0 = f0;
              pc.kt1 = f1;
              pc.a0 = max(f0, g.lo / kKeys);
              pc.a1 = nt == 1 ? max(pc.a0, min(f1, (g.hi + kKeys - 1) / kKeys)) : pc.a0;
            } else {
              pc.kt0 = t;
              pc.kt1 = t + 1;
              pc.a0 = t;
              pc.a1 = n > 0 ? t + 1 : t;
              if (n > 0 && (f0 > 0 || f1 < n)) {
                pc.cut = f0 == 0 ? 2 : 1;
                if (f0 == 0 && lane == 0) {
                  WeightsCut c = {static_cast<int>((at + n - 1) / per) - static_cast<int>(blockIdx.x) + 1,
                                  g.s.own, g.s.row, gi, t, g.s.len};
                  cuts[blockIdx.x] = c;
                }
                pc.t1 = pc.t0 + f1;
                pc.t0 += f0;
              }
            }
            ok = publish(pc);
          }
          a = at + n;
        }
      }
    }
    WPiece last = {};
    last.row = -1;
    if (ok) publish(last);
  } else if (warp >= 12) {
    // ------------------------------------------------------------ Q rows
    // A Q tile that stays is fetched by the four warps together; of several that
    // stream by, each warp fetches every fourth, so that as many are on their
    // way as there are stages (one after the other, each took 3000 clk).  A
    // parity wait tells a phase only from the ones next to it, and with two or
    // three places for four warps a place changes hands more often than a warp
    // has a tile of its own.  So every warp waits for the place of every tile, in
    // order, and arrives for every tile, its own or not: no product starts
    // before all four have seen its place free, so none is ever a phase behind
    // or ahead.
    uint32_t nt = 0, qs = 0, qph = 0, loaded = 0;
    const int wi = warp - 12;
    WPiece pc;
    bool ok = true;
    while (ok && take(nt, pc)) {
      if (pc.a0 >= pc.a1) continue;
      const bool many = pc.t1 - pc.t0 > 1;
      const int first = many ? 0 : wi, each = many ? 1 : 4;  // this warp's runs of 32 rows
      for (int t = pc.t0; t < pc.t1; ++t) {
        if (loaded >= S::kQS && !(ok = mbar_wait_warp(&bars->q_empty[qs], qph ^ 1, s_abort))) break;
        if (!many || static_cast<int>(loaded & 3) == wi) {
          const uint32_t x0 = static_cast<uint32_t>(t) * kRows;
          const int i0 = static_cast<int>(x0 / static_cast<uint32_t>(p.R));
          const int h0 = static_cast<int>(x0) - i0 * p.R;
          const int n = min(kRows, pc.rows - static_cast<int>(x0));
          uint8_t* dst = sQ + qs * S::kT;
          copy_q_rows<HD>(p, dst, pc.g, pc.tok0 + i0, h0, n, many ? 0 : wi, many ? 1 : 4);
          // the rows' scalars: all loads first
          float nlse[4], nslope[4];
          int pos[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = (first + k * each) * 32 + lane;
            nlse[k] = -INFINITY;
            nslope[k] = 0.f;
            pos[k] = 0;
            if (first + k * each < 4 && r < n) {
              const int dt = head_div(p, h0 + r), tok = pc.tok0 + i0 + dt;
              const int h = pc.g * p.R + h0 + r - dt * p.R;
              nlse[k] = __ldg(p.lse + static_cast<int64_t>(tok) * p.Hq + h);
              if (POS) {
                int b = pc.row;
                if (!pc.own) {
                  const int b0 = __ldg(p.cu_prefix + pc.row), b1 = __ldg(p.cu_prefix + pc.row + 1);
                  b = b1 - b0 == pc.ntok && __ldg(p.cu_q + b0 + tok - pc.tok0) == tok &&
                              __ldg(p.cu_q + b0 + tok - pc.tok0 + 1) > tok
                          ? b0 + tok - pc.tok0
                          : seq_of(p.cu_q, b0, b1, tok);
                }
                if (p.slopes) nslope[k] = -__ldg(p.slopes + b * p.slopes_bs + h) * kLog2e;
                if (p.q_pos)
                  pos[k] = __ldg(p.q_pos + tok);
                else if (pc.own)
                  pos[k] = pc.plen + pc.len - pc.ntok + tok - pc.tok0;
                else
                  pos[k] = pc.plen + seg_len(p, true, b) - (__ldg(p.cu_q + b + 1) - tok);
              }
            }
          }
          // The scalars' place, once the sums have read those of kIS tiles before.  A
          // warp may pass over places here: the product kQS tiles before is done,
          // which needed the step four before it summed, and the groups take steps
          // in turn, so both have read all tiles up to kQS + 6 before.
          static_assert(2 * S::kIS >= S::kQS + 6, "a wait for row scalars could be a phase behind");
          const int is = loaded & (S::kIS - 1);
          if (loaded >= S::kIS &&
              !(ok = mbar_wait_warp(&bars->info_read[is], ((loaded / S::kIS) & 1) ^ 1, s_abort)))
            break;
          RowInfo& info = sInfo[is];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int run = first + k * each, r = run * 32 + lane;
            if (run >= 4) break;
            info.nlse[r] = nlse[k] > -INFINITY ? -nlse[k] * kLog2e : -INFINITY;
            if (POS) {
              info.nslope[r] = nslope[k];
              info.pos[r] = pos[k];
              info.fpos[r] = static_cast<float>(pos[k]);
              const int lo = __reduce_min_sync(0xffffffffu, r < n ? pos[k] : INT32_MAX);
              const int hi = __reduce_max_sync(0xffffffffu, r < n ? pos[k] : INT32_MIN);
              if (lane == 0) {
                info.least[run] = lo;
                info.most[run] = hi;
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_n(&bars->info_full[is], many ? 4 : 1);
          // rows up to the next multiple of 16 take part in the product
          const int pad = (n + 15) / 16 * 16 - n;
          for (int i = (many ? 0 : wi * 32) + lane; i < pad * (HD / 8); i += many ? 32 : 128) {
            const int q = i / (HD / 8);
            *reinterpret_cast<uint4*>(dst + kmajor_unit(n + q, i - q * (HD / 8))) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&bars->q_full[qs]);
        ++loaded;
        if (++qs == S::kQS) {
          qs = 0;
          qph ^= 1;
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ sums
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int r = quad * 32 + lane;  // key of the tile
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    const float in_scale = CAP ? p.sigma / p.softcap : p.sigma * kLog2e;
    const float sc = CAP ? p.softcap * kLog2e : in_scale;
    uint32_t nt = 0, step = 0, used = 0, npair = 0;  // used: row infos
    WPiece pc;
    bool ok = true;
    while (ok && take(nt, pc)) {
      const float* in = p.w_in[pc.own];
      if (in) in += pc.row * p.wi_rs[pc.own] + pc.g * p.wi_hs[pc.own];
      float* out = p.w_out[pc.own] + pc.row * p.wo_rs[pc.own] + pc.g * p.wo_hs[pc.own];
      // keys that no row reads keep their sum
      for (int kt = pc.kt0; kt < pc.kt1; ++kt) {
        if ((kt < pc.a0 || kt >= pc.a1) && (kt & 1) == half) {
          const int key = kt * kKeys + r;
          if (key < pc.len) out[key] = in ? in[key] : 0.f;
        }
      }
      const bool many = pc.t1 - pc.t0 > 1;
      for (int kt = pc.a0; ok && kt < pc.a1; ++kt) {
        const int key = kt * kKeys + r;
        const bool there = key < pc.len;
        float before = 0.f;  // read while the products run
        if (there && in && !pc.cut) before = in[key];
        const Table& t = pc.own ? p.own : p.prefix;
        // a key whose page is out of the pool receives nothing
        const bool gone = there && static_cast<unsigned>(__ldg(t.pages + pc.row * t.rs + (key >> p.page_log2))) >=
                                       static_cast<unsigned>(p.num_pages);
        int kpos = 0;
        if (POS) {
          kpos = t.pos ? __ldg(t.pos + pc.row * t.pos_rs + pc.g * t.pos_hs + min(key, pc.len - 1))
                       : (pc.own ? pc.plen : 0) + key;
        }
        float total = 0.f;
        for (int t = pc.t0; t < pc.t1; ++t, ++step) {
          const bool last_q = many || kt == pc.a1 - 1;
          if (static_cast<int>(step & 1) == half) {
            const int cols = min(kRows, pc.rows - t * kRows);
            const RowInfo& info = sInfo[used & (S::kIS - 1)];
            if (!(ok = mbar_wait_warp(&bars->info_full[used & (S::kIS - 1)], (used / S::kIS) & 1, s_abort)))
              break;
            if (!(ok = mbar_wait_warp(&bars->s_full[step & 3], (step >> 2) & 1, s_abort))) break;
            tc_fence_after();
            bool free = true;  // no key of this warp is masked for any row
            bool near = true;  // positions are exact in fp32
            if (POS) {
              const int least = min(min(info.least[0], info.least[1]), min(info.least[2], info.least[3]));
              const int most = max(max(info.most[0], info.most[1]), max(info.most[2], info.most[3]));
              free = __all_sync(0xffffffffu, !there || ((p.wl < 0 || kpos >= most - p.wl) &&
                                                        (p.wr < 0 || kpos <= least + p.wr)));
              near = __all_sync(0xffffffffu, max(kpos, most) < (1 << 24) && min(kpos, least) >= 0);
            }
            uint64_t sum = f2_make(0.f, 0.f);
            const uint32_t sb = tmem + (step & 3) * 128 + lane_addr;
#pragma unroll 1
            for (int c0 = 0; c0 < cols; c0 += 16) {
              float x[16];
              tmem_ld16(sb + c0, x);
              float nl[16];
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(nl + i) = *reinterpret_cast<const float4*>(info.nlse + c0 + i);
              if (POS && free && near) {
                if (p.slopes) {
                  const float kf = static_cast<float>(kpos);
#pragma unroll
                  for (int i = 0; i < 16; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(info.fpos + c0 + i);
                    const float4 s = *reinterpret_cast<const float4*>(info.nslope + c0 + i);
                    nl[i] = fmaf(fabsf(f.x - kf), s.x, nl[i]);
                    nl[i + 1] = fmaf(fabsf(f.y - kf), s.y, nl[i + 1]);
                    nl[i + 2] = fmaf(fabsf(f.z - kf), s.z, nl[i + 2]);
                    nl[i + 3] = fmaf(fabsf(f.w - kf), s.w, nl[i + 3]);
                  }
                }
              } else if (POS) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const int d = info.pos[c0 + i] - kpos;
                  const bool cut = (p.wl >= 0 && d > p.wl) || (p.wr >= 0 && -d > p.wr);
                  const float b = p.slopes ? fmaf(static_cast<float>(abs(d)), info.nslope[c0 + i], info.nlse[c0 + i])
                                           : info.nlse[c0 + i];
                  nl[i] = cut ? -INFINITY : b;
                }
              }
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                uint64_t z = f2_make(x[i], x[i + 1]);
                if (CAP) z = tanh2_fp32(f2_mul(z, f2_make(in_scale, in_scale)));
                z = f2_fma(z, f2_make(sc, sc), f2_make(nl[i], nl[i + 1]));
                sum = f2_add(sum, f2_make(ex2_approx(f2_lo(z)), ex2_approx(f2_hi(z))));
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->s_read[step & 3]);
            total += f2_lo(sum) + f2_hi(sum);
            if (!many) {  // one row tile
              if (gone) total = 0.f;
              if (pc.cut)
                parts[(2 * blockIdx.x + (pc.cut == 2)) * 128 + r] = total;
              else if (there)
                out[key] = before + total;
            }
          } else if (last_q && !(ok = mbar_wait_warp(&bars->info_full[used & (S::kIS - 1)],
                                                     (used / S::kIS) & 1, s_abort))) {
            break;  // (not ahead of the entry's filling, or two arrivals would count as one)
          }
          if (last_q) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->info_read[used & (S::kIS - 1)]);
            ++used;
          }
        }
        if (!ok || !many) continue;
        // both groups' shares of the row tiles
        float* mine = sSum + (npair & 1) * 128;
        if (half) mine[r] = total;
        if (!(ok = warp_exchange(&bars->pair[quad], npair & 1, s_abort))) break;
        ++npair;
        if (!half) {
          total = gone ? 0.f : total + mine[r];
          if (pc.cut)
            parts[(2 * blockIdx.x + (pc.cut == 2)) * 128 + r] = total;
          else if (there)
            out[key] = before + total;
        }
      }
    }
  }
  __syncthreads();
  if (tid == 0 && *s_abort) report(p.status, ATTN_DEV_TIMEOUT_FWD);
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <bool B, int HD>
auto pick_weights(const CacheParams& p) {
  const bool pos = p.slopes || p.wl >= 0 || p.wr >= 0 || p.own.pos || (p.P && p.prefix.pos);
  if (p.softcap > 0.f)
    return pos ? cache_weights_kernel<B, HD, true, true> : cache_weights_kernel<B, HD, true, false>;
  return pos ? cache_weights_kernel<B, HD, false, true> : cache_weights_kernel<B, HD, false, false>;
}

template <int HD>
cudaError_t launch_weights_d(const CacheParams& p, const WeightsWs& w, const CUtensorMap& tk,
                             const CUtensorMap& tkt, int grid, cudaStream_t s) {
  constexpr uint32_t smem = WShape<HD>::kOffBar + sizeof(WBars);
  static_assert(smem <= 232448, "shared memory");
  auto k = p.dtype == 1 ? pick_weights<true, HD>(p) : pick_weights<false, HD>(p);
  cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  k<<<grid, kThreadsW, smem, s>>>(p, w, tk, tkt);
  return cudaGetLastError();
}

}  // namespace kv
}  // namespace attn
