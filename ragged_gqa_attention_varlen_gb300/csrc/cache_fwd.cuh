// cache_fwd.cuh -- attention of packed query rows over the paged K/V cache
// (the tile kernel; cache_sched.cuh cuts the work, the merge kernel in
// cache_fwd.cu joins cut rows).
//
// Per step (128 rows x 128 keys), with z the base-2 logit and m the row's
// reference (a running maximum, or a bound known beforehand):
//   S = Q K^T            tcgen05.mma, fp32 in TMEM
//   P = 2^(z - m)        softmax warps, one TMEM lane per row; the 16-bit pairs
//                        overwrite S, whose buffer is free again after P V
//   O += P V             tcgen05.mma with P from TMEM
//   L += P 1             the same product with a tile of ones: the row sums of
//                        the rounded P, which divide O (one key then gives
//                        exactly its V row) without an element's instruction
// and l = sum of P in fp32 in the softmax warps (for lse).
//
// Single-token calls read every K and V row once for R <= 128 rows of a group,
// so the copies bound them; calls with many rows behind a shared prefix are
// bound by the softmax warps' MUFU work and the hand-offs between them and
// the tensor core, as the packed forward is.
//
// Warps (384 threads): 0 loads K (lanes 0-15) and V (lanes 16-31) by TMA, a
// box of min(page_size, 128) rows x 64 features each; 1 issues S, 2 issues O
// and clears the V rows of a cut tile that no row reads (the pages may hold
// anything there, and 0 * NaN would reach O); 3 plans the CTA's pieces and
// copies Q rows (a row is any (token, head), so Q is gathered with cp.async
// into the swizzled layout rather than boxed by TMA); 4-11 softmax, two per
// TMEM lane quadrant, each taking 64 of a step's keys.
#pragma once
#include "../../include/attn_varlen.h"
#include "cache_tile.cuh"

namespace attn {
namespace kv {

// Partial results of the forward in its workspace: byte offsets.
struct FwdWs {
  size_t info, meta, stats, rows, total;
  int64_t cut_rows;  // rows of one CTA's border piece
};
struct FwdHead {  // at offset 0
  int ok;
};
inline FwdWs fwd_ws(int B, int P, int Hq, int Hkv, int d, int64_t total_q) {
  FwdWs w;
  const int64_t R = Hq / Hkv, x = total_q * R;
  const int64_t tiles = static_cast<int64_t>(Hkv) * (x / kRows + B + (P ? x / kRows + P : 0));
  w.cut_rows = ((x < kRows ? x : kRows) + 7) / 8 * 8;
  const int64_t rows = (2 * kMaxCtas * w.cut_rows + (P ? 2 * total_q * Hq : 0) + 7) / 8 * 8;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  w.info = 256;
  w.meta = w.info + up(static_cast<size_t>(B + P) * sizeof(int2));
  w.stats = w.meta + up(static_cast<size_t>(tiles) * sizeof(int2));
  w.rows = w.stats + up(static_cast<size_t>(rows) * sizeof(float4));
  w.total = w.rows + up(static_cast<size_t>(rows) * d * sizeof(float));
  return w;
}
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
  int first;        // mode 1: the tile's first part
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

template <int HD>
struct FwdShape {
  static constexpr uint32_t kQ = HD == 160 ? 40960 : HD * 256;  // a K-major tile
  static constexpr uint32_t kV = HD == 160 ? 49152 : HD * 256;  // V: 64-feature chunks of 16 KB
  static constexpr int kChunksK = (HD + 63) / 64;
  static constexpr int kKS = HD == 160 ? 2 : (HD == 128 ? 3 : 6);  // K stages
  static constexpr int kVS = HD == 160 ? 2 : (HD == 128 ? 2 : 6);  // V stages
  static constexpr uint32_t kOffK = kQ;
  static constexpr uint32_t kOffV = kOffK + kKS * kQ;
  static constexpr uint32_t kOffMax = kOffV + kVS * kV;          // [2 steps][2 halves][128]
  static constexpr uint32_t kOffSum = kOffMax + 2 * 2 * 128 * 4;  // [2 pieces][2 halves][128] l
  static constexpr uint32_t kOffOne = kOffSum + 2 * 2 * 128 * 4;  // 16 x 16 ones in any layout (1 KB)
  static constexpr uint32_t kOffBar = kOffOne + 1024;
};

struct FwdBars {
  uint64_t q_first, q_full, q_empty;
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t o_full, o_empty, drain;
  uint64_t mx_x[4][2], l_x[4];
  PieceRing ring;
  Plan plan;
  uint32_t tmem;
  int abort;
};

constexpr uint32_t kColOv = 256;  // TMEM: S0 / P0 [0,128), S1 / P1 [128,256), O [256, 256 + d), L 16 more
constexpr float kLazy = 8.f;                    // rescale when the maximum grows by more (base 2)
constexpr float kFixedCap = 9.5f;               // largest cap with a reference known beforehand
constexpr int kCh = 16;                         // columns of a softmax pass

// CAP: the call has a softcap; FIXED: of at most kFixedCap and default key
// positions, so P is taken against a bound and no maximum is tracked; POS:
// the call has ALiBi, a mask or key positions.
template <bool BF16, int HD, bool CAP, bool FIXED, bool POS>
__global__ void __launch_bounds__(kThreads, 1)
    cache_fwd_kernel(const __grid_constant__ CacheParams p, const __grid_constant__ FwdWs w,
                     const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tkt, const __grid_constant__ CUtensorMap tv) {
  using S = FwdShape<HD>;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t* sQ = sm;
  uint8_t* sK = sm + S::kOffK;
  uint8_t* sV = sm + S::kOffV;
  float* sMax = reinterpret_cast<float*>(sm + S::kOffMax);
  float* sSum = reinterpret_cast<float*>(sm + S::kOffSum);
  FwdBars* bars = reinterpret_cast<FwdBars*>(sm + S::kOffBar);
  volatile int* s_abort = &bars->abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int2* info = reinterpret_cast<int2*>(p.ws + w.info);
  int2* meta = reinterpret_cast<int2*>(p.ws + w.meta);
  if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's share of the steps
  Plan* pl = &bars->plan;
  const bool busy = make_plan(
      p, pl, info,
      [&](int s) { return seg_plan(p, s); },
      [&](const SegPlan& g) -> int64_t { return seg_cost(p, g) * p.Hkv; },
      [&](const SegPlan& g) -> int { return g.tiles * p.Hkv; });
  if (blockIdx.x == 0 && tid == 0) {
    FwdHead* head = reinterpret_cast<FwdHead*>(p.ws);
    int ok = pl->bad == 0;
    if (smem_addr(sm) & 1023u) {
      report(p.status, ATTN_DEV_SMEM_ALIGN);
      ok = 0;
    }
    if (pl->bad) report(p.status, pl->bad);
    head->ok = ok;
  }
  if (!busy || (smem_addr(sm) & 1023u)) return;  // uniform

  if (tid == 0) {
    mbar_init(&bars->q_first, 8);
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int b = 0; b < S::kKS; ++b) {
      mbar_init(&bars->k_full[b], 1);
      mbar_init(&bars->k_empty[b], 1);
    }
    for (int b = 0; b < S::kVS; ++b) {
      mbar_init(&bars->v_full[b], 1);
      mbar_init(&bars->v_empty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->p_full[b], 8);
      mbar_init(&bars->pv_done[b], 1);
    }
    mbar_init(&bars->o_full, 1);
    mbar_init(&bars->o_empty, 8);
    mbar_init(&bars->drain, 2);
    for (int q = 0; q < 4; ++q) {
      mbar_init(&bars->mx_x[q][0], 2);
      mbar_init(&bars->mx_x[q][1], 2);
      mbar_init(&bars->l_x[q], 2);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bars->ring.full[s], 1);
      mbar_init(&bars->ring.empty[s], 12);  // K and V loads, two MMA issuers, 8 softmax warps
    }
    fence_barrier_init();
    bars->abort = 0;
  }
  for (int i = tid; i < 256; i += kThreads)
    reinterpret_cast<uint32_t*>(sm + S::kOffOne)[i] = Pack<BF16>::two(1.f, 1.f);
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  const int box = min(p.page_size, kKeys);  // rows of a load box
  const int pieces = kKeys / box;           // boxes of a key tile and chunk

  if (warp < 4) {
    warpgroup_reg_dealloc<kRegsLow>();
    if (warp == 0) {
      // ------------------------------------------------------------ K and V loads
      const bool is_k = lane < 16;
      const int gl = lane & 15;
      const unsigned gmask = is_k ? 0x0000ffffu : 0xffff0000u;
      const int lead = is_k ? 0 : 16;
      if (gl == 0) {
        prefetch_tensormap(is_k ? &tk : &tv);
        if (is_k && HD == 160) prefetch_tensormap(&tkt);
      }
      const int stages = is_k ? S::kKS : S::kVS;
      const uint32_t bytes = is_k ? S::kQ : S::kV;  // of a whole tile
      uint64_t* full = is_k ? bars->k_full : bars->v_full;
      uint64_t* empty = is_k ? bars->k_empty : bars->v_empty;
      uint8_t* dst0 = is_k ? sK : sV;
      uint32_t take = 0, st = 0, ph = 0, loaded = 0;
      Piece pc;
      for (;;) {
        if (!__all_sync(gmask, piece_take(&bars->ring, take, &pc, s_abort))) break;
        __syncwarp(gmask);
        if (gl == 0) piece_done(&bars->ring, take);
        if (pc.row < 0) break;
        const Table& t = pc.own ? p.own : p.prefix;
        const int32_t* row = t.pages + pc.row * t.rs;
        const int total = S::kChunksK * pieces;  // boxes of a tile: (chunk, row block)
        bool ok = true;
        for (int kt = pc.kt0; kt < pc.kt1; ++kt) {
          const int key0 = kt * kKeys;
          const int have = min(pieces, (pc.len - key0 + box - 1) / box);  // row blocks in use
          // page numbers before the wait for a free stage
          int pages[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int x = gl + 16 * i, pi = x % pieces;
            if (x < total && pi < have) pages[i] = tile_page(p, row, key0 + pi * box);
          }
          if (loaded >= static_cast<uint32_t>(stages) &&
              !(ok = __all_sync(gmask, mbar_wait(&empty[st], ph ^ 1, s_abort))))
            break;
          if (gl == 0) mbar_arrive_expect_tx(&full[st], bytes / pieces * have);
          __syncwarp(gmask);
          uint8_t* dst = dst0 + st * bytes;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int x = gl + 16 * i, ch = x / pieces, pi = x % pieces;
            if (x < total && pi < have) {
              const int slot = p.page_size > kKeys ? key0 & (p.page_size - 1) : 0;
              if (is_k && HD == 160 && ch == 2)
                tma_load_4d(dst + 2 * 16384 + pi * box * 64, &tkt, &full[st], 128, pc.g, slot,
                            pages[i]);
              else
                tma_load_4d(dst + ch * 16384 + pi * box * 128, is_k ? &tk : &tv, &full[st],
                            ch * kChunk, pc.g, slot, pages[i]);
            }
          }
          ++loaded;
          if (++st == static_cast<uint32_t>(stages)) {
            st = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
      }
      if (*s_abort && lane == lead) {
        // let every load of this group land before the CTA exits
        const uint32_t n = min(loaded, static_cast<uint32_t>(stages));
        for (uint32_t f = loaded - n; f < loaded; ++f) wait_drain(&full[f % stages], (f / stages) & 1);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ S = Q K^T
      if (lane == 0) {
        constexpr uint32_t kIdS = idesc_f16(128, 128, BF16, false, false);
        uint32_t take = 0, step = 0, st = 0, ph = 0, tiles = 0;
        Piece pc;
        bool ok = true;
        while (ok && piece_take(&bars->ring, take, &pc, s_abort)) {
          piece_done(&bars->ring, take);
          if (pc.row < 0) break;
          if (!(tiles == 0 ? mbar_wait(&bars->q_first, 0, s_abort)
                           : mbar_wait(&bars->q_full, (tiles - 1) & 1, s_abort)))
            break;
          for (int kt = pc.kt0; kt < pc.kt1; ++kt, ++step) {
            if (!(ok = mbar_wait(&bars->k_full[st], ph, s_abort))) break;
            // the product with the P that took the buffer's previous S (step - 2) is done
            if (step >= 2 && !(ok = mbar_wait(&bars->pv_done[step & 1], ((step - 2) >> 1) & 1, s_abort)))
              break;
            tc_fence_after();
            const uint32_t kb = smem_addr(sK + st * S::kQ), qb = smem_addr(sQ);
#pragma unroll
            for (int k = 0; k < HD / 16; ++k)
              umma_ss(tmem + (step & 1) * 128, kmajor_desc(qb, k), kmajor_desc(kb, k), kIdS, k > 0);
            umma_commit(&bars->s_full[step & 1]);
            umma_commit(&bars->k_empty[st]);
            if (kt == pc.kt1 - 1) umma_commit(&bars->q_empty);
            if (++st == S::kKS) {
              st = 0;
              ph ^= 1;
            }
          }
          ++tiles;
        }
        umma_commit(&bars->drain);
        wait_drain(&bars->drain, 0);
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------ O += P V
      constexpr uint32_t kIdO = idesc_f16(128, HD, BF16, false, true);
      constexpr uint32_t kIdL = idesc_f16(128, 16, BF16, false, false);
      const uint64_t ones = sdesc_sw64(smem_addr(sm + S::kOffOne));
      uint32_t take = 0, step = 0, st = 0, ph = 0, tiles = 0;
      Piece pc;
      bool ok = true;
      while (ok) {
        if (!__all_sync(0xffffffffu, piece_take(&bars->ring, take, &pc, s_abort))) break;
        __syncwarp();
        if (lane == 0) piece_done(&bars->ring, take);
        if (pc.row < 0) break;
        for (int kt = pc.kt0; kt < pc.kt1; ++kt, ++step) {
          const int key0 = kt * kKeys;
          const int nk = min(kKeys, pc.len - key0);        // keys of the tile that exist
          const int z0 = min(max(pc.klo - key0, 0), nk);   // those [z0, z1) that some row reads
          const int z1 = max(min(pc.khi - key0, nk), z0);
          const int ksteps = (nk + 15) / 16;
          if (!(ok = mbar_wait_warp(&bars->v_full[st], ph, s_abort))) break;
          if (z0 > 0 || z1 < ksteps * 16) {
            // clear the other rows: they may hold anything, and P is 0 there
            uint8_t* v = sV + st * S::kV;
            const int rows = z0 + ksteps * 16 - z1;
            for (int i = lane; i < rows * 8; i += 32) {
              const int r0 = i >> 3, r = r0 < z0 ? r0 : r0 - z0 + z1;
#pragma unroll
              for (int c = 0; c < S::kChunksK; ++c)
                *reinterpret_cast<uint4*>(v + c * 16384 + r * 128 + (i & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (!(ok = mbar_wait_warp(&bars->p_full[step & 1], (step >> 1) & 1, s_abort))) break;
          if (kt == pc.kt0 && tiles > 0 &&
              !(ok = mbar_wait_warp(&bars->o_empty, (tiles - 1) & 1, s_abort)))
            break;
          if (lane == 0) {
            tc_fence_after();
            const uint32_t vb = smem_addr(sV + st * S::kV);
            // keys 16k .. 16k + 15: pair columns 8 (k mod 4) of half k / 4
            for (int k = 0; k < ksteps; ++k)
              umma_ts(tmem + kColOv, tmem + (step & 1) * 128 + (k >> 2) * 64 + (k & 3) * 8,
                      sdesc_sw128(vb + k * 2048, 16384, 1024), kIdO, (kt > pc.kt0 || k > 0));
            for (int k = 0; k < ksteps; ++k)
              umma_ts(tmem + kColOv + HD, tmem + (step & 1) * 128 + (k >> 2) * 64 + (k & 3) * 8, ones,
                      kIdL, (kt > pc.kt0 || k > 0));
            umma_commit(&bars->pv_done[step & 1]);
            umma_commit(&bars->v_empty[st]);
            if (kt == pc.kt1 - 1) umma_commit(&bars->o_full);
          }
          __syncwarp();
          if (++st == S::kVS) {
            st = 0;
            ph ^= 1;
          }
        }
        ++tiles;
      }
      if (lane == 0) {
        umma_commit(&bars->drain);
        wait_drain(&bars->drain, 0);
      }
    } else {
      // ------------------------------------------------------------ plan and Q rows
      uint32_t npub = 0;
      bool ok = true;
      // the next piece for the whole CTA, and its Q rows
      auto publish = [&](const Piece& pc) -> bool {
        const int slot = npub & 3;
        if (npub >= 4 && !mbar_wait_warp(&bars->ring.empty[slot], ((npub >> 2) - 1) & 1, s_abort))
          return false;
        if (lane == 0) {
          bars->ring.piece[slot] = pc;
          mbar_arrive(&bars->ring.full[slot]);
        }
        __syncwarp();
        if (pc.row >= 0 && npub > 0) {  // (the softmax warps fetch the first piece's)
          if (!mbar_wait_warp(&bars->q_empty, (npub - 1) & 1, s_abort)) return false;
          copy_q_rows<HD>(p, sQ, pc.g, pc.tok, pc.head, pc.rows, 0, 1);
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->q_full);
        }
        ++npub;
        return true;
      };
      const int64_t per = pl->per, begin = pl->begin, end = pl->end;
      int64_t first = pl->seg_begin;
      int tile0 = pl->seg_tile;
      const int s0 = pl->seg, known = pl->window;
      for (int s = s0; ok && first < end && s < p.P + p.B; ++s) {
        if (s - s0 >= known && ((s - s0) & 31) == 0) {  // the next 32 segments
          __syncwarp();
          if (s + lane < p.P + p.B) pl->segs[lane] = seg_plan(p, s + lane);
          __syncwarp();
        }
        const SegPlan g = pl->segs[(s - s0) & 31];
        const int nt = g.tiles;
        const bool varies = g.each < 0;
        int lo = g.lo, hi = g.hi;
        int64_t a = first;  // first unit of the row tile
        int gi = 0, t = 0;
        if (!varies) {
          if (g.each > 0 && begin > a) {  // skip whole row tiles before this CTA's share
            const int cost = tile_cost(g.each);
            const int64_t skip = min((begin - a) / cost, static_cast<int64_t>(nt) * p.Hkv);
            a += skip * cost;
            gi = static_cast<int>(skip / nt);
            t = static_cast<int>(skip - static_cast<int64_t>(gi) * nt);
          }
          if (g.each == 0) gi = p.Hkv;
        }
        for (; ok && gi < p.Hkv && a < end; ++gi, t = 0) {
          int64_t x0 = static_cast<int64_t>(t) * kRows;  // the tile's first row
          int i0 = static_cast<int>(x0 / p.R), h0 = static_cast<int>(x0 - static_cast<int64_t>(i0) * p.R);
          for (; ok && t < nt && a < end; ++t) {
            if (varies) tile_keys(p, g.s, t, lo, hi);
            const int n = varies ? tile_steps(lo, hi) : g.each;
            // units [a, a + kTileCost) carry no step
            const int64_t at = a + kTileCost;  // of step 0
            const int f0 = static_cast<int>(max(begin - at, static_cast<int64_t>(0)));
            const int f1 = static_cast<int>(min(end - at, static_cast<int64_t>(n)));
            if (f0 < f1) {
              Piece pc;
              pc.row = g.s.row;
              pc.own = g.s.own;
              pc.g = gi;
              pc.tok = g.s.tok0 + i0;
              pc.head = h0;
              pc.rows = static_cast<int>(min(static_cast<int64_t>(kRows), static_cast<int64_t>(g.s.ntok) * p.R - x0));
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
              if (f0 == 0 && lane == 0)
                meta[tile0 + gi * nt + t] = make_int2(
                    blockIdx.x, f1 < n ? static_cast<int>((at + n - 1) / per) - static_cast<int>(blockIdx.x) + 1 : 1);
              ok = publish(pc);
            }
            a += tile_cost(n);
            x0 += kRows;
            h0 += kRows;
            if (p.R < 2 * kRows) {
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
        first = varies ? a : first + static_cast<int64_t>(tile_cost(g.each)) * nt * p.Hkv;
        tile0 += nt * p.Hkv;
      }
      Piece last = {};
      last.row = -1;
      if (ok) publish(last);
    }
  } else {
    warpgroup_reg_alloc<kRegsHigh>();
    // ------------------------------------------------------------ softmax
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int r = quad * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    // z = out_scale * tanh(in_scale * x), or in_scale * x, in base-2 units
    const float in_scale = CAP ? p.sigma / p.softcap : p.sigma * kLog2e;
    const float out_scale = CAP ? p.softcap * kLog2e : 1.f;
    const float exp_scale = 2.f * kLog2e * in_scale;
    uint32_t take = 0, step = 0, tiles = 0;
    Piece pc;
    bool ok = true;
    while (ok) {
      if (!__all_sync(0xffffffffu, piece_take(&bars->ring, take, &pc, s_abort))) break;
      __syncwarp();
      if (lane == 0) piece_done(&bars->ring, take);
      if (pc.row < 0) break;
      if (tiles == 0) {
        copy_q_rows<HD>(p, sQ, pc.g, pc.tok, pc.head, pc.rows, warp - 4, 8);
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_first);
      }
      const bool valid = r < pc.rows;
      const bool any = quad * 32 < pc.rows;  // some row of this warp
      int tok = pc.tok, h = pc.head + r;     // packed token, head
      {
        const int dt = head_div(p, h);
        tok += dt;
        h += (pc.g - dt) * p.R;
      }
      // the row's own slope, and the keys [jlo, jhi] it may attend to; default
      // positions are counted from the segment's slot 0
      float slope2 = 0.f;
      int jlo = 0, jhi = pc.len - 1, pos = 0;
      bool kpos = false;
      const int32_t* kp = nullptr;
      if (POS) {
        const Table& t = pc.own ? p.own : p.prefix;
        const int base = pc.own ? pc.plen : 0;  // position of slot 0
        kpos = !FIXED && t.pos != nullptr;
        if (kpos) kp = t.pos + pc.row * t.pos_rs + pc.g * t.pos_hs;
        if (valid) {
          int b = pc.row;
          if (!pc.own) {
            const int b0 = __ldg(p.cu_prefix + pc.row), b1 = __ldg(p.cu_prefix + pc.row + 1);
            // one token each: no search
            b = b1 - b0 == pc.ntok && __ldg(p.cu_q + b0 + tok - pc.tok0) == tok &&
                        __ldg(p.cu_q + b0 + tok - pc.tok0 + 1) > tok
                    ? b0 + tok - pc.tok0
                    : seq_of(p.cu_q, b0, b1, tok);
          }
          if (p.slopes) slope2 = __ldg(p.slopes + b * p.slopes_bs + h) * kLog2e;
          if (p.q_pos)
            pos = __ldg(p.q_pos + tok) - (kpos ? 0 : base);
          else if (pc.own)
            pos = pc.len - pc.ntok + tok - pc.tok0;
          else
            pos = pc.plen + __ldg(p.own.lens + b) - (__ldg(p.cu_q + b + 1) - tok);
        }
        if (!kpos) {
          if (p.wl >= 0) jlo = max(jlo, pos - p.wl);
          if (p.wr >= 0) jhi = min(jhi, pos + p.wr);
        }
      }
      float m_run = -INFINITY;
      if (FIXED) {
        m_run = 0.f;
        if (POS && jlo <= jhi) {
          // the ALiBi term of the nearest (or, rising, the farthest) key: every
          // logit lies within the cap of it
          const int d = slope2 >= 0.f ? (pos < jlo ? jlo - pos : (pos > jhi ? pos - jhi : 0))
                                      : max(abs(pos - jlo), abs(pos - jhi));
          m_run = -slope2 * static_cast<float>(d);
        }
      }
      // subtracted from the logits; with FIXED they come without their constant c
      const float bref = FIXED ? m_run - out_scale : 0.f;
      uint64_t l2 = f2_make(0.f, 0.f);

      for (int kt = pc.kt0; kt < pc.kt1; ++kt, ++step) {
        const int key0 = kt * kKeys + half * 64;
        const uint32_t sb = tmem + (step & 1) * 128 + half * 64 + lane_addr;
        int kpa = 0, kpb = 0;
        if (POS && kpos) {
          kpa = __ldg(kp + min(key0 + lane, pc.len - 1));
          kpb = __ldg(kp + min(key0 + 32 + lane, pc.len - 1));
        }
        // the bounds are applied per key only where they cut some row's keys
        const bool edge = __any_sync(0xffffffffu, valid && (key0 < jlo || key0 + 63 > jhi));
        const bool behind = POS && __all_sync(0xffffffffu, !valid || pos >= key0 + 63);
        // base-2 logits (less bref) of columns [c0, c0 + 16) from their products
        auto logits16 = [&](float (&x)[kCh], int c0) {
          if (CAP) {
#pragma unroll
            for (int i = 0; i < kCh; i += 2) {
              if (FIXED) {
                // c - 2c / (1 + e^2x): the cap is small, so its absolute error of
                // c 2^-22 is that of the logit itself; the constant c is in bref
                const float d0 = 1.f + ex2_approx(fminf(x[i] * exp_scale, 60.f));
                const float d1 = 1.f + ex2_approx(fminf(x[i + 1] * exp_scale, 60.f));
                const float rc = rcp_approx(d0 * d1);
                x[i] = rc * d1;
                x[i + 1] = rc * d0;
                continue;
              }
              const uint64_t th = tanh2_fp32(f2_mul(f2_make(x[i], x[i + 1]), f2_make(in_scale, in_scale)));
              x[i] = f2_lo(th);
              x[i + 1] = f2_hi(th);
            }
          }
          const float sc = FIXED ? -2.f * out_scale : (CAP ? out_scale : in_scale);
          if (POS && kpos) {
#pragma unroll
            for (int i = 0; i < kCh; ++i) {
              const int kq = __shfl_sync(0xffffffffu, c0 < 32 ? kpa : kpb, (c0 & 31) + i);
              const bool adm = key0 + c0 + i < pc.len && (p.wl < 0 || kq >= pos - p.wl) &&
                               (p.wr < 0 || kq <= pos + p.wr);
              x[i] = adm ? fmaf(x[i], sc, -slope2 * static_cast<float>(abs(pos - kq))) : -INFINITY;
            }
            return;
          }
          if (POS && behind) {
            // every key stands at or before the row: the distance is linear
            const float a = fmaf(static_cast<float>(pos - key0 - c0), -slope2, -bref);
#pragma unroll
            for (int i = 0; i < kCh; i += 2) {
              const uint64_t z = f2_fma(f2_make(x[i], x[i + 1]), f2_make(sc, sc),
                                        f2_fma(f2_make(i, i + 1), f2_make(slope2, slope2), f2_make(a, a)));
              x[i] = f2_lo(z);
              x[i + 1] = f2_hi(z);
            }
          } else if (POS) {
            const float pos0 = static_cast<float>(pos - key0 - c0);
#pragma unroll
            for (int i = 0; i < kCh; i += 2) {
              const uint64_t dist = f2_make(fabsf(pos0 - i), fabsf(pos0 - (i + 1)));
              const uint64_t z = f2_fma(f2_make(x[i], x[i + 1]), f2_make(sc, sc),
                                        f2_fma(dist, f2_make(-slope2, -slope2), f2_make(-bref, -bref)));
              x[i] = f2_lo(z);
              x[i + 1] = f2_hi(z);
            }
          } else {
#pragma unroll
            for (int i = 0; i < kCh; i += 2) {
              const uint64_t z = f2_fma(f2_make(x[i], x[i + 1]), f2_make(sc, sc), f2_make(-bref, -bref));
              x[i] = f2_lo(z);
              x[i + 1] = f2_hi(z);
            }
          }
          if (edge) {
#pragma unroll
            for (int i = 0; i < kCh; ++i)
              x[i] = key0 + c0 + i >= jlo && key0 + c0 + i <= jhi ? x[i] : -INFINITY;
          }
        };
        if (!(ok = mbar_wait_warp(&bars->s_full[step & 1], (step >> 1) & 1, s_abort))) break;
        tc_fence_after();
        float alpha = 1.f;
        bool need = false;
        // without logits to keep, the second pass scales the products itself
        const bool keep = CAP || (POS && (kpos || p.slopes)) || edge || !(in_scale > 0.f);
        if (!FIXED) {
          float* mxs = sMax + (step & 1) * 256;
          float mx = -INFINITY;
          if (any) {
#pragma unroll 1
            for (int c0 = 0; c0 < 64; c0 += kCh) {
              float x[kCh];
              tmem_ld16(sb + c0, x);
              tmem_wait_ld();
              if (keep) {
                logits16(x, c0);
                tmem_st16(sb + c0, reinterpret_cast<uint32_t(&)[16]>(x));
              }
#pragma unroll
              for (int i = 0; i < kCh; ++i) mx = fmaxf(mx, x[i]);
            }
            if (keep)
              tmem_wait_st();
            else
              mx *= in_scale;
            mxs[half * 128 + r] = mx;
          }
          // the row's maximum over both halves
          if (!(ok = warp_exchange(&bars->mx_x[quad][step & 1], (step >> 1) & 1, s_abort))) break;
          if (any) {
            mx = fmaxf(mx, mxs[(half ^ 1) * 128 + r]);
            need = mx > m_run + kLazy;
            if (need) {
              alpha = ex2_approx(m_run - mx);
              m_run = mx;
            }
            l2 = f2_mul(l2, f2_make(alpha, alpha));
          }
        }
        if (any) {
          const float m_use = FIXED || m_run == -INFINITY ? 0.f : m_run;
          const float sc = keep ? 1.f : in_scale;
#pragma unroll 1
          for (int c0 = 0; c0 < 64; c0 += kCh) {
            float x[kCh];
            tmem_ld16(sb + c0, x);
            tmem_wait_ld();
            if (FIXED) logits16(x, c0);
            uint32_t pk[kCh / 2];
#pragma unroll
            for (int i = 0; i < kCh; i += 2) {
              uint64_t z = f2_make(x[i], x[i + 1]);
              if (!FIXED) z = f2_fma(z, f2_make(sc, sc), f2_make(-m_use, -m_use));
              const float e0 = ex2_approx(f2_lo(z)), e1 = ex2_approx(f2_hi(z));
              pk[i >> 1] = Pack<BF16>::two(e0, e1);
              l2 = f2_add(l2, f2_make(e0, e1));
            }
            tmem_st8(sb + c0 / 2, pk);
          }
          if (!FIXED && kt > pc.kt0 && __any_sync(0xffffffffu, need)) {
            // O follows the new reference, once the previous products are in
            // it: this half's features
            if (!(ok = mbar_wait_warp(&bars->pv_done[(step - 1) & 1], ((step - 1) >> 1) & 1, s_abort)))
              break;
            tc_fence_after();
            constexpr int kC = HD / 2;
            const uint32_t ob = tmem + kColOv + half * kC + lane_addr;
#pragma unroll 1
            for (int c = 0; c < kC; c += 16) {
              float o[16];
              tmem_ld16(ob + c, o);
              tmem_wait_ld();
              uint32_t u[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i] * alpha);
              tmem_st16(ob + c, u);
            }
            if (half) {  // and L
              uint32_t u[8];
              tmem_ld8(tmem + kColOv + HD + lane_addr, u);
              tmem_wait_ld();
              u[0] = __float_as_uint(__uint_as_float(u[0]) * alpha);
              tmem_st8(tmem + kColOv + HD + lane_addr, u);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[step & 1]);
      }
      if (!ok) break;
      // ---- the row's sum over both halves, then O
      float l = f2_lo(l2) + f2_hi(l2);
      float* sums = sSum + (tiles & 1) * 256;
      sums[half * 128 + r] = l;
      if (!(ok = warp_exchange(&bars->l_x[quad], tiles & 1, s_abort))) break;
      l = sums[r] + sums[128 + r];
      if (!(ok = mbar_wait_warp(&bars->o_full, tiles & 1, s_abort))) break;
      tc_fence_after();
      constexpr int kC = HD / 2;
      float o[kC], lr = 0.f;
      if (any) {
        uint32_t u[8];
        tmem_ld8(tmem + kColOv + HD + lane_addr, u);
        const uint32_t ob = tmem + kColOv + half * kC + lane_addr;
#pragma unroll
        for (int c = 0; c < kC; c += 16) tmem_ld16(ob + c, *reinterpret_cast<float(*)[16]>(o + c));
        tmem_wait_ld();
        lr = __uint_as_float(u[0]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->o_empty);
      ++tiles;
      if (!valid) continue;
      if (pc.mode == 0) {
        const float inv = lr > 0.f ? 1.f / lr : 0.f;
        if (half == 0)
          p.lse[static_cast<int64_t>(tok) * p.Hq + h] = l > 0.f ? (m_run + log2f(l)) * kLn2 : -INFINITY;
        uint16_t* orow = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(tok) * p.out_ts +
                         static_cast<int64_t>(h) * p.out_hs + half * kC;
#pragma unroll
        for (int u = 0; u < kC / 8; ++u) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = o[8 * u + i] * inv;
          *reinterpret_cast<uint4*>(orow + u * 8) = pack8<BF16>(v);
        }
      } else {
        const int64_t pr = pc.mode == 1 ? cut_row(w, blockIdx.x, pc.first, r)
                                        : whole_row(w, p.total_q, p.Hq, pc.own, tok, h);
        if (half == 0) reinterpret_cast<float4*>(p.ws + w.stats)[pr] = make_float4(m_run, l, lr, 0.f);
        float4* part = reinterpret_cast<float4*>(p.ws + w.rows) + part_at<HD>(pr, half * kC / 4);
#pragma unroll
        for (int u = 0; u < kC / 4; ++u)
          part[u * 8] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
      }
    }
  }
  __syncthreads();
  if (tid == 0 && *s_abort) report(p.status, ATTN_DEV_TIMEOUT_FWD);
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <bool B, int HD>
auto pick_fwd(const CacheParams& p) {
  const bool moved = p.own.pos || (p.P && p.prefix.pos);
  const bool pos = p.slopes || p.wl >= 0 || p.wr >= 0 || moved;
  if (!(p.softcap > 0.f))
    return pos ? cache_fwd_kernel<B, HD, false, false, true>
               : cache_fwd_kernel<B, HD, false, false, false>;
  if (p.softcap <= kFixedCap && !moved)
    return pos ? cache_fwd_kernel<B, HD, true, true, true>
               : cache_fwd_kernel<B, HD, true, true, false>;
  return pos ? cache_fwd_kernel<B, HD, true, false, true>
             : cache_fwd_kernel<B, HD, true, false, false>;
}

template <int HD>
cudaError_t launch_fwd_d(const CacheParams& p, const FwdWs& w, const CUtensorMap& tk, const CUtensorMap& tkt,
                         const CUtensorMap& tv, int grid, cudaStream_t s) {
  constexpr uint32_t smem = FwdShape<HD>::kOffBar + sizeof(FwdBars);
  static_assert(smem <= 232448, "shared memory");
  auto k = p.dtype == 1 ? pick_fwd<true, HD>(p) : pick_fwd<false, HD>(p);
  cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  k<<<grid, kThreads, smem, s>>>(p, w, tk, tkt, tv);
  return cudaGetLastError();
}

}  // namespace kv
}  // namespace attn
