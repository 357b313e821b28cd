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
// and two row sums in fp32 in the softmax warps: l of P, which gives lse, and lr
// of the rounded P that multiplies V, which divides O, so that out is a weighted
// mean of V rows whatever the roundings: equal rows come out exactly.  (lr takes 8
// % of a capped call of drafts, nothing of one with short steps; as a product
// with a tile of ones it doubled the time of P V.)  P has V's 16-bit type because
// the tensor core takes one type for both: out's error against 64 bits is 0.0023
// of its size with bf16 weights all alike (0.0019 where few are large), of which
// 0.0017 are the rounding of out itself.
//
// Single-token calls read every K and V row once for R <= 128 rows of a group,
// so the copies bound them; calls with many rows behind a shared prefix are
// bound by the softmax warps' MUFU work and the hand-offs between them and
// the tensor core, as the packed forward is.
//
// Warps (512 threads): 0 loads K and 12 loads V by TMA, a box of min(page_size,
// 128) rows x 64 features per lane; 1 issues S, 2 issues O and L and clears the
// V rows of a cut tile that no row reads (the pages may hold anything there,
// and 0 * NaN would reach O); 3 plans the CTA's pieces; 13-15 gather Q rows with
// cp.async into the swizzled layout (a row is any (token, head), so TMA boxes
// do not fit); 4-11 softmax, two per TMEM lane quadrant, each taking 64 of a
// step's keys in passes of 16.  The passes are rolled loops: straight-line code
// for all columns cost 8000 to 11000 clk of instruction fetches on a CTA's
// first step and slowed the rest; four warps per quadrant with 32 keys each
// gained nothing.
//
// Measured with the join: 64 single tokens over 270000 keys in 16-row pages 54.5
// us (3.2 TB/s; 26 us would be the copy's rate), 128 behind an 8200-key prefix 101
// us, 144 drafted tokens behind two prefixes of 12001 keys 178 us (691 TFLOP/s).
#pragma once
#include "cache_piece.cuh"

namespace attn {
namespace kv {

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
  static constexpr uint32_t kOffSum = kOffMax + 2 * 2 * 128 * 4;  // [2 pieces][2 halves][128] (l, lr)
  static constexpr uint32_t kOffBar = kOffSum + 2 * 2 * 128 * 8;
};

struct FwdBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint32_t gone[8];  // of a step's key tile: load boxes whose page is out of the pool
  uint64_t o_full, o_empty, drain;
  uint64_t mx_x[4][2], l_x[4];
  PieceRing ring;
  Plan plan;
  uint32_t tmem;
  int abort;
};

constexpr int kThreadsF = 512;
// registers per thread of warps 0-3, 4-11 and 12-15 (launched at 128)
constexpr int kRegsPlan = 96, kRegsSoft = 168, kRegsLoad = 80;
static_assert(kRegsPlan + 2 * kRegsSoft + kRegsLoad <= 4 * 128, "register split exceeds the launch");
constexpr uint32_t kColOv = 256;  // TMEM: S0 / P0 [0,128), S1 / P1 [128,256), O [256, 256 + d)
constexpr float kLazy = 8.f;                    // rescale when the maximum grows by more (base 2)
constexpr float kFixedCap = 9.5f;               // largest cap with a reference known beforehand

// One warp: the key tiles of every piece into the K (or V) stages, a box per
// lane.
template <int HD, bool K>
__device__ __forceinline__ void load_pages(const CacheParams& p, FwdBars* bars, uint8_t* dst0,
                                           const CUtensorMap* map, const CUtensorMap* tail, int box,
                                           volatile int* s_abort) {
  using S = FwdShape<HD>;
  constexpr int kStages = K ? S::kKS : S::kVS;
  constexpr uint32_t kBytes = K ? S::kQ : S::kV;  // of a whole tile
  const int lane = threadIdx.x & 31;
  uint64_t* full = K ? bars->k_full : bars->v_full;
  uint64_t* empty = K ? bars->k_empty : bars->v_empty;
  const int pieces = kKeys / box, ch = lane / pieces, pi = lane - ch * pieces;  // (chunk, row block)
  uint32_t take = 0, st = 0, ph = 0, loaded = 0;
  Piece pc;
  bool ok = true;
  while (ok) {
    if (!__all_sync(0xffffffffu, piece_take(&bars->ring, take, &pc, s_abort))) break;
    __syncwarp();
    if (lane == 0) piece_done(&bars->ring, take);
    if (pc.row < 0) break;
    const Table& t = pc.own ? p.own : p.prefix;
    const int32_t* row = t.pages + pc.row * t.rs;
    auto page_of = [&](int kt) {  // this lane's page of key tile kt, or -1: no box
      const int key = kt * kKeys + pi * box;
      return ch < S::kChunksK && kt >= pc.kt0 && key < pc.len ? tile_page(p, row, key) : -1;
    };
    int page = page_of(pc.kt1 - 1);
    for (int kt = pc.kt1 - 1; kt >= pc.kt0; --kt) {
      const int key0 = kt * kKeys;
      const int have = min(pieces, (pc.len - key0 + box - 1) / box);  // row blocks in use
      const int next = page_of(kt - 1);  // read while this tile's stage is waited for
      if (loaded >= kStages && !(ok = mbar_wait_warp(&empty[st], ph ^ 1, s_abort))) break;
      if (K) {
        // Pages out of the pool are loaded as zeros; their keys are masked by this.
        // Eight entries: the load of a step waits for the product at most six before,
        // which waited for the softmax two before that.
        static_assert(!K || kStages + 2 <= 8, "an entry could still be read");
        const uint32_t gone = __ballot_sync(0xffffffffu, ch == 0 && page == p.num_pages);
        if (lane == 0) bars->gone[loaded & 7] = gone;
      }
      if (lane == 0) mbar_arrive_expect_tx(&full[st], kBytes / pieces * have);
      __syncwarp();
      if (page >= 0) {
        uint8_t* dst = dst0 + st * kBytes;
        const int slot = p.page_size > kKeys ? key0 & (p.page_size - 1) : 0;
        if (K && HD == 160 && ch == 2)
          tma_load_4d(dst + 2 * 16384 + pi * box * 64, tail, &full[st], 128, pc.g, slot, page);
        else
          tma_load_4d(dst + ch * 16384 + pi * box * 128, map, &full[st], ch * kChunk, pc.g, slot, page);
      }
      page = next;
      ++loaded;
      if (++st == kStages) {
        st = 0;
        ph ^= 1;
      }
    }
  }
  if (*s_abort && lane == 0) {  // let every load land before the CTA exits
    const uint32_t n = min(loaded, static_cast<uint32_t>(kStages));
    for (uint32_t f = loaded - n; f < loaded; ++f) wait_drain(&full[f % kStages], (f / kStages) & 1);
  }
}

// CAP: the call has a softcap; FIXED: of at most kFixedCap and default key
// positions, so P is taken against a bound and no maximum is tracked; POS:
// the call has ALiBi, a mask or key positions.
template <bool BF16, int HD, bool CAP, bool FIXED, bool POS>
__global__ void __launch_bounds__(kThreadsF, 1)
    cache_fwd_kernel(const __grid_constant__ CacheParams p, const __grid_constant__ FwdWs w,
                     const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tkt, const __grid_constant__ CUtensorMap tv) {
  using S = FwdShape<HD>;
  constexpr int kCh = 16;  // columns of a softmax pass
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t* sQ = sm;
  uint8_t* sK = sm + S::kOffK;
  uint8_t* sV = sm + S::kOffV;
  float* sMax = reinterpret_cast<float*>(sm + S::kOffMax);
  float2* sSum = reinterpret_cast<float2*>(sm + S::kOffSum);
  FwdBars* bars = reinterpret_cast<FwdBars*>(sm + S::kOffBar);
  volatile int* s_abort = &bars->abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int2* meta = reinterpret_cast<int2*>(p.ws + w.meta);
  if (tid == 0) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    mbar_init(&bars->q_full, 3);
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
      mbar_init(&bars->s_full[b], 2);  // the products, and the issuer (which has seen `gone`)
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
      mbar_init(&bars->ring.empty[s], 15);  // K and V loads, two MMA issuers, 8 softmax, 3 Q warps
    }
    fence_barrier_init();
    bars->abort = 0;
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  if (warp == 13 && lane == 0) {
    prefetch_tensormap(&tk);
    prefetch_tensormap(&tv);
    if (HD == 160) prefetch_tensormap(&tkt);
  }
  tc_fence_before();

  // ---- this CTA's share of the steps
  Plan* pl = &bars->plan;
  const bool busy = make_plan(
      p, pl, [&](int s) { return seg_plan(p, s); },
      [&](const SegPlan& g) -> int64_t { return seg_cost(p, g) * p.Hkv; });
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  if (blockIdx.x == 0 && tid == 0) {
    FwdHead* head = reinterpret_cast<FwdHead*>(p.ws);
    int ok = pl->bad == 0;
    if (smem_addr(sm) & 1023u) {
      report(p.status, ATTN_DEV_SMEM_ALIGN);
      ok = 0;
    }
    head->ok = ok;
  }
  if (!busy || (smem_addr(sm) & 1023u)) {  // uniform
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }
  const int box = min(p.page_size, kKeys), box_log2 = min(p.page_log2, 7);  // rows of a load box

  if (warp < 4) {
    warpgroup_reg_dealloc<kRegsPlan>();
    if (warp == 0) {
      // ------------------------------------------------------------ K loads
      load_pages<HD, true>(p, bars, sK, &tk, &tkt, box, s_abort);
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
          if (!mbar_wait(&bars->q_full, tiles & 1, s_abort)) break;
          for (int kt = pc.kt1 - 1; kt >= pc.kt0; --kt, ++step) {
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
            mbar_arrive(&bars->s_full[step & 1]);
            umma_commit(&bars->k_empty[st]);
            if (kt == pc.kt0) umma_commit(&bars->q_empty);
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
      uint32_t take = 0, step = 0, st = 0, ph = 0, tiles = 0;
      Piece pc;
      bool ok = true;
      while (ok) {
        if (!__all_sync(0xffffffffu, piece_take(&bars->ring, take, &pc, s_abort))) break;
        __syncwarp();
        if (lane == 0) piece_done(&bars->ring, take);
        if (pc.row < 0) break;
        for (int kt = pc.kt1 - 1; kt >= pc.kt0; --kt, ++step) {
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
          const bool first = kt == pc.kt1 - 1;
          if (first && tiles > 0 &&
              !(ok = mbar_wait_warp(&bars->o_empty, (tiles - 1) & 1, s_abort)))
            break;
          if (lane == 0) {
            tc_fence_after();
            const uint32_t vb = smem_addr(sV + st * S::kV);
            // keys 16k .. 16k + 15: pair columns 8 (k mod 4) of half k / 4
            for (int k = 0; k < ksteps; ++k)
              umma_ts(tmem + kColOv, tmem + (step & 1) * 128 + (k >> 2) * 64 + (k & 3) * 8,
                      sdesc_sw128(vb + k * 2048, 16384, 1024), kIdO, (!first || k > 0));
            umma_commit(&bars->pv_done[step & 1]);
            umma_commit(&bars->v_empty[st]);
            if (kt == pc.kt0) umma_commit(&bars->o_full);
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
      // ------------------------------------------------------------ plan
      plan_pieces(p, pl, &bars->ring, s_abort);
    }
  } else if (warp < 12) {
    warpgroup_reg_alloc<kRegsSoft>();
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
      const bool valid = r < pc.rows;
      const bool any = quad * 32 < pc.rows;  // some row of this warp
      int tok = pc.tok, h = pc.head + r;     // packed token, head
      {
        const int dt = head_div(p, h);
        tok += dt;
        h += (pc.g - dt) * p.R;
      }
      if (pc.first && valid && half == 0)
        meta[(static_cast<int64_t>(pc.own ? 0 : p.total_q) + tok) * p.Hq + h] = make_int2(blockIdx.x, pc.parts);
      // the row's own slope, and the keys [jlo, jhi] it may attend to; default
      // positions are counted from the segment's slot 0
      float slope2 = 0.f, m0 = 0.f;  // m0: ALiBi term common to all keys
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
            pos = pc.plen + seg_len(p, true, b) - (__ldg(p.cu_q + b + 1) - tok);
        }
        if (!kpos) {
          if (p.wl >= 0) jlo = max(jlo, pos - p.wl);
          if (p.wr >= 0) jhi = min(jhi, pos + p.wr);
          // A row that stands beyond its keys is moved up to them (their tile's
          // end), and what that takes off every distance is added to the result: the
          // distances of far positions would lose their last bits in fp32, and
          // logits near 2^24 the reference's.
          if (p.slopes && jlo <= jhi) {
            const int to = min(max(pos, jlo), jhi | (kKeys - 1));
            m0 = -slope2 * static_cast<float>(abs(pos - to));
            pos = to;
          }
        }
      }
      const int32_t* pages = pc.own ? p.own.pages + pc.row * p.own.rs : p.prefix.pages + pc.row * p.prefix.rs;
      auto no_page = [&](int j) {
        return static_cast<unsigned>(__ldg(pages + (j >> p.page_log2))) >= static_cast<unsigned>(p.num_pages);
      };
      float m_run = -INFINITY;
      if (FIXED) {
        m_run = 0.f;
        if (POS && p.slopes && jlo <= jhi) {
          // the ALiBi term of the nearest (or, rising, the farthest) key that has a
          // page: every logit lies within the cap of it
          const bool near = slope2 >= 0.f;
          int a = near ? min(pos, jhi) : jhi, b = near ? max(pos, jlo) : jlo;
          while (a >= jlo && no_page(a)) a = (a >> p.page_log2 << p.page_log2) - 1;
          while (b <= jhi && no_page(b)) b = ((b >> p.page_log2) + 1) << p.page_log2;
          const int da = a >= jlo ? abs(pos - a) : -1, db = b <= jhi ? abs(pos - b) : -1;
          const int d = near && da >= 0 && db >= 0 ? min(da, db) : max(max(da, db), 0);
          m_run = -slope2 * static_cast<float>(d);
        }
      }
      // subtracted from the logits; with FIXED they come without their constant c
      float bref = FIXED ? m_run - out_scale : 0.f;
      uint64_t l2 = f2_make(0.f, 0.f), lr2 = l2;  // of P, and of the rounded P

      for (int kt = pc.kt1 - 1; kt >= pc.kt0; --kt, ++step) {
        const int key0 = kt * kKeys + half * 64;
        const uint32_t sb = tmem + (step & 1) * 128 + half * 64 + lane_addr;
        int kpa = 0, kpb = 0;
        if (POS && kpos) {
          kpa = __ldg(kp + min(key0 + lane, pc.len - 1));
          kpb = __ldg(kp + min(key0 + 32 + lane, pc.len - 1));
        }
        // the bounds are applied per key only where they cut some row's keys
        bool edge = __any_sync(0xffffffffu, valid && (key0 < jlo || key0 + 63 > jhi));
        uint32_t gone = 0;  // a bit per load box of keys without a page
        const bool behind = POS && __all_sync(0xffffffffu, !valid || pos >= key0 + 63);
        // without logits to keep, both passes read the products and scale themselves
        const bool keep = CAP || (POS && (kpos || p.slopes)) || !(in_scale > 0.f);
        auto no_box = [&](int c0) { return gone >> ((half * 64 + c0) >> box_log2) & 1; };
        auto mask = [&](auto& x, int c0, int n) {
          const int lo = no_box(c0) ? n : jlo - key0 - c0, hi = jhi - key0 - c0;
#pragma unroll
          for (int i = 0; i < n; ++i) x[i] = i >= lo && i <= hi ? x[i] : -INFINITY;
        };
        // base-2 logits (less bref) of columns [c0, c0 + 16) from their products
        auto logits16 = [&](float (&x)[16], int c0) {
          if (CAP) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
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
            const int len = no_box(c0) ? 0 : pc.len;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int kq = __shfl_sync(0xffffffffu, c0 < 32 ? kpa : kpb, (c0 & 31) + i);
              const bool adm = key0 + c0 + i < len && (p.wl < 0 || kq >= pos - p.wl) &&
                               (p.wr < 0 || kq <= pos + p.wr);
              x[i] = adm ? fmaf(x[i], sc, -slope2 * static_cast<float>(abs(pos - kq))) : -INFINITY;
            }
            return;
          }
          if (POS && behind) {
            // every key stands at or before the row: the distance is linear
            const float a = fmaf(static_cast<float>(pos - key0 - c0), -slope2, -bref);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const uint64_t z = f2_fma(f2_make(x[i], x[i + 1]), f2_make(sc, sc),
                                        f2_fma(f2_make(i, i + 1), f2_make(slope2, slope2), f2_make(a, a)));
              x[i] = f2_lo(z);
              x[i + 1] = f2_hi(z);
            }
          } else if (POS) {
            const float pos0 = static_cast<float>(pos - key0 - c0);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const uint64_t dist = f2_make(fabsf(pos0 - i), fabsf(pos0 - (i + 1)));
              const uint64_t z = f2_fma(f2_make(x[i], x[i + 1]), f2_make(sc, sc),
                                        f2_fma(dist, f2_make(-slope2, -slope2), f2_make(-bref, -bref)));
              x[i] = f2_lo(z);
              x[i + 1] = f2_hi(z);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const uint64_t z = f2_fma(f2_make(x[i], x[i + 1]), f2_make(sc, sc), f2_make(-bref, -bref));
              x[i] = f2_lo(z);
              x[i + 1] = f2_hi(z);
            }
          }
          if (edge) mask(x, c0, 16);
        };
        if (!(ok = mbar_wait_warp(&bars->s_full[step & 1], (step >> 1) & 1, s_abort))) break;
        tc_fence_after();
        gone = bars->gone[step & 7];
        edge = edge || gone;
        float alpha = 1.f;
        bool need = false;
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
              } else if (edge) {
                mask(x, c0, kCh);
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
            lr2 = f2_mul(lr2, f2_make(alpha, alpha));
          }
        }
        // With FIXED, the first tile's maximum becomes the reference: the largest
        // weight of most rows is then exactly 1.  The tile is passed over twice
        // for that.  A later logit may lie as high as the cap above the ALiBi
        // term of the nearest key, so the reference stays within 15 of that and
        // no P passes 2^15; the row's largest is at least 2^-12.5 then (caps up to
        // 9.5), which 16 bits hold.
        if (FIXED && kt == pc.kt1 - 1) {
          float mx = -INFINITY;
          if (any) {
#pragma unroll 1
            for (int c0 = 0; c0 < 64; c0 += kCh) {
              float x[kCh];
              tmem_ld16(sb + c0, x);
              tmem_wait_ld();
              logits16(x, c0);
#pragma unroll
              for (int i = 0; i < kCh; ++i) mx = fmaxf(mx, x[i]);
            }
          }
          float* mxs = sMax + (tiles & 1) * 256;
          mxs[half * 128 + r] = mx;
          if (!(ok = warp_exchange(&bars->mx_x[quad][tiles & 1], (tiles >> 1) & 1, s_abort))) break;
          const float up = fmaxf(fmaxf(mx, mxs[(half ^ 1) * 128 + r]), out_scale - 15.f);
          m_run += up;
          bref += up;
        }
        if (any) {
          const float m_use = FIXED || m_run == -INFINITY ? 0.f : m_run;
          const float sc = keep ? 1.f : in_scale;
#pragma unroll 1
          for (int c0 = 0; c0 < 64; c0 += kCh) {
            float x[kCh];
            tmem_ld16(sb + c0, x);
            tmem_wait_ld();
            if constexpr (FIXED) logits16(x, c0);
            if (!keep && edge) mask(x, c0, kCh);
            uint32_t pk[kCh / 2];
#pragma unroll
            for (int i = 0; i < kCh; i += 2) {
              uint64_t z = f2_make(x[i], x[i + 1]);
              if (!FIXED) z = f2_fma(z, f2_make(sc, sc), f2_make(-m_use, -m_use));
              const float e0 = ex2_approx(f2_lo(z)), e1 = ex2_approx(f2_hi(z));
              pk[i >> 1] = Pack<BF16>::two(e0, e1);
              l2 = f2_add(l2, f2_make(e0, e1));
              lr2 = f2_add(lr2, Pack<BF16>::unpack(pk[i >> 1]));
            }
            tmem_st8(sb + c0 / 2, pk);
          }
          if (!FIXED && kt < pc.kt1 - 1 && __any_sync(0xffffffffu, need)) {
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
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[step & 1]);
      }
      if (!ok) break;
      // ---- the row's sums over both halves, then O
      float2* sums = sSum + (tiles & 1) * 256;
      sums[half * 128 + r] = make_float2(f2_lo(l2) + f2_hi(l2), f2_lo(lr2) + f2_hi(lr2));
      if (!(ok = warp_exchange(&bars->l_x[quad], tiles & 1, s_abort))) break;
      const float l = sums[r].x + sums[128 + r].x, lr = sums[r].y + sums[128 + r].y;
      if (!(ok = mbar_wait_warp(&bars->o_full, tiles & 1, s_abort))) break;
      tc_fence_after();
      if (any) {
        constexpr int kC = HD / 2;
        const float inv = lr > 0.f ? 1.f / lr : 0.f;
        int64_t pr = 0;
        if (pc.mode)
          pr = pc.mode == 1 ? cut_row(w, blockIdx.x, pc.first, r) : whole_row(w, p.total_q, p.Hq, pc.own, tok, h);
        if (valid && half == 0) {
          if (pc.mode)
            reinterpret_cast<float4*>(p.ws + w.stats)[pr] = make_float4(m_run, l, lr, m0);
          else
            p.lse[static_cast<int64_t>(tok) * p.Hq + h] = l > 0.f ? (m_run + log2f(l) + m0) * kLn2 : -INFINITY;
        }
        uint16_t* orow = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(tok) * p.out_ts +
                         static_cast<int64_t>(h) * p.out_hs + half * kC;
        float4* part = reinterpret_cast<float4*>(p.ws + w.rows) + part_at<HD>(pr, half * kC / 4);
#pragma unroll 1
        for (int c = 0; c < kC; c += 16, part += 32) {
          float o[16];
          tmem_ld16(tmem + kColOv + half * kC + c + lane_addr, o);
          tmem_wait_ld();
          if (!valid) continue;
          if (pc.mode == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= inv;
            *reinterpret_cast<uint4*>(orow + c) = pack8<BF16>(o);
            *reinterpret_cast<uint4*>(orow + c + 8) = pack8<BF16>(o + 8);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              part[i * 8] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->o_empty);
      ++tiles;
    }
  } else {
    warpgroup_reg_dealloc<kRegsLoad>();
    if (warp == 12) {
      // ------------------------------------------------------------ V loads
      load_pages<HD, false>(p, bars, sV, &tv, nullptr, box, s_abort);
    } else {
      // ------------------------------------------------------------ Q rows
      uint32_t take = 0, tiles = 0;
      Piece pc;
      for (;;) {
        if (!__all_sync(0xffffffffu, piece_take(&bars->ring, take, &pc, s_abort))) break;
        __syncwarp();
        if (lane == 0) piece_done(&bars->ring, take);
        if (pc.row < 0) break;
        if (tiles > 0 && !mbar_wait_warp(&bars->q_empty, (tiles - 1) & 1, s_abort)) break;
        copy_q_rows<HD>(p, sQ, pc.g, pc.tok, pc.head, pc.rows, warp - 13, 3);
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_full);
        ++tiles;
      }
    }
  }
  __syncthreads();
  if (tid == 0 && *s_abort) report(p.status, ATTN_DEV_TIMEOUT_FWD);
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// A softcap of at most kFixedCap at default key positions.
inline bool fixed_reference(const CacheParams& p) {
  return p.softcap > 0.f && p.softcap <= kFixedCap && !p.own.pos && !(p.P && p.prefix.pos);
}

template <bool B, int HD>
auto pick_fwd(const CacheParams& p) {
  const bool moved = p.own.pos || (p.P && p.prefix.pos);
  const bool pos = p.slopes || p.wl >= 0 || p.wr >= 0 || moved;
  if (!(p.softcap > 0.f))
    return pos ? cache_fwd_kernel<B, HD, false, false, true>
               : cache_fwd_kernel<B, HD, false, false, false>;
  if (fixed_reference(p))
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
  k<<<grid, kThreadsF, smem, s>>>(p, w, tk, tkt, tv);
  return cudaGetLastError();
}

}  // namespace kv
}  // namespace attn
