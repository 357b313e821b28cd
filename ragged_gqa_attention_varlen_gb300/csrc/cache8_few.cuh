// cache8_few.cuh -- attention over the 8-bit cache for few query rows a key: the
// single tokens of grouped heads.
//
// With up to 16 rows a key, the tiles of cache8_fwd.cuh are nearly empty, and
// their hand-offs between loads, tensor core, softmax and conversion, not the
// pages' bytes, are what a step waits for (3700 clk a step of 128 keys where the
// copy's rate would take 1400).  Here a warp does everything for 32 keys at a time,
// in registers, with the warp-level product m16n8k16:
//   S^T = K Q^T     16 keys x 8 rows: a lane's 16 bytes of a key row widen to its
//                   operands of four products; the features of a product may stand
//                   in any order, as long as Q's do too
//   P = 2^(z - m)   turned over eight by eight (movmatrix)
//   O^T += V^T P^T  16 features x 8 rows: bytes of two keys' rows are interleaved
//                   and widened; which features a lane holds is free again
// Keys and features lie along the 16 because these products run at 1/16 of
// tcgen05's rate here: with the rows along the 16 the tensor pipe took 420 clk for
// 32 keys, above the 350 of the copy's rate.  The warps of a CTA take its 32-key
// chunks in turn.  At the end of a piece they leave their O to a warp that adds them
// up while they go on.  Keys 2i and 2i + 1 of a product are rows 2i and (2i + 5) mod
// 8 of eight: with the copies' 128-byte swizzle, K's and V's loads then meet no bank
// twice.
//
// Bound by the pages' bytes: no value is touched by more than one warp, and the
// loads run up to 16 chunks (131 KB at d = 128) ahead.
//
// q enters in fp16, bf16 rows times a power of two for each (their 8 bits fit);
// K's scale goes to the logits and V's to the weights, over a power of two that
// follows the largest of them; where that would take the weights below 2^-12, O is
// scaled up around the product instead.
//
// Warps: 8 compute, four load in turn (one takes 1900 clk for 64 keys), one joins and
// one plans the pieces.
//
// Measured with the join: 96 single tokens of 32 heads over 8 (d = 128, bf16, 490 MB)
// 103 us, 4.8 TB/s; by the tiles of 128 rows 268 us.  One loading warp 249, three 151.
#pragma once
#include <cuda_fp8.h>

#include "cache8_wait.cuh"

namespace attn {
namespace kv {

constexpr int kFewRows = 8;   // rows of a tile
constexpr int kFewKeys = 32;  // keys of a chunk
constexpr int kFewLoad = 64;  // keys that are loaded together
constexpr int kFewLoads = 4;  // loading warps
constexpr int kFewWarps = 8, kFewThreads = (kFewWarps + kFewLoads + 2) * 32;

template <int HD>
struct FewShape {
  static constexpr uint32_t kBytes = kFewLoad * HD;           // of K or V of a stage
  static constexpr int kStages = HD == 64 ? 16 : 8;
  // A wait tells phases of a barrier apart by their parity, so it may only wait for
  // the phase after the last one it has seen: every half of a stage is always the
  // same warp's, and every stage the same loading warp's.  (With stages that went
  // from warp to warp, a warp could meet a stage whose previous load had not landed
  // and take the one before that for its own.)
  static_assert(2 * kStages % kFewWarps == 0 && kStages % kFewLoads == 0, "a stage's warps change");
  static constexpr uint32_t kOffPart = kStages * 2 * kBytes;  // [warps][8 rows][HD] fp32
  static constexpr uint32_t kOffBar = kOffPart + kFewWarps * 8 * HD * 4;
  static constexpr int kSteps = HD / 16;  // products of S along the features
  static constexpr int kCols = HD / 16;   // tiles of features of O
};

struct FewBars {
  uint64_t full[16], empty[16];
  uint64_t done, taken;            // O of a piece's warps: left, added up
  alignas(16) float scale[16][8];  // of a stage: K scales of its four 16 keys, V scales
  uint32_t gone[16];               // of a stage: bit i: its i-th 16 keys have no page
  alignas(16) float4 stat[kFewWarps][8];  // (reference, sum, sum of the rounded weights, -) of a row in each warp
  float m0[8];                     // ALiBi term common to a row's keys
  PieceRing ring;
  Plan plan;
  int abort;
};

// An 8 x 8 matrix of 16-bit values, two of a row in a lane, turned over.
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The two halves of a word of e4m3 in fp16.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Four warps in turn: the 64 keys of every fourth stage, in boxes of min(page_size,
// 64) rows; lanes 0 .. 7 take a scale each.  The pages of 8 stages ahead are looked up
// together, 16 keys a lane.  One lane issues all boxes: lanes that issue one each go
// through the copy instruction one by one (500 clk a box).
template <int HD>
__device__ __forceinline__ void few_load(const Cache8Params& p8, FewBars* bars, uint8_t* sm, const CUtensorMap* tk,
                                         const CUtensorMap* tkt, const CUtensorMap* tv, const CUtensorMap* tvt, int wi,
                                         volatile int* s_abort) {
  using S = FewShape<HD>;
  const CacheParams& p = p8.c;
  const int lane = threadIdx.x & 31;
  const int box = min(p.page_size, kFewLoad), boxes = kFewLoad / box;  // rows of a box; boxes of a stage
  uint32_t take = 0, i = 0;
  Piece pc;
  bool ok = true;
  while (ok) {
    if (!__all_sync(0xffffffffu, piece_take8(&bars->ring, take, &pc, s_abort))) break;
    __syncwarp();
    if (lane == 0) piece_done(&bars->ring, take);
    if (pc.row < 0) break;
    const Table& t = pc.own ? p.own : p.prefix;
    const int32_t* row = t.pages + pc.row * t.rs;
    const int c0 = pc.kt0 * 2, c1 = min(pc.kt1 * 2, (pc.len + kFewLoad - 1) / kFewLoad);
    int pages = 0;
    for (int c = c1 - 1; c >= c0; --c, ++i) {
      const int ahead = (c1 - 1 - c) & 7;
      if (ahead == 0) {  // of stage c - lane / 4: the page of its 16 keys lane mod 4, -1 beyond the end
        const int key = (c - (lane >> 2)) * kFewLoad + (lane & 3) * 16;
        pages = c - (lane >> 2) >= c0 && key < pc.len ? tile_page(p, row, key) : -1;
      }
      if (i % kFewLoads != static_cast<uint32_t>(wi)) continue;
      const int mine16 = __shfl_sync(0xffffffffu, pages, ahead * 4 + (lane & 3));  // of 16 keys lane mod 4
      const uint32_t st = i % S::kStages;
      if (i >= S::kStages && !(ok = mbar_wait8_warp(&bars->empty[st], (i / S::kStages - 1) & 1, s_abort))) break;
      const int key0 = c * kFewLoad;
      const uint32_t gone = __ballot_sync(0xffffffffu, mine16 == p.num_pages) & 15u;
      if (lane < 8) {
        const int key = key0 + (lane & 3) * 16;
        const Scales& sc = lane < 4 ? p8.ks : p8.vs;
        const bool there = mine16 >= 0 && mine16 < p.num_pages;
        const int64_t at = there ? mine16 * sc.page + static_cast<int64_t>((key & (p.page_size - 1)) >> p8.block_log2) * sc.block + pc.g * sc.head : 0;
        cp_async4_or_zero(&bars->scale[st][lane], sc.base + at, there);
        cp_async_arrive(&bars->full[st]);
      }
      const int have = min(boxes, (pc.len - key0 + box - 1) / box);  // boxes in use
      if (lane == 0) {
        bars->gone[st] = gone;
        mbar_arrive_expect_tx(&bars->full[st], have * box * HD * 2);
      }
      __syncwarp();
      for (int b = 0; b < have; ++b) {
        const int page = __shfl_sync(0xffffffffu, mine16, b * box >> 4);
        if (lane == 0) {
          uint8_t* dst = sm + st * 2 * S::kBytes;
          const int slot = key0 & (p.page_size - 1) & ~(box - 1);
          constexpr int kRow = HD == 64 ? 64 : 128;
          tma_load_4d(dst + b * box * kRow, tk, &bars->full[st], 0, pc.g, slot, page);
          tma_load_4d(dst + S::kBytes + b * box * kRow, tv, &bars->full[st], 0, pc.g, slot, page);
          if (HD == 160) {
            tma_load_4d(dst + kFewLoad * 128 + b * box * 32, tkt, &bars->full[st], 128, pc.g, slot, page);
            tma_load_4d(dst + S::kBytes + kFewLoad * 128 + b * box * 32, tvt, &bars->full[st], 128, pc.g, slot, page);
          }
        }
        __syncwarp();
      }
    }
  }
  if (*s_abort && lane == 0) {  // let every load land before the CTA exits
    const uint32_t n = min(i, static_cast<uint32_t>(S::kStages));
    for (uint32_t f = i - n; f < i; ++f)
      if (f % kFewLoads == static_cast<uint32_t>(wi)) wait_drain(&bars->full[f % S::kStages], (f / S::kStages) & 1);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// One warp: adds up what a piece's warps left, in their order.
template <bool BF16, int HD>
__device__ __forceinline__ void few_join(const CacheParams& p, const FwdWs& w, FewBars* bars, const float* part,
                                         volatile int* s_abort) {
  const int lane = threadIdx.x & 31;
  uint32_t take = 0, round = 0;
  Piece pc;
  for (;;) {
    if (!__all_sync(0xffffffffu, piece_take8(&bars->ring, take, &pc, s_abort))) return;
    __syncwarp();
    if (lane == 0) piece_done(&bars->ring, take);
    if (pc.row < 0) return;
    if (!mbar_wait8_warp(&bars->done, round++ & 1, s_abort)) return;
    {
      for (int r8 = 0; r8 < pc.rows; ++r8) {
        const float4 mine = lane < kFewWarps ? bars->stat[lane][r8] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        float top = mine.x;
#pragma unroll
        for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        if (top == -INFINITY) top = 0.f;
        const float f = mine.x == -INFINITY ? 0.f : ex2_approx(mine.x - top);
        float sum = mine.y * f, rounded = mine.z * f;
#pragma unroll
        for (int x = 16; x; x >>= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, x);
          rounded += __shfl_xor_sync(0xffffffffu, rounded, x);
        }
        int h = pc.head + r8;
        const int dt = head_div(p, h);
        const int64_t tok = pc.tok + dt;
        h += (pc.g - dt) * p.R;
        const float m0 = bars->m0[r8];
        int64_t pr = 0;
        if (pc.mode)
          pr = pc.mode == 1 ? cut_row(w, blockIdx.x, pc.first, r8) : whole_row(w, p.total_q, p.Hq, pc.own, tok, h);
        const float inv = rounded > 0.f ? 1.f / rounded : 0.f;
#pragma unroll
        for (int u = 0; u < (HD / 4 + 31) / 32; ++u) {
          const int f4 = lane + 32 * u;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int x = 0; x < kFewWarps; ++x) {
            const float fx = __shfl_sync(0xffffffffu, f, x);
            if (f4 < HD / 4) {
              const float4 y = *reinterpret_cast<const float4*>(part + (x * 8 + r8) * HD + f4 * 4);
              acc.x = fmaf(y.x, fx, acc.x);
              acc.y = fmaf(y.y, fx, acc.y);
              acc.z = fmaf(y.z, fx, acc.z);
              acc.w = fmaf(y.w, fx, acc.w);
            }
          }
          if (f4 >= HD / 4) continue;
          if (pc.mode)
            reinterpret_cast<float4*>(p.ws + w.rows)[part_at<HD>(pr, f4)] = acc;
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + tok * p.out_ts + static_cast<int64_t>(h) * p.out_hs + f4 * 4) =
                make_uint2(Pack<BF16>::two(acc.x * inv, acc.y * inv), Pack<BF16>::two(acc.z * inv, acc.w * inv));
        }
        if (lane == 0) {
          if (pc.mode)
            reinterpret_cast<float4*>(p.ws + w.stats)[pr] = make_float4(top, sum, rounded, m0);
          else
            p.lse[tok * p.Hq + h] = sum > 0.f ? (top + log2f(sum) + m0) * kLn2 : -INFINITY;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->taken);
    }
  }
}

template <bool BF16, int HD, bool CAP, bool POS>
__global__ void __launch_bounds__(kFewThreads, 1)
    cache8_few_kernel(const __grid_constant__ Cache8Params p8, const __grid_constant__ FwdWs w,
                      const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tkt,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tvt) {
  using S = FewShape<HD>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const CacheParams& p = p8.c;
  FewBars* bars = reinterpret_cast<FewBars*>(sm + S::kOffBar);
  float* part = reinterpret_cast<float*>(sm + S::kOffPart);
  volatile int* s_abort = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int2* meta = reinterpret_cast<int2*>(p.ws + w.meta);
  if (tid == 0) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int b = 0; b < S::kStages; ++b) {
      mbar_init(&bars->full[b], 1 + 8);  // the boxes' bytes, and each scale
      mbar_init(&bars->empty[b], 2);     // its chunks' warps
    }
    mbar_init(&bars->done, kFewWarps);
    mbar_init(&bars->taken, 1);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bars->ring.full[s], 1);
      mbar_init(&bars->ring.empty[s], kFewWarps + kFewLoads + 1);
    }
    fence_barrier_init();
    bars->abort = 0;
  }
  if (warp == kFewWarps && lane == 0) {
    prefetch_tensormap(&tk);
    prefetch_tensormap(&tv);
    if (HD == 160) {
      prefetch_tensormap(&tkt);
      prefetch_tensormap(&tvt);
    }
  }
  Plan* pl = &bars->plan;
  const bool busy = make_plan(
      p, pl, [&](int s) { return seg_plan<kFewRows>(p, s); },
      [&](const SegPlan& g) -> int64_t { return seg_cost<kFewRows>(p, g) * p.Hkv; });
  if (blockIdx.x == 0 && tid == 0) {
    int ok = pl->bad == 0;
    if (smem_addr(sm) & 1023u) {
      report(p.status, ATTN_DEV_SMEM_ALIGN);
      ok = 0;
    }
    reinterpret_cast<FwdHead*>(p.ws)->ok = ok;
  }
  if (!busy || (smem_addr(sm) & 1023u)) return;  // uniform

  if (warp >= kFewWarps) {
    if (warp < kFewWarps + kFewLoads)
      few_load<HD>(p8, bars, sm, &tk, &tkt, &tv, &tvt, warp - kFewWarps, s_abort);
    else if (warp == kFewWarps + kFewLoads)
      few_join<BF16, HD>(p, w, bars, part, s_abort);
    else
      plan_pieces<kFewRows>(p, pl, &bars->ring, s_abort);
  } else {
    const int g = lane >> 2, t = lane & 3;
    const float call_scale = CAP ? p.sigma / p.softcap : p.sigma * kLog2e;
    const float out_scale = CAP ? p.softcap * kLog2e : 1.f;
    const int rg = (g & 1) ? (g + 4) & 7 : g;      // this lane's key of eight, as a row of S^T
    const int ka = 2 * t, kb = (2 * t + 5) & 7;    // its keys of eight in O's products
    uint32_t take = 0, round = 0;
    uint32_t stages = 0, first = 0;  // of the CTA before this piece; the warp that takes its first chunk
    Piece pc;
    bool ok = true;
    while (ok) {
      if (!__all_sync(0xffffffffu, piece_take8(&bars->ring, take, &pc, s_abort))) break;
      __syncwarp();
      if (lane == 0) piece_done(&bars->ring, take);
      if (pc.row < 0) break;
      // ---- the rows 2t and 2t + 1 of this lane: columns of S^T and O^T
      float slope2[2] = {0.f, 0.f}, m0[2] = {0.f, 0.f};
      int jlo[2], jhi[2], pos[2] = {0, 0};
      bool kpos = false;
      const int32_t* kp = nullptr;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int r = 2 * t + n;
        jlo[n] = 0;
        jhi[n] = r < pc.rows ? pc.len - 1 : -1;
        if (!POS) continue;
        int h = pc.head + r;
        const int dt = head_div(p, h), tok = pc.tok + dt;
        h += (pc.g - dt) * p.R;
        const Table& tb = pc.own ? p.own : p.prefix;
        const int base = pc.own ? pc.plen : 0;  // position of slot 0
        kpos = tb.pos != nullptr;
        if (kpos) kp = tb.pos + pc.row * tb.pos_rs + pc.g * tb.pos_hs;
        if (r >= pc.rows) continue;
        int b = pc.row;
        if (!pc.own) b = seq_of(p.cu_q, __ldg(p.cu_prefix + pc.row), __ldg(p.cu_prefix + pc.row + 1), tok);
        if (p.slopes) slope2[n] = __ldg(p.slopes + b * p.slopes_bs + h) * kLog2e;
        if (p.q_pos)
          pos[n] = __ldg(p.q_pos + tok) - (kpos ? 0 : base);
        else if (pc.own)
          pos[n] = pc.len - pc.ntok + tok - pc.tok0;
        else
          pos[n] = pc.plen + seg_len(p, true, b) - (__ldg(p.cu_q + b + 1) - tok);
        if (kpos) continue;
        if (p.wl >= 0) jlo[n] = max(jlo[n], pos[n] - p.wl);
        if (p.wr >= 0) jhi[n] = min(jhi[n], pos[n] + p.wr);
        // a row beyond its keys is moved up to them (cache_fwd.cuh)
        if (p.slopes && jlo[n] <= jhi[n]) {
          const int to = min(max(pos[n], jlo[n]), jhi[n] | (kKeys - 1));
          m0[n] = -slope2[n] * static_cast<float>(abs(pos[n] - to));
          pos[n] = to;
        }
      }
      // keys [elo, ehi] that both of this lane's rows may attend to
      const int elo = max(2 * t < pc.rows ? jlo[0] : 0, 2 * t + 1 < pc.rows ? jlo[1] : 0);
      const int ehi = min(2 * t < pc.rows ? jhi[0] : INT32_MAX, 2 * t + 1 < pc.rows ? jhi[1] : INT32_MAX);
      // ---- Q as operands, row g: step k takes features 64c + 16t + 4s .. + 3 (s = k mod 4)
      uint32_t qb[S::kSteps][2];
      float in_scale[2] = {call_scale, call_scale};
      {
        int h = pc.head + g;
        const int dt = head_div(p, h), tok = pc.tok + dt;
        h += (pc.g - dt) * p.R;
        if (pc.first && warp == 0 && t == 0 && g < pc.rows)
          meta[(static_cast<int64_t>(pc.own ? 0 : p.total_q) + tok) * p.Hq + h] = make_int2(blockIdx.x, pc.parts);
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + static_cast<int64_t>(tok) * p.q_ts + static_cast<int64_t>(h) * p.q_hs;
#pragma unroll
        for (int k = 0; k < S::kSteps; ++k) {
          const int f = k < 8 ? (k >> 2) * 64 + t * 16 + (k & 3) * 4 : 128 + t * 8 + (k - 8) * 4;
          const uint2 x = g < pc.rows ? __ldg(reinterpret_cast<const uint2*>(src + f)) : make_uint2(0, 0);
          qb[k][0] = x.x;
          qb[k][1] = x.y;
        }
        if (BF16) {
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < S::kSteps; ++k) top = __vmaxu2(top, __vmaxu2(qb[k][0] & 0x7fff7fffu, qb[k][1] & 0x7fff7fffu));
          top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // the largest to [2^14, 2^15)
          const int e = static_cast<int>(max(top >> 16, top & 0xffffu) >> 7);
          const int up = min(max(268 - e, 1), 253);
          const float by = __int_as_float(up << 23), back = __int_as_float((254 - up) << 23);
#pragma unroll
          for (int n = 0; n < 2; ++n) in_scale[n] = call_scale * __shfl_sync(0xffffffffu, back, (2 * t + n) * 4);
#pragma unroll
          for (int k = 0; k < S::kSteps; ++k)
#pragma unroll
            for (int q = 0; q < 2; ++q)
              qb[k][q] = Pack<false>::two(__uint_as_float(qb[k][q] << 16) * by, __uint_as_float(qb[k][q] & 0xffff0000u) * by);
        }
      }
      float o[S::kCols][4];
#pragma unroll
      for (int j = 0; j < S::kCols; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      float m_run[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, lr[2] = {0.f, 0.f};
      float vref = 0.f, vinv = 0.f;

      // Chunks from the last keys back, each stage's upper half first.  A stage whose
      // upper half lies beyond the keys counts as two chunks all the same: the warp
      // that meets it only gives the stage back.
      const int c0 = pc.kt0 * 2, c1 = min(pc.kt1 * 2, (pc.len + kFewLoad - 1) / kFewLoad);
      const int n_chunks = (c1 - c0) * 2;
      int q = warp - static_cast<int>(first);
      if (q < 0) q += kFewWarps;
      for (; q < n_chunks; q += kFewWarps) {
        const uint32_t i = stages + (q >> 1), st = i % S::kStages;
        const int upper = (q & 1) ^ 1;
        const int key0 = (c1 - 1 - (q >> 1)) * kFewLoad + upper * kFewKeys;
        const uint8_t* sk = sm + st * 2 * S::kBytes;
        const uint8_t* sv = sk + S::kBytes;
        const int r0 = upper * kFewKeys;  // its rows in the stage
        if (!(ok = mbar_wait8_warp(&bars->full[st], (i / S::kStages) & 1, s_abort))) break;
        if (key0 >= pc.len) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->empty[st]);
          continue;
        }
        // ---- S^T: two tiles of 16 keys, side by side
        float s[2][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) s[mt][0] = s[mt][1] = s[mt][2] = s[mt][3] = 0.f;
#pragma unroll
        for (int c = 0; c < (HD == 64 ? 1 : 2); ++c) {
          alignas(16) uint32_t words[4][4];  // of keys rg + 8i
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = r0 + rg + e * 8;
            *reinterpret_cast<uint4*>(words[e]) = *reinterpret_cast<const uint4*>(
                HD == 64 ? sk + r * 64 + ((t ^ ((r >> 1) & 3)) << 4) : sk + r * 128 + (((c * 4 + t) ^ (r & 7)) << 4));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              uint32_t a[4];
              widen4(words[2 * mt][k], a[0], a[2]);
              widen4(words[2 * mt + 1][k], a[1], a[3]);
              mma16816(s[mt], a, qb[c * 4 + k][0], qb[c * 4 + k][1]);
            }
        }
        if (HD == 160) {
          uint2 tail[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = r0 + rg + e * 8;
            tail[e] = *reinterpret_cast<const uint2*>(sk + kFewLoad * 128 + r * 32 + (((t >> 1) ^ ((r >> 2) & 1)) << 4) + (t & 1) * 8);
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            uint32_t a[4];
            widen4(tail[2 * mt].x, a[0], a[2]);
            widen4(tail[2 * mt + 1].x, a[1], a[3]);
            mma16816(s[mt], a, qb[S::kSteps - 2][0], qb[S::kSteps - 2][1]);
            widen4(tail[2 * mt].y, a[0], a[2]);
            widen4(tail[2 * mt + 1].y, a[1], a[3]);
            mma16816(s[mt], a, qb[S::kSteps - 1][0], qb[S::kSteps - 1][1]);
          }
        }
        // ---- base-2 logits and their maximum
        const float2 ks = *reinterpret_cast<const float2*>(bars->scale[st] + upper * 2);
        const float2 vs = *reinterpret_cast<const float2*>(bars->scale[st] + 4 + upper * 2);
        const uint32_t gone = bars->gone[st] >> (upper * 2) & 3u;
        const bool edge = __any_sync(0xffffffffu, gone || key0 < elo || key0 + kFewKeys - 1 > ehi);
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const float in[2] = {in_scale[0] * (mt ? ks.y : ks.x), in_scale[1] * (mt ? ks.y : ks.x)};
          const bool no = gone >> mt & 1;
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // keys rg and rg + 8 of the tile
            const int j = key0 + mt * 16 + e * 8 + rg;
            float z[2] = {s[mt][2 * e] * in[0], s[mt][2 * e + 1] * in[1]};
            if (CAP) {
              const uint64_t th = tanh2_fp32(f2_make(z[0], z[1]));
              z[0] = f2_lo(th) * out_scale;
              z[1] = f2_hi(th) * out_scale;
            }
            if (POS && kpos) {
              const int kq = __ldg(kp + min(j, pc.len - 1));
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const bool adm = j <= jhi[n] && (p.wl < 0 || kq >= pos[n] - p.wl) && (p.wr < 0 || kq <= pos[n] + p.wr) && !no;
                z[n] = adm ? fmaf(-slope2[n], static_cast<float>(abs(pos[n] - kq)), z[n]) : -INFINITY;
              }
            } else {
              if (POS && p.slopes) {
#pragma unroll
                for (int n = 0; n < 2; ++n) z[n] = fmaf(-slope2[n], static_cast<float>(abs(pos[n] - j)), z[n]);
              }
              if (edge) {
#pragma unroll
                for (int n = 0; n < 2; ++n) z[n] = !no && j >= jlo[n] && j <= jhi[n] ? z[n] : -INFINITY;
              }
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              s[mt][2 * e + n] = z[n];
              mx[n] = fmaxf(mx[n], z[n]);
            }
          }
        }
        bool move = false;
        float alpha[2] = {1.f, 1.f};
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], x));
          mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], x));
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          if (mx[n] > m_run[n] + kLazy8) {
            alpha[n] = ex2_approx(m_run[n] - mx[n]);
            m_run[n] = mx[n];
            move = true;
          }
          l[n] *= alpha[n];
          lr[n] *= alpha[n];
        }
        const float vtop = fmaxf(vs.x, vs.y);
        if (vtop > vref) {  // the power of two at or above it, within [2^-126, 2^126]
          const int e = min(max(((__float_as_int(vtop) + 0x7fffff) >> 23) & 0xff, 1), 253);
          const float was = vref;
          vref = __int_as_float(e << 23);
          vinv = __int_as_float((254 - e) << 23);
          alpha[0] *= was * vinv;
          alpha[1] *= was * vinv;
          move = true;
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int j = 0; j < S::kCols; ++j) {
            o[j][0] *= alpha[0];
            o[j][1] *= alpha[1];
            o[j][2] *= alpha[0];
            o[j][3] *= alpha[1];
          }
        }
        // ---- P and O, 16 keys at a time
        const int last = pc.len - key0;  // rows from here on hold anything
        const float m_use[2] = {m_run[0] == -INFINITY ? 0.f : m_run[0] - kShift8, m_run[1] == -INFINITY ? 0.f : m_run[1] - kShift8};
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          float by = (mt ? vs.y : vs.x) * vinv, down = 1.f;
          if (by < 1.f / 4096 && by > 0.f) {  // (rare, the same in all lanes) far below the largest
            // to [1/2, 1), but by 2^59 at most: O may be 2^60 already
            const int e = max((__float_as_int(by) >> 23) & 0xff, 67);
            const float up = __int_as_float((253 - e) << 23);
            down = __int_as_float((e + 1) << 23);
            by *= up;
#pragma unroll
            for (int j = 0; j < S::kCols; ++j)
#pragma unroll
              for (int n = 0; n < 4; ++n) o[j][n] *= up;
          }
          // The rounded weights count as what they stand for (out is a weighted mean then),
          // unless a far block's lose bits that its own keys do not need and the sum does.
          const float back = by >= 1.f / 64 && down == 1.f ? rcp_approx(by) : 0.f;
          uint32_t pb[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float e0 = ex2_approx(s[mt][2 * e] - m_use[0]), e1 = ex2_approx(s[mt][2 * e + 1] - m_use[1]);
            pb[e] = Pack<false>::two(e0 * by, e1 * by);
            const uint64_t seen = Pack<false>::unpack(pb[e]);
            l[0] += e0;
            l[1] += e1;
            lr[0] += back > 0.f ? f2_lo(seen) * back : e0;
            lr[1] += back > 0.f ? f2_hi(seen) * back : e1;
            pb[e] = turn8x8(pb[e]);
          }
          constexpr int kWords = HD == 64 ? 2 : (HD == 128 ? 4 : 5);  // of four features a lane holds of a row
          uint32_t v[4][kWords];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int in = mt * 16 + (u >> 1) * 8 + ((u & 1) ? kb : ka), r = r0 + in;
            if (HD == 64) {
              const uint2 x = *reinterpret_cast<const uint2*>(sv + r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
              v[u][0] = x.x;
              v[u][1] = x.y;
            } else {
              const uint4 x = *reinterpret_cast<const uint4*>(sv + r * 128 + ((g ^ (r & 7)) << 4));
              v[u][0] = x.x;
              v[u][1] = x.y;
              v[u][kWords > 2 ? 2 : 0] = x.z;
              v[u][kWords > 2 ? 3 : 0] = x.w;
              if (HD == 160)
                v[u][kWords - 1] = *reinterpret_cast<const uint32_t*>(sv + kFewLoad * 128 + r * 32 + (((g >> 2) ^ ((r >> 2) & 1)) << 4) + (g & 3) * 4);
            }
          }
          if (last < kFewKeys) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (mt * 16 + (u >> 1) * 8 + ((u & 1) ? kb : ka) >= last) {
#pragma unroll
                for (int x = 0; x < kWords; ++x) v[u][x] = 0;
              }
          }
#pragma unroll
          for (int x = 0; x < kWords; ++x) {  // features 4x .. 4x + 3 of this lane's: rows g, g + 8 of two tiles
            uint32_t a[4], b[4];
            widen4(__byte_perm(v[0][x], v[1][x], 0x5140), a[0], a[1]);
            widen4(__byte_perm(v[2][x], v[3][x], 0x5140), a[2], a[3]);
            widen4(__byte_perm(v[0][x], v[1][x], 0x7362), b[0], b[1]);
            widen4(__byte_perm(v[2][x], v[3][x], 0x7362), b[2], b[3]);
            mma16816(o[2 * x], a, pb[0], pb[1]);
            mma16816(o[2 * x + 1], b, pb[0], pb[1]);
          }
          if (down != 1.f) {
#pragma unroll
            for (int j = 0; j < S::kCols; ++j)
#pragma unroll
              for (int n = 0; n < 4; ++n) o[j][n] *= down;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->empty[st]);
      }
      if (!ok) break;
      stages += c1 - c0;
      first = (first + n_chunks) % kFewWarps;
      // ---- leave O and the sums to the joining warp
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          l[n] += __shfl_xor_sync(0xffffffffu, l[n], x);
          lr[n] += __shfl_xor_sync(0xffffffffu, lr[n], x);
        }
      }
      if (round > 0 && !(ok = mbar_wait8_warp(&bars->taken, (round - 1) & 1, s_abort))) break;
      ++round;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int r = 2 * t + n;
        if (g == 0) {
          bars->stat[warp][r] = make_float4(m_run[n] == -INFINITY ? -INFINITY : m_run[n] - kShift8, l[n], lr[n], 0.f);
          if (warp == 0) bars->m0[r] = m0[n];
        }
        if (r >= pc.rows) continue;
        float* dst = part + (warp * 8 + r) * HD;
#pragma unroll
        for (int x = 0; x < S::kCols / 2; ++x) {
          const int at = HD == 64 ? g * 8 + x * 4 : (x < 4 ? g * 16 + x * 4 : 128 + g * 4);
          *reinterpret_cast<float4*>(dst + at) =
              make_float4(o[2 * x][n] * vref, o[2 * x][2 + n] * vref, o[2 * x + 1][n] * vref, o[2 * x + 1][2 + n] * vref);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->done);
    }
  }
  __syncthreads();
  if (tid == 0 && *s_abort) report(p.status, ATTN_DEV_TIMEOUT_FWD);
}

template <int HD>
cudaError_t launch_few_d(const Cache8Params& p, const FwdWs& w, const CUtensorMap& tk, const CUtensorMap& tkt,
                         const CUtensorMap& tv, const CUtensorMap& tvt, int grid, cudaStream_t s) {
  constexpr uint32_t smem = FewShape<HD>::kOffBar + sizeof(FewBars);
  static_assert(smem <= 232448, "shared memory");
  const bool cap = p.c.softcap > 0.f, bf = p.c.dtype == 1;
  const bool pos = p.c.slopes || p.c.wl >= 0 || p.c.wr >= 0 || p.c.own.pos || (p.c.P && p.c.prefix.pos);
  auto k = bf ? (cap ? (pos ? cache8_few_kernel<true, HD, true, true> : cache8_few_kernel<true, HD, true, false>)
                     : (pos ? cache8_few_kernel<true, HD, false, true> : cache8_few_kernel<true, HD, false, false>))
              : (cap ? (pos ? cache8_few_kernel<false, HD, true, true> : cache8_few_kernel<false, HD, true, false>)
                     : (pos ? cache8_few_kernel<false, HD, false, true> : cache8_few_kernel<false, HD, false, false>));
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  k<<<grid, kFewThreads, smem, s>>>(p, w, tk, tkt, tv, tvt);
  return cudaGetLastError();
}

}  // namespace kv
}  // namespace attn
