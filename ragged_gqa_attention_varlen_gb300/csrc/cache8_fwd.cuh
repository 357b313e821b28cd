// cache8_fwd.cuh -- attention of packed query rows over the paged cache held in
// 8 bits: e4m3 values with a scale for each block of slots and head.
//
// Per step (128 rows x 128 keys), with z the base-2 logit and m the row's
// reference (a running maximum, or a bound known beforehand):
//   S = sum_i Q_i K8^T   tcgen05.mma kind::f8f6f4 on K's own bytes, fp32 in TMEM
//   P = 2^(z - m)        softmax warps, one TMEM lane per row; z takes the K
//                        scale of its 16 columns' block.  fp16 pairs over S
//   V16 = V8 * scale / vref in fp16 (conversion warps)
//   O += P V16           tcgen05.mma kind::f16 with P from TMEM
// and out = vref O / l with l the sum of P.
//
// K is never converted: a row of Q, times a power of two that takes its largest
// value to (224, 448], is the sum of two (bf16) or three (fp16) e4m3 numbers, each
// the rounding of what the ones before leave.  Every piece takes four significant
// bits off, so the sum is exact down to 2^-9, the last bit of e4m3's smallest
// numbers: an element of q is off by at most 2^-10 where the row's largest is above
// 224, 2^-17.8 of it.  The products run at twice the rate of fp16 ones, so two pieces
// cost what an fp16 product would; converting K as well took the conversion warps
// to 6000 clk a step.  The fp8 product keeps fp32's accuracy (2^-22 of the sum of
// magnitudes, measured over 128 products with and without cancellation).
// P is not split like that: weights range further than e4m3 reaches.
//
// vref, a power of two, is a sixteenth of the largest V scale met when it was set:
// while a block's scale is at most 64 vref, V16 stays below 2^15; beyond that vref
// moves and O with it.  Every warp that needs it follows the scales by itself.  A
// block enters V16 with the power of two at or above scale / vref, 2^-15 at least,
// and its weights take the rest: e4m3 times a power of two from 2^-15 to 2^6 is exact
// in fp16, so V is never rounded, whatever the scales are, and blocks lose nothing
// however far their scales lie apart, until the weights do.  P lies up to 2^15 (a
// shift of 7 above the usual 1, and 8 for the lazy reference), so the smallest weights
// that fp16 still holds are 2^-31 of the largest.
// out divides by the sum of the rounded weights (as in cache_fwd.cuh, so it is a
// weighted mean of V rows whatever the roundings), lse by that of the unrounded ones.
//
// The pages' bytes bound calls of few rows a key; the softmax's MUFU work, the
// conversion and the hand-offs bound those of many.
//
// Warps (640 threads): 0 loads K (TMA boxes of min(page_size, 128) rows per lane)
// and the scales, 16 loads V, 1 issues S, 2 issues O, 3 plans the CTA's pieces,
// 17-19 bring in Q rows (with 4-11 the first tile's), 12-15 convert V, 64 keys at a
// time (rows that no row of the tile reads become zeros: the pages may hold anything
// there, and 0 * NaN would reach O), 4-11 softmax as in cache_fwd.cuh.
//
// Measured with the join: 144 drafted tokens of 96 heads behind two prefixes of 12001
// keys 226 us (546 TFLOP/s of the logits' and outputs' products), 64 single tokens of
// 80 heads over 277000 keys in 16-row pages 61 us (1.45 TB/s), one token of 96 heads
// over 700 keys 19 us.  The second row sum is 11 and 2.5 us of the first two; without it
// a step took about 4000 clk: 3600 of softmax (four passes of
// 16 columns, two warps in each sub-partition, at half of the issue slots; the fetch
// of instructions is the largest stall that is not a dependency), the rest the
// hand-offs to the products (1300 clk of tensor work) and back.  Loading the next
// pass's products ahead (254 us), passes of 32 columns (281), descriptors kept as
// halves and sleeping waits (no change) were tried.  A CTA's first product stands
// 20000 clk behind its start: plan, page and row lookups, first instructions.
#pragma once
#include <cuda_fp8.h>

#include "cache8_wait.cuh"

namespace attn {
namespace kv {

template <bool BF16, int HD>
struct Fwd8Shape {
  static constexpr int kPieces = BF16 ? 2 : 3;                  // of Q
  static constexpr uint32_t kTile = 128 * HD;                   // a tile of bytes: K, V, a piece of Q
  static constexpr uint32_t kV = (HD + 63) / 64 * 8192;         // V16 of 64 keys: 64-feature chunks of 8 KB
  static constexpr int kRK = HD == 160 ? (BF16 ? 3 : 2) : (HD == 128 ? (BF16 ? 4 : 3) : 6);  // stages of K,
  static constexpr int kRV = HD == 160 ? 2 : (HD == 128 ? 3 : 5);                             // V
  static constexpr int kVS = HD == 160 ? 3 : (HD == 128 ? 4 : 6);                             // and V16
  static constexpr uint32_t kOffV = kPieces * kTile;
  static constexpr uint32_t kOffRK = kOffV + kVS * kV;
  static constexpr uint32_t kOffRV = kOffRK + kRK * kTile;
  static constexpr uint32_t kOffMax = kOffRV + kRV * kTile;       // [2 steps][2 halves][128]
  static constexpr uint32_t kOffSum = kOffMax + 2 * 2 * 128 * 4;  // [2 pieces][2 halves][128]
  static constexpr uint32_t kOffQs = kOffSum + 2 * 2 * 128 * 8;   // [4 pieces][128] row factors of Q
  static constexpr uint32_t kOffBar = kOffQs + 4 * 128 * 4;
};

// K-major tiles of bytes: 128-byte rows (128-byte swizzle) and, at d = 160,
// features 128 and up in 32-byte rows behind them (32-byte swizzle); at d = 64
// 64-byte rows (64-byte swizzle).  Byte offset of 16-byte unit u of row r:
template <int HD>
__device__ __forceinline__ uint32_t byte_unit(int r, int u) {
  if (HD == 64) return r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
  return u < 8 ? r * 128 + ((u ^ (r & 7)) << 4) : 16384 + r * 32 + (((u - 8) ^ ((r >> 2) & 1)) << 4);
}
// Descriptor of the 32 features from 32k on.
template <int HD>
__device__ __forceinline__ uint64_t byte_desc(uint32_t base, int k) {
  if (HD == 64) return sdesc_sw64(base + k * 32);
  return k < 4 ? sdesc_sw128(base + k * 32, 16, 1024) : sdesc_sw32(base + 16384);
}

constexpr int kStepsHeld = 16;  // steps whose scales are kept

struct Fwd8Bars {
  uint64_t q_full, q_empty, q_more;
  uint64_t rk_full[6], rk_empty[6], rv_full[6], rv_empty[6];
  uint64_t v_full[6], v_empty[6];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t o_full, o_empty, drain;
  uint64_t mx_x[4][2], l_x[4];
  alignas(16) float scale[kStepsHeld][2][8];  // K and V scales of the 16-key blocks of a step
  alignas(16) float v_scale[kStepsHeld][8];   // V's, once more, along with its bytes
  uint32_t gone[kStepsHeld];      // load boxes whose page is out of the pool
  PieceRing ring;
  Plan plan;
  uint32_t tmem;
  int abort;
};

constexpr int kThreads8 = 640;
// registers per thread of warps 0-3, 4-11, 12-15 and 16-19 (launched at 96)
constexpr int kRegsPlan8 = 88, kRegsSoft8 = 128, kRegsConv8 = 64, kRegsQ8 = 72;
static_assert(kRegsPlan8 + 2 * kRegsSoft8 + kRegsConv8 + kRegsQ8 <= 5 * 96, "register split exceeds the launch");
constexpr uint32_t kColO8 = 256;  // TMEM: S0 / P0 [0,128), S1 / P1 [128,256), O [256, 256 + d)
constexpr float kFixedCap8 = 9.5f;

// The reference of the V scales, as every warp that needs it follows it.
struct VRef {
  float ref, inv;
  __device__ __forceinline__ void start() { ref = inv = 0.f; }
  // Takes a step's scales; the factor that O takes (1: none).
  __device__ __forceinline__ float step(const float* vs) {
    const float4 a = *reinterpret_cast<const float4*>(vs), b = *reinterpret_cast<const float4*>(vs + 4);
    const float top = fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
    if (!(top > ref * 64.f)) return 1.f;
    // a sixteenth of the power of two at or above it, within [2^-126, 2^126]
    const int e = ((__float_as_int(top) + 0x7fffff) >> 23) & 0xff;
    const int ce = min(max(e - 4, 1), 253);
    const float was = ref;
    ref = __int_as_float(ce << 23);
    inv = __int_as_float((254 - ce) << 23);
    return was * inv;
  }
  // What of a block's scale V16 takes, and the weights.
  __device__ __forceinline__ float of_v(float scale) const {
    const float by = scale * inv;
    return by > 0.f ? above(by) : 0.f;
  }
  __device__ __forceinline__ float of_p(float scale) const {
    const float by = scale * inv;
    return by * __int_as_float(0x7f000000 - __float_as_int(above(by)));
  }
  // The power of two at or above it, kLeastV at least.
  __device__ __forceinline__ static float above(float by) {
    return fmaxf(__int_as_float((__float_as_int(by) + 0x7fffff) & 0x7f800000), kLeastV);
  }
  static constexpr float kLeastV = 1.f / 32768.f;
};

// One warp: the bytes of every key tile of the pieces into the stages, a box per
// lane, and the scales: V's with both, since the warps that convert V and those
// that scale O stand at different steps.
template <bool BF16, int HD, bool K>
__device__ __forceinline__ void load_pages8(const Cache8Params& p8, Fwd8Bars* bars, uint8_t* dst0,
                                            const CUtensorMap* map, const CUtensorMap* tail, int box,
                                            volatile int* s_abort) {
  using S = Fwd8Shape<BF16, HD>;
  const CacheParams& p = p8.c;
  constexpr int kStages = K ? S::kRK : S::kRV;
  const int lane = threadIdx.x & 31;
  uint64_t* full = K ? bars->rk_full : bars->rv_full;
  uint64_t* empty = K ? bars->rk_empty : bars->rv_empty;
  const int pieces = kKeys / box;
  const int pi = lane & (pieces - 1), part = lane / pieces;  // row block; features from 128 part on
  constexpr int kParts = K && HD == 160 ? 2 : 1;
  const int sj = lane & 7, my_box = sj * 16 / box;  // scales: block of 16 keys, its load box
  uint32_t take = 0, st = 0, ph = 0, loaded = 0;
  Piece pc;
  bool ok = true;
  while (ok) {
    if (!__all_sync(0xffffffffu, piece_take8(&bars->ring, take, &pc, s_abort))) break;
    __syncwarp();
    if (lane == 0) piece_done(&bars->ring, take);
    if (pc.row < 0) break;
    const Table& t = pc.own ? p.own : p.prefix;
    const int32_t* row = t.pages + pc.row * t.rs;
    auto page_of = [&](int kt) {  // this lane's page of key tile kt, or -1: no box
      const int key = kt * kKeys + pi * box;
      return part < kParts && kt >= pc.kt0 && key < pc.len ? tile_page(p, row, key) : -1;
    };
    int page = page_of(pc.kt1 - 1);
    for (int kt = pc.kt1 - 1; kt >= pc.kt0; --kt) {
      const int key0 = kt * kKeys;
      const int have = min(pieces, (pc.len - key0 + box - 1) / box);  // row blocks in use
      const int next = page_of(kt - 1);  // read while this tile's stage is waited for
      if (loaded >= kStages && !(ok = mbar_wait8_warp(&empty[st], ph ^ 1, s_abort))) break;
      const int sp = __shfl_sync(0xffffffffu, page, my_box), key = key0 + sj * 16;
      if (K) {
        const uint32_t gone = __ballot_sync(0xffffffffu, part == 0 && page == p.num_pages);
        if (lane == 0) bars->gone[loaded % kStepsHeld] = gone;
      }
      if (lane < (K ? 16 : 8)) {
        // The entry of sixteen steps ago.  Of K: this tile's stage was free, so S of
        // the tile kRK before is done, and P of the second before that has been
        // multiplied.  Of V: the tile kRV before is converted.
        static_assert(S::kRK + 2 < kStepsHeld && S::kRV < kStepsHeld, "an entry could still be read");
        const Scales& sc = K && lane < 8 ? p8.ks : p8.vs;
        const bool there = key < pc.len && sp >= 0 && sp < p.num_pages;
        const int64_t at = there ? sp * sc.page + static_cast<int64_t>((key & (p.page_size - 1)) >> p8.block_log2) * sc.block + pc.g * sc.head : 0;
        float* dst = K ? &bars->scale[loaded % kStepsHeld][lane >> 3][sj] : &bars->v_scale[loaded % kStepsHeld][sj];
        cp_async4_or_zero(dst, sc.base + at, there);
      }
      cp_async_arrive(&full[st]);
      if (lane == 0) mbar_arrive_expect_tx(&full[st], S::kTile / pieces * have);
      __syncwarp();
      if (page >= 0) {
        const int slot = p.page_size > kKeys ? key0 & (p.page_size - 1) : 0;
        uint8_t* dst = dst0 + st * S::kTile;
        if (kParts == 2 && part == 1)
          tma_load_4d(dst + 16384 + pi * box * 32, tail, &full[st], 128, pc.g, slot, page);
        else
          tma_load_4d(dst + pi * box * (kParts == 2 ? 128 : HD), map, &full[st], 0, pc.g, slot, page);
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
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// e4m3 values in fp16: two, eight.
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint4 widen8(uint2 q) {
  uint4 r;
  asm("{\n\t.reg .b16 a, b, c, d;\n\tmov.b32 {a, b}, %4;\n\tmov.b32 {c, d}, %5;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t"
      "cvt.rn.f16x2.e4m3x2 %2, c;\n\tcvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
      : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
      : "r"(q.x), "r"(q.y));
  return r;
}
__device__ __forceinline__ uint32_t mul2_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t sub2_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t narrow2(uint32_t h) {  // to e4m3, in the low half
  __half2_raw x;
  x.x = static_cast<unsigned short>(h & 0xffff);
  x.y = static_cast<unsigned short>(h >> 16);
  return __nv_cvt_halfraw2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
}

// Four warps: V's bytes to fp16 tiles of 64 keys in the swizzled layout of the
// product, times scale / vref; 16 keys (a scale) each.  A lane's units of 8 values
// lie at the same places of every 16 keys, so their offsets are worked out once,
// and all loads of 16 keys go out before the first store (which the compiler could
// not tell from the loads of the next).
template <bool BF16, int HD>
__device__ __forceinline__ void convert_v(Fwd8Bars* bars, const uint8_t* raw0, uint8_t* dst0, volatile int* s_abort) {
  using S = Fwd8Shape<BF16, HD>;
  constexpr int kUnits = HD / 8;           // of a row
  constexpr int kLane = 16 * kUnits / 32;  // of a lane
  const int lane = threadIdx.x & 31, wi = (threadIdx.x >> 5) & 3;
  uint32_t off[kLane];
#pragma unroll
  for (int i = 0; i < kLane; ++i) {
    const int u = lane + 32 * i, r = u / kUnits, c = u - r * kUnits;
    off[i] = (c >> 3) * 8192 + wi * 2048 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  }
  uint32_t take = 0, step = 0, rst = 0, rph = 0, st = 0, ph = 0, made = 0;
  VRef vref;
  Piece pc;
  bool ok = true;
  while (ok) {
    if (!__all_sync(0xffffffffu, piece_take8(&bars->ring, take, &pc, s_abort))) break;
    __syncwarp();
    if (lane == 0) piece_done(&bars->ring, take);
    if (pc.row < 0) break;
    vref.start();
    for (int kt = pc.kt1 - 1; kt >= pc.kt0; --kt, ++step) {
      const int key0 = kt * kKeys;
      const int nk = min(kKeys, pc.len - key0);        // keys of the tile that exist
      const int z0 = min(max(pc.klo - key0, 0), nk);   // those [z0, z1) that some row reads
      const int z1 = max(min(pc.khi - key0, nk), z0);
      const int blocks = (nk + 15) / 16;               // the product takes 16 at a time
      if (!(ok = mbar_wait8_warp(&bars->rv_full[rst], rph, s_abort))) break;
      vref.step(bars->v_scale[step % kStepsHeld]);
      const uint8_t* raw = raw0 + rst * S::kTile + lane * 8;
#pragma unroll 1
      for (int half = 0; half * 4 < blocks; ++half) {
        const int blk = half * 4 + wi;
        uint2 q[kLane];
        if (blk < blocks) {
#pragma unroll
          for (int i = 0; i < kLane; ++i) q[i] = *reinterpret_cast<const uint2*>(raw + blk * 16 * HD + i * 256);
        }
        if (made >= S::kVS && !(ok = mbar_wait8_warp(&bars->v_empty[st], ph ^ 1, s_abort))) break;
        if (blk < blocks) {
          const float by = vref.of_v(bars->v_scale[step % kStepsHeld][blk]);
          const uint32_t f = Pack<false>::two(by, by);
          const bool cut = blk * 16 < z0 || blk * 16 + 16 > z1;
          uint8_t* dst = dst0 + st * S::kV;
#pragma unroll
          for (int i = 0; i < kLane; ++i) {
            uint4 x = widen8(q[i]);
            x = make_uint4(mul2_f16(x.x, f), mul2_f16(x.y, f), mul2_f16(x.z, f), mul2_f16(x.w, f));
            if (cut) {
              const int r = blk * 16 + (lane + 32 * i) / kUnits;
              if (r < z0 || r >= z1) x = make_uint4(0, 0, 0, 0);
            }
            *reinterpret_cast<uint4*>(dst + off[i]) = x;
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->v_full[st]);
        ++made;
        if (++st == S::kVS) {
          st = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(&bars->rv_empty[rst]);
      if (++rst == S::kRV) {
        rst = 0;
        rph ^= 1;
      }
    }
  }
}

// Rows of Q as pieces of e4m3 (above); the inverse of the row's factor goes to
// `qs`.  Warp wi of nw; four lanes a row, the next row of a lane in flight.
// Scaled values and what the pieces leave are exact in fp16 but for what lies below
// its smallest numbers, 2^-33 of the row's largest.  The units are a rolled loop:
// this code is short because its fetch is what a CTA's first product waits for and
// what the softmax loops lose from the instruction cache (drafts / ragged batch /
// one user: remainders in fp32, all unrolled 242 / 66 / 19.5 us; in fp16, unrolled
// 236 / 60 / 18.3; rolled 214 / 58 / 18.7).
template <bool BF16, int HD>
__device__ __forceinline__ void split_q_rows(const CacheParams& p, uint8_t* dst, float* qs, const Piece& pc, int wi,
                                             int nw) {
  using S = Fwd8Shape<BF16, HD>;
  constexpr int kPer = HD / 32;  // 16-byte units of q of a lane
  const int lane = threadIdx.x & 31, u0 = lane & 3;
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + static_cast<int64_t>(pc.g) * p.R * p.q_hs + u0 * 8;
  auto row_at = [&](int r) {
    const int hh = pc.head + r, dt = head_div(p, hh);
    return q + static_cast<int64_t>(pc.tok + dt) * p.q_ts + static_cast<int64_t>(hh - dt * p.R) * p.q_hs;
  };
  uint4 next[kPer];
  auto load = [&](int r) {
    const uint16_t* src = row_at(r);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      next[k] = r < pc.rows ? __ldg(reinterpret_cast<const uint4*>(src + k * 32)) : make_uint4(0, 0, 0, 0);
  };
  int r = wi * 8 + (lane >> 2);
  load(r);
#pragma unroll 1
  for (; r - (lane >> 2) < pc.rows; r += nw * 8) {
    uint4 x[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) x[k] = next[k];
    load(r + nw * 8);
    uint32_t top = 0;  // the largest magnitude's bits, in both halves
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu),
                                   __vmaxu2(x[k].z & 0x7fff7fffu, x[k].w & 0x7fff7fffu)));
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (r >= pc.rows) continue;
    const int bits = __float_as_int(to_float<BF16>(static_cast<uint16_t>(max(top >> 16, top & 0xffffu))));
    // 1.m 2^e times 2^(8 - e), or 2^(7 - e) above 1.75
    const int up = min(max(262 - (bits >> 23) - ((bits & 0x7fffff) > 0x600000 ? 1 : 0), 1), 253);
    const uint64_t by = f2_make(__int_as_float(up << 23), __int_as_float(up << 23));
    if (u0 == 0) qs[r] = __int_as_float((254 - up) << 23);
#pragma unroll 1
    for (int k = 0; k < kPer; ++k) {
      const uint32_t w[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
#pragma unroll
      for (int j = 1; j < kPer; ++j) x[j - 1] = x[j];
      const int u = u0 + 4 * k;  // 8 values: half of a 16-byte unit of bytes
      uint8_t* y = dst + byte_unit<HD>(r, u >> 1) + (u & 1) * 8;
      uint32_t left[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t z = f2_mul(Pack<BF16>::unpack(w[i]), by);
        left[i] = Pack<false>::two(f2_lo(z), f2_hi(z));
      }
#pragma unroll
      for (int piece = 0; piece < S::kPieces; ++piece) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          b[i] = narrow2(left[i]);
          if (piece + 1 < S::kPieces) left[i] = sub2_f16(left[i], widen2(b[i]));
        }
        *reinterpret_cast<uint2*>(y + piece * S::kTile) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
      }
    }
  }
}

// CAP, FIXED and POS as in cache_fwd.cuh; BF16: the type of q and out.
template <bool BF16, int HD, bool CAP, bool FIXED, bool POS>
__global__ void __launch_bounds__(kThreads8, 1)
    cache8_fwd_kernel(const __grid_constant__ Cache8Params p8, const __grid_constant__ FwdWs w,
                      const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tkt,
                      const __grid_constant__ CUtensorMap tv) {
  using S = Fwd8Shape<BF16, HD>;
  // Columns of a softmax pass: they share a K scale.  (Twice as many in a pass took
  // drafts from 233 to 276 us: the longer loop body misses the instruction cache.)
  constexpr int kCh = 16;
  extern __shared__ __align__(1024) uint8_t sm[];
  const CacheParams& p = p8.c;
  uint8_t* sQ = sm;
  uint8_t* sV = sm + S::kOffV;
  uint8_t* sK = sm + S::kOffRK;
  float* sMax = reinterpret_cast<float*>(sm + S::kOffMax);
  float2* sSum = reinterpret_cast<float2*>(sm + S::kOffSum);
  float* sQs = reinterpret_cast<float*>(sm + S::kOffQs);
  Fwd8Bars* bars = reinterpret_cast<Fwd8Bars*>(sm + S::kOffBar);
  volatile int* s_abort = &bars->abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int2* meta = reinterpret_cast<int2*>(p.ws + w.meta);
  if (tid == 0) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    mbar_init(&bars->q_full, 3);
    mbar_init(&bars->q_empty, 1);
    mbar_init(&bars->q_more, 8);  // the first tile: the softmax warps' rows
    for (int b = 0; b < S::kRK; ++b) {
      mbar_init(&bars->rk_full[b], 1 + 32);  // the boxes' bytes, and each lane's scales
      mbar_init(&bars->rk_empty[b], 1);
    }
    for (int b = 0; b < S::kRV; ++b) {
      mbar_init(&bars->rv_full[b], 1 + 32);
      mbar_init(&bars->rv_empty[b], 4);
    }
    for (int b = 0; b < S::kVS; ++b) {
      mbar_init(&bars->v_full[b], 4);
      mbar_init(&bars->v_empty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->s_full[b], 2);  // the products, and the issuer (which has seen the scales)
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
      mbar_init(&bars->ring.empty[s], 19);  // K and V loads, two MMA issuers, 8 softmax, 4 conversion, 3 Q warps
    }
    fence_barrier_init();
    bars->abort = 0;
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  if (warp == 17 && lane == 0) {
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
  // Where the kernel for few rows took a part of the sequences, this one starts beside
  // its last CTAs and reads nothing of it, but ends behind it: the join waits for this
  // one alone.
  auto behind_few = [&] {
    if (p.most_rows) asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  if (!busy || (smem_addr(sm) & 1023u)) {  // uniform
    if (warp == 1) tmem_dealloc(tmem, 512);
    behind_few();
    return;
  }
  const int box = min(p.page_size, kKeys), box_log2 = min(p.page_log2, 7);  // rows of a load box

  if (warp < 4) {
    warpgroup_reg_dealloc<kRegsPlan8>();
    if (warp == 0) {
      // ------------------------------------------------------------ K bytes and scales
      load_pages8<BF16, HD, true>(p8, bars, sK, &tk, &tkt, box, s_abort);
    } else if (warp == 1) {
      // ------------------------------------------------------------ S = Q K^T
      if (lane == 0) {
        constexpr uint32_t kIdS = idesc_e4m3(128, 128);
        uint32_t take = 0, step = 0, st = 0, ph = 0, tiles = 0;
        Piece pc;
        bool ok = true;
        while (ok && piece_take8(&bars->ring, take, &pc, s_abort)) {
          piece_done(&bars->ring, take);
          if (pc.row < 0) break;
          if (!mbar_wait8(&bars->q_full, tiles & 1, s_abort)) break;
          if (tiles == 0 && !mbar_wait8(&bars->q_more, 0, s_abort)) break;
          for (int kt = pc.kt1 - 1; kt >= pc.kt0; --kt, ++step) {
            if (!(ok = mbar_wait8(&bars->rk_full[st], ph, s_abort))) break;
            // the product with the P that took the buffer's previous S (step - 2) is done
            if (step >= 2 && !(ok = mbar_wait8(&bars->pv_done[step & 1], ((step - 2) >> 1) & 1, s_abort)))
              break;
            tc_fence_after();
            const uint32_t kb = smem_addr(sK + st * S::kTile), qb = smem_addr(sQ);
#pragma unroll
            for (int i = 0; i < S::kPieces; ++i)
#pragma unroll
              for (int k = 0; k < HD / 32; ++k)
                umma_ss_f8(tmem + (step & 1) * 128, byte_desc<HD>(qb + i * S::kTile, k), byte_desc<HD>(kb, k), kIdS,
                           i + k > 0);
            umma_commit(&bars->s_full[step & 1]);
            mbar_arrive(&bars->s_full[step & 1]);
            umma_commit(&bars->rk_empty[st]);
            if (kt == pc.kt0) umma_commit(&bars->q_empty);
            if (++st == S::kRK) {
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
      if (lane == 0) {
        constexpr uint32_t kIdO = idesc_f16(128, HD, false, false, true);
        uint32_t take = 0, step = 0, st = 0, ph = 0, tiles = 0;
        Piece pc;
        bool ok = true;
        while (ok && piece_take8(&bars->ring, take, &pc, s_abort)) {
          piece_done(&bars->ring, take);
          if (pc.row < 0) break;
          for (int kt = pc.kt1 - 1; kt >= pc.kt0; --kt, ++step) {
            const int ksteps = (min(kKeys, pc.len - kt * kKeys) + 15) / 16;
            if (!(ok = mbar_wait8(&bars->p_full[step & 1], (step >> 1) & 1, s_abort))) break;
            const bool first = kt == pc.kt1 - 1;
            if (first && tiles > 0 && !(ok = mbar_wait8(&bars->o_empty, (tiles - 1) & 1, s_abort))) break;
            for (int half = 0; half * 4 < ksteps; ++half) {
              if (!(ok = mbar_wait8(&bars->v_full[st], ph, s_abort))) break;
              tc_fence_after();
              const uint32_t vb = smem_addr(sV + st * S::kV);
              // keys 64 half + 16k .. + 15: pair columns 8k of that half
              for (int k = 0; k < min(4, ksteps - half * 4); ++k)
                umma_ts(tmem + kColO8, tmem + (step & 1) * 128 + half * 64 + k * 8,
                        sdesc_sw128(vb + k * 2048, 8192, 1024), kIdO, (!first || half + k > 0));
              umma_commit(&bars->v_empty[st]);
              if (++st == S::kVS) {
                st = 0;
                ph ^= 1;
              }
            }
            if (!ok) break;
            umma_commit(&bars->pv_done[step & 1]);
            if (kt == pc.kt0) umma_commit(&bars->o_full);
          }
          ++tiles;
        }
        umma_commit(&bars->drain);
        wait_drain(&bars->drain, 0);
      }
    } else {
      // ------------------------------------------------------------ plan
      plan_pieces(p, pl, &bars->ring, s_abort);
    }
  } else if (warp < 12) {
    warpgroup_reg_alloc<kRegsSoft8>();
    // ------------------------------------------------------------ softmax
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int r = quad * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    // z = out_scale * tanh(in_scale * x), or in_scale * x, in base-2 units
    const float call_scale = CAP ? p.sigma / p.softcap : p.sigma * kLog2e;
    const float out_scale = CAP ? p.softcap * kLog2e : 1.f;
    uint32_t take = 0, step = 0, tiles = 0;
    Piece pc;
    VRef vref;
    bool ok = true;
    while (ok) {
      if (!__all_sync(0xffffffffu, piece_take8(&bars->ring, take, &pc, s_abort))) break;
      __syncwarp();
      if (lane == 0) piece_done(&bars->ring, take);
      if (pc.row < 0) break;
      // the first tile's rows: nothing to do but wait for them (three warps had them
      // ready 24000 clk after the kernel's start, eleven 18000)
      if (tiles == 0) {
        split_q_rows<BF16, HD>(p, sQ, sQs, pc, warp - 1, 11);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_more);
      }
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
          // A row that stands beyond its keys is moved up to them, and what that
          // takes off every distance is added to the result (cache_fwd.cuh).
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
      float in_scale = call_scale;
      uint64_t l2 = f2_make(0.f, 0.f), lr2 = l2;  // of P, and of P as V sees it
      vref.start();

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
        const bool keep = CAP || (POS && (kpos || p.slopes));
        auto no_box = [&](int c0) { return gone >> ((half * 64 + c0) >> box_log2) & 1; };
        auto mask = [&](float* x, int c0, int n) {
          const int lo = no_box(c0) ? n : jlo - key0 - c0, hi = jhi - key0 - c0;
#pragma unroll
          for (int i = 0; i < n; ++i) x[i] = i >= lo && i <= hi ? x[i] : -INFINITY;
        };
        const float* ks = bars->scale[step % kStepsHeld][0] + half * 4;
        const float* vs = bars->scale[step % kStepsHeld][1] + half * 4;
        // base-2 logits (less bref) of columns [c0, c0 + 16) from their products
        auto logits16 = [&](float* x, int c0) {
          const float in = in_scale * ks[c0 >> 4];
          if (CAP) {
            const float exp_scale = 2.f * kLog2e * in;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              if (FIXED) {
                // c - 2c / (1 + e^2x): the cap is small, so its absolute error of
                // c 2^-22 is that of the logit itself; the constant c is in bref.  (One
                // reciprocal for two needs clamps and four products: 244 against 242 us.)
                const uint64_t y = f2_mul(f2_make(x[i], x[i + 1]), f2_make(exp_scale, exp_scale));
                const uint64_t d = f2_add(f2_make(ex2_approx(f2_lo(y)), ex2_approx(f2_hi(y))), f2_make(1.f, 1.f));
                x[i] = rcp_approx(f2_lo(d));
                x[i + 1] = rcp_approx(f2_hi(d));
                continue;
              }
              const uint64_t th = tanh2_fp32(f2_mul(f2_make(x[i], x[i + 1]), f2_make(in, in)));
              x[i] = f2_lo(th);
              x[i + 1] = f2_hi(th);
            }
          }
          const float sc = FIXED ? -2.f * out_scale : (CAP ? out_scale : in);
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
        if (!(ok = mbar_wait8_warp(&bars->s_full[step & 1], (step >> 1) & 1, s_abort))) break;
        tc_fence_after();
        gone = bars->gone[step % kStepsHeld];
        edge = edge || gone;
        if (kt == pc.kt1 - 1) in_scale = call_scale * (valid ? sQs[(tiles & 3) * 128 + r] : 1.f);
        const float v_alpha = vref.step(bars->scale[step % kStepsHeld][1]);  // the same in every warp
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
              } else {
                const float in = in_scale * ks[c0 >> 4];
#pragma unroll
                for (int i = 0; i < kCh; ++i) x[i] *= in;
                if (edge) mask(x, c0, kCh);
              }
#pragma unroll
              for (int i = 0; i < kCh; ++i) mx = fmaxf(mx, x[i]);
            }
            if (keep) tmem_wait_st();
            mxs[half * 128 + r] = mx;
          }
          // the row's maximum over both halves
          if (!(ok = warp_exchange8(&bars->mx_x[quad][step & 1], (step >> 1) & 1, s_abort))) break;
          if (any) {
            mx = fmaxf(mx, mxs[(half ^ 1) * 128 + r]);
            need = mx > m_run + kLazy8;
            if (need) {
              alpha = ex2_approx(m_run - mx);
              m_run = mx;
            }
            l2 = f2_mul(l2, f2_make(alpha, alpha));
            lr2 = f2_mul(lr2, f2_make(alpha, alpha));
          }
        }
        // With FIXED, the first tile's maximum becomes the reference.  The tile is
        // passed over twice for that.  A later logit may lie as high as the cap
        // above the ALiBi term of the nearest key, so the reference stays within 15
        // of that and no P passes 2^15.
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
          if (!(ok = warp_exchange8(&bars->mx_x[quad][tiles & 1], (tiles >> 1) & 1, s_abort))) break;
          const float up = fmaxf(fmaxf(mx, mxs[(half ^ 1) * 128 + r]) - kShift8, out_scale - 15.f);
          m_run += up;
          bref += up;
        }
        if (any) {
          const float m_use = FIXED ? 0.f : (m_run == -INFINITY ? 0.f : m_run - kShift8);
#pragma unroll 1
          for (int c0 = 0; c0 < 64; c0 += kCh) {
            float x[kCh];
            tmem_ld16(sb + c0, x);
            tmem_wait_ld();
            if constexpr (FIXED) {
              logits16(x, c0);
            } else {
              const float sc = keep ? 1.f : in_scale * ks[c0 >> 4];
#pragma unroll
              for (int i = 0; i < kCh; i += 2) {
                const uint64_t z = f2_fma(f2_make(x[i], x[i + 1]), f2_make(sc, sc), f2_make(-m_use, -m_use));
                x[i] = f2_lo(z);
                x[i + 1] = f2_hi(z);
              }
              if (!keep && edge) mask(x, c0, kCh);
            }
            uint32_t pk[kCh / 2];
            const uint64_t l_was = l2, lr_was = lr2;
#pragma unroll
            for (int i = 0; i < kCh; i += 2) {
              x[i] = ex2_approx(x[i]);
              x[i + 1] = ex2_approx(x[i + 1]);
              l2 = f2_add(l2, f2_make(x[i], x[i + 1]));
              if constexpr (CAP) {
                pk[i >> 1] = Pack<false>::two(x[i], x[i + 1]);
                lr2 = f2_add(lr2, Pack<false>::unpack(pk[i >> 1]));
              } else {
                // Cut to fp16's 11 bits (those below 2^-14 are rounded once more, by 2^-25 at
                // most): the sum that divides takes the bias out again.  Rounded and widened as
                // above 413 us (192 rows a key) and 609 (a prompt), so 388 and 569; with a cap
                // the same, drafts 228 and 230.
                const float a = __int_as_float(__float_as_int(x[i]) & 0xffffe000);
                const float b = __int_as_float(__float_as_int(x[i + 1]) & 0xffffe000);
                pk[i >> 1] = Pack<false>::two(a, b);
                lr2 = f2_add(lr2, f2_make(a, b));
              }
            }
            const float rest = vref.of_p(vs[c0 >> 4]);
            if (rest < 1.f) {  // (a scale that is no power of two, or far below the others)
              // The rounded weights count as what they stand for, unless a far block's lose
              // bits that its own keys do not need and the sum does.
              uint64_t rb = f2_make(0.f, 0.f);
#pragma unroll
              for (int i = 0; i < kCh; i += 2) {
                pk[i >> 1] = Pack<false>::two(x[i] * rest, x[i + 1] * rest);
                rb = f2_add(rb, Pack<false>::unpack(pk[i >> 1]));
              }
              const float back = rcp_approx(rest);
              lr2 = rest < 0.5f ? f2_add(lr_was, f2_add(l2, f2_mul(l_was, f2_make(-1.f, -1.f)))) : f2_fma(rb, f2_make(back, back), lr_was);
            }
            tmem_st8(sb + c0 / 2, pk);
          }
          if (kt < pc.kt1 - 1 && (v_alpha != 1.f || (!FIXED && __any_sync(0xffffffffu, need)))) {
            // O follows the new references, once the previous products are in
            // it: this half's features
            if (!(ok = mbar_wait8_warp(&bars->pv_done[(step - 1) & 1], ((step - 1) >> 1) & 1, s_abort)))
              break;
            tc_fence_after();
            constexpr int kC = HD / 2;
            const uint32_t ob = tmem + kColO8 + half * kC + lane_addr;
            const float by = alpha * v_alpha;
#pragma unroll 1
            for (int c = 0; c < kC; c += 16) {
              float o[16];
              tmem_ld16(ob + c, o);
              tmem_wait_ld();
              uint32_t u[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i] * by);
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
      if (!(ok = warp_exchange8(&bars->l_x[quad], tiles & 1, s_abort))) break;
      const float l = sums[r].x + sums[128 + r].x, lr = sums[r].y + sums[128 + r].y;
      if (!(ok = mbar_wait8_warp(&bars->o_full, tiles & 1, s_abort))) break;
      tc_fence_after();
      if (any) {
        constexpr int kC = HD / 2;
        const float m_ref = FIXED ? m_run : (m_run == -INFINITY ? 0.f : m_run - kShift8);
        const float inv = pc.mode ? vref.ref : (lr > 0.f ? vref.ref / lr : 0.f);
        int64_t pr = 0;
        if (pc.mode)
          pr = pc.mode == 1 ? cut_row(w, blockIdx.x, pc.first, r) : whole_row(w, p.total_q, p.Hq, pc.own, tok, h);
        if (valid && half == 0) {
          if (pc.mode)
            reinterpret_cast<float4*>(p.ws + w.stats)[pr] = make_float4(m_ref, l, lr, m0);
          else
            p.lse[static_cast<int64_t>(tok) * p.Hq + h] = l > 0.f ? (m_ref + log2f(l) + m0) * kLn2 : -INFINITY;
        }
        uint16_t* orow = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(tok) * p.out_ts +
                         static_cast<int64_t>(h) * p.out_hs + half * kC;
        float4* part = reinterpret_cast<float4*>(p.ws + w.rows) + part_at<HD>(pr, half * kC / 4);
#pragma unroll 1
        for (int c = 0; c < kC; c += 16, part += 32) {
          float o[16];
          tmem_ld16(tmem + kColO8 + half * kC + c + lane_addr, o);
          tmem_wait_ld();
          if (!valid) continue;
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] *= inv;
          if (pc.mode == 0) {
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
  } else if (warp < 16) {
    warpgroup_reg_dealloc<kRegsConv8>();
    // ------------------------------------------------------------ V's bytes to fp16
    convert_v<BF16, HD>(bars, sm + S::kOffRV, sV, s_abort);
  } else {
    warpgroup_reg_dealloc<kRegsQ8>();
    if (warp == 16) {
      // ------------------------------------------------------------ V bytes
      load_pages8<BF16, HD, false>(p8, bars, sm + S::kOffRV, &tv, nullptr, box, s_abort);
    } else {
      // ------------------------------------------------------------ Q rows
      uint32_t take = 0, tiles = 0;
      Piece pc;
      for (;;) {
        if (!__all_sync(0xffffffffu, piece_take8(&bars->ring, take, &pc, s_abort))) break;
        __syncwarp();
        if (lane == 0) piece_done(&bars->ring, take);
        if (pc.row < 0) break;
        if (tiles > 0 && !mbar_wait8_warp(&bars->q_empty, (tiles - 1) & 1, s_abort)) break;
        // (the factors of four tiles ago are not read any more: S of the last tile
        // is done, so P of two steps before it has been multiplied)
        split_q_rows<BF16, HD>(p, sQ, sQs + (tiles & 3) * 128, pc, warp - 17, tiles ? 3 : 11);
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
  behind_few();
}

// A softcap of at most kFixedCap8 at default key positions.
inline bool fixed_reference8(const CacheParams& p) {
  return p.softcap > 0.f && p.softcap <= kFixedCap8 && !p.own.pos && !(p.P && p.prefix.pos);
}

template <bool B, int HD>
auto pick_fwd8(const CacheParams& p) {
  const bool moved = p.own.pos || (p.P && p.prefix.pos);
  const bool pos = p.slopes || p.wl >= 0 || p.wr >= 0 || moved;
  if (!(p.softcap > 0.f))
    return pos ? cache8_fwd_kernel<B, HD, false, false, true>
               : cache8_fwd_kernel<B, HD, false, false, false>;
  if (fixed_reference8(p))
    return pos ? cache8_fwd_kernel<B, HD, true, true, true>
               : cache8_fwd_kernel<B, HD, true, true, false>;
  return pos ? cache8_fwd_kernel<B, HD, true, false, true>
             : cache8_fwd_kernel<B, HD, true, false, false>;
}

template <int HD>
cudaError_t launch_fwd8_d(const Cache8Params& p, const FwdWs& w, const CUtensorMap& tk, const CUtensorMap& tkt,
                          const CUtensorMap& tv, int grid, cudaStream_t s) {
  constexpr uint32_t kBf = Fwd8Shape<true, HD>::kOffBar + sizeof(Fwd8Bars);
  constexpr uint32_t kHf = Fwd8Shape<false, HD>::kOffBar + sizeof(Fwd8Bars);
  static_assert(kBf <= 232448 && kHf <= 232448, "shared memory");
  const uint32_t smem = p.c.dtype == 1 ? kBf : kHf;
  auto k = p.c.dtype == 1 ? pick_fwd8<true, HD>(p.c) : pick_fwd8<false, HD>(p.c);
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads8);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.c.most_rows ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, p, w, tk, tkt, tv);
}

}  // namespace kv
}  // namespace attn
