// append8.cu -- new tokens into a paged cache held in 8 bits: K rows normed and
// turned on the way, K and V rows quantised to e4m3 with a scale for each block of
// slots and head.
//
// A value is scale * q with q an e4m3 number (|q| <= 448).  Scales are powers of
// two: a product with one is exact, so a block whose scale has to grow when a
// larger token arrives loses nothing of its held values but what falls below
// e4m3's smallest step, and with e4m3's own exponent a finer scale would gain
// nothing.  For the new rows of a block, top = their largest |value|:
//   was = the block's scale if it holds slots already, else 0
//   now = was if top <= 448 was, else the smallest power of two (2^-126 at least)
//         with top <= 448 now; 0 when all is 0
//   q = rn(x / now), and held values become rn(q was / now).
//
// Rows are fp32 from the load to the one rounding (values near a border of e4m3 in twice
// the digits, below).  A block of threads takes a run
// of tokens of one head of K or of V: the tokens that begin a block of slots (or a
// sequence) own that block and bring in its other new tokens, so every block of
// slots has one writer.  All its rows stay in registers between the maximum and
// the rounding (NIT passes of 16 warps), nothing is read twice.
//
// Bound by a block's own latency: its rows, positions and held scales are three
// dependent reads before the first product.  Measured: a token each of 64 sequences,
// 8 heads of 128, normed and turned (bf16): 8.6 us; 9 prompts of up to 12000 tokens
// (17 thousand in all), one head of 160: 17.2 us, 1 TB/s of its 16.5 MB.
#include <cuda_fp8.h>

#include "../../include/attn_varlen.h"
#include "rowfrag.cuh"

namespace attn {
namespace kv {
namespace {

constexpr int kWarpsQ = 16, kThreadsQ = kWarpsQ * 32;
constexpr int kMaxTokensQ = 64;  // of a block: two for each lane of a warp
constexpr int kCuQ = 256;        // entries of cu_new that a block keeps
constexpr float kLeastScale = 1.1754943508222875e-38f;  // 2^-126
constexpr float kFarUp = 18446744073709551616.f;        // 2^64

template <int D>
constexpr int pass_rows() { return kWarpsQ * RowShape<D>::kRowsWarp; }

__device__ __forceinline__ float pow2_scale(float top) {
  if (!(top > 0.f)) return 0.f;
  const int bits = __float_as_int(fminf(top, 3.402823466e38f));
  // top = 1.m 2^e: above 1.75 2^e it takes 2^(e-7), else 2^(e-8)
  const int e = (bits >> 23) - ((bits & 0x7fffff) > 0x600000 ? 7 : 8);
  return __int_as_float(max(e, 1) << 23);
}

// A value that lies within fp32's error of a border of e4m3 falls to one side or the
// other by chance, a sixteenth apart: of the K rows of 17 thousand tokens, a few.  So
// K rows are normed and turned in fp32 first, by at most kOffTurn or kOffNorm of their
// size off, and the pairs with a value nearer than that to a border once more in twice
// the digits (rows that turn through shared memory are not: they may be off by that).
// Borders, e4m3's and those of its smallest numbers, are numbers of four bits after the
// leading one, whatever the block's factor (a power of two): between two of them the
// other bits count up.
//
// Two: two numbers that stand for their sum, |l| at most half a step of h.
struct Two {
  float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {  // |a| >= |b|
  const float h = __fadd_rn(a, b);
  return {h, __fsub_rn(b, __fsub_rn(h, a))};
}
__device__ __forceinline__ Two two_product(float a, float b) {
  const float h = __fmul_rn(a, b);
  return {h, __fmaf_rn(a, b, -h)};
}
// a c + b s.
__device__ __forceinline__ Two two_dot(float a, Two c, float b, Two s) {
  const Two p = two_product(a, c.h), q = two_product(b, s.h);
  const float d = __fadd_rn(p.h, q.h), z = __fsub_rn(d, p.h);
  const float off = __fadd_rn(__fsub_rn(p.h, __fsub_rn(d, z)), __fsub_rn(q.h, z));
  return two_sum(d, off + (p.l + q.l) + fmaf(a, c.l, b * s.l));
}
// In fp32, with an odd last bit if it is not exact: a later rounding to fewer bits then
// goes the way that the pair's own would.
__device__ __forceinline__ float to_odd(Two x) {
  const int b = __float_as_int(x.h);
  return __int_as_float(x.l == 0.f || (b & 1) ? b : ((x.l > 0.f) == (x.h > 0.f) ? b + 1 : b - 1));
}

struct Turn {
  Two c, s;
};
// (cos, sin) of `pos` times a turn fraction, off by less than 2^-27: the angle's distance
// from the nearest quarter turn, at most pi / 4, into the Taylor series.
__device__ __forceinline__ Turn turn_two(int64_t pos, uint64_t per_pos) {
  const uint32_t u = static_cast<uint32_t>((static_cast<uint64_t>(pos) * per_pos + 0x80000000u) >> 32);
  const uint32_t quarter = (u + 0x20000000u) >> 30;
  const int32_t d = static_cast<int32_t>(u - (quarter << 30));
  const float dh = static_cast<float>(d), dl = static_cast<float>(d - static_cast<int32_t>(dh));
  constexpr double kTurn = 6.283185307179586477 / 4294967296.0;
  constexpr float kHi = static_cast<float>(kTurn), kLo = static_cast<float>(kTurn - kHi);
  Two t = two_product(dh, kHi);
  t.l += fmaf(dh, kLo, dl * kHi);
  const Two q = two_product(t.h, t.h);
  float p = fmaf(q.h, 1.f / 362880, -1.f / 5040);
  p = fmaf(q.h, fmaf(q.h, p, 1.f / 120), -1.f / 6);
  Two sn = two_sum(t.h, t.h * q.h * p);
  sn.l += fmaf(-0.5f * q.h, t.l, t.l);
  float r = fmaf(q.h, -1.f / 3628800, 1.f / 40320);
  r = fmaf(q.h, fmaf(q.h, r, -1.f / 720), 1.f / 24);
  Two cn = two_sum(1.f, -0.5f * q.h);
  cn.l += fmaf(q.h * q.h, r, -fmaf(t.h, t.l, 0.5f * q.l));
  Turn x = quarter & 1 ? Turn{sn, cn} : Turn{cn, sn};
  if ((quarter + 1) & 2) x.c = {-x.c.h, -x.c.l};
  if (quarter & 2) x.s = {-x.s.h, -x.s.l};
  return x;
}
__device__ __forceinline__ void turn_pair(const Turn& t, float& a, float& b) {
  const float x = a;
  a = to_odd(two_dot(x, t.c, -b, t.s));
  b = to_odd(two_dot(b, t.c, x, t.s));
}

// turn_of (rotary.cuh) to fp32's accuracy.  The angle goes to fp32 as its distance from
// the nearest quarter turn (off by 2^-27 of a half turn).
__device__ __forceinline__ float2 turn_fp32(int64_t pos, uint64_t per_pos) {
  const uint32_t u = static_cast<uint32_t>((static_cast<uint64_t>(pos) * per_pos) >> 32);
  const uint32_t quarter = (u + 0x20000000u) >> 30;
  float sn, cn;
  sincospif(static_cast<float>(static_cast<int32_t>(u - (quarter << 30))) * 4.656612873077393e-10f, &sn, &cn);
  const float a = quarter & 1 ? sn : cn, b = quarter & 1 ? cn : sn;
  return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

// x w / the row's size.
__device__ __forceinline__ float normed(float x, float w, float r0, float r1) {
  const Two rw = two_product(r0, w), y = two_product(x, rw.h);
  return to_odd(two_sum(y.h, fmaf(x, fmaf(r1, w, rw.l), y.l)));
}

// fp32's error of a turned pair, relative to the sum of its magnitudes, in 2^-24: sine and
// cosine 1, the angle 0.6, the products and the sum 1/2 each; with a norm 2 for its factor
// and products.
constexpr float kOffTurn = 3.f / (1 << 24), kOffNorm = 6.f / (1 << 24);
// Whether a value may lie on the other side of a border.
__device__ __forceinline__ uint32_t near_border(float y, float off) {
  return (__float_as_int(y + off) ^ __float_as_int(y - off)) & 0xfff80000u;
}
// Features fa and fb of a row once more.  A call, so that the rows keep their registers:
// inlined, the kernel of prompts spilled (18.2 us; so 17.1, without any of this 15.1, all
// pairs in twice the digits 19.8).
template <bool BF16>
__device__ __noinline__ float2 redo_pair(const uint16_t* row, int fa, int fb, int norm, const float* w, float r0, float r1, bool turned,
                                         const int32_t* pos, uint64_t per_pos) {
  float a = to_float<BF16>(row[fa]), b = to_float<BF16>(row[fb]);
  if (norm) {
    a = normed(a, w ? __ldg(w + fa) : 1.f, r0, r1);
    b = normed(b, w ? __ldg(w + fb) : 1.f, r0, r1);
  }
  if (turned) turn_pair(turn_two(__ldg(pos), per_pos), a, b);
  return make_float2(a, b);
}
// Turns pair e of a lane and notes it in `near` if a value is near a border.
__device__ __forceinline__ void turn_checked(float& a, float& b, int e, float off, const float2& c, uint32_t& near) {
  off *= fabsf(a) + fabsf(b);
  turn2<true>(c, a, b);
  if (near_border(a, off) | near_border(b, off)) near |= 1u << e;
}

__device__ __forceinline__ uint2 pack_e4m3(const float (&v)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

struct Job {         // a block of slots with new tokens
  int tok, start;    // its first new token, and that token's row here
  int held;          // slots it holds already
  int64_t at, scale; // its first slot's place in the pool (elements), its scale's
  float was, now, up, inv;  // inv: 1 / (now up)
  int top;           // bits of the largest |value|
};

struct Append8Smem {
  int cu[kCuQ + 1];
  Job job[kMaxTokensQ];
  int jobs, rows;
  int seq[kMaxTokensQ], slot[kMaxTokensQ];  // seq -1: not taken
  uint64_t per_pos[kMaxPairs];
  int64_t axis_row[kMaxPairs];
};

template <bool BF16, int D, bool VEC, int NIT>
__global__ void __launch_bounds__(kThreadsQ, NIT <= 2 ? 2 : 1)
    append8_kernel(const __grid_constant__ Append8Params p8, int ntok) {
  using S = RowShape<D>;
  __shared__ Append8Smem sm;
  __shared__ float rowbuf[VEC ? 1 : kWarpsQ * (S::kRowsWarp + 1)][VEC ? 1 : D + 4];
  const AppendParams& p = p8.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.y >> 1, is_v = blockIdx.y & 1;  // head, tensor
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * ntok;
  ntok = static_cast<int>(min(static_cast<int64_t>(ntok), p.T - tok0));
  const Pages& pool = is_v ? p.v : p.k;
  const Scales& sc = is_v ? p8.vs : p8.ks;
  const int sb = p8.block;
  const int pairs = !is_v && p.r.inv_freq ? p.r.pairs : 0;

  int bad = 0;
  const bool kept = p.B <= kCuQ;  // (searched in shared memory then: a chain of loads otherwise)
  for (int b = tid; b < p.B; b += kThreadsQ) {
    const int c0 = __ldg(p.cu_new + b), c1 = __ldg(p.cu_new + b + 1);
    bad |= c0 < 0 || c1 < c0 || c1 > p.T || (b == 0 && c0 != 0);
    if (kept) {
      sm.cu[b] = c0;
      if (b == p.B - 1) sm.cu[p.B] = c1;
    }
  }
  // the rows that the lookups below will ask for
  if (tid >= 32 && tid - 32 < ntok)
    for (int f = 0; f < D; f += 64)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint16_t*>(is_v ? p.vx : p.kx) + (tok0 + tid - 32) * (is_v ? p.v_ts : p.k_ts) + g * (is_v ? p.v_hs : p.k_hs) + f));
  if (tid >= 128 && tid - 128 < pairs) {
    const int i = tid - 128, ax = p.r.pair_axis ? __ldg(p.r.pair_axis + i) : 0;
    sm.per_pos[i] = turn_fraction(__ldg(p.r.inv_freq + i));
    sm.axis_row[i] = min(max(ax, 0), p.r.axes - 1) * p.r.axis_stride;
  }
  if (kept) __syncthreads();
  if (warp == 0) {
    int jobs = 0, rows = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int t = half * 32 + lane, tok = static_cast<int>(tok0) + t;
      int seq = -1, slot = 0, n = 0, held = 0;
      int64_t at = 0, scale = 0;
      float was = 0.f;
      const int* cu = kept ? sm.cu : p.cu_new;
      if (t < ntok && tok < cu[p.B]) {  // tokens behind the last sequence are left out
        int b = 0;  // the last sequence that starts at or before the token
        for (int end = p.B; end - b > 1;) {
          const int mid = (b + end) >> 1;
          if (cu[mid] <= tok)
            b = mid;
          else
            end = mid;
        }
        const int c0 = cu[b], c1 = cu[b + 1];
        // (cu_new may be anything still: only a token of its own run is looked up)
        const int first = c0 >= 0 && c0 <= tok && tok < c1 ? append_at(p, b, c1 - c0) : -1;
        int page = -1;
        if (first >= 0) {
          slot = first + tok - c0;
          page = __ldg(p.table + b * p.table_rs + (slot >> p.page_log2));
        }
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) {
          seq = b;
          const int in_block = slot & (sb - 1), in_page = slot & (p.page_size - 1);
          if (in_block == 0 || tok == c0) {
            held = in_block;
            n = min(sb - in_block, c1 - tok);
            at = page * pool.page + static_cast<int64_t>(in_page - in_block) * pool.slot + g * pool.head;
            scale = page * sc.page + static_cast<int64_t>(in_page >> p8.block_log2) * sc.block + g * sc.head;
            if (held) was = sc.base[scale];
          }
        } else if (blockIdx.y == 0) {
          seq = -2;
        }
      }
      if (t < kMaxTokensQ) {
        sm.seq[t] = seq;
        sm.slot[t] = slot;
      }
      const uint32_t lead = __ballot_sync(0xffffffffu, n > 0);
      int upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      if (n > 0) {
        Job& job = sm.job[jobs + __popc(lead & ((1u << lane) - 1u))];
        job.tok = tok;
        job.start = rows + upto - n;
        job.held = held;
        job.at = at;
        job.scale = scale;
        job.was = was;
        job.top = 0;
      }
      jobs += __popc(lead);
      rows += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) {
      sm.jobs = jobs;
      sm.rows = rows;
    }
  }
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (bad && tid == 0) report(p.status, ATTN_DEV_BAD_CU);
    for (int b = tid; b < p.B && (p.lens_out || !bad); b += kThreadsQ) {
      const int n = bad ? 0 : __ldg(p.cu_new + b + 1) - __ldg(p.cu_new + b);
      const int at = append_at(p, b, n);
      if (!bad && at < 0) report(p.status, ATTN_DEV_BAD_CACHE);
      if (p.lens_out) p.lens_out[b] = at < 0 ? __ldg(p.lens + b) : at + n;
    }
  }
  if (bad) return;
  if (blockIdx.y == 0) {
    if (tid < ntok && sm.seq[tid] == -2) report(p.status, ATTN_DEV_BAD_CACHE);
    if (p.key_pos)
      for (int i = tid; i < ntok * p.Hkv; i += kThreadsQ) {
        const int t = i / p.Hkv, h = i - t * p.Hkv;
        if (sm.seq[t] >= 0)
          p.key_pos[sm.seq[t] * p.kp_rs + h * p.kp_hs + sm.slot[t]] =
              p.r.positions ? __ldg(p.r.positions + tok0 + t) : sm.slot[t];
      }
  }
  const int jobs = sm.jobs, rows = sm.rows;
  if (jobs == 0) return;

  // ---- the rows, turned, and the largest value of each block of slots
  const int j = lane % S::kLanes, rg = lane / S::kLanes;
  const Units u = item_units<VEC>(j, pairs, p.r.interleaved);
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? p.vx : p.kx) + g * (is_v ? p.v_hs : p.k_hs);
  const int64_t src_ts = is_v ? p.v_ts : p.k_ts;
  float v[NIT][2][8];
  int of[NIT], tok[NIT];  // the row's job (-1: none) and token
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    const int row = it * pass_rows<D>() + warp * S::kRowsWarp + rg;
    of[it] = -1;
    tok[it] = 0;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (rg < S::kRowsWarp && row < rows) {
      int lo = 0, hi = jobs;  // the last job that starts at or before the row
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sm.job[mid].start <= row)
          lo = mid;
        else
          hi = mid;
      }
      of[it] = lo;
      tok[it] = sm.job[lo].tok + row - sm.job[lo].start;
      const uint16_t* x = src + tok[it] * src_ts;
      a = __ldcs(reinterpret_cast<const uint4*>(x + u.a));
      b = __ldcs(reinterpret_cast<const uint4*>(x + u.b));
    }
    unpack8<BF16>(a, v[it][0]);
    unpack8<BF16>(b, v[it][1]);
  }
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    float(&x)[2][8] = v[it];
    float r0 = 1.f, r1 = 0.f;  // 1 / the row's size, in two terms
    uint32_t near = 0;         // pairs of this lane with a value near a border
    const int n = min(max(pairs - 8 * j, 0), 8);  // its pairs that turn
    if (!is_v && p8.norm) {
      float sq[4] = {};  // (four short sums: half the roundings of one)
#pragma unroll
      for (int e = 0; e < 8; ++e) sq[e & 3] = fmaf(x[0][e], x[0][e], fmaf(x[1][e], x[1][e], sq[e & 3]));
      const float mean = row_sum<D>((sq[0] + sq[1]) + (sq[2] + sq[3])) / D + p8.eps;
      r0 = rsqrtf(mean);
      const Two m = two_product(mean, r0);  // a step of Newton's: r0 + r0 (1 - mean r0^2) / 2
      r1 = 0.5f * r0 * (__fmaf_rn(-m.h, r0, 1.f) - m.l * r0);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[0][e] *= (r0 + r1) * (p8.k_weight ? __ldg(p8.k_weight + u.a + e) : 1.f);
        x[1][e] *= (r0 + r1) * (p8.k_weight ? __ldg(p8.k_weight + u.b + e) : 1.f);
      }
      if (VEC && n < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // (of an interleaved lane the last four pairs alone may stay as they are)
          const float a = p.r.interleaved ? x[e >> 2][2 * (e & 3)] : x[0][e], b = p.r.interleaved ? x[e >> 2][2 * (e & 3) + 1] : x[1][e];
          if (e >= n && (near_border(a, fabsf(a) * kOffNorm) | near_border(b, fabsf(b) * kOffNorm))) near |= 1u << e;
        }
      }
    }
    if (pairs) {
      auto turn = [&](int i) { return turn_fp32(__ldg(p.r.positions + sm.axis_row[i] + tok[it]), sm.per_pos[i]); };
      if (VEC) {
        const float off = p8.norm ? kOffNorm : kOffTurn;
        if (!p.r.interleaved) {
          if (n > 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) turn_checked(x[0][e], x[1][e], e, off, turn(8 * j + e), near);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (n > 4 * h) {
#pragma unroll
              for (int e = 0; e < 4; ++e) turn_checked(x[h][2 * e], x[h][2 * e + 1], 4 * h + e, off, turn(8 * j + 4 * h + e), near);
            }
        }
      } else {
        turn_row(x, rowbuf[warp * (S::kRowsWarp + 1) + rg], j, pairs, p.r.interleaved, turn);
      }
    }
    if (of[it] < 0) near = 0;
    while (near) {  // (a pair in some ten thousand)
      const int e = __ffs(near) - 1;
      near &= near - 1;
      const int fa = p.r.interleaved ? 16 * j + 2 * e : u.a + e, fb = p.r.interleaved ? fa + 1 : u.b + e;
      const int i = 8 * j + e;
      const float2 y = redo_pair<BF16>(src + tok[it] * src_ts, fa, fb, p8.norm, p8.k_weight, r0, r1, e < n,
                                       e < n ? p.r.positions + sm.axis_row[i] + tok[it] : nullptr, sm.per_pos[i]);
#pragma unroll
      for (int k = 0; k < 16; ++k) {  // (features of this lane: units a and b)
        const int f = (k & 8 ? u.b : u.a) + (k & 7);
        if (f == fa) x[k >> 3][k & 7] = y.x;
        if (f == fb) x[k >> 3][k & 7] = y.y;
      }
    }
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(x[0][e]), fabsf(x[1][e])));
    top = row_max<D>(top);
    if (of[it] >= 0 && j == 0) atomicMax(&sm.job[of[it]].top, __float_as_int(top));
  }
  __syncthreads();
  if (tid < jobs) {
    Job& job = sm.job[tid];
    const float top = __int_as_float(job.top);
    job.now = top <= 448.f * job.was ? job.was : pow2_scale(top);
    // (another quantiser's factor may be too small for its reciprocal: value 2^64 / (now 2^64))
    job.up = job.now < kLeastScale ? kFarUp : 1.f;
    job.inv = job.now > 0.f ? 1.f / (job.now * job.up) : 0.f;
    sc.base[job.scale] = job.now;
  }
  __syncthreads();

  // ---- the new values
  uint8_t* dst = static_cast<uint8_t*>(const_cast<void*>(pool.base));
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    if (of[it] < 0) continue;
    const Job& job = sm.job[of[it]];
    uint8_t* y = dst + job.at + static_cast<int64_t>(job.held + tok[it] - job.tok) * pool.slot;
    if (job.up != 1.f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[it][0][e] *= job.up;
        v[it][1][e] *= job.up;
      }
    }
    *reinterpret_cast<uint2*>(y + u.a) = pack_e4m3(v[it][0], job.inv);
    *reinterpret_cast<uint2*>(y + u.b) = pack_e4m3(v[it][1], job.inv);
  }
  // ---- held values of blocks whose scale grew
  for (int i = 0; i < jobs; ++i) {
    const Job& job = sm.job[i];
    if (job.held == 0 || job.now == job.was) continue;
    const float by = job.now > 0.f ? job.was / job.now : 0.f;
    for (int w = tid; w < job.held * (D / 8); w += kThreadsQ) {
      const int s = w / (D / 8), f = (w - s * (D / 8)) * 8;
      uint2* y = reinterpret_cast<uint2*>(dst + job.at + static_cast<int64_t>(s) * pool.slot + f);
      const uint2 q = *y;
      float x[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t word = k < 2 ? q.x : q.y;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(k & 1 ? word >> 16 : word & 0xffffu), __NV_E4M3);
        const float2 two = __half22float2(*reinterpret_cast<const __half2*>(&h));
        x[2 * k] = two.x;
        x[2 * k + 1] = two.y;
      }
      *y = pack_e4m3(x, by);
    }
  }
}

template <int D>
cudaError_t launch_d(const Append8Params& p, cudaStream_t s) {
  // passes: enough for the block's other tokens and 16 to begin one
  const int one = pass_rows<D>(), need = p.block + 15;
  int nit = need <= one ? 1 : (need <= 2 * one ? 2 : 4);
  // Two passes also where one would take more blocks than are resident: each block is
  // a chain of lookups of about 4 us however many rows it takes.
  if (nit == 1 && p.a.T * 2 * p.a.Hkv > static_cast<int64_t>(one - p.block + 1) * 304) nit = 2;
  static_assert(4 * pass_rows<D>() >= 128 + 15, "four passes hold the largest blocks");
  int64_t ntok = nit * one - p.block + 1;
  if (ntok > kMaxTokensQ) ntok = kMaxTokensQ;
  // few tokens: over more blocks of threads
  const int64_t spread = p.a.T * 2 * p.a.Hkv / 152;
  if (ntok > spread) ntok = spread < 1 ? 1 : spread;
  const dim3 grid(p.a.T > 0 ? static_cast<unsigned>((p.a.T + ntok - 1) / ntok) : 1u, 2 * p.a.Hkv);
  const bool vec = vector_pairs(p.a.r.inv_freq ? p.a.r.pairs : 0, p.a.r.interleaved), b = p.a.dtype == 1;
#define ATTN_GO(NIT)                                                                                          \
  if (nit == NIT) {                                                                                           \
    auto k = b ? (vec ? append8_kernel<true, D, true, NIT> : append8_kernel<true, D, false, NIT>)             \
               : (vec ? append8_kernel<false, D, true, NIT> : append8_kernel<false, D, false, NIT>);          \
    k<<<grid, kThreadsQ, 0, s>>>(p, static_cast<int>(ntok));                                                  \
  }
  ATTN_GO(1)
  ATTN_GO(2)
  if constexpr (pass_rows<D>() * 2 < 128 + 15) {
    ATTN_GO(4)
  }
#undef ATTN_GO
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append8(const Append8Params& p, cudaStream_t s) {
  return p.a.d == 160 ? launch_d<160>(p, s) : (p.a.d == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s));
}

}  // namespace kv
}  // namespace attn
