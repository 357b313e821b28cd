// norm.cu -- norms of the rows of q and k with the turn by rotary positions in
// the same pass, and the gradients.
//
// A row x of d features (one head of one token) with weights w:
//   r = (mean(x^2) + eps)^(-1/2),  n_i = x_i r w_i,  y = turn(n)
// and with g = turn^-1(dy), h_i = g_i w_i:
//   dx_i = r (h_i - x_i r mean(h x r)),  dw_i = sum over the rows of g_i x_i r.
// Everything between the load and the store is fp32; a row is rounded once.
//
// Bound by memory: the forward reads and writes each row once, the backward
// reads x and dy and writes dx.  A row lies in the registers of four to ten
// lanes (rowfrag.cuh), so its sums take a few shuffles and nothing is read
// twice; a block takes runs of tokens with all their heads, so one pair's sine
// serves them all.  The weights' gradients are summed per lane over the rows of a
// block, then over the lanes and warps, and a second kernel adds the blocks in
// their order: no atomics, the same bits every time.
//
// Measured (bf16, turned): forward, 16000 tokens x 97 heads of 160: 190 us, 5.2 TB/s
// of its 0.99 GB; backward, 9999 tokens x 40 heads of 128: 72 us, 4.3 TB/s; 64 tokens
// x 81 heads of 160: 4.2 us, one launch.  The forward spends 0.6 of its issue slots,
// most on the values themselves, and three resident blocks (80 registers) beat two
// (85: 228 against 209 us); two rows in flight a lane took 244 us.
#include "../../include/attn_varlen.h"
#include "rowfrag.cuh"

namespace attn {
namespace kv {
namespace {

constexpr int kSms = 152;
// Warps of a block: rows that are turned through shared memory (VEC false) need
// a buffer each.
template <bool VEC>
constexpr int warps_n() { return VEC ? 8 : 4; }

// How one tensor's rows are cut into jobs: runs of ntok tokens x hs heads.
struct Jobs {
  int ntok, hs, splits;  // splits: head ranges of a run
  int64_t count;
};
Jobs jobs_of(int64_t T, int H, int rows_min) {
  Jobs j = {1, 1, 1, 0};
  if (H < 1) return j;
  // rows of a job: enough jobs for four rounds of the SMs, or as few rows as one
  // pass of a block takes
  int64_t rows = T * H / (4 * kSms);
  rows = rows < rows_min ? rows_min : (rows > 512 ? 512 : rows);
  if (H <= rows) {
    const int64_t n = rows / H;
    j.ntok = static_cast<int>(n > kMaxTokensR ? kMaxTokensR : n);
    j.hs = H;
  } else {
    j.splits = static_cast<int>((H + rows - 1) / rows);
    j.hs = (H + j.splits - 1) / j.splits;
    j.splits = (H + j.hs - 1) / j.hs;
  }
  j.count = (T + j.ntok - 1) / j.ntok * j.splits;
  return j;
}

struct NormPlan {
  Jobs job[2];
  int blocks[2];  // backward: blocks of each tensor
};

// A lane's part of a row.
template <bool BF16, bool VEC>
struct RowOps {
  uint4 raw[2];
  __device__ __forceinline__ void load(const uint16_t* x, const Units& u) {
    raw[0] = __ldcs(reinterpret_cast<const uint4*>(x + u.a));
    raw[1] = __ldcs(reinterpret_cast<const uint4*>(x + u.b));
  }
  __device__ __forceinline__ void fill(uint32_t v) { raw[0] = raw[1] = make_uint4(v, v, v, v); }
  // The 16 values as pairs.
  __device__ __forceinline__ void unpack(uint64_t (&v)[8]) const {
    const uint32_t u[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = Pack<BF16>::unpack(u[e]);
  }
  __device__ __forceinline__ static void store(uint16_t* y, const float (&v)[2][8], const Units& u) {
    __stcs(reinterpret_cast<uint4*>(y + u.a), pack8<BF16>(v[0]));
    __stcs(reinterpret_cast<uint4*>(y + u.b), pack8<BF16>(v[1]));
  }
  __device__ __forceinline__ static void weights(const float* w, uint64_t (&v)[8], const Units& u) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = w ? f2_make(__ldg(w + u.a + 2 * e), __ldg(w + u.a + 2 * e + 1)) : f2_make(1.f, 1.f);
      v[4 + e] = w ? f2_make(__ldg(w + u.b + 2 * e), __ldg(w + u.b + 2 * e + 1)) : f2_make(1.f, 1.f);
    }
  }
  __device__ __forceinline__ static void turn(float (&v)[2][8], float* row, int j, int pairs, bool interleaved,
                                              const float2* cs) {
    if (VEC)
      turn_item(v[0], v[1], j, pairs, interleaved, [&](int i, float2& a, float2& b) {
        const float4 x = *reinterpret_cast<const float4*>(cs + spread_pair(i));
        a = make_float2(x.x, x.y);
        b = make_float2(x.z, x.w);
      });
    else
      turn_row(v, row, j, pairs, interleaved, [&](int i) { return cs[i]; });
  }
};

struct Run {
  int64_t tok0;
  int ntok, h0, nh;
};
__device__ __forceinline__ Run run_of(const Jobs& j, int64_t T, int H, int64_t i) {
  Run r;
  const int64_t run = j.splits > 1 ? i / j.splits : i;
  r.tok0 = run * j.ntok;
  r.ntok = static_cast<int>(min(static_cast<int64_t>(j.ntok), T - r.tok0));
  r.h0 = static_cast<int>(i - run * j.splits) * j.hs;
  r.nh = min(j.hs, H - r.h0);
  return r;
}

// The lane's row of a run, by passes of the block: its token in the run, its head,
// and its place in N tensors, in elements from the run's first row.  Steps are
// additions: a division and the products of the strides for every row took a fifth
// of the forward's instructions.  Off: uint32_t where a run spans less than 2^31
// elements of every tensor (short_runs): 190 us for the forward above, 64-bit ones
// spill and take 204, the products 197.
template <int D, int STEP, class Off, int N>
struct Rows {
  int tok, h, left;  // left: rows from this one to the run's end
  Off off[N];
  int nh, dtok, dh;
  Off by[N], wrap[N];
  __device__ __forceinline__ Rows(const Run& run, int r0) {
    using S = RowShape<D>;
    const int g = (threadIdx.x & 31) / S::kLanes, row = r0 + g;
    nh = run.nh;
    left = g < S::kRowsWarp ? run.ntok * run.nh - row : 0;
    tok = left > 0 ? quotient(row, 1.f / nh) : 0;
    h = left > 0 ? row - tok * nh : 0;
    dtok = quotient(STEP, 1.f / nh);
    dh = STEP - dtok * nh;
  }
  __device__ __forceinline__ void tensor(int n, int h0, int64_t ts, int64_t hs) {
    off[n] = static_cast<Off>(tok * ts + (h0 + h) * hs);
    by[n] = static_cast<Off>(dtok * ts + dh * hs);
    wrap[n] = static_cast<Off>(ts - nh * hs);
  }
  __device__ __forceinline__ bool valid() const { return left > 0; }
  __device__ __forceinline__ void step() {
    left -= STEP;
    tok += dtok;
    h += dh;
#pragma unroll
    for (int n = 0; n < N; ++n) off[n] += by[n];
    if (h >= nh) {
      h -= nh;
      ++tok;
#pragma unroll
      for (int n = 0; n < N; ++n) off[n] += wrap[n];
    }
  }
};

template <int D, bool VEC>
struct NormSmem {
  Turns turns;
  // rows that are turned through shared memory (one more a warp for idle lanes)
  float rows[VEC ? 1 : warps_n<VEC>() * (RowShape<D>::kRowsWarp + 1)][VEC ? 1 : D + 4];
  __device__ __forceinline__ float* row() {
    using S = RowShape<D>;
    if (VEC) return nullptr;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    return rows[warp * (S::kRowsWarp + 1) + lane / S::kLanes];
  }
};

template <bool BF16, int D, bool VEC, class Off>
__global__ void __launch_bounds__(warps_n<VEC>() * 32, VEC ? 3 : 1)
    norm_kernel(const __grid_constant__ NormParams p, const __grid_constant__ NormPlan plan) {
  using S = RowShape<D>;
  using Ops = RowOps<BF16, VEC>;
  constexpr int kStep = warps_n<VEC>() * S::kRowsWarp;
  __shared__ NormSmem<D, VEC> sm;
  const int j = (threadIdx.x & 31) % S::kLanes;
  const bool inter = p.r.interleaved;
  const int pairs = p.r.inv_freq ? p.r.pairs : 0;
  const Units at = item_units<VEC>(j, pairs, inter);
  for (int64_t i = blockIdx.x; i < plan.job[0].count + plan.job[1].count; i += gridDim.x) {
    const int which = i >= plan.job[0].count;
    const NormTensor& t = p.t[which];
    const Run run = run_of(plan.job[which], p.T, t.H, which ? i - plan.job[0].count : i);
    const uint16_t* x0 = static_cast<const uint16_t*>(t.x) + run.tok0 * t.ts;
    uint16_t* y0 = static_cast<uint16_t*>(t.out) + run.tok0 * t.ots;
    const int all = run.ntok * run.nh;
    int r0 = (threadIdx.x >> 5) * S::kRowsWarp;
    Ops next;
    Rows<D, kStep, Off, 2> row(run, r0);
    row.tensor(0, run.h0, t.ts, t.hs);
    row.tensor(1, run.h0, t.ots, t.ohs);
    next.fill(0);
    if (row.valid()) next.load(x0 + row.off[0], at);
    if (pairs) {
      __syncthreads();
      fill_turns<VEC>(p.r, run.tok0, run.ntok, sm.turns);
    }
    uint64_t w[8];
    Ops::weights(t.weight, w, at);
    if (pairs) __syncthreads();
    for (; r0 < all; r0 += kStep) {
      uint64_t x[8];
      next.unpack(x);
      const bool valid = row.valid();
      const int tok = valid ? row.tok : 0;
      uint16_t* y = y0 + row.off[1];
      row.step();
      if (row.valid()) next.load(x0 + row.off[0], at);
      uint64_t sq = f2_mul(x[0], x[0]);
#pragma unroll
      for (int e = 1; e < 8; ++e) sq = f2_fma(x[e], x[e], sq);
      const float r = rsqrtf(row_sum<D>(f2_lo(sq) + f2_hi(sq)) * (1.f / D) + p.eps);
      float v[2][8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint64_t z = f2_mul(x[e], f2_mul(w[e], f2_make(r, r)));
        v[e >> 2][(e & 3) * 2] = f2_lo(z);
        v[e >> 2][(e & 3) * 2 + 1] = f2_hi(z);
      }
      if (pairs) Ops::turn(v, sm.row(), j, pairs, inter, sm.turns.cs[tok]);
      if (valid) Ops::store(y, v, at);
    }
  }
}

// Blocks [0, blocks[0]) take q, the others k.
template <bool BF16, int D, bool VEC, class Off>
__global__ void __launch_bounds__(warps_n<VEC>() * 32, VEC ? 2 : 1)
    norm_bwd_kernel(const __grid_constant__ NormParams p, const __grid_constant__ NormPlan plan) {
  using S = RowShape<D>;
  using Ops = RowOps<BF16, VEC>;
  constexpr int kWarps = warps_n<VEC>(), kStep = kWarps * S::kRowsWarp;
  __shared__ NormSmem<D, VEC> sm;
  __shared__ float sums[kWarps][D];
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = lane % S::kLanes;
  const bool inter = p.r.interleaved;
  const int pairs = p.r.inv_freq ? p.r.pairs : 0;
  const Units at = item_units<VEC>(j, pairs, inter);
  const int which = static_cast<int>(blockIdx.x) >= plan.blocks[0];
  const NormTensor& t = p.t[which];
  const Jobs& jobs = plan.job[which];
  uint64_t w[8], dw[8];
  Ops::weights(t.weight, w, at);
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = f2_make(0.f, 0.f);
  for (int64_t i = blockIdx.x - (which ? plan.blocks[0] : 0); i < jobs.count; i += plan.blocks[which]) {
    const Run run = run_of(jobs, p.T, t.H, i);
    const uint16_t* x0 = static_cast<const uint16_t*>(t.x) + run.tok0 * t.ts;
    const uint16_t* d0 = static_cast<const uint16_t*>(t.dy) + run.tok0 * t.dts;
    uint16_t* y0 = static_cast<uint16_t*>(t.out) + run.tok0 * t.ots;
    const int all = run.ntok * run.nh;
    int r0 = warp * S::kRowsWarp;
    Ops next, dnext;
    Rows<D, kStep, Off, 3> row(run, r0);
    row.tensor(0, run.h0, t.ts, t.hs);
    row.tensor(1, run.h0, t.ots, t.ohs);
    row.tensor(2, run.h0, t.dts, t.dhs);
    auto load = [&] {
      if (row.valid()) {
        next.load(x0 + row.off[0], at);
        dnext.load(d0 + row.off[2], at);
      } else {  // nothing of it may reach the sums: ones, whose r is finite with eps = 0 too, times zeros
        next.fill(BF16 ? 0x3f803f80u : 0x3c003c00u);
        dnext.fill(0);
      }
    };
    load();
    if (pairs) {
      __syncthreads();
      fill_turns<VEC>(p.r, run.tok0, run.ntok, sm.turns);
      __syncthreads();
    }
    for (; r0 < all; r0 += kStep) {
      uint64_t x[8], g[8];
      next.unpack(x);
      const bool valid = row.valid();
      const int tok = valid ? row.tok : 0;
      uint16_t* y = y0 + row.off[1];
      if (pairs) {
        float v[2][8];
        unpack8<BF16>(dnext.raw[0], v[0]);
        unpack8<BF16>(dnext.raw[1], v[1]);
        row.step();
        load();
        Ops::turn(v, sm.row(), j, pairs, inter, sm.turns.cs[tok]);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = f2_make(v[e >> 2][(e & 3) * 2], v[e >> 2][(e & 3) * 2 + 1]);
      } else {
        dnext.unpack(g);
        row.step();
        load();
      }
      uint64_t sq = f2_mul(x[0], x[0]), hx = f2_mul(f2_mul(g[0], w[0]), x[0]);
#pragma unroll
      for (int e = 1; e < 8; ++e) {
        sq = f2_fma(x[e], x[e], sq);
        hx = f2_fma(f2_mul(g[e], w[e]), x[e], hx);
      }
      const float r = rsqrtf(row_sum<D>(f2_lo(sq) + f2_hi(sq)) * (1.f / D) + p.eps);
      // dx = r h - x^ (r mean(h x^)), x^ = x r: r^3 in one factor would pass fp32's range
      // for rows below 2^-42 with eps = 0
      const float rc = -row_sum<D>(f2_lo(hx) + f2_hi(hx)) * (1.f / D) * r * r;  // -r mean(h x^)
      float v[2][8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint64_t gr = f2_mul(g[e], f2_make(r, r));
        dw[e] = f2_fma(gr, x[e], dw[e]);
        const uint64_t z = f2_fma(gr, w[e], f2_mul(f2_mul(x[e], f2_make(r, r)), f2_make(rc, rc)));
        v[e >> 2][(e & 3) * 2] = f2_lo(z);
        v[e >> 2][(e & 3) * 2 + 1] = f2_hi(z);
      }
      if (valid) Ops::store(y, v, at);
    }
  }
  if (!t.dweight) return;
  // over the warp's rows, then over the warps, each in a fixed order
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < S::kRowsWarp; ++g)
        s += __shfl_sync(0xffffffffu, e & 1 ? f2_hi(dw[u * 4 + e / 2]) : f2_lo(dw[u * 4 + e / 2]), g * S::kLanes + j);
      if (lane < S::kLanes) sums[warp][(u ? at.b : at.a) + e] = s;
    }
  __syncthreads();
  for (int f = threadIdx.x; f < D; f += kWarps * 32) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) s += sums[q][f];
    p.partial[static_cast<int64_t>(blockIdx.x) * D + f] = s;
  }
}

// dweight of tensor blockIdx.y, features 32 blockIdx.x and up: 32 warps add a
// part of the blocks each, then one adds the warps.
__global__ void __launch_bounds__(1024)
    norm_join_kernel(const __grid_constant__ NormParams p, const __grid_constant__ NormPlan plan) {
  __shared__ float sums[32][33];
  const int which = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int f = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float* out = p.t[which].dweight;
  if (!out) return;
  const float* part = p.partial + static_cast<int64_t>(which ? plan.blocks[0] : 0) * p.d + f;
  float s = 0.f;
  for (int b = warp; b < plan.blocks[which]; b += 32) s += part[static_cast<int64_t>(b) * p.d];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp) return;
  s = 0.f;
#pragma unroll
  for (int q = 0; q < 32; ++q) s += sums[q][lane];
  out[f] = s;
}

// (rows that are turned through shared memory have the one form)
template <template <bool, int, bool, class> class F, class... A>
void pick(const NormParams& p, bool vec, bool near, A... a, unsigned grid, cudaStream_t s) {
  const bool b = p.dtype == 1;
#define ATTN_GO(B, D)                                            \
  vec ? (near ? F<B, D, true, uint32_t>::go(a..., grid, s) : F<B, D, true, int64_t>::go(a..., grid, s)) \
      : F<B, D, false, int64_t>::go(a..., grid, s)
#define ATTN_PICK(D) \
  if (p.d == D) b ? (ATTN_GO(true, D)) : (ATTN_GO(false, D));
  ATTN_PICK(64)
  ATTN_PICK(128)
  ATTN_PICK(160)
#undef ATTN_PICK
#undef ATTN_GO
}
template <bool B, int D, bool V, class Off>
struct Fwd {
  static void go(const NormParams& p, const NormPlan& n, unsigned grid, cudaStream_t s) {
    norm_kernel<B, D, V, Off><<<grid, warps_n<V>() * 32, 0, s>>>(p, n);
  }
};
template <bool B, int D, bool V, class Off>
struct Bwd {
  static void go(const NormParams& p, const NormPlan& n, unsigned grid, cudaStream_t s) {
    norm_bwd_kernel<B, D, V, Off><<<grid, warps_n<V>() * 32, 0, s>>>(p, n);
  }
};

// Whether offsets within a run fit 32 bits (rows of heads far apart do not: one head
// behind the other's tokens).
bool short_runs(const NormParams& p) {
  for (const NormTensor& t : p.t) {
    const __int128 H = t.H > 1 ? t.H - 1 : 0, T = p.T > 1 ? kMaxTokensR : 0;
    auto far = [&](int64_t ts, int64_t hs) { return T * ts + H * hs + p.d >= (1ll << 31); };
    if (t.H > 0 && (far(t.ts, t.hs) || far(t.ots, t.ohs) || far(t.dts, t.dhs))) return false;
  }
  return true;
}

NormPlan plan_of(int64_t T, int Hq, int Hkv, int d) {
  NormPlan n;
  const int rows = 8 * (32 / (d / 16));  // of a pass
  n.job[0] = jobs_of(T, Hq, rows);
  n.job[1] = jobs_of(T, Hkv, rows);
  // backward: the blocks in proportion to the rows, one at least
  const int most = 2 * kSms;  // as many as are resident
  int64_t k = Hkv > 0 ? (static_cast<int64_t>(most) * Hkv + Hq + Hkv - 1) / (Hq + Hkv) : 0;
  const int64_t q = most - k < 1 ? 1 : most - k;
  n.blocks[0] = static_cast<int>(n.job[0].count < q ? n.job[0].count : q);
  n.blocks[1] = static_cast<int>(n.job[1].count < k ? n.job[1].count : k);
  return n;
}

}  // namespace

size_t norm_bwd_workspace(int64_t T, int Hq, int Hkv, int d) {
  const NormPlan n = plan_of(T, Hq, Hkv, d);
  const size_t bytes = static_cast<size_t>(n.blocks[0] + n.blocks[1]) * d * sizeof(float);
  return bytes < 256 ? 256 : bytes;
}

cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  const NormPlan n = plan_of(p.T, p.t[0].H, p.t[1].H, p.d);
  const int64_t all = n.job[0].count + n.job[1].count, most = 16 * kSms;
  pick<Fwd, const NormParams&, const NormPlan&>(p, vector_pairs(p.r.inv_freq ? p.r.pairs : 0, p.r.interleaved), short_runs(p), p, n,
                                                static_cast<unsigned>(all < most ? all : most), s);
  return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormParams& p, cudaStream_t s) {
  const NormPlan n = plan_of(p.T, p.t[0].H, p.t[1].H, p.d);
  if (p.T > 0) pick<Bwd, const NormParams&, const NormPlan&>(p, vector_pairs(p.r.inv_freq ? p.r.pairs : 0, p.r.interleaved), short_runs(p), p, n,
                                                static_cast<unsigned>(n.blocks[0] + n.blocks[1]), s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!p.t[0].dweight && !p.t[1].dweight)) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.d / 32, 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_join_kernel, p, n);
}

}  // namespace kv
}  // namespace attn
