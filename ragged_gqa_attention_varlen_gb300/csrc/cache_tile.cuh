// cache_tile.cuh -- operand tiles and element arithmetic shared by the kernels
// over the paged cache.
#pragma once
#include "cache_sched.cuh"

namespace attn {
namespace kv {

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh of a pair to a few units of 2^-24 relative (3e-7 at most, 6e-8 in the
// mean): x P(x^2) / Q(x^2), both of degree 4, fitted to tanh(x) / x on [0, 8.5]
// by reweighted least squares on the relative error (2e-8), |x| cut at 8.5,
// where tanh is 1 to 8e-8.  The pair shares one reciprocal, of the product of
// its denominators.  tanh.approx (2^-11) would leave a sum of weights in fp32
// with an error of 16 bits, and 1 - 2 / (1 + e^2x) loses small x and takes an
// exponential more.
__device__ __forceinline__ uint64_t tanh2_fp32(uint64_t x) {
  auto c = [](float v) { return f2_make(v, v); };
  auto cut = [](float v) {
    float r;
    asm("min.xorsign.abs.f32 %0, %1, 0f41080000;" : "=f"(r) : "f"(v));  // 8.5 with v's sign
    return r;
  };
  x = f2_make(cut(f2_lo(x)), cut(f2_hi(x)));
  const uint64_t y = f2_mul(x, x);
  uint64_t n = f2_fma(y, c(1.42689628674e-8f), c(2.1250905809e-5f));
  uint64_t d = f2_fma(y, c(8.14503033431e-7f), c(3.34885330616e-4f));
  n = f2_fma(y, n, c(3.5340209526e-3f));
  d = f2_fma(y, d, c(2.60227318807e-2f));
  n = f2_fma(y, n, c(0.134132429775f));
  d = f2_fma(y, d, c(0.467465658106f));
  n = f2_mul(f2_fma(y, n, c(0.999999988432f)), x);
  d = f2_fma(y, d, c(1.f));
  const float d0 = f2_lo(d), d1 = f2_hi(d), r = rcp_approx(d0 * d1);
  return f2_mul(n, f2_make(r * d1, r * d0));
}

__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > kWaitLimitNs) break;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Byte offset of 16-byte unit u of row r in a K-major tile: 64-feature chunks
// of 128-byte rows (128-byte swizzle), features 128..159 in 64-byte rows
// (64-byte swizzle).
__device__ __forceinline__ uint32_t kmajor_unit(int r, int u) {
  return u < 16 ? static_cast<uint32_t>((u >> 3) * 16384 + r * 128 + (((u & 7) ^ (r & 7)) << 4))
                : static_cast<uint32_t>(32768 + r * 64 + (((u - 16) ^ ((r >> 1) & 3)) << 4));
}
// Descriptor of K step k (16 features) of such a tile.
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t base, int k) {
  return k < 8 ? sdesc_sw128(base + (k >> 2) * 16384 + (k & 3) * 32, 16, 1024)
               : sdesc_sw64(base + 32768 + (k - 8) * 32);
}

// Copy `rows` Q rows, from (token tok, head `head` of group g) on, into shared
// memory (warp wi of nw; asynchronous): four lanes a row, eight rows at a time.
template <int HD>
__device__ __forceinline__ void copy_q_rows(const CacheParams& p, uint8_t* dst, int g, int tok,
                                            int head, int rows, int wi, int nw) {
  const int lane = threadIdx.x & 31, u0 = lane & 3;
  const uint32_t base = smem_addr(dst);
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + static_cast<int64_t>(g) * p.R * p.q_hs;
#pragma unroll 2
  for (int r = wi * 8 + (lane >> 2); r < rows; r += nw * 8) {
    const int hh = head + r, dt = head_div(p, hh);
    const uint16_t* src = q + static_cast<int64_t>(tok + dt) * p.q_ts +
                          static_cast<int64_t>(hh - dt * p.R) * p.q_hs;
#pragma unroll
    for (int k = 0; k < HD / 32; ++k)
      cp_async16(base + kmajor_unit(r, u0 + 4 * k), src + (u0 + 4 * k) * 8);
  }
}

// Pages of a key tile, one per box: lane `i` of a load group returns the page
// of box row block i (of `pieces`), or the pool's size (reads as zeros) when
// its number is out of the pool.
__device__ __forceinline__ int tile_page(const CacheParams& p, const int32_t* row, int key) {
  const int page = __ldg(row + (key >> p.page_log2));
  if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) return page;
  report(p.status, ATTN_DEV_BAD_CACHE);
  return p.num_pages;
}

}  // namespace kv
}  // namespace attn
