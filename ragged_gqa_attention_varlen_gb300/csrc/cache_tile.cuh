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

// tanh of a pair to a few units of 2^-24 relative: an odd polynomial below
// 0.55 (least squares at Chebyshev nodes, 7e-8), 1 - 2 / (1 + e^2x) above, the
// two reciprocals from one of the product (the exponent is cut at 2^60, where
// tanh is 1).  tanh.approx (2^-11) would leave a sum of weights in fp32 with an
// error of 16 bits.  `small`: every |x| of the warp is below 0.55.
__device__ __forceinline__ uint64_t tanh2_fp32(uint64_t x, bool small) {
  const uint64_t y = f2_mul(x, x);
  auto c = [](float v) { return f2_make(v, v); };
  uint64_t s = f2_fma(y, c(-0.006615754682570696f), c(0.021312745288014412f));
  s = f2_fma(y, s, c(-0.053910065442323685f));
  s = f2_fma(y, s, c(0.13333117961883545f));
  s = f2_fma(y, s, c(-0.3333333134651184f));
  s = f2_fma(f2_mul(x, y), s, x);
  if (small) return s;
  const uint64_t e = f2_mul(x, c(2.8853900817779268f));  // 2 log2 e
  const float d0 = 1.f + ex2_approx(fminf(f2_lo(e), 60.f)), d1 = 1.f + ex2_approx(fminf(f2_hi(e), 60.f));
  const float r = rcp_approx(d0 * d1);
  const uint64_t b = f2_fma(f2_make(r * d1, r * d0), c(-2.f), c(1.f));
  return f2_make(fabsf(f2_lo(x)) < 0.55f ? f2_lo(s) : f2_lo(b),
                 fabsf(f2_hi(x)) < 0.55f ? f2_hi(s) : f2_hi(b));
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
