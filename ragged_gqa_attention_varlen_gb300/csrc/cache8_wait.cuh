// cache8_wait.cuh -- waits, small copies and constants that the kernels over the
// 8-bit cache share.
#pragma once
#include "cache_piece.cuh"

namespace attn {
namespace kv {

constexpr float kLazy8 = 8.f;     // rescale when the maximum grows by more (base 2)
constexpr float kShift8 = 7.f;    // P of a row's maximum, as an exponent

// Waits as in sm103.cuh, by a try that may suspend the warp for longer: twenty warps
// that poll took a third of the issue slots.
__device__ __forceinline__ bool mbar_try_long(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool mbar_wait8(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_long(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_long(bar, parity)) {
    if (*abort) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool mbar_wait8_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait8(bar, parity, abort));
}
__device__ __forceinline__ bool warp_exchange8(uint64_t* bar, uint32_t parity, volatile int* abort) {
  __threadfence_block();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
  return mbar_wait8_warp(bar, parity, abort);
}
__device__ __forceinline__ bool piece_take8(PieceRing* r, uint32_t& k, Piece* out, volatile int* abort) {
  const int s = k & 3;
  if (!mbar_wait8(&r->full[s], (k >> 2) & 1, abort)) return false;
  *out = r->piece[s];
  ++k;
  return true;
}

__device__ __forceinline__ void cp_async4_or_zero(float* dst, const float* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 4 : 0)
               : "memory");
}
// Arrives on `bar` (which counts this thread) when the thread's copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

}  // namespace kv
}  // namespace attn
