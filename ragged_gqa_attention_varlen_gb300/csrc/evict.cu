// evict.cu -- eviction from the paged K/V cache by accumulated weight.
//
// Of the n = lens[s] slots of sequence s, K/V head g keeps the k = min(n,
// budget) that rank first by (position >= next_pos[s] - recent, score, lowest
// slot).  The kept keys behind the new end move into the evicted slots before
// it: the i-th evicted slot below k takes the i-th kept slot at or above k.
// Every destination is an evicted slot below k and every source lies at or
// above k, so the moves never meet, run in any order and touch only the rows
// that have to move (attention does not care about the order of its keys;
// their positions travel with them).
//
// select_kernel: one block per (sequence, K/V head).  The k-th largest rank is
// found digit by digit (8-bit histograms in shared memory, eight copies because
// scores crowd into few exponents; the ranks of the first kSmemKeys slots stay
// there; as soon as a digit's keys are wanted all, the rest is left out), then
// counting passes over contiguous slot ranges per warp number the ties (only if
// some of them go), the holes and the movers in slot order: no atomics decide an order, so results
// are repeatable.  Latencies bound it: loads go out four at a time.
// move_kernel: the listed K and V rows with their scores and positions, over
// the whole GPU: a row is found through three dependent scattered reads (list,
// page table, row), so a warp takes four rows through each of them together
// (both kernels, 12 prompts of up to 20000 keys, 91 MB: 46 to 48 us; with a thread
// per 16-byte unit, two in flight, 10 more.  Eight rows: the same, and the call
// for one key goes from 8.6 to 10.6).
#include "../../include/attn_varlen.h"
#include "cache.cuh"

namespace attn {
namespace kv {
namespace {

constexpr int kThreadsE = 1024;
constexpr int kWarpsE = kThreadsE / 32;
constexpr int kSmemKeys = 48 * 1024;  // ranks held in shared memory (192 KB)
constexpr int kThreadsM = 256;
constexpr int kCopies = 8;  // of the histogram
constexpr int kMoves = 4;   // rows a warp moves at a time

struct EvictWs {
  size_t newlen, counts, lists, total;
  int64_t list_cap;
};

__host__ __device__ inline EvictWs evict_ws(int S, int Hkv, int64_t slots, int budget) {
  EvictWs w;
  const int64_t rest = slots > budget ? slots - budget : 0;
  w.list_cap = rest < budget ? rest : budget;
  w.newlen = 0;
  w.counts = (static_cast<size_t>(S) * 4 + 255) / 256 * 256;
  w.lists = w.counts + (static_cast<size_t>(S) * Hkv * 4 + 255) / 256 * 256;
  w.total = w.lists + static_cast<size_t>(S) * Hkv * 2 * w.list_cap * 4 + 256;
  return w;
}

// Scores as unsigned integers in the same order: NaN lowest, -0 = +0.  The
// protected (recent) slots come above all.
__device__ __forceinline__ uint32_t rank_key(float score, bool safe) {
  if (safe) return 0xFFFFFFFFu;
  if (!(score == score)) return 0u;
  const uint32_t u = __float_as_uint(score + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kThreadsE)
    select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t skey[];
  __shared__ uint32_t hist[kCopies][256];
  __shared__ int s_digit, s_above;
  __shared__ int cnt[3][kWarpsE];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int s = blockIdx.x / p.Hkv, g = blockIdx.x - s * p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t slots = static_cast<int64_t>(p.width) << p.page_log2;
  const EvictWs w = evict_ws(p.S, p.Hkv, slots, p.budget);
  int32_t* counts = reinterpret_cast<int32_t*>(p.ws + w.counts);
  int32_t* newlen = reinterpret_cast<int32_t*>(p.ws + w.newlen);
  int32_t* holes = reinterpret_cast<int32_t*>(p.ws + w.lists) + 2 * w.list_cap * blockIdx.x;
  int32_t* movers = holes + w.list_cap;
  const float* sc = p.scores + s * p.sc_rs + g * p.sc_hs;
  const int32_t* kp = p.key_pos + s * p.kp_rs + g * p.kp_hs;
  float* so = p.scores_out + s * p.so_rs + g * p.so_hs;
  int32_t* po = p.pos_out + s * p.po_rs + g * p.po_hs;
  const int n0 = __ldg(p.lens + s);
  const bool bad = n0 < 0 || n0 > slots;
  const int n = bad ? 0 : n0;
  const int k = min(n, p.budget);
  if (tid == 0) {
    if (bad) report(p.status, ATTN_DEV_BAD_CACHE);
    if (g == 0) newlen[s] = bad ? n0 : k;
    if (n <= k) counts[blockIdx.x] = 0;
  }
  // the slots below the new end (evicted ones are replaced by the moves)
  if (so != sc || po != kp) {
    for (int j0 = tid; j0 < k; j0 += 4 * kThreadsE) {
      float x[4];
      int32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j0 + i * kThreadsE < k) {
          x[i] = sc[j0 + i * kThreadsE];
          y[i] = kp[j0 + i * kThreadsE];
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j0 + i * kThreadsE < k) {
          if (so != sc) so[j0 + i * kThreadsE] = x[i];
          if (po != kp) po[j0 + i * kThreadsE] = y[i];
        }
    }
  }
  if (n <= k) return;  // nothing to evict
  const int from = __ldg(p.next_pos + s) - p.recent;
  auto load_key = [&](int j) { return rank_key(sc[j], kp[j] >= from); };
  if (n - k == 1) {
    // One key leaves, as in every step of a full cache: the lowest rank, of
    // equal ones the highest slot, found in one pass (32 caches of 1025 keys: 8.5
    // us for the call, against 12.8 with the histograms).  Slot k is the only one
    // behind the new end.
    uint64_t least = ~0ull;
    for (int j0 = tid; j0 < n; j0 += 4 * kThreadsE) {
      float x[4];
      int32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j0 + i * kThreadsE < n) {
          x[i] = sc[j0 + i * kThreadsE];
          y[i] = kp[j0 + i * kThreadsE];
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * kThreadsE;
        if (j < n)
          least = min(least, static_cast<uint64_t>(rank_key(x[i], y[i] >= from)) << 32 |
                                 (0xFFFFFFFFu - static_cast<uint32_t>(j)));
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
      least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    __shared__ uint64_t lows[kWarpsE];
    if (lane == 0) lows[warp] = least;
    __syncthreads();
    if (warp == 0) {
      least = lows[lane];
#pragma unroll
      for (int o = 16; o; o >>= 1)
        least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
      const int slot = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(least));
      if (lane == 0) {
        counts[blockIdx.x] = slot < k;
        holes[0] = slot;
        movers[0] = k;
      }
    }
    return;
  }
  auto key = [&](int j) { return j < kSmemKeys ? skey[j] : load_key(j); };

  // the k-th largest key: its digits from the top
  uint32_t prefix = 0;
  int need = k;  // how many keys with the digits found so far are still to take
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < kCopies * 256; i += kThreadsE) hist[i >> 8][i & 255] = 0;
    __syncthreads();
    uint32_t* mine = hist[warp & (kCopies - 1)];
    if (shift == 24) {
      for (int j0 = tid; j0 < n; j0 += 4 * kThreadsE) {
        float x[4];
        int32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j0 + i * kThreadsE < n) {
            x[i] = sc[j0 + i * kThreadsE];
            y[i] = kp[j0 + i * kThreadsE];
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = j0 + i * kThreadsE;
          if (j < n) {
            const uint32_t u = rank_key(x[i], y[i] >= from);
            if (j < kSmemKeys) skey[j] = u;
            atomicAdd(&mine[u >> 24], 1u);
          }
        }
      }
    } else {
#pragma unroll 4
      for (int j = tid; j < n; j += kThreadsE) {
        const uint32_t x = key(j);
        if (((x ^ prefix) >> (shift + 8)) == 0) atomicAdd(&mine[(x >> shift) & 255], 1u);
      }
    }
    __syncthreads();
    if (tid < 256) {
      uint32_t sum = 0;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) sum += hist[i][tid];
      hist[0][tid] = sum;
    }
    __syncthreads();
    if (warp == 0) {  // lane l: digits 255 - 8l down to 248 - 8l
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i] = static_cast<int>(hist[0][255 - 8 * lane - i]);
      int above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, above, o);
        if (lane >= o) above += y;
      }
      above -= sum;  // keys with a digit above this lane's
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (above < need && above + c[i] >= need) {
          s_digit = 255 - 8 * lane - i;
          s_above = above + c[i] == need ? -1 : above;
        }
        above += c[i];
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    if (s_above < 0) {  // all keys with these digits are wanted: key >= prefix
      need = INT32_MAX;
      break;
    }
    need -= s_above;
    __syncthreads();
  }
  // kept: key > prefix, or key == prefix and among the first `need` such slots

  const int span = ((n + kThreadsE - 1) / kThreadsE) * 32;  // slots of a warp, a multiple of 32
  const int j0 = min(n, warp * span), j1 = min(n, j0 + span);
  auto total_before = [&](int (&c)[kWarpsE]) {
    int t = 0;
    for (int i = 0; i < warp; ++i) t += c[i];
    return t;
  };
  const bool ties = need != INT32_MAX;  // some of the keys equal to prefix go
  int eq0 = 0;
  if (ties) {
    int c0 = 0;
    for (int j = j0 + lane; j - lane < j1; j += 32)
      c0 += __popc(__ballot_sync(0xffffffffu, j < j1 && key(j) == prefix));
    if (lane == 0) cnt[0][warp] = c0;
    __syncthreads();
    eq0 = total_before(cnt[0]);
  }
  const uint32_t below = (1u << lane) - 1u;
  // f(slot, kept) for this warp's slots in order, whole warps at a time
  auto walk = [&](auto f) {
    if (!ties) {
#pragma unroll 4
      for (int j = j0 + lane; j - lane < j1; j += 32) {
        const bool in = j < j1;
        f(j, in, in && key(j) >= prefix);
      }
      return;
    }
    int eq = eq0;
    for (int j = j0 + lane; j - lane < j1; j += 32) {
      const bool in = j < j1;
      const uint32_t x = in ? key(j) : 0u;
      const uint32_t e = __ballot_sync(0xffffffffu, in && x == prefix);
      const bool keep = in && (x > prefix || (x == prefix && eq + __popc(e & below) < need));
      eq += __popc(e);
      f(j, in, keep);
    }
  };
  int nh = 0, nm = 0;
  walk([&](int j, bool in, bool keep) {
    nh += __popc(__ballot_sync(0xffffffffu, in && !keep && j < k));
    nm += __popc(__ballot_sync(0xffffffffu, in && keep && j >= k));
  });
  if (lane == 0) {
    cnt[1][warp] = nh;
    cnt[2][warp] = nm;
  }
  __syncthreads();
  int ih = total_before(cnt[1]), im = total_before(cnt[2]);
  if (tid == kThreadsE - 1) counts[blockIdx.x] = im + nm;  // as many as holes
  walk([&](int j, bool in, bool keep) {
    const bool hole = in && !keep && j < k, mover = in && keep && j >= k;
    const uint32_t bh = __ballot_sync(0xffffffffu, hole), bm = __ballot_sync(0xffffffffu, mover);
    if (hole) holes[ih + __popc(bh & below)] = j;
    if (mover) movers[im + __popc(bm & below)] = j;
    ih += __popc(bh);
    im += __popc(bm);
  });
}

__global__ void __launch_bounds__(kThreadsM)
    move_kernel(const __grid_constant__ EvictParams p) {
  const int sg = blockIdx.x, s = sg / p.Hkv, g = sg - s * p.Hkv;
  const EvictWs w =
      evict_ws(p.S, p.Hkv, static_cast<int64_t>(p.width) << p.page_log2, p.budget);
  const int32_t* holes = reinterpret_cast<const int32_t*>(p.ws + w.lists) + 2 * w.list_cap * sg;
  const int32_t* movers = holes + w.list_cap;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int count = reinterpret_cast<const int32_t*>(p.ws + w.counts)[sg];
  if (g == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    p.lens_out[s] = reinterpret_cast<const int32_t*>(p.ws + w.newlen)[s];
  const int units = p.d / 8;  // 16-byte units of a K or V row
  const int32_t* row = p.table + s * p.table_rs;
  const float* sc = p.scores + s * p.sc_rs + g * p.sc_hs;
  const int32_t* kp = p.key_pos + s * p.kp_rs + g * p.kp_hs;
  float* so = p.scores_out + s * p.so_rs + g * p.so_hs;
  int32_t* po = p.pos_out + s * p.po_rs + g * p.po_hs;
  const uint16_t* kb = static_cast<const uint16_t*>(p.k.base) + g * p.k.head;
  const uint16_t* vb = static_cast<const uint16_t*>(p.v.base) + g * p.v.head;
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.y * (kThreadsM / 32);
  // kMoves rows a warp at a time: lanes 0 .. kMoves-1 look them up, then all
  // lanes copy, the units of every row on their way before the first is stored
  for (int64_t m0 = (static_cast<int64_t>(blockIdx.y) * (kThreadsM / 32) + (threadIdx.x >> 5)) * kMoves;
       m0 < count; m0 += static_cast<int64_t>(warps) * kMoves) {
    int ps = -1, pd = -1, src = 0, dst = 0;
    if (lane < kMoves && m0 + lane < count) {
      src = movers[m0 + lane];
      dst = holes[m0 + lane];
      ps = __ldg(row + (src >> p.page_log2));
      pd = __ldg(row + (dst >> p.page_log2));
      const float score = sc[src];
      const int32_t pos = kp[src];
      if (static_cast<unsigned>(ps) >= static_cast<unsigned>(p.num_pages) ||
          static_cast<unsigned>(pd) >= static_cast<unsigned>(p.num_pages)) {
        // nothing of this move: the slot keeps its key, score and position
        report(p.status, ATTN_DEV_BAD_CACHE);
        ps = -1;
      } else {
        so[dst] = score;
        po[dst] = pos;
      }
      src &= p.page_size - 1;
      dst &= p.page_size - 1;
    }
    for (int u = lane; u - lane < 2 * units; u += 32) {
      const bool k = u < units;
      const Pages& pg = k ? p.k : p.v;
      const uint16_t* base = (k ? kb : vb) + (k ? u : u - units) * 8;
      uint4 v[kMoves];
#pragma unroll
      for (int i = 0; i < kMoves; ++i) {
        const int page = __shfl_sync(0xffffffffu, ps, i), at = __shfl_sync(0xffffffffu, src, i);
        if (page >= 0 && u < 2 * units)
          v[i] = *reinterpret_cast<const uint4*>(base + page * pg.page + at * pg.slot);
      }
#pragma unroll
      for (int i = 0; i < kMoves; ++i) {
        const int ok = __shfl_sync(0xffffffffu, ps, i), page = __shfl_sync(0xffffffffu, pd, i);
        const int at = __shfl_sync(0xffffffffu, dst, i);
        if (ok >= 0 && u < 2 * units)
          *reinterpret_cast<uint4*>(const_cast<uint16_t*>(base) + page * pg.page + at * pg.slot) = v[i];
      }
    }
  }
}

}  // namespace

size_t evict_workspace(int S, int Hkv, int64_t slots, int budget) {
  return evict_ws(S, Hkv, slots, budget).total;
}

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
  const int64_t slots = static_cast<int64_t>(p.width) << p.page_log2;
  const int smem = static_cast<int>(slots < kSmemKeys ? slots : kSmemKeys) * 4;
  cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemKeys * 4);
  select_kernel<<<p.S * p.Hkv, kThreadsE, smem, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  constexpr int kPerBlock = kThreadsM / 32 * kMoves;
  int64_t x = (evict_ws(p.S, p.Hkv, slots, p.budget).list_cap + kPerBlock - 1) / kPerBlock;
  const int64_t most = 152 * 32 / (p.S * p.Hkv) + 1;
  x = x < 1 ? 1 : (x > most ? most : x);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.S * p.Hkv, static_cast<unsigned>(x));
  cfg.blockDim = dim3(kThreadsM);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, move_kernel, p);
}

}  // namespace kv
}  // namespace attn
