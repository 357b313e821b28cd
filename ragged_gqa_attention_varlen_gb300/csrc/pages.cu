// pages.cu -- the pages of a cache: forking and freeing rows of its table,
// packing its live pages together, copying pages.
//
// What a page holds is moved by one kernel over a list of moves, for all pools of
// a model's layers at once (bound by memory: the moved rows are read and written
// once).  What the tables, reference counts and lists become is worked out before
// by one cluster of blocks that meet at cluster barriers between the steps: the
// steps depend on one another and touch little, so a launch for each of them
// would cost more than they do, and one block alone takes long for a pool of a
// million pages.
//
// Everything has one answer whatever runs first: reference counts are integer
// sums, free pages are taken lowest first in the order of the rows.
#include "../../include/attn_varlen.h"
#include "cache.cuh"

namespace attn {
namespace kv {
namespace {

constexpr int kThreadsP = 1024;
constexpr int kCtasP = 8;  // of the cluster, at most

struct PagesHead {  // of both workspaces, at offset 0
  int bad, lacking, moves;  // (status bits of the inputs; of the pages and their counts)
  int count[kCtasP][3];  // of each block: sums of its part
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The block's sum of a value per thread, and the sum of the threads before
// this one (whole block).
__device__ __forceinline__ int block_before(int v, int* tmp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  __syncthreads();  // (tmp may still be read)
  if (lane == 31) tmp[warp] = upto;
  __syncthreads();
  const int mine = tmp[lane];
  int w = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += x;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  return __shfl_sync(0xffffffffu, w - mine, warp) + upto - v;
}

// This block's part [lo, hi) of n values, in runs of whole passes.
struct Part {
  int lo, hi;
};
__device__ __forceinline__ Part part_of(int n) {
  const int per = (n + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  Part p;
  p.lo = min(n, per * static_cast<int>(blockIdx.x));
  p.hi = min(n, p.lo + per);
  return p;
}

struct ForkWs {
  size_t delta, uses, times, lowest, lens, held, fresh, start, free, table, moves, total;
};
ForkWs fork_ws(int R, int W, int N) {
  ForkWs w;
  size_t at = 256;
  auto take = [&](int64_t n, size_t e) {
    const size_t here = at;
    at += (static_cast<size_t>(n) * e + 255) / 256 * 256;
    return here;
  };
  w.delta = take(N, 4);
  w.uses = take(N, 4);
  w.times = take(R, 4);
  w.lowest = take(R, 4);
  w.lens = take(R, 4);
  w.held = take(R, 4);
  w.fresh = take(R, 4);
  w.start = take(R, 4);
  w.free = take(N, 4);
  w.table = take(static_cast<int64_t>(R) * W, 4);
  w.moves = take(R, sizeof(Move));
  w.total = at;
  return w;
}

// Row r of the new table goes on from row parents[r] of the old one (-1: empty).
// All that do share its full pages; the first of them (lowest r) also keeps its
// other pages, the others get a copy of the part that is used.  A row that nobody
// goes on from gives its pages back.  Rows then get pages for `room` more slots.
//
// Either everything is done or, with any input out of range or too few pages,
// nothing: the outputs are the inputs then.
__global__ void __launch_bounds__(kThreadsP)
    fork_kernel(const __grid_constant__ ForkParams p, const __grid_constant__ ForkWs w) {
  __shared__ int tmp[32];
  __shared__ int sums[3];
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, nt = blockDim.x * gridDim.x, at = blockIdx.x * blockDim.x + tid;
  const int ps = 1 << p.page_log2;
  PagesHead* head = reinterpret_cast<PagesHead*>(p.ws);
  int* delta = reinterpret_cast<int*>(p.ws + w.delta);
  int* uses = reinterpret_cast<int*>(p.ws + w.uses);
  int* times = reinterpret_cast<int*>(p.ws + w.times);
  int* lowest = reinterpret_cast<int*>(p.ws + w.lowest);
  int* lens = reinterpret_cast<int*>(p.ws + w.lens);
  int* held = reinterpret_cast<int*>(p.ws + w.held);
  int* fresh = reinterpret_cast<int*>(p.ws + w.fresh);
  int* start = reinterpret_cast<int*>(p.ws + w.start);
  int* freed = reinterpret_cast<int*>(p.ws + w.free);
  int* table = reinterpret_cast<int*>(p.ws + w.table);
  Move* moves = reinterpret_cast<Move*>(p.ws + w.moves);
  const int64_t cells = static_cast<int64_t>(p.R) * p.W;

  // ---- copies of what the outputs may overwrite, and what is out of range
  if (at == 0) {
    head->bad = 0;
    head->lacking = 0;
    head->moves = 0;
  }
  for (int i = at; i < p.N; i += nt) delta[i] = uses[i] = 0;
  for (int r = at; r < p.R; r += nt) {
    times[r] = 0;
    lowest[r] = p.R;
  }
  cluster_sync();
  int bad = 0;
  for (int r = at; r < p.R; r += nt) {
    const int n = p.lens[r], h = p.held[r], up = p.parents[r], room = p.room ? p.room[r] : 0;
    lens[r] = n;
    held[r] = h;
    if (h < 0 || h > p.W || n < 0 || n > static_cast<int64_t>(max(h, 0)) << p.page_log2 || up < -1 || up >= p.R || room < 0) {
      bad |= ATTN_DEV_BAD_CACHE;
    } else if (up >= 0) {
      atomicAdd(times + up, 1);
      atomicMin(lowest + up, r);
    }
  }
  for (int64_t i = at; i < cells; i += nt) {
    const int r = static_cast<int>(i / p.W), c = static_cast<int>(i - static_cast<int64_t>(r) * p.W);
    const int page = p.table[r * p.table_rs + c];
    table[i] = page;
    if (c >= p.held[r]) continue;
    if (static_cast<unsigned>(page) < static_cast<unsigned>(p.N))
      atomicAdd(uses + page, 1);
    else
      bad |= ATTN_DEV_BAD_CACHE;
  }
  if (bad) atomicOr(&head->bad, bad);
  cluster_sync();
  const bool sound = head->bad == 0;  // (nothing changes it from here on)

  // ---- the change of every page's count, and the pages that every row lacks
  const Part rows = part_of(p.R);
  int need = 0;
  if (sound) {
    for (int64_t i = at; i < cells; i += nt) {
      const int r = static_cast<int>(i / p.W), c = static_cast<int>(i - static_cast<int64_t>(r) * p.W);
      if (c >= held[r]) continue;
      const int change = c < lens[r] >> p.page_log2 ? times[r] - 1 : (times[r] > 0 ? 0 : -1);
      if (change) atomicAdd(delta + table[i], change);
    }
    int wide = 0;
    for (int r0 = rows.lo; r0 < rows.hi; r0 += kThreadsP) {
      const int r = r0 + tid;
      int n = 0;
      if (r < rows.hi) {
        const int up = p.parents[r];
        if (up >= 0) {
          const int had = lowest[up] == r ? held[up] : lens[up] >> p.page_log2;
          const int64_t want = (static_cast<int64_t>(lens[up]) + (p.room ? p.room[r] : 0) + ps - 1) >> p.page_log2;
          if (want > p.W)
            wide = 1;
          else
            n = max(0, static_cast<int>(want) - had);
        }
        fresh[r] = n;
      }
      int sum;
      const int before = block_before(n, tmp, sum);
      if (r < rows.hi) start[r] = need + before;  // (its part's start is added below)
      need += sum;
    }
    if (wide) atomicOr(&head->lacking, ATTN_DEV_NO_PAGES);
  }
  cluster_sync();
  // ---- the free pages, lowest first
  const Part pages = part_of(p.N);
  int free_here = 0, first_free = 0, wrong = 0;
  if (sound) {
    for (int i0 = pages.lo; i0 < pages.hi; i0 += kThreadsP) {
      const int i = i0 + tid;
      const int n = i < pages.hi ? p.refs[i] : 0;
      // held by more rows than it counts: it could pass for free while a row keeps it
      if (i < pages.hi && uses[i] > 0 && n < uses[i]) wrong = 1;
      free_here += __syncthreads_count(i < pages.hi && n + delta[i] == 0);
    }
    if (wrong) atomicOr(&head->lacking, ATTN_DEV_BAD_CACHE);
    if (tid == 0) {
      head->count[blockIdx.x][0] = need;
      head->count[blockIdx.x][1] = free_here;
    }
  }
  cluster_sync();
  if (tid == 0) {
    int a = 0, b = 0, all = 0, space = 0;
    for (int c = 0; c < static_cast<int>(gridDim.x); ++c) {
      if (c == static_cast<int>(blockIdx.x)) a = all, b = space;
      all += head->count[c][0];
      space += head->count[c][1];
    }
    sums[0] = a;
    sums[1] = b;
    sums[2] = all;
    if (sound && all > space) atomicOr(&head->lacking, ATTN_DEV_NO_PAGES);
  }
  __syncthreads();
  if (sound) {
    first_free = sums[1];
    for (int i0 = pages.lo; i0 < pages.hi && first_free < sums[2]; i0 += kThreadsP) {
      const int i = i0 + tid;
      const int is = i < pages.hi && p.refs[i] + delta[i] == 0;
      int sum;
      const int before = block_before(is, tmp, sum);
      if (is && first_free + before < sums[2]) {
        freed[first_free + before] = i;
        delta[i] += 1 << 30;  // taken (told from a count by its size)
      }
      first_free += sum;
    }
    for (int r = rows.lo + tid; r < rows.hi; r += kThreadsP) start[r] += sums[0];
  }
  cluster_sync();
  bad = head->bad | head->lacking;
  if (bad) {  // the outputs are the inputs
    if (at == 0) report(p.status, bad);
    for (int64_t i = at; i < cells; i += nt) {
      const int r = static_cast<int>(i / p.W), c = static_cast<int>(i - static_cast<int64_t>(r) * p.W);
      p.table_out[r * p.to_rs + c] = table[i];
    }
    for (int r = at; r < p.R; r += nt) {
      p.lens_out[r] = lens[r];
      p.held_out[r] = held[r];
    }
    for (int i = at; i < p.N; i += nt) p.refs_out[i] = p.refs[i];
    return;
  }
  // ---- the outputs
  for (int i = at; i < p.N; i += nt) p.refs_out[i] = delta[i] >= 1 << 29 ? 1 : p.refs[i] + delta[i];
  for (int64_t i = at; i < cells; i += nt) {
    const int r = static_cast<int>(i / p.W), c = static_cast<int>(i - static_cast<int64_t>(r) * p.W);
    const int up = p.parents[r];
    if (up < 0) continue;
    const int had = lowest[up] == r ? held[up] : lens[up] >> p.page_log2;
    if (c < had)
      p.table_out[r * p.to_rs + c] = table[static_cast<int64_t>(up) * p.W + c];
    else if (c < had + fresh[r])
      p.table_out[r * p.to_rs + c] = freed[start[r] + c - had];
  }
  for (int r = at; r < p.R; r += nt) {
    const int up = p.parents[r];
    if (up < 0) {
      p.lens_out[r] = p.held_out[r] = 0;
      continue;
    }
    const bool first = lowest[up] == r;
    const int full = lens[up] >> p.page_log2, used = lens[up] & (ps - 1);
    p.lens_out[r] = lens[up];
    p.held_out[r] = (first ? held[up] : full) + fresh[r];
    if (!first && used) {
      Move m;
      m.src = table[static_cast<int64_t>(up) * p.W + full];
      m.dst = freed[start[r]];
      m.used = used;
      m.pad = 0;
      moves[atomicAdd(&head->moves, 1)] = m;
    }
  }
}

struct CompactWs {
  size_t to, holes, moves, total;
};
CompactWs compact_ws(int N) {
  CompactWs w;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  w.to = 256;
  w.holes = w.to + up(static_cast<size_t>(N) * 4);
  w.moves = w.holes + up(static_cast<size_t>(N / 2 + 1) * 4);
  w.total = w.moves + up(static_cast<size_t>(N / 2 + 1) * sizeof(Move));
  return w;
}

// The i-th free page below the number of live ones takes the place of the i-th
// live page at or above it.
__global__ void __launch_bounds__(kThreadsP)
    compact_kernel(const __grid_constant__ CompactParams p, const __grid_constant__ CompactWs w) {
  __shared__ int tmp[32];
  __shared__ int sums[3];
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, nt = blockDim.x * gridDim.x, at = blockIdx.x * blockDim.x + tid;
  PagesHead* head = reinterpret_cast<PagesHead*>(p.ws);
  int* to = reinterpret_cast<int*>(p.ws + w.to);
  int* holes = reinterpret_cast<int*>(p.ws + w.holes);
  Move* moves = reinterpret_cast<Move*>(p.ws + w.moves);
  const Part part = part_of(p.N);
  auto is_live = [&](int i) { return i < part.hi && p.refs[i] > 0; };
  int here = 0;
  for (int i0 = part.lo; i0 < part.hi; i0 += kThreadsP) here += __syncthreads_count(is_live(i0 + tid));
  if (tid == 0) head->count[blockIdx.x][0] = here;
  cluster_sync();
  if (tid == 0) {
    int before = 0, all = 0;
    for (int c = 0; c < static_cast<int>(gridDim.x); ++c) {
      if (c == static_cast<int>(blockIdx.x)) before = all;
      all += head->count[c][0];
    }
    sums[0] = before;
    sums[1] = all;
  }
  __syncthreads();
  const int live = sums[1];
  // Rank of a live page among the live ones = x: of a hole i below `live`, i - x
  // holes lie before it; of a mover, x - (live pages below `live`) movers do.
  // The two lists meet at equal ranks, so the movers need the number of holes:
  // live pages below `live` = live - movers, known once all parts have counted.
  int rank = sums[0];
  int low = 0;  // live pages below `live` in this part
  for (int i0 = part.lo; i0 < part.hi; i0 += kThreadsP) {
    const int i = i0 + tid, is = is_live(i);
    low += __syncthreads_count(is && i < live);
    int sum;
    const int x = rank + block_before(is, tmp, sum);
    if (i < part.hi) {
      if (i < live && !is) holes[i - x] = i;
      to[i] = is ? (i < live ? i : -2 - x) : -1;  // movers: their rank, for now
    }
    rank += sum;
  }
  if (tid == 0) head->count[blockIdx.x][1] = low;
  cluster_sync();
  if (tid == 0) {
    int all = 0;
    for (int c = 0; c < static_cast<int>(gridDim.x); ++c) all += head->count[c][1];
    sums[2] = all;
    if (at == 0) {
      head->moves = live - all;
      *p.live = live;
    }
  }
  __syncthreads();
  const int stay = sums[2];
  for (int i = part.lo + tid; i < part.hi; i += kThreadsP) {
    const int n = p.refs[i];
    if (to[i] >= 0) p.refs_out[i] = n;
    if (to[i] > -2) continue;
    const int k = -2 - to[i] - stay, hole = holes[k];
    Move m;
    m.src = i;
    m.dst = hole;
    m.used = 1 << p.page_log2;
    m.pad = 0;
    moves[k] = m;
    to[i] = hole;
    p.refs_out[hole] = n;  // (in place: the hole's own count, 0 or less, is not read any more)
  }
  cluster_sync();
  for (int i = part.lo + tid; i < part.hi; i += kThreadsP)
    if (i >= live) p.refs_out[i] = 0;
  int bad = 0;
  for (int k = 0; k < 2; ++k) {
    const CompactTable& t = p.t[k];
    const int64_t cells = static_cast<int64_t>(t.R) * t.W;
    for (int64_t i = at; i < cells; i += nt) {
      const int r = static_cast<int>(i / t.W), c = static_cast<int>(i - static_cast<int64_t>(r) * t.W);
      const int h = t.held[r];
      if (h < 0 || h > t.W) bad = ATTN_DEV_BAD_CACHE;
      if (c >= min(h, t.W)) continue;
      const int page = t.table[r * t.rs + c];
      int now = page;
      if (static_cast<unsigned>(page) < static_cast<unsigned>(p.N) && to[page] >= 0)
        now = to[page];
      else
        bad = ATTN_DEV_BAD_CACHE;  // out of the pool, or a page that nobody counts: left as it is
      t.out[r * t.out_rs + c] = now;
    }
  }
  if (bad) report(p.status, bad);
}

// ------------------------------------------------------------------ moving pages

constexpr int kThreadsM = 256;
constexpr int kUnroll = 4;
constexpr int kChunkBytes = kThreadsM * kUnroll * 16;  // of a block's turn

struct MoveList {
  const PagesHead* head;  // null: `count` pairs of two arrays
  const Move* moves;
  const int32_t *src, *dst;
  int count, src_pages, dst_pages, page_log2;
  int32_t* status;
};

// Work is cut into (move, pool, chunk of a page); a thread has kUnroll units of
// T in flight.
template <class T>
__device__ __forceinline__ void move_chunk(const MovedPool& q, int src, int dst, int rows, int chunk) {
  constexpr int kUnit = sizeof(T);
  const int per_piece = q.bytes / kUnit, per_row = per_piece * q.pieces, units = rows * per_row;
  const char* s = static_cast<const char*>(q.src) + src * q.src_page;
  char* d = static_cast<char*>(q.dst) + dst * q.dst_page;
  const int u_end = min(units, (chunk + 1) * (kChunkBytes / kUnit));
#pragma unroll 1
  for (int u0 = chunk * (kChunkBytes / kUnit) + static_cast<int>(threadIdx.x); u0 < u_end; u0 += kThreadsM * kUnroll) {
    T v[kUnroll];
    int64_t to[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int u = u0 + i * kThreadsM;
      to[i] = -1;
      if (u >= u_end) continue;
      int64_t from;
      if (q.flat) {
        from = to[i] = static_cast<int64_t>(u) * kUnit;
      } else {
        const int row = u / per_row, rest = u - row * per_row, piece = rest / per_piece;
        const int64_t in = static_cast<int64_t>(rest - piece * per_piece) * kUnit;
        from = row * q.src_row + piece * q.src_piece + in;
        to[i] = row * q.dst_row + piece * q.dst_piece + in;
      }
      v[i] = __ldcs(reinterpret_cast<const T*>(s + from));
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (to[i] >= 0) __stcs(reinterpret_cast<T*>(d + to[i]), v[i]);
  }
}

__global__ void __launch_bounds__(kThreadsM)
    move_kernel(const __grid_constant__ MovedPools pools, const __grid_constant__ MoveList list, int chunks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool made = list.head != nullptr;
  const int count = made ? list.head->moves : list.count;
  const int64_t per_move = static_cast<int64_t>(pools.n) * chunks, all = count * per_move;
  const int slots = 1 << list.page_log2;
  for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
    const int m = static_cast<int>(i / per_move), rest = static_cast<int>(i - m * per_move);
    const int pool = rest / chunks, chunk = rest - pool * chunks;
    const MovedPool& q = pools.pool[pool];
    int src, dst, used = slots;
    if (made) {
      const int4 x = *reinterpret_cast<const int4*>(list.moves + m);
      src = x.x;
      dst = x.y;
      used = x.z;
    } else {
      src = __ldg(list.src + m);
      dst = __ldg(list.dst + m);
      if (static_cast<unsigned>(src) >= static_cast<unsigned>(list.src_pages) ||
          static_cast<unsigned>(dst) >= static_cast<unsigned>(list.dst_pages)) {
        if (rest == 0 && threadIdx.x == 0) report(list.status, ATTN_DEV_BAD_CACHE);
        continue;
      }
      if (q.src == q.dst && src == dst) continue;
    }
    // the rows that the used slots take (a pool of scales has one for several)
    const int rows = static_cast<int>((static_cast<int64_t>(used) * q.rows + slots - 1) >> list.page_log2);
    if (q.wide)
      move_chunk<uint4>(q, src, dst, rows, chunk);
    else
      move_chunk<uint32_t>(q, src, dst, rows, chunk);
  }
}

cudaError_t launch_moves(const MoveList& list, const MovedPool* pools, int n, bool dependent, cudaStream_t s) {
  for (int at = 0; at < n; at += kPoolsPerLaunch) {
    MovedPools m;
    m.n = n - at < kPoolsPerLaunch ? n - at : kPoolsPerLaunch;
    int64_t most = 0;
    for (int i = 0; i < m.n; ++i) {
      m.pool[i] = pools[at + i];
      const MovedPool& q = m.pool[i];
      const int64_t bytes = static_cast<int64_t>(q.rows) * q.pieces * q.bytes;
      most = bytes > most ? bytes : most;
    }
    const int chunks = static_cast<int>((most + kChunkBytes - 1) / kChunkBytes);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(152 * 8);
    cfg.blockDim = dim3(kThreadsM);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, move_kernel, m, list, chunks);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <class K, class P, class W>
cudaError_t launch_cluster(K kernel, int64_t values, const P& p, const W& w, cudaStream_t s) {
  // a block alone needs no cluster; it is enough for what it reads in a few passes
  const int ctas = values <= 8 * kThreadsP ? 1 : kCtasP;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreadsP);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, w);
}

}  // namespace

size_t fork_workspace(int R, int W, int N) { return fork_ws(R, W, N).total; }
size_t compact_workspace(int N) { return compact_ws(N).total; }

cudaError_t launch_fork(const ForkParams& p, const MovedPool* pools, int n, cudaStream_t s) {
  const ForkWs w = fork_ws(p.R, p.W, p.N);
  const cudaError_t e = launch_cluster(fork_kernel, static_cast<int64_t>(p.R) * p.W + p.N, p, w, s);
  if (e != cudaSuccess) return e;
  const MoveList list = {reinterpret_cast<const PagesHead*>(p.ws), reinterpret_cast<const Move*>(p.ws + w.moves),
                         nullptr, nullptr, 0, p.N, p.N, p.page_log2, p.status};
  return launch_moves(list, pools, n, true, s);
}

cudaError_t launch_compact(const CompactParams& p, const MovedPool* pools, int n, cudaStream_t s) {
  const CompactWs w = compact_ws(p.N);
  const int64_t cells = static_cast<int64_t>(p.t[0].R) * p.t[0].W + static_cast<int64_t>(p.t[1].R) * p.t[1].W;
  const cudaError_t e = launch_cluster(compact_kernel, cells + p.N, p, w, s);
  if (e != cudaSuccess) return e;
  const MoveList list = {reinterpret_cast<const PagesHead*>(p.ws), reinterpret_cast<const Move*>(p.ws + w.moves),
                         nullptr, nullptr, 0, p.N, p.N, p.page_log2, p.status};
  return launch_moves(list, pools, n, true, s);
}

cudaError_t launch_copy_pages(const int32_t* src, const int32_t* dst, int count, int src_pages, int dst_pages,
                              const MovedPool* pools, int n, int32_t* status, cudaStream_t s) {
  const MoveList list = {nullptr, nullptr, src, dst, count, src_pages, dst_pages, 0, status};
  return launch_moves(list, pools, n, false, s);
}

}  // namespace kv
}  // namespace attn
