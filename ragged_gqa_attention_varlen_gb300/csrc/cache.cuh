// cache.cuh -- the paged K/V cache: parameters of its kernels and the device
// helpers they share.
//
// A cache is a pool of pages [num_pages, page_size, Hkv, d] for K and one for
// V.  Slot j of sequence b is row j % page_size of page table[b][j /
// page_size], for j < lens[b].  A run of consecutive sequences may share a
// prefix: further slots, listed once in a table of their own, that precede
// each of these sequences' own slots.  Both kinds are "segments" here: a page
// table row, a length and the run of query tokens that read it.  Segments 0 ..
// P-1 are the prefixes, P .. P+B-1 the sequences' own slots.
#pragma once
#include "common.cuh"

namespace attn {
namespace kv {

// K or V pages; strides in elements.
struct Pages {
  const void* base;
  int64_t page, slot, head;
};

// One kind of segment (the prefixes, or the sequences' own slots).
struct Table {
  const int32_t* pages;  // [rows, width] with row stride `rs`; null: no such segments
  int64_t rs;
  int width;
  const int32_t* lens;    // [rows]
  const int32_t* pos;     // positions [rows, Hkv, >= width * page_size], or null
  int64_t pos_rs, pos_hs;
};

struct CacheParams {
  int dtype;  // 0 fp16, 1 bf16
  int B, P, Hq, Hkv, d;
  int R;      // query heads per K/V head
  float inv_R;
  int64_t total_q;
  const void* q;
  int64_t q_ts, q_hs;
  Pages k, v;
  int num_pages, page_size, page_log2;
  Table own, prefix;
  const int32_t* cu_prefix;  // [P+1] over the sequences
  const int32_t* cu_q;       // [B+1]
  const int32_t* q_pos;      // [total_q], or null: position Lk - Lq + i
  const float* slopes;       // [B, Hq] with batch stride, or null
  int64_t slopes_bs;
  int wl, wr;                // window limits, < 0: none (wr = 0 when causal)
  float softcap, sigma;
  int tile_cost;             // what a tile's start costs, in steps (cache_sched.cuh)
  int least_rows, most_rows; // the sequences that this kernel takes, by their rows of a K/V head (most 0: all)
  void* out;                 // forward
  int64_t out_ts, out_hs;
  float* lse;                // [total_q, Hq]; the forward writes it, the weights call reads it
  // key weights: rows [rows, Hkv, >= len] of the two kinds of segments
  const float* w_in[2];      // accumulated so far, or null (0: prefixes, 1: own)
  int64_t wi_rs[2], wi_hs[2];
  float* w_out[2];           // null: this kind is not wanted
  int64_t wo_rs[2], wo_hs[2];
  uint8_t* ws;
  int32_t* status;           // caller's sticky status word, or null
};

__device__ __forceinline__ void report(int32_t* status, int bits) {
  if (status) atomicOr(status, bits);
}

// The prefix that sequence b reads, or -1.
__device__ __forceinline__ int prefix_of(const CacheParams& p, int b) {
  int lo = 0, hi = p.P;  // the last group that starts at or before b
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu_prefix + mid + 1) <= b)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo < p.P && __ldg(p.cu_prefix + lo) <= b ? lo : -1;
}

// The sequence of packed query token t (cu_q is known to be monotone and to
// hold t): the last b in [b0, b1) with cu_q[b] <= t.
__device__ __forceinline__ int seq_of(const int32_t* cu, int b0, int b1, int t) {
  int lo = b0, hi = b1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Whether a key at position kpos is admissible for a query at qpos, and the
// bounds of that range (positions lie in [0, 2^30), so nothing overflows).
__device__ __forceinline__ int pos_lo(const CacheParams& p, int qpos) {
  return p.wl < 0 ? INT32_MIN : qpos - p.wl;
}
__device__ __forceinline__ int pos_hi(const CacheParams& p, int qpos) {
  return p.wr < 0 ? INT32_MAX : qpos + p.wr;
}

// The row of slot j of a segment inside a page pool, in elements, or -1 when
// its page is outside of the pool.
__device__ __forceinline__ int64_t slot_row(const CacheParams& p, const Pages& pg,
                                            const int32_t* row, int j) {
  const int page = __ldg(row + (j >> p.page_log2));
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) return -1;
  return page * pg.page + static_cast<int64_t>(j & (p.page_size - 1)) * pg.slot;
}

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t x) {
  return BF16 ? __uint_as_float(static_cast<uint32_t>(x) << 16)
              : __half2float(__ushort_as_half(x));
}
template <bool BF16>
__device__ __forceinline__ uint16_t from_float(float x) {
  return BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

// Tensor maps of a page pool: 64-feature boxes (128-byte swizzle), and with
// `tail` the 32 features from 128 on (64-byte swizzle).
bool encode_pages(CUtensorMap* m, const CacheParams& p, const Pages& pg, bool tail);
int device_ctas();  // CTAs of a persistent kernel on the current device

size_t fwd_workspace(int B, int P, int Hq, int Hkv, int d, int64_t total_q);
size_t fwd8_workspace(int B, int P, int Hq, int Hkv, int d, int64_t total_q);
size_t weights_workspace();
cudaError_t launch_fwd(const CacheParams& p, cudaStream_t s);
cudaError_t launch_weights(const CacheParams& p, cudaStream_t s);

// Scales of a pool held in 8 bits: [num_pages, page_size / block, Hkv].
struct Scales {
  float* base;
  int64_t page, block, head;
};

// Attention over a cache held in 8 bits (k, v of `c`: pages of e4m3 values).
struct Cache8Params {
  CacheParams c;
  Scales ks, vs;
  int block_log2;
};
cudaError_t launch_fwd8(const Cache8Params& p, cudaStream_t s);

// Rotary positions: x[H][d] rows of up to two tensors, or new K rows on their
// way into the cache.
struct RotaryTable {
  const double* inv_freq;    // [pairs] on the device; null: no rotation
  const int32_t* pair_axis;  // [pairs], or null (every pair: axis 0)
  const int32_t* positions;  // [axes, tokens] with axis stride
  int64_t axis_stride;
  int axes, pairs, interleaved, inverse;
};

struct RotaryTensor {
  const void* x;
  int64_t ts, hs;
  void* out;
  int64_t ots, ohs;
  int H;
};

struct RotaryParams {
  int dtype, d;
  int64_t T;
  RotaryTable r;
  RotaryTensor t[2];  // t[1].H = 0: only one
};

// Norms of the rows of up to two tensors, with the turn in the same pass.
struct NormTensor {
  const void* x;
  int64_t ts, hs;
  const void* dy;        // backward: the gradient of the output
  int64_t dts, dhs;
  const float* weight;   // [d], or null: ones
  void* out;             // the output, or (backward) the gradient of x
  int64_t ots, ohs;
  float* dweight;        // backward: [d], or null
  int H;
};

struct NormParams {
  int dtype, d;
  int64_t T;
  float eps;
  RotaryTable r;  // r.inv_freq null: no turn
  NormTensor t[2];
  float* partial;  // backward: sums of a block [blocks, d]
};

struct AppendParams {
  int dtype, B, Hkv, d;
  int64_t T;
  const void *kx, *vx;
  int64_t k_ts, k_hs, v_ts, v_hs;
  Pages k, v;  // written
  int num_pages, page_size, page_log2;
  const int32_t* table;
  int64_t table_rs;
  int width;
  const int32_t* lens;
  const int32_t* cu_new;
  RotaryTable r;
  int32_t* key_pos;
  int64_t kp_rs, kp_hs;
  float* scores;
  int64_t sc_rs, sc_hs;
  int32_t* lens_out;
  int32_t* status;
};

struct Append8Params {
  AppendParams a;  // (k, v: pages of e4m3 values; strides in elements)
  Scales ks, vs;
  int block, block_log2;
  const float* k_weight;  // [d]: K rows are normed first; null: not, unless `norm`
  int norm;
  float eps;
};

struct EvictParams {
  int S, Hkv, d;
  Pages k, v;  // moved in place
  int num_pages, page_size, page_log2;
  const int32_t* table;
  int64_t table_rs;
  int width;
  const int32_t* lens;
  const float* scores;
  int64_t sc_rs, sc_hs;
  const int32_t* key_pos;
  int64_t kp_rs, kp_hs;
  const int32_t* next_pos;
  int budget, recent;
  float* scores_out;
  int64_t so_rs, so_hs;
  int32_t* pos_out;
  int64_t po_rs, po_hs;
  int32_t* lens_out;
  uint8_t* ws;
  int32_t* status;
};

// A pool of pages as the kernels that move whole pages see it: `rows` rows a
// page, each of `pieces` runs of `bytes` contiguous bytes; strides in bytes.
struct MovedPool {
  const void* src;
  void* dst;
  int64_t src_page, src_row, src_piece, dst_page, dst_row, dst_piece;
  int rows, pieces, bytes;
  int flat;  // a page is one run of bytes in both
  int wide;  // everything is a multiple of 16 bytes (of 4 otherwise)
};
constexpr int kPoolsPerLaunch = 32;
struct MovedPools {
  MovedPool pool[kPoolsPerLaunch];
  int n;
};

// One move of the list in a workspace: page dst takes the first `used` of the
// page_size slots of page src.
struct Move {
  int src, dst, used, pad;
};

struct ForkParams {
  int R, W, N;  // rows and width of the table, pages
  int page_log2;
  const int32_t* table;
  int64_t table_rs;
  const int32_t *lens, *held, *refs, *parents, *room;
  int32_t* table_out;
  int64_t to_rs;
  int32_t *lens_out, *held_out, *refs_out;
  uint8_t* ws;
  int32_t* status;
};

// Tables whose pages a compaction renumbers.
struct CompactTable {
  int R, W;
  const int32_t* table;
  int64_t rs;
  const int32_t* held;
  int32_t* out;
  int64_t out_rs;
};
struct CompactParams {
  int N, page_log2;
  const int32_t* refs;
  int32_t* refs_out;
  int32_t* live;
  CompactTable t[2];  // t[1].R = 0: only one
  uint8_t* ws;
  int32_t* status;
};

size_t fork_workspace(int R, int W, int N);
size_t compact_workspace(int N);
// pools: n of them in host memory, moved within themselves (src = dst)
cudaError_t launch_fork(const ForkParams& p, const MovedPool* pools, int n, cudaStream_t s);
cudaError_t launch_compact(const CompactParams& p, const MovedPool* pools, int n, cudaStream_t s);
// count pairs (src[i], dst[i]) on the device
cudaError_t launch_copy_pages(const int32_t* src, const int32_t* dst, int count, int src_pages,
                              int dst_pages, const MovedPool* pools, int n, int32_t* status,
                              cudaStream_t s);
size_t evict_workspace(int S, int Hkv, int64_t slots, int budget);
cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t s);
size_t norm_bwd_workspace(int64_t T, int Hq, int Hkv, int d);
cudaError_t launch_norm(const NormParams& p, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormParams& p, cudaStream_t s);
cudaError_t launch_append(const AppendParams& p, cudaStream_t s);
cudaError_t launch_append8(const Append8Params& p, cudaStream_t s);
cudaError_t launch_evict(const EvictParams& p, cudaStream_t s);

}  // namespace kv
}  // namespace attn
