// Blocks and pages of a cache after gdn_batch_maps has handed them out:
// sharing a request's blocks with new branches of it, giving blocks up,
// moving the blocks in use to the low end of the pool, and the copies of
// pages that these ask for (TokenSpeed Qwen3.5 page, "Scheduler dual" and
// "Ciclo de vida de slots": requests hold block indices, checkpoints are
// block-aligned, a shared prefix is kept once).
//
// Whole numbers but for the page copies, which are HBM streams.  Every result
// is the same whatever the order in which the threads run: new blocks go out
// in the requests' order, given-up ones go back by id.
#include "gdn_common.cuh"
#include "decode_tma.cuh"  // sm_count

#include <cooperative_groups.h>

namespace gdn {
namespace {

// ---------------------------------------------------------------------------
// page copy
// ---------------------------------------------------------------------------
// A CTA walks the pairs y, y + gridDim.y, ... of one piece (16 KB) of one plane:
// it reads its pairs' ids 256 at a time, keeps the usable ones, and moves two
// pairs' pieces at once with eight 16-byte accesses in flight per thread.
constexpr int kCopyThreads = 256, kCopyVec = 4, kCopyPairs = 2;
constexpr int64_t kPiece = (int64_t)kCopyThreads * kCopyVec * 16;

struct CopyArgs {
  void* const* planes;
  int32_t n_planes, n, num_pages;
  int64_t page_bytes, page_stride;
  const int32_t* src_ids;
  const int32_t* dst_ids;
  uint32_t* err;
  int32_t pieces;
};

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const CopyArgs a) {
  __shared__ int2 pair[kCopyThreads];
  __shared__ int n_pair;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int plane = blockIdx.x / a.pieces, piece = blockIdx.x % a.pieces;
  const int64_t begin = piece * kPiece, end = min(a.page_bytes, begin + kPiece);
  const auto src_ids = GDN_GV(a.src_ids, a.n), dst_ids = GDN_GV(a.dst_ids, a.n);
  char* const base = reinterpret_cast<char*>(GDN_GV(a.planes, a.n_planes)[plane]);
  const auto pages = GDN_GV(base, a.num_pages > 0 ? (a.num_pages - 1) * a.page_stride + a.page_bytes : 0);
  const int64_t mine = (a.n - (int64_t)blockIdx.y + gridDim.y - 1) / gridDim.y;  // pairs of this CTA
  for (int64_t j0 = 0; j0 < mine; j0 += kCopyThreads) {
    if (tid == 0) n_pair = 0;
    __syncthreads();
    const int64_t j = j0 + tid;
    if (j < mine) {
      const int64_t i = blockIdx.y + j * gridDim.y;
      const int32_t s = src_ids[i], d = dst_ids[i];
      const int cs = slot_class(s, a.num_pages), cd = slot_class(d, a.num_pages);
      if ((cs == 2 || cd == 2) && blockIdx.x == 0) report(a.err, GDN_DEV_ERR_SLOT_OOB);
      if (!cs && !cd) pair[atomicAdd(&n_pair, 1)] = make_int2(s, d);  // any order: the destinations are distinct
    }
    __syncthreads();
    const int np = n_pair;
    for (int p = 0; p < np; p += kCopyPairs) {
      uint4 v[kCopyPairs][kCopyVec];
#pragma unroll
      for (int k = 0; k < kCopyPairs; ++k)
#pragma unroll
        for (int i = 0; i < kCopyVec; ++i) {
          const int64_t off = begin + ((int64_t)i * kCopyThreads + tid) * 16;
          if (p + k < np && off < end) v[k][i] = __ldcs(&vec_at<const uint4>(pages, pair[p + k].x * a.page_stride + off));
        }
#pragma unroll
      for (int k = 0; k < kCopyPairs; ++k)
#pragma unroll
        for (int i = 0; i < kCopyVec; ++i) {
          const int64_t off = begin + ((int64_t)i * kCopyThreads + tid) * 16;
          if (p + k < np && off < end) __stcs(&vec_at<uint4>(pages, pair[p + k].y * a.page_stride + off), v[k][i]);
        }
    }
    __syncthreads();  // pair and n_pair may be replaced
  }
}

// ---------------------------------------------------------------------------
// scans
// ---------------------------------------------------------------------------
constexpr int kThreads = 1024;
// inclusive scan of one value per thread of a CTA of kThreads; total: the sum
__device__ __forceinline__ int scan_cta(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int s = warp_sums[lane];  // 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  const int before = warp ? __shfl_sync(0xffffffffu, s, warp - 1) : 0;
  total = __shfl_sync(0xffffffffu, s, 31);
  __syncthreads();  // warp_sums may be written again
  return v + before;
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
struct ForkArgs {
  const int32_t* src_rows;
  const int32_t* dst_rows;
  const int64_t* lens;
  int32_t n, shift;
  int32_t* table;
  int32_t n_rows, max_blocks;
  int32_t* refs;
  int32_t num_blocks;
  const int32_t* free_ids;
  int32_t free_cap;
  const int32_t* n_free;
  int32_t* n_free_out;
  int32_t* copy_src;
  int32_t* copy_dst;
  uint32_t* err;
};

// fork i's rows and blocks; false: it is padding or wrong (bits in bad)
struct Fork {
  int32_t src, dst;
  int64_t full;  // whole blocks
  bool part;     // and a partly filled one
};
__device__ __forceinline__ bool load_fork(const ForkArgs& a, int i, Fork& f, uint32_t& bad) {
  f.src = GDN_GV(a.src_rows, a.n)[i];
  f.dst = GDN_GV(a.dst_rows, a.n)[i];
  const int64_t len = GDN_GV(a.lens, a.n)[i];
  const int cs = slot_class(f.src, a.n_rows), cd = slot_class(f.dst, a.n_rows);
  if (cs == 2 || cd == 2 || (!cs && !cd && f.src == f.dst)) bad |= GDN_DEV_ERR_SLOT_OOB;
  if (cs || cd || f.src == f.dst) return false;
  if (len < 0 || len > ((int64_t)a.max_blocks << a.shift)) {
    bad |= GDN_DEV_ERR_SEQLENS;
    return false;
  }
  f.full = len >> a.shift;
  f.part = (len & (((int64_t)1 << a.shift) - 1)) != 0;
  return true;
}

// one CTA: the new blocks, in the forks' order, and the pairs to copy
__device__ __forceinline__ void fork_alloc(const ForkArgs& a, int* warp_sums) {
  const int tid = threadIdx.x;
  const int32_t n_free = min(max(*a.n_free, 0), a.free_cap);
  uint32_t bad = 0;
  int carry = 0;
  for (int i0 = 0; i0 < a.n; i0 += kThreads) {
    const int i = i0 + tid;
    Fork f;
    bool some = false;
    int32_t from = -1;
    if (i < a.n) {
      some = load_fork(a, i, f, bad) && f.part;
      if (some) {
        from = GDN_GV(a.table, (long long)a.n_rows * a.max_blocks)[(int64_t)f.src * a.max_blocks + f.full];
        if (slot_class(from, a.num_blocks)) {  // nothing to copy from
          bad |= GDN_DEV_ERR_SLOT_OOB;
          some = false;
        }
      }
    }
    int total;
    const int rank = carry + scan_cta(some, warp_sums, total) - 1;
    carry += total;
    if (i < a.n) {
      int32_t to = -1;
      if (some && rank < n_free) {
        to = GDN_GV(a.free_ids, a.free_cap)[n_free - 1 - rank];
        if (slot_class(to, a.num_blocks)) {
          bad |= GDN_DEV_ERR_SLOT_OOB;
          to = -1;
        }
      } else if (some) {
        bad |= GDN_DEV_ERR_BLOCKS;
      }
      GDN_GV(a.copy_src, a.n)[i] = to < 0 ? -1 : from;
      GDN_GV(a.copy_dst, a.n)[i] = to;
    }
  }
  if (bad) report(a.err, bad);
  if (tid == 0) *a.n_free_out = max(n_free - carry, 0);
}

// forks first, first + step, ..: their rows of the table, by `threads` threads of
// which this is number t, and one more holder per shared block
__device__ __forceinline__ void fork_rows(const ForkArgs& a, int64_t first, int64_t step, int t, int threads) {
  const auto table = GDN_GV(a.table, (long long)a.n_rows * a.max_blocks);
  for (int64_t i = first; i < a.n; i += step) {
    Fork f;
    uint32_t bad = 0;
    if (!load_fork(a, (int)i, f, bad)) continue;  // reported by fork_alloc
    for (int64_t j = t; j < f.full + f.part; j += threads) {
      int32_t id;
      if (j < f.full) {
        id = table[(int64_t)f.src * a.max_blocks + j];
        if (slot_class(id, a.num_blocks)) {
          bad |= GDN_DEV_ERR_SLOT_OOB;
          id = -1;
        } else {
          atomicAdd(&GDN_GV(a.refs, a.num_blocks)[id], 1);
        }
      } else {
        id = GDN_GV(a.copy_dst, a.n)[i];
      }
      table[(int64_t)f.dst * a.max_blocks + j] = id;
    }
    if (bad) report(a.err, bad);
  }
}

// Small batches: one cluster, a warp per fork.  Larger ones in two launches, the
// second with a CTA per fork on the whole GPU.
constexpr int kCluster = 8;
constexpr int kRowThreads = 256;
__global__ void __launch_bounds__(kThreads) fork_small_kernel(const ForkArgs a) {
  __shared__ int warp_sums[32];
  pdl_wait();
  pdl_trigger();
  const int rank = (int)cluster_ctarank();
  if (rank == 0) fork_alloc(a, warp_sums);
  cluster_arrive_release();
  cluster_wait_acquire();  // copy_dst complete
  fork_rows(a, rank * (kThreads / 32) + (threadIdx.x >> 5), kCluster * (kThreads / 32), threadIdx.x & 31, 32);
}
__global__ void __launch_bounds__(kThreads) fork_alloc_kernel(const ForkArgs a) {
  __shared__ int warp_sums[32];
  pdl_wait();
  pdl_trigger();
  fork_alloc(a, warp_sums);
}
__global__ void __launch_bounds__(kRowThreads) fork_rows_kernel(const ForkArgs a) {
  pdl_wait();
  pdl_trigger();
  fork_rows(a, blockIdx.x, gridDim.x, threadIdx.x, kRowThreads);
}
// Whether one cluster does a call over n rows of max_blocks entries: up to one
// entry per thread of it (256 rows of 128 in a graph: fork, copy and release 26 us so, 21 with the GPU).
bool one_cluster(int64_t n, int64_t max_blocks) { return n * max_blocks <= (int64_t)kCluster * kThreads; }

// ---------------------------------------------------------------------------
// release
// ---------------------------------------------------------------------------
struct ReleaseArgs {
  const int32_t* rows;
  const int64_t* old_lens;
  const int64_t* new_lens;
  int32_t n, shift;
  int32_t* table;
  int32_t n_rows, max_blocks;
  int32_t* refs;
  int32_t num_blocks;
  int32_t* free_ids;
  int32_t free_cap;
  const int32_t* n_free;
  int32_t* n_free_out;
  uint32_t* err;
};

// Requests first, first + step, ..: one holder less for every block behind a
// request's new length.  A block that nobody holds any more ends at -1.
__device__ __forceinline__ void release_rows(const ReleaseArgs& a, int64_t first, int64_t step, int t, int threads) {
  const auto table = GDN_GV(a.table, (long long)a.n_rows * a.max_blocks);
  const auto refs = GDN_GV(a.refs, a.num_blocks);
  const int64_t up = ((int64_t)1 << a.shift) - 1;
  for (int64_t i = first; i < a.n; i += step) {
    const int32_t row = GDN_GV(a.rows, a.n)[i];
    const int cls = slot_class(row, a.n_rows);
    uint32_t bad = cls == 2 ? GDN_DEV_ERR_SLOT_OOB : 0;
    const int64_t from = GDN_GV(a.new_lens, a.n)[i], to = GDN_GV(a.old_lens, a.n)[i];
    if (!cls && (from < 0 || to < from || to > ((int64_t)a.max_blocks << a.shift))) bad |= GDN_DEV_ERR_SEQLENS;
    if (!cls && !bad)
      for (int64_t j = ((from + up) >> a.shift) + t; j < (to + up) >> a.shift; j += threads) {
        const int64_t at = (int64_t)row * a.max_blocks + j;
        const int32_t id = table[at];
        table[at] = -1;
        if (slot_class(id, a.num_blocks)) bad |= GDN_DEV_ERR_SLOT_OOB;
        else if (atomicSub(&refs[id], 1) < 0) bad |= GDN_DEV_ERR_SLOT_OOB;  // given up more often than held
      }
    if (bad) report(a.err, bad);
  }
}
__global__ void __launch_bounds__(kRowThreads) release_rows_kernel(const ReleaseArgs a) {
  pdl_wait();
  pdl_trigger();
  release_rows(a, blockIdx.x, gridDim.x, threadIdx.x, kRowThreads);
}

// One cluster: the blocks at -1, in ascending order, onto the stack; ROWS: the
// requests' rows before that, a warp each.
constexpr int kPer = 4;  // consecutive blocks per thread and pass
template <bool ROWS>
__global__ void __launch_bounds__(kThreads) release_push_kernel(const ReleaseArgs a) {
  __shared__ int warp_sums[32];
  __shared__ int counts[kCluster];  // in CTA 0: every CTA's
  pdl_wait();
  pdl_trigger();
  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = (int)cluster_ctarank();
  const auto refs = GDN_GV(a.refs, a.num_blocks);
  constexpr int kTile = kThreads * kPer;
  const int64_t tiles = ((int64_t)a.num_blocks + kTile - 1) / kTile, per = (tiles + kCluster - 1) / kCluster;
  const int64_t b0 = rank * per * kTile, b1 = min((int64_t)a.num_blocks, b0 + per * kTile);
  if (ROWS) release_rows(a, rank * (kThreads / 32) + (tid >> 5), kCluster * (kThreads / 32), tid & 31, 32);
  cluster.sync();  // the counts are final; every CTA has begun, so that its shared memory may be written
  int mine = 0;
  for (int64_t b = b0 + tid; b < b1; b += kThreads) mine += refs[b] < 0;
  int total;
  scan_cta(mine, warp_sums, total);
  if (tid < kCluster) *cluster.map_shared_rank(&counts[rank], tid) = total;
  cluster.sync();
  int64_t at = min(max(*a.n_free, 0), a.free_cap);
  int64_t all = at;
  for (int k = 0; k < kCluster; ++k) {
    if (k < rank) at += counts[k];
    all += counts[k];
  }
  cluster.sync();  // everyone has read *n_free and the counts
  if (total)
    for (int64_t t0 = b0; t0 < b1; t0 += kTile) {
      int f = 0;
      const int64_t b = t0 + (int64_t)tid * kPer;
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (b + e < b1 && refs[b + e] < 0) f |= 1 << e;
      int here;
      int64_t to = at + scan_cta(__popc(f), warp_sums, here) - __popc(f);
      at += here;
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (f >> e & 1) {
          refs[b + e] = 0;
          if (to < a.free_cap) GDN_GV(a.free_ids, a.free_cap)[to] = (int32_t)(b + e);
          ++to;
        }
    }
  if (rank == 0 && tid == 0) {
    if (all > a.free_cap) report(a.err, GDN_DEV_ERR_BLOCKS);
    *a.n_free_out = (int32_t)min(all, (int64_t)a.free_cap);
  }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
struct CompactArgs {
  const int32_t* table;
  int32_t* table_out;
  int64_t n_entries;
  const int32_t* refs;
  int32_t* refs_out;
  int32_t num_blocks;
  const int32_t* free_ids;
  int32_t* free_out;
  int32_t free_cap;
  const int32_t* n_free;
  int32_t* move_src;
  int32_t* move_dst;
  int32_t max_moves;
  int32_t* n_moves;
  int32_t* remap;    // [num_blocks]
  uint32_t* bitmap;  // [words]: the free blocks
  int32_t* wrong;    // whether the stack is inconsistent
  int32_t words;
  uint32_t* err;
};

// the tables' entries, by `step` threads of which this is number `first`
__device__ __forceinline__ void remap_entries(const CompactArgs& a, int64_t first, int64_t step) {
  const auto table = GDN_GV(a.table, a.n_entries);
  const auto out = GDN_GV(a.table_out, a.n_entries);
  const auto remap = GDN_GV(a.remap, a.num_blocks);
  for (int64_t i = first; i < a.n_entries; i += step) {
    const int32_t id = table[i];
    out[i] = slot_class(id, a.num_blocks) ? id : remap[id];
  }
}

// `live` blocks are in use; the k-th highest of those at or above `live` goes to
// the k-th lowest free one below it.
//
// One CTA with everything but the tensors in its shared memory, 8 blocks and 8
// table entries per thread: a few dependent global accesses and eight
// barriers.  512 blocks 4.8 us (by one cluster 13.4), 8192 blocks 11.9 (19.2).
constexpr int kSmallBlocks = 8 * kThreads, kSmallEntries = 8 * kThreads;
template <bool REMAP>
__global__ void __launch_bounds__(kThreads) compact_small_kernel(const CompactArgs a) {
  constexpr int kWords = kSmallBlocks / 32, kPer = 8;
  __shared__ uint32_t bits_s[kWords], was_s[kWords];                // the free blocks: now, before the moves
  __shared__ uint16_t to_s[kSmallBlocks];                           // where a block goes
  __shared__ uint16_t src_s[kSmallBlocks / 2], dst_s[kSmallBlocks / 2];  // (as many movers as holes)
  __shared__ int warp_sums[32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, N = a.num_blocks;
  const auto bits = GDN_SV(bits_s, kWords), was = GDN_SV(was_s, kWords);
  const auto to = GDN_SV(to_s, kSmallBlocks), src = GDN_SV(src_s, kSmallBlocks / 2), dst = GDN_SV(dst_s, kSmallBlocks / 2);
  const auto free_ids = GDN_GV(a.free_ids, a.free_cap);
  const auto free_out = GDN_GV(a.free_out, a.free_cap);
  const auto refs = GDN_GV(a.refs, N);
  const auto refs_out = GDN_GV(a.refs_out, N);
  const auto table = GDN_GV(a.table, a.n_entries);
  const auto table_out = GDN_GV(a.table_out, a.n_entries);
  const auto move_src = GDN_GV(a.move_src, a.max_moves), move_dst = GDN_GV(a.move_dst, a.max_moves);
  const int32_t nf0 = *a.n_free;
  int32_t entry[kPer];
  if (REMAP) {
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (e * kThreads + tid < a.n_entries) entry[e] = table[e * kThreads + tid];
  }
  if (tid < kWords) bits[tid] = 0;
  for (int b = tid; b < N; b += kThreads) to[b] = (uint16_t)b;
  __syncthreads();
  const bool bad_count = nf0 < 0 || nf0 > a.free_cap || nf0 > N;
  const int32_t n_free = bad_count ? 0 : nf0;
  bool wrong = false;
  for (int i = tid; i < n_free; i += kThreads) {
    const int32_t id = free_ids[i];
    if (id < 0 || id >= N) wrong = true;
    else if (atomicOr(&bits[id >> 5], 1u << (id & 31)) >> (id & 31) & 1) wrong = true;  // twice on the stack
  }
  if (wrong) report(a.err, GDN_DEV_ERR_SLOT_OOB);
  if (bad_count && tid == 0) report(a.err, GDN_DEV_ERR_BLOCKS);
  const bool skip = __syncthreads_or(wrong || bad_count) != 0;
  // this thread's blocks 8 tid .. 8 tid + 7
  const int b0 = kPer * tid, live = N - n_free;
  auto first = [&](int n) { return (1u << min(max(n - b0, 0), kPer)) - 1; };  // those below n
  auto mine = [&]() { return bits[tid / 4] >> (kPer * (tid % 4)) & 0xffu; };
  int moves = 0;
  if (!skip) {
    uint32_t h = mine() & first(live), m = ~mine() & first(N) & ~first(live);
    const int nh = __popc(h), nm = __popc(m);
    int total;
    const int upto = scan_cta(nh | nm << 16, warp_sums, total), all = total >> 16;
    moves = min(all, a.max_moves);
    int k = (upto & 0xffff) - nh;
    for (; h; h &= h - 1, ++k)
      if (k < moves) dst[k] = (uint16_t)(b0 + __ffs(h) - 1);
    k = all - (upto >> 16);  // movers above this thread's
    for (; m; ++k) {
      const int b = 31 - __clz(m);
      if (k < moves) src[k] = (uint16_t)(b0 + b);
      m &= ~(1u << b);
    }
    if (tid < kWords) was[tid] = bits[tid];
    __syncthreads();
  }
  for (int64_t k = tid; k < a.max_moves; k += kThreads) {
    if (k < moves) {
      const int s = src[k], d = dst[k];
      const int32_t c = refs[s];
      move_src[k] = s;
      move_dst[k] = d;
      to[s] = (uint16_t)d;
      atomicOr(&bits[s >> 5], 1u << (s & 31));
      atomicAnd(&bits[d >> 5], ~(1u << (d & 31)));
      refs_out[d] = c;  // a moved block's count goes along
      refs_out[s] = 0;
    } else {
      move_src[k] = move_dst[k] = -1;
    }
  }
  if (tid == 0) *a.n_moves = moves;
  __syncthreads();
  if (a.refs_out != a.refs)  // the others; a free block has none
    for (int b = tid; b < N; b += kThreads) {
      const uint32_t now = bits[b >> 5] >> (b & 31) & 1;
      if (skip) refs_out[b] = refs[b];
      else if (now == (was[b >> 5] >> (b & 31) & 1)) refs_out[b] = now ? 0 : refs[b];
    }
  if (a.free_out != a.free_ids)
    for (int64_t i = (skip ? 0 : n_free) + tid; i < a.free_cap; i += kThreads) free_out[i] = free_ids[i];
  if (REMAP) {
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (e * kThreads + tid < a.n_entries)
        table_out[e * kThreads + tid] = slot_class(entry[e], N) ? entry[e] : (int32_t)to[entry[e]];
  } else {
    const auto remap = GDN_GV(a.remap, N);
    for (int b = tid; b < N; b += kThreads) remap[b] = to[b];
  }
  if (skip) return;
  // the stack: the free blocks, the lowest on top
  uint32_t f = mine();
  int all;
  int k = scan_cta(__popc(f), warp_sums, all) - __popc(f);
  for (; f; f &= f - 1, ++k) free_out[n_free - 1 - k] = (int32_t)(b0 + __ffs(f) - 1);
}

// The same by one cluster, for pools beyond a CTA's shared memory.
template <bool REMAP>
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a) {
  __shared__ int warp_sums[32];
  __shared__ int counts[2][kCluster];
  pdl_wait();
  pdl_trigger();
  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = (int)cluster_ctarank(), gt = rank * kThreads + tid, gn = kCluster * kThreads;
  const auto free_ids = GDN_GV(a.free_ids, a.free_cap);
  const auto free_out = GDN_GV(a.free_out, a.free_cap);
  const auto refs = GDN_GV(a.refs, a.num_blocks);
  const auto refs_out = GDN_GV(a.refs_out, a.num_blocks);
  const auto remap = GDN_GV(a.remap, a.num_blocks);
  const auto bitmap = GDN_GV(a.bitmap, a.words);
  const auto move_src = GDN_GV(a.move_src, a.max_moves), move_dst = GDN_GV(a.move_dst, a.max_moves);
  const int32_t nf0 = *a.n_free;
  const bool bad_count = nf0 < 0 || nf0 > a.free_cap || nf0 > a.num_blocks;
  const int32_t n_free = bad_count ? 0 : nf0;
  for (int w = gt; w < a.words; w += gn) bitmap[w] = 0;
  if (gt == 0) *a.wrong = bad_count;
  for (int64_t b = gt; b < a.num_blocks; b += gn) remap[b] = (int32_t)b;
  for (int64_t k = gt; k < a.max_moves; k += gn) move_src[k] = move_dst[k] = -1;
  cluster.sync();  // (every CTA has begun, too: see the stores to their shared memory below)
  bool wrong = false;
  for (int i = gt; i < n_free; i += gn) {
    const int32_t id = free_ids[i];
    if (id < 0 || id >= a.num_blocks) wrong = true;
    else if (atomicOr(&bitmap[id >> 5], 1u << (id & 31)) >> (id & 31) & 1) wrong = true;  // twice on the stack
  }
  if (wrong) {
    report(a.err, GDN_DEV_ERR_SLOT_OOB);
    atomicExch(a.wrong, 1);
  }
  cluster.sync();
  const bool skip = *reinterpret_cast<volatile int32_t*>(a.wrong) != 0;
  if (bad_count && gt == 0) report(a.err, GDN_DEV_ERR_BLOCKS);
  const int64_t live = a.num_blocks - n_free;
  // this CTA's words, one per thread and pass
  const int passes = (a.words + gn - 1) / gn, w0 = rank * passes * kThreads;
  // a word's free blocks; bits outside the pool count as neither free nor used
  auto inside = [&](int64_t w) -> uint32_t {
    const int64_t left = a.num_blocks - 32 * w;
    return w >= a.words || left <= 0 ? 0u : left >= 32 ? 0xffffffffu : (1u << left) - 1;
  };
  auto below = [&](int64_t w) -> uint32_t {  // the bits of blocks below `live`
    const int64_t left = live - 32 * w;
    return left <= 0 ? 0u : left >= 32 ? 0xffffffffu : (1u << left) - 1;
  };
  auto holes = [&](int64_t w) -> uint32_t { return w < a.words ? bitmap[w] & below(w) : 0u; };
  auto movers = [&](int64_t w) -> uint32_t { return w < a.words ? ~bitmap[w] & inside(w) & ~below(w) : 0u; };
  int moves = 0;
  if (!skip) {
    int nh = 0, nm = 0;
    for (int p = 0; p < passes; ++p) {
      nh += __popc(holes(w0 + p * kThreads + tid));
      nm += __popc(movers(w0 + p * kThreads + tid));
    }
    int th, tm;
    scan_cta(nh, warp_sums, th);
    scan_cta(nm, warp_sums, tm);
    if (tid < kCluster) {
      *cluster.map_shared_rank(&counts[0][rank], tid) = th;
      *cluster.map_shared_rank(&counts[1][rank], tid) = tm;
    }
    cluster.sync();
    int at_h = 0, above = 0, all = 0;
    for (int k = 0; k < kCluster; ++k) {
      if (k < rank) at_h += counts[0][k];
      if (k > rank) above += counts[1][k];
      all += counts[1][k];
    }
    moves = min(all, a.max_moves);
    int left = above + tm;  // movers from this pass's first word on
    for (int p = 0; p < passes; ++p) {
      const int64_t w = w0 + p * kThreads + tid;
      uint32_t h = holes(w), m = movers(w);
      int here;
      int k = at_h + scan_cta(__popc(h), warp_sums, here) - __popc(h);
      at_h += here;
      for (; h; h &= h - 1, ++k)
        if (k < moves) move_dst[k] = (int32_t)(32 * w + __ffs(h) - 1);
      k = left - scan_cta(__popc(m), warp_sums, here);  // movers above this word
      left -= here;
      for (; m; ++k) {
        const int b = 31 - __clz(m);
        if (k < moves) move_src[k] = (int32_t)(32 * w + b);
        m &= ~(1u << b);
      }
    }
    cluster.sync();  // both lists complete, the bitmap read
    for (int k = gt; k < moves; k += gn) {
      const int32_t s = move_src[k], d = move_dst[k];
      remap[s] = d;
      atomicOr(&bitmap[s >> 5], 1u << (s & 31));
      atomicAnd(&bitmap[d >> 5], ~(1u << (d & 31)));
    }
    cluster.sync();
  }
  if (gt == 0) *a.n_moves = moves;
  // reference counts: a moved block's go along, a free block has none
  if (a.refs_out != a.refs)
    for (int64_t b = gt; b < a.num_blocks; b += gn)
      if (skip) refs_out[b] = refs[b];
      else if (remap[b] == b && !(bitmap[b >> 5] >> (b & 31) & 1)) refs_out[b] = refs[b];
      else if (bitmap[b >> 5] >> (b & 31) & 1) refs_out[b] = 0;
  if (!skip) {
    if (a.refs_out != a.refs) cluster.sync();  // before the moved blocks' own counts
    for (int k = gt; k < moves; k += gn) {
      const int32_t c = refs[move_src[k]];
      refs_out[move_dst[k]] = c;
      refs_out[move_src[k]] = 0;
    }
  }
  // the stack: the free blocks, the lowest on top
  if (skip) {
    if (a.free_out != a.free_ids)
      for (int64_t i = gt; i < a.free_cap; i += gn) free_out[i] = free_ids[i];
    if (REMAP) remap_entries(a, gt, gn);  // the identity
    return;
  }
  if (a.free_out != a.free_ids)
    for (int64_t i = n_free + gt; i < a.free_cap; i += gn) free_out[i] = free_ids[i];
  if (REMAP) remap_entries(a, gt, gn);  // remap has been final since the last barrier
  int nf = 0;
  for (int p = 0; p < passes; ++p) {
    const int64_t w = w0 + p * kThreads + tid;
    nf += w < a.words ? __popc(bitmap[w]) : 0;
  }
  int tf;
  scan_cta(nf, warp_sums, tf);
  if (tid < kCluster) *cluster.map_shared_rank(&counts[0][rank], tid) = tf;
  cluster.sync();
  int before = 0;
  for (int k = 0; k < rank; ++k) before += counts[0][k];
  for (int p = 0; p < passes; ++p) {
    const int64_t w = w0 + p * kThreads + tid;
    uint32_t f = w < a.words ? bitmap[w] : 0u;
    int here;
    int k = before + scan_cta(__popc(f), warp_sums, here) - __popc(f);
    before += here;
    for (; f; f &= f - 1, ++k) free_out[n_free - 1 - k] = (int32_t)(32 * w + __ffs(f) - 1);
  }
}

// the tables' entries where they are too many for the cluster
__global__ void __launch_bounds__(kRowThreads) remap_kernel(const CompactArgs a) {
  pdl_wait();
  pdl_trigger();
  remap_entries(a, (int64_t)blockIdx.x * kRowThreads + threadIdx.x, (int64_t)gridDim.x * kRowThreads);
}

int shift_of(int32_t block) {
  int s = 0;
  while ((1 << s) < block) ++s;
  return s;
}
bool pow2(int32_t block) { return block > 0 && !(block & (block - 1)); }
constexpr int64_t up16(int64_t x) { return (x + 15) & ~(int64_t)15; }

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_page_copy(void* const* planes, int32_t n_planes, int64_t page_bytes, int64_t page_stride,
                                    int32_t num_pages, const int32_t* src_ids, const int32_t* dst_ids, int32_t n,
                                    uint32_t* dev_err, void* stream) {
  using namespace gdn;
  if (n_planes < 0 || n < 0 || num_pages < 0 || page_bytes <= 0 || page_stride < page_bytes) return GDN_ERR_INVALID_ARG;
  if (page_bytes % 16 || page_stride % 16) return GDN_ERR_UNSUPPORTED;
  if (n == 0 || n_planes == 0) return GDN_OK;
  if (!planes || !src_ids || !dst_ids) return GDN_ERR_INVALID_ARG;
  const int64_t pieces = (page_bytes + kPiece - 1) / kPiece;
  if (pieces * n_planes > 2147483647LL) return GDN_ERR_UNSUPPORTED;
  CopyArgs a = {planes, n_planes, n, num_pages, page_bytes, page_stride, src_ids, dst_ids, dev_err, (int32_t)pieces};
  // as many CTAs per piece as fill the GPU, each walking its share of the pairs
  const int64_t x = pieces * n_planes, fill = std::max<int64_t>(1, 8LL * sm_count() / x);
  const unsigned y = (unsigned)std::min<int64_t>(std::min<int64_t>(n, fill), 65535);
  if (launch_pdl(page_copy_kernel, dim3((unsigned)x, y), dim3(kCopyThreads), 0, reinterpret_cast<cudaStream_t>(stream),
                 dim3(1), a) != cudaSuccess)
    return GDN_ERR_CUDA;
  count_launch(GDN_K_PAGE_COPY);
  return GDN_OK;
}

extern "C" gdn_status gdn_block_fork(const int32_t* src_rows, const int32_t* dst_rows, const int64_t* lens, int32_t n,
                                     int32_t block, int32_t* block_table, int32_t n_rows, int32_t max_blocks,
                                     int32_t* refs, int32_t num_blocks, const int32_t* free_ids, int32_t free_cap,
                                     const int32_t* n_free, int32_t* n_free_out, int32_t* copy_src, int32_t* copy_dst,
                                     uint32_t* dev_err, void* stream) {
  using namespace gdn;
  if (n < 0 || n_rows < 0 || max_blocks < 0 || num_blocks < 0 || free_cap < 0 || !pow2(block)) return GDN_ERR_INVALID_ARG;
  if (!n_free || !n_free_out || (free_cap > 0 && !free_ids)) return GDN_ERR_INVALID_ARG;
  if (n > 0 && (!src_rows || !dst_rows || !lens || !copy_src || !copy_dst)) return GDN_ERR_INVALID_ARG;
  if ((n_rows > 0 && max_blocks > 0 && !block_table) || (num_blocks > 0 && !refs)) return GDN_ERR_INVALID_ARG;
  ForkArgs a = {src_rows, dst_rows, lens,     n,        shift_of(block), block_table, n_rows,   max_blocks, refs,
                num_blocks, free_ids, free_cap, n_free, n_free_out,      copy_src,    copy_dst, dev_err};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (one_cluster(n, max_blocks)) {
    e = launch_pdl(fork_small_kernel, dim3(kCluster), dim3(kThreads), 0, s, dim3(kCluster), a);
  } else {
    e = launch_pdl(fork_alloc_kernel, dim3(1), dim3(kThreads), 0, s, dim3(1), a);
    if (e == cudaSuccess)
      e = launch_pdl(fork_rows_kernel, dim3((unsigned)std::min<int64_t>(n, 8LL * sm_count())), dim3(kRowThreads), 0, s,
                     dim3(1), a);
  }
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  count_launch(GDN_K_BLOCK_FORK);
  return GDN_OK;
}

extern "C" gdn_status gdn_block_release(const int32_t* rows, const int64_t* old_lens, const int64_t* new_lens, int32_t n,
                                        int32_t block, int32_t* block_table, int32_t n_rows, int32_t max_blocks,
                                        int32_t* refs, int32_t num_blocks, int32_t* free_ids, int32_t free_cap,
                                        const int32_t* n_free, int32_t* n_free_out, uint32_t* dev_err, void* stream) {
  using namespace gdn;
  if (n < 0 || n_rows < 0 || max_blocks < 0 || num_blocks < 0 || free_cap < 0 || !pow2(block)) return GDN_ERR_INVALID_ARG;
  if (!n_free || !n_free_out || (free_cap > 0 && !free_ids)) return GDN_ERR_INVALID_ARG;
  if (n > 0 && (!rows || !old_lens || !new_lens)) return GDN_ERR_INVALID_ARG;
  if ((n_rows > 0 && max_blocks > 0 && !block_table) || (num_blocks > 0 && !refs)) return GDN_ERR_INVALID_ARG;
  ReleaseArgs a = {rows, old_lens, new_lens, n, shift_of(block), block_table, n_rows, max_blocks, refs, num_blocks,
                   free_ids, free_cap, n_free, n_free_out, dev_err};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (one_cluster(n, max_blocks)) {
    e = launch_pdl(release_push_kernel<true>, dim3(kCluster), dim3(kThreads), 0, s, dim3(kCluster), a);
  } else {
    e = launch_pdl(release_rows_kernel, dim3((unsigned)std::min<int64_t>(n, 8LL * sm_count())), dim3(kRowThreads), 0, s,
                   dim3(1), a);
    if (e == cudaSuccess)
      e = launch_pdl(release_push_kernel<false>, dim3(kCluster), dim3(kThreads), 0, s, dim3(kCluster), a);
  }
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  count_launch(GDN_K_BLOCK_RELEASE);
  return GDN_OK;
}

extern "C" size_t gdn_block_compact_workspace_size(int32_t num_blocks) {
  if (num_blocks <= 0) return 256;
  const int64_t words = ((int64_t)num_blocks + 31) / 32;
  return (size_t)((gdn::up16(4LL * num_blocks) + gdn::up16(4 * words) + 16 + 255) & ~255LL);
}

extern "C" gdn_status gdn_block_compact(const int32_t* block_table, int32_t* table_out, int64_t n_entries,
                                        const int32_t* refs, int32_t* refs_out, int32_t num_blocks,
                                        const int32_t* free_ids, int32_t* free_out, int32_t free_cap,
                                        const int32_t* n_free, int32_t* move_src, int32_t* move_dst, int32_t max_moves,
                                        int32_t* n_moves, void* workspace, size_t workspace_bytes, uint32_t* dev_err,
                                        void* stream) {
  using namespace gdn;
  if (n_entries < 0 || num_blocks < 0 || free_cap < 0 || max_moves < 0) return GDN_ERR_INVALID_ARG;
  if (!n_free || !n_moves || (free_cap > 0 && (!free_ids || !free_out))) return GDN_ERR_INVALID_ARG;
  if (n_entries > 0 && (!block_table || !table_out)) return GDN_ERR_INVALID_ARG;
  if (num_blocks > 0 && (!refs || !refs_out)) return GDN_ERR_INVALID_ARG;
  if (max_moves > 0 && (!move_src || !move_dst)) return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < gdn_block_compact_workspace_size(num_blocks))
    return GDN_ERR_INVALID_ARG;
  CompactArgs a = {};
  a.table = block_table;
  a.table_out = table_out;
  a.n_entries = n_entries;
  a.refs = refs;
  a.refs_out = refs_out;
  a.num_blocks = num_blocks;
  a.free_ids = free_ids;
  a.free_out = free_out;
  a.free_cap = free_cap;
  a.n_free = n_free;
  a.move_src = move_src;
  a.move_dst = move_dst;
  a.max_moves = max_moves;
  a.n_moves = n_moves;
  a.words = (int32_t)(((int64_t)num_blocks + 31) / 32);
  char* ws = reinterpret_cast<char*>(workspace);
  a.remap = reinterpret_cast<int32_t*>(ws);
  a.bitmap = reinterpret_cast<uint32_t*>(ws + up16(4LL * num_blocks));
  a.wrong = reinterpret_cast<int32_t*>(ws + up16(4LL * num_blocks) + up16(4LL * a.words));
  a.err = dev_err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  const bool small = num_blocks <= kSmallBlocks, whole = n_entries <= kSmallEntries;
  const unsigned ctas = small ? 1 : kCluster;
  if (whole) {
    e = launch_pdl(small ? compact_small_kernel<true> : compact_kernel<true>, dim3(ctas), dim3(kThreads), 0, s,
                   dim3(ctas), a);
  } else {
    e = launch_pdl(small ? compact_small_kernel<false> : compact_kernel<false>, dim3(ctas), dim3(kThreads), 0, s,
                   dim3(ctas), a);
    if (e == cudaSuccess)
      e = launch_pdl(remap_kernel, dim3(4u * (unsigned)sm_count()), dim3(kRowThreads), 0, s, dim3(1), a);
  }
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  count_launch(GDN_K_BLOCK_COMPACT);
  return GDN_OK;
}
