// Upkeep of a paged cache: fork, free, compact and copy pages.
//
// A pool holds n_blocks pages of block_size tokens; sequences name pages in
// block tables, and refs[b] counts the table entries that name page b (0:
// free).  The bookkeeping (fork, free, compact) works on tables and counts
// alone and leaves a list of page moves; fuse_pages_copy applies the list to
// the pools of every layer, whose tables are the same.
//
// Fork and compact run as one cluster of 8 CTAs: every step is a count, a
// scan or a scatter over at most a few hundred KB, bound by latency, and the
// cluster barrier (with the counts exchanged through distributed shared
// memory) replaces the launches that separate grids would need between the
// steps.  Sums and scans take two counts at a time, and a thread keeps the counts
// of its first four pages.  36 branches of 12 sequences in a pool of 4 096 pages:
// 8 us; packing such a pool 10 us, its copies (133 MB) 43 us.
#include <cooperative_groups.h>

#include <algorithm>

#include "checks.h"
#include "common.cuh"
#include "launch.h"
#include "trace.h"

namespace fusekv {

namespace {

namespace cg = cooperative_groups;

constexpr int kCtas = 8;            // CTAs of the bookkeeping cluster (the portable limit)
constexpr int kThreads = 1024;
constexpr int kMoveHead = 2;        // moves[0] count, moves[1] live pages, then (src, dst) pairs

struct TableArgs {
  const fuse_chunk_t* src;
  const fuse_chunk_t* dst;          // fork only
  int32_t n_chunks;
  int32_t block_size;
  int32_t n_blocks;
  int32_t cap;                      // pairs that moves has room for
  int32_t* refs;
  int32_t* moves;
  int32_t* list;                    // scratch: fork: free pages; compact: holes
  int32_t* map;                     // scratch: compact: new id of each tail page
  uint32_t* err;
};

// Two counts in one word: sums and scans take both at once.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(int lo, int hi) { return (Pair)(uint32_t)hi << 32 | (uint32_t)lo; }
__device__ __forceinline__ int lo_of(Pair p) { return (int)(uint32_t)p; }
__device__ __forceinline__ int hi_of(Pair p) { return (int)(p >> 32); }

// Sum of x over the block, in every thread.
__device__ __forceinline__ Pair block_sum(Pair x, Pair* s_warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();                                  // s_warp may still be read
  if (threadIdx.x % 32 == 0) s_warp[threadIdx.x / 32] = x;
  __syncthreads();
  Pair t = s_warp[threadIdx.x % 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// Exclusive prefix sum of x over the block; *total receives the sum.
__device__ __forceinline__ Pair block_scan(Pair x, Pair* s_warp, Pair* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  Pair inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  Pair w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const Pair before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + inc - x;
}

// A CTA's counts and whether it met a bad entry; the other CTAs read them.
struct Counts {
  Pair n;
  int bad;
};

// Sum of the counts over the cluster's CTAs, and over the CTAs before this
// one; whether any met a bad entry.  Call between two cluster barriers.
__device__ __forceinline__ bool cluster_counts(cg::cluster_group& cl, Counts* s_cnt, int rank,
                                               Pair* before, Pair* total) {
  Pair b = 0, t = 0;
  int bad = 0;
#pragma unroll
  for (int r = 0; r < kCtas; ++r) {
    const Counts v = *cl.map_shared_rank(s_cnt, r);
    t += v.n;
    bad |= v.bad;
    if (r < rank) b += v.n;
  }
  *before = b;
  *total = t;
  return bad != 0;
}

__device__ __forceinline__ int n_entries(const fuse_chunk_t& c, int bs) {
  return (int)(((int64_t)c.len + bs - 1) / bs);
}

// The pages of this CTA: a range of ids, a multiple of four long.
__device__ __forceinline__ void slice(int n, int rank, int* lo, int* hi) {
  const int per = ((n + kCtas - 1) / kCtas + 3) / 4 * 4;
  *lo = min((int64_t)n, (int64_t)per * rank);
  *hi = min((int64_t)n, (int64_t)per * (rank + 1));
}

// Counts of four consecutive pages; pages past hi read as -1 (neither free nor live).
__device__ __forceinline__ void load_refs4(const int32_t* refs, int b, int hi, int (&r)[4]) {
  if (b + 3 < hi) {
    const int4 v = *reinterpret_cast<const int4*>(refs + b);
    r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = b + i < hi ? refs[b + i] : -1;
  }
}

// Whether any of the counts that load_refs4 read is negative (reported): such a
// page is neither free nor live, and a compaction would have more pages to move
// than places for them.
__device__ __forceinline__ int negative_count(uint32_t* err, int b, int hi, const int (&r)[4]) {
  int bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r[i] < 0 && b + i < hi) {
      bad = 1;
      report_error(err, FUSE_ERR_DEVICE_BOUNDS, SITE_PAGE_COUNT, (uint32_t)(b + i));
    }
  return bad;
}

// Fork: dst[i] shares the full pages of src[i] and gets a page of its own
// for the last, partly filled one: the lowest-numbered free pages, in table
// order.  Nothing changes unless every source entry names a live page, no count
// is negative, the free pages suffice and the move list has room.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1)
    pages_fork_kernel(const TableArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), tid = threadIdx.x;
  const int lane = tid % 32, warp = rank * (kThreads / 32) + tid / 32;
  constexpr int kWarps = kCtas * kThreads / 32;
  __shared__ Pair s_warp[32];
  __shared__ Counts s_cnt;                          // free pages, partly filled last pages
  pdl_trigger();
  pdl_wait();
  int lo, hi;
  slice(a.n_blocks, rank, &lo, &hi);
  int free_n = 0, bad = 0;
  for (int b = lo + 4 * tid; b < hi; b += 4 * kThreads) {
    int r[4];
    load_refs4(a.refs, b, hi, r);
    bad |= negative_count(a.err, b, hi, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) free_n += r[i] == 0;
  }
  const int c_per = (a.n_chunks + kCtas - 1) / kCtas;
  const int c_lo = min(a.n_chunks, c_per * rank), c_hi = min(a.n_chunks, c_per * (rank + 1));
  int need_n = 0;
  for (int c = c_lo + tid; c < c_hi; c += kThreads) need_n += a.src[c].len % a.block_size != 0;
  for (int c = warp; c < a.n_chunks; c += kWarps) {
    const fuse_chunk_t s = a.src[c];
    const int n = n_entries(s, a.block_size);
#pragma unroll 4
    for (int j = lane; j < n; j += 32) {
      const int b = s.block_table[j];
      if (b < 0 || b >= a.n_blocks || a.refs[b] <= 0) {
        bad = 1;
        report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_PAGE_ENTRY, (uint32_t)c);
      }
    }
  }
  const Pair mine = block_sum(pair(free_n, need_n), s_warp);
  bad = __syncthreads_or(bad);
  if (tid == 0) s_cnt = {mine, bad};
  cl.sync();
  Pair before, all;
  const bool any_bad = cluster_counts(cl, &s_cnt, rank, &before, &all);
  const int f_total = lo_of(all), need = hi_of(all);
  const bool ok = !any_bad && need <= f_total && need <= a.cap;
  if (rank == 0 && tid == 0) {
    if (!any_bad && need > f_total)
      report_error(a.err, FUSE_ERR_NO_PAGES, SITE_PAGE_FREE, (uint32_t)(need - f_total));
    else if (!any_bad && need > a.cap)
      report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_PAGE_MOVES, (uint32_t)need);
    a.moves[0] = ok ? need : 0;
    a.moves[1] = a.n_blocks - f_total + (ok ? need : 0);
  }
  // the first `need` free pages, ascending
  int at = lo_of(before);
  for (int b0 = lo; ok && b0 < hi && at < need; b0 += 4 * kThreads) {
    int r[4], cnt = 0;
    Pair total;
    load_refs4(a.refs, b0 + 4 * tid, hi, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) cnt += r[i] == 0;
    int p = at + lo_of(block_scan(cnt, s_warp, &total));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r[i] == 0) {
        if (p < need) a.list[p] = b0 + 4 * tid + i;
        ++p;
      }
    at += lo_of(total);
  }
  cl.sync();                                        // every count read, the list written
  if (!ok) return;
  int rank0 = hi_of(before);
  for (int c0 = c_lo; c0 < c_hi; c0 += kThreads) {
    const int c = c0 + tid;
    const bool mine = c < c_hi && a.src[c].len % a.block_size != 0;
    Pair total;
    const int p = rank0 + lo_of(block_scan(mine ? 1 : 0, s_warp, &total));
    if (mine) {
      const int j = a.src[c].len / a.block_size;
      const int b = a.list[p];
      a.moves[kMoveHead + 2 * p] = a.src[c].block_table[j];
      a.moves[kMoveHead + 2 * p + 1] = b;
      const_cast<int32_t*>(a.dst[c].block_table)[j] = b;
      a.refs[b] = 1;
    }
    rank0 += lo_of(total);
  }
  for (int c = warp; c < a.n_chunks; c += kWarps) {
    const fuse_chunk_t s = a.src[c];
    int32_t* d = const_cast<int32_t*>(a.dst[c].block_table);
    const int n = s.len / a.block_size;
#pragma unroll 4
    for (int j = lane; j < n; j += 32) {
      const int b = s.block_table[j];
      d[j] = b;
      atomicAdd(a.refs + b, 1);
    }
  }
}

// Compact: the live pages at ids >= n_live move into the free ids below it
// (both ascending), so sources and destinations are disjoint, as few pages
// move as can, and every table entry is rewritten.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1)
    pages_compact_kernel(const TableArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), tid = threadIdx.x;
  const int lane = tid % 32, warp = rank * (kThreads / 32) + tid / 32;
  constexpr int kWarps = kCtas * kThreads / 32;
  __shared__ Pair s_warp[32];
  __shared__ Counts s_live, s_cnt;                  // live pages; holes and tail pages
  pdl_trigger();
  pdl_wait();
  int lo, hi;
  slice(a.n_blocks, rank, &lo, &hi);
  int first[4];                                     // the counts of this thread's first four pages
  load_refs4(a.refs, lo + 4 * tid, hi, first);
  auto refs4 = [&](int b, int (&r)[4]) {
    if (b < lo + 4 * kThreads) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = first[i];
    } else {
      load_refs4(a.refs, b, hi, r);
    }
  };
  int live = 0, bad = 0;
  for (int c = warp; c < a.n_chunks; c += kWarps) {
    const fuse_chunk_t s = a.src[c];
    const int n = n_entries(s, a.block_size);
#pragma unroll 4
    for (int j = lane; j < n; j += 32) {
      const int b = s.block_table[j];
      if (b < 0 || b >= a.n_blocks || a.refs[b] <= 0) {
        bad = 1;
        report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_PAGE_ENTRY, (uint32_t)c);
      }
    }
  }
  for (int b = lo + 4 * tid; b < hi; b += 4 * kThreads) {
    int r[4];
    refs4(b, r);
    bad |= negative_count(a.err, b, hi, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) live += r[i] > 0;
  }
  const Pair here = block_sum(live, s_warp);
  bad = __syncthreads_or(bad);
  if (tid == 0) s_live = {here, bad};
  cl.sync();
  Pair before, all;
  const bool any_bad = cluster_counts(cl, &s_live, rank, &before, &all);
  const int n_live = lo_of(all);
  int holes = 0, tails = 0;
  for (int b = lo + 4 * tid; b < hi; b += 4 * kThreads) {
    int r[4];
    refs4(b, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      holes += r[i] == 0 && b + i < n_live;
      tails += r[i] > 0 && b + i >= n_live;
    }
  }
  const Pair both = block_sum(pair(holes, tails), s_warp);
  if (tid == 0) s_cnt = {both, 0};
  cl.sync();
  Pair at;
  cluster_counts(cl, &s_cnt, rank, &at, &all);
  const int n_moves = lo_of(all);
  const bool ok = !any_bad && n_moves <= a.cap;
  if (rank == 0 && tid == 0) {
    if (!any_bad && !ok)
      report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_PAGE_MOVES, (uint32_t)n_moves);
    a.moves[0] = ok ? n_moves : 0;
    a.moves[1] = n_live;
  }
  for (int b0 = lo; ok && b0 < hi; b0 += 4 * kThreads) {
    int r[4], hc = 0, tc = 0;
    Pair total;
    const int b = b0 + 4 * tid;
    refs4(b, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hc += r[i] == 0 && b + i < n_live;
      tc += r[i] > 0 && b + i >= n_live;
    }
    const Pair p = at + block_scan(pair(hc, tc), s_warp, &total);
    int hp = lo_of(p), tp = hi_of(p);
    at += total;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (r[i] == 0 && b + i < n_live) a.list[hp++] = b + i;
      if (r[i] > 0 && b + i >= n_live) {
        a.map[b + i] = tp;                          // rank of the tail page
        a.moves[kMoveHead + 2 * tp] = b + i;
        ++tp;
      }
    }
  }
  cl.sync();
  if (!ok) return;
  // the tables by the cluster's last warps, the moves by its first ones.  Two
  // tables may be the same buffer: an entry rewritten already is below n_live
  for (int c = kWarps - 1 - warp; c < a.n_chunks; c += kWarps) {
    const fuse_chunk_t s = a.src[c];
    int32_t* t = const_cast<int32_t*>(s.block_table);
    const int n = n_entries(s, a.block_size);
#pragma unroll 4
    for (int j = lane; j < n; j += 32) {
      const int b = t[j];
      if (b >= n_live) t[j] = a.list[a.map[b]];
    }
  }
  for (int m = rank * kThreads + tid; m < n_moves; m += kCtas * kThreads) {
    const int from = a.moves[kMoveHead + 2 * m], to = a.list[m];
    a.moves[kMoveHead + 2 * m + 1] = to;
    a.refs[to] = a.refs[from];
    a.refs[from] = 0;
  }
}

// Free: every entry of the tables gives up one reference.  An entry past the
// references there are is reported and leaves the count as it was.
__global__ void __launch_bounds__(256) pages_free_kernel(const TableArgs a) {
  pdl_trigger();
  pdl_wait();
  for (int c = blockIdx.x; c < a.n_chunks; c += gridDim.x) {
    const fuse_chunk_t s = a.src[c];
    const int n = n_entries(s, a.block_size);
    for (int j = threadIdx.x; j < n; j += 256) {
      const int b = s.block_table[j];
      if (b < 0 || b >= a.n_blocks) {
        report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_PAGE_ENTRY, (uint32_t)c);
      } else if (atomicSub(a.refs + b, 1) <= 0) {
        atomicAdd(a.refs + b, 1);
        report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_PAGE_ENTRY, (uint32_t)c);
      }
    }
  }
}

// Pools of one launch (parameter space): up to 8 in a short list, which costs
// the host 0.5 us less than one of 64 (4.5 against 5.1 us for one layer).
constexpr int kMaxPools = 64, kFewPools = 8;

template <int N> struct CopyArgs {
  fuse_pool_t pool[N];
  int32_t n_pools;
  int32_t cap;
  int32_t n_blocks;
  int32_t scale_bytes;              // bytes of a page's v_scale (and v_zero); 0: none
  int64_t page_bytes;               // bytes of a page's K (and V), a multiple of 16
  const int32_t* moves;
  uint32_t* err;
};

constexpr int kCopyThreads = 256;
constexpr int kVecs = 4;                            // 16-byte loads of a thread in flight
constexpr int kPiece = kCopyThreads * kVecs * 16;   // 16 KB

// Copy pages: every (pool, move, K or V) page in pieces of 16 KB, one piece a
// CTA at a time, four 16-byte loads of a thread in flight before the first
// store.  Bound by HBM: every byte is read once and written once (64 pages of
// 64 KB in 16 layers: 20.8 us, 6.4 TB/s; a plain copy reaches 6.8).
template <int N>
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ CopyArgs<N> a) {
  pdl_trigger();
  pdl_wait();
  const int n = a.moves[0];
  if (n < 0 || n > a.cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0)
      report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_PAGE_MOVES, (uint32_t)n);
    return;
  }
  const int pieces = (int)((a.page_bytes + kPiece - 1) / kPiece);
  const int64_t total = (int64_t)n * a.n_pools * 2 * pieces;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int piece = (int)(w % pieces);
    const int64_t q = w / pieces;
    const bool value = q & 1;
    const int64_t mp = q >> 1;
    const int m = (int)(mp % n), p = (int)(mp / n);
    const int src = a.moves[kMoveHead + 2 * m], dst = a.moves[kMoveHead + 2 * m + 1];
    if (src < 0 || src >= a.n_blocks || dst < 0 || dst >= a.n_blocks) {
      if (threadIdx.x == 0)
        report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_PAGE_MOVES, (uint32_t)m);
      continue;
    }
    const fuse_pool_t& P = a.pool[p];
    char* base = reinterpret_cast<char*>(value ? P.v : P.k);
    const int64_t off = (int64_t)piece * kPiece;
    const int64_t left = a.page_bytes - off;
    const uint4* s = reinterpret_cast<const uint4*>(base + src * a.page_bytes + off);
    uint4* d = reinterpret_cast<uint4*>(base + dst * a.page_bytes + off);
    uint4 x[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = i * kCopyThreads + threadIdx.x;
      if ((int64_t)e * 16 < left) x[i] = s[e];
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = i * kCopyThreads + threadIdx.x;
      if ((int64_t)e * 16 < left) d[e] = x[i];
    }
    if (a.scale_bytes > 0 && piece == 0) {          // with K the scales, with V the zeros
      char* sb = reinterpret_cast<char*>(value ? P.v_zero : P.v_scale);
      const uint16_t* ss = reinterpret_cast<const uint16_t*>(sb + (int64_t)src * a.scale_bytes);
      uint16_t* sd = reinterpret_cast<uint16_t*>(sb + (int64_t)dst * a.scale_bytes);
      for (int e = threadIdx.x; e < a.scale_bytes / 2; e += kCopyThreads) sd[e] = ss[e];
    }
  }
}

// ---- host side ---------------------------------------------------------------

fuse_status_t check_tables(const fuse_chunks_t* c, bool entries_on_device = true) {
  if (!c || c->n_chunks < 0) return FUSE_ERR_INVALID_ARG;
  if (c->kv_layout != FUSE_KV_PAGED) return FUSE_ERR_UNSUPPORTED;
  if (c->block_size <= 0 || c->n_pool_blocks <= 0) return FUSE_ERR_INVALID_ARG;
  if (c->n_pool_blocks > INT32_MAX / 4) return FUSE_ERR_UNSUPPORTED;
  if (c->n_chunks == 0) return FUSE_OK;
  if (!c->h_chunks || (entries_on_device && !c->d_chunks)) return FUSE_ERR_INVALID_ARG;
  for (int i = 0; i < c->n_chunks; ++i) {
    if (c->h_chunks[i].len < 0) return FUSE_ERR_INVALID_ARG;
    if (entries_on_device && c->h_chunks[i].len > 0 && !c->h_chunks[i].block_table)
      return FUSE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(c->h_chunks[i].block_table) & 3u) return FUSE_ERR_MISALIGNED;
  }
  return FUSE_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct PagesWs {
  size_t list, map, total;
};

// list: a fork's new pages (one per table at most) or a compaction's holes
// (at most half the pages); map: an entry per page.
PagesWs pages_ws(const fuse_chunks_t* c) {
  PagesWs L;
  L.list = sizeof(WsHeader);
  L.map = L.total = L.list;
  if (!c) return L;
  const size_t n = std::max<size_t>((size_t)c->n_chunks, (size_t)c->n_pool_blocks / 2 + 1);
  L.map = align_up(L.list + n * sizeof(int32_t), 256);
  L.total = align_up(L.map + (size_t)c->n_pool_blocks * sizeof(int32_t), 256);
  return L;
}

template <typename T> T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(ws) + off);
}

fuse_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? FUSE_OK : FUSE_ERR_CUDA; }

TableArgs table_args(const fuse_chunks_t& c, int32_t* refs, int32_t* moves, int32_t max_moves,
                     void* ws) {
  const PagesWs L = pages_ws(&c);
  TableArgs a;
  a.src = c.d_chunks;
  a.dst = nullptr;
  a.n_chunks = c.n_chunks;
  a.block_size = c.block_size;
  a.n_blocks = (int32_t)c.n_pool_blocks;
  a.cap = max_moves;
  a.refs = refs;
  a.moves = moves;
  a.list = at<int32_t>(ws, L.list);
  a.map = at<int32_t>(ws, L.map);
  a.err = at<uint32_t>(ws, 0);
  return a;
}

}  // namespace
}  // namespace fusekv

using namespace fusekv;

extern "C" {

fuse_status_t fuse_pages_workspace_size(const fuse_chunks_t* tables, size_t* bytes) {
  if (!bytes) return FUSE_ERR_INVALID_ARG;
  if (tables) {
    const fuse_status_t st = check_tables(tables, false);
    if (st != FUSE_OK) return st;
  }
  *bytes = pages_ws(tables).total;
  return FUSE_OK;
}

fuse_status_t fuse_pages_fork(const fuse_chunks_t* src, const fuse_chunks_t* dst, int32_t* refs,
                              int32_t* moves, int32_t max_moves, void* ws, size_t ws_bytes,
                              fuse_stream_t stream) {
  fuse_status_t st = check_tables(src);
  if (st == FUSE_OK) st = check_tables(dst);
  if (st != FUSE_OK) return st;
  if (src->n_chunks != dst->n_chunks || src->block_size != dst->block_size ||
      src->n_pool_blocks != dst->n_pool_blocks)
    return FUSE_ERR_INVALID_ARG;
  if (!refs || !moves || max_moves < 0) return FUSE_ERR_INVALID_ARG;
  if (!aligned16(refs) || !aligned4(moves)) return FUSE_ERR_MISALIGNED;
  int64_t need = 0;
  for (int i = 0; i < src->n_chunks; ++i) {
    const fuse_chunk_t &s = src->h_chunks[i], &d = dst->h_chunks[i];
    if (s.len != d.len || (s.len > 0 && s.block_table == d.block_table)) return FUSE_ERR_INVALID_ARG;
    need += s.len % src->block_size != 0;
  }
  if (need > max_moves) return FUSE_ERR_WORKSPACE;
  st = check_ws(ws, ws_bytes, pages_ws(src).total);
  if (st != FUSE_OK) return st;
  TableArgs a = table_args(*src, refs, moves, max_moves, ws);
  a.dst = dst->d_chunks;
  cudaStream_t s = (cudaStream_t)stream;
  return cuda_status(traced("pages_fork", s, [&] {
    return launch_pdl(pages_fork_kernel, dim3(kCtas), dim3(kThreads), 0, s, a);
  }));
}

fuse_status_t fuse_pages_free(const fuse_chunks_t* tables, int32_t* refs, void* ws, size_t ws_bytes,
                              fuse_stream_t stream) {
  fuse_status_t st = check_tables(tables);
  if (st != FUSE_OK) return st;
  if (!refs) return FUSE_ERR_INVALID_ARG;
  if (!aligned16(refs)) return FUSE_ERR_MISALIGNED;
  st = check_ws(ws, ws_bytes, sizeof(WsHeader));
  if (st != FUSE_OK) return st;
  if (tables->n_chunks == 0) return FUSE_OK;
  const TableArgs a = table_args(*tables, refs, nullptr, 0, ws);
  cudaStream_t s = (cudaStream_t)stream;
  return cuda_status(traced("pages_free", s, [&] {
    return launch_pdl(pages_free_kernel, dim3(std::min(a.n_chunks, 4096)), dim3(256), 0, s, a);
  }));
}

fuse_status_t fuse_pages_compact(const fuse_chunks_t* tables, int32_t* refs, int32_t* moves,
                                 int32_t max_moves, void* ws, size_t ws_bytes,
                                 fuse_stream_t stream) {
  fuse_status_t st = check_tables(tables);
  if (st != FUSE_OK) return st;
  if (!refs || !moves || max_moves < 0) return FUSE_ERR_INVALID_ARG;
  if (!aligned16(refs) || !aligned4(moves)) return FUSE_ERR_MISALIGNED;
  if (max_moves < tables->n_pool_blocks / 2) return FUSE_ERR_WORKSPACE;
  st = check_ws(ws, ws_bytes, pages_ws(tables).total);
  if (st != FUSE_OK) return st;
  const TableArgs a = table_args(*tables, refs, moves, max_moves, ws);
  cudaStream_t s = (cudaStream_t)stream;
  return cuda_status(traced("pages_compact", s, [&] {
    return launch_pdl(pages_compact_kernel, dim3(kCtas), dim3(kThreads), 0, s, a);
  }));
}

fuse_status_t fuse_pages_copy(const fuse_layer_desc_t* desc, const fuse_pools_t* pools,
                              const int32_t* moves, int32_t max_moves, void* ws, size_t ws_bytes,
                              fuse_stream_t stream) {
  fuse_status_t st = check_desc(desc);
  if (st != FUSE_OK) return st;
  if (!pools || pools->n_pools < 0 || pools->reserved != 0 || !moves || max_moves < 0)
    return FUSE_ERR_INVALID_ARG;
  if (!aligned4(moves)) return FUSE_ERR_MISALIGNED;
  const int kind = pools->kv_storage;
  if (kind != FUSE_F32 && kind != FUSE_BF16 && kind != FUSE_U8_ASYM && kind != FUSE_U4_ASYM)
    return FUSE_ERR_INVALID_ARG;
  if (pools->block_size <= 0 || pools->n_blocks <= 0) return FUSE_ERR_INVALID_ARG;
  if (pools->n_blocks > INT32_MAX / 4) return FUSE_ERR_UNSUPPORTED;
  if (pools->n_pools > 0 && !pools->h_pools) return FUSE_ERR_INVALID_ARG;
  const bool quant = kind == FUSE_U8_ASYM || kind == FUSE_U4_ASYM;
  for (int i = 0; i < pools->n_pools; ++i) {
    const fuse_pool_t& p = pools->h_pools[i];
    if (!p.k || !p.v) return FUSE_ERR_INVALID_ARG;
    if (!aligned16(p.k) || !aligned16(p.v)) return FUSE_ERR_MISALIGNED;
    if (quant && (!p.v_scale || !p.v_zero)) return FUSE_ERR_INVALID_ARG;
    if (quant &&
        ((reinterpret_cast<uintptr_t>(p.v_scale) | reinterpret_cast<uintptr_t>(p.v_zero)) & 1u))
      return FUSE_ERR_MISALIGNED;
  }
  st = check_ws(ws, ws_bytes, sizeof(WsHeader));
  if (st != FUSE_OK) return st;
  const int64_t rows = (int64_t)pools->block_size * desc->n_kv_heads;
  const int64_t bits = kind == FUSE_F32 ? 32 : kind == FUSE_BF16 ? 16 : kind == FUSE_U8_ASYM ? 8 : 4;
  const int64_t page = rows * desc->head_dim * bits / 8;
  if (rows * 2 > INT32_MAX || page > INT32_MAX) return FUSE_ERR_UNSUPPORTED;
  if (max_moves == 0) return FUSE_OK;
  cudaStream_t s = (cudaStream_t)stream;
  int dev = 0, sms = 1;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t pieces = (page + kPiece - 1) / kPiece;
  auto go = [&](auto a, int p0, int n) {
    a.n_pools = n;
    std::copy(pools->h_pools + p0, pools->h_pools + p0 + n, a.pool);
    a.cap = max_moves;
    a.n_blocks = (int32_t)pools->n_blocks;
    a.page_bytes = page;
    a.scale_bytes = quant ? (int32_t)(rows * 2) : 0;
    a.moves = moves;
    a.err = at<uint32_t>(ws, 0);
    const int grid = (int)std::min<int64_t>((int64_t)max_moves * n * 2 * pieces, (int64_t)sms * 8);
    return cuda_status(traced("pages_copy", s, [&] {
      constexpr int N = sizeof(a.pool) / sizeof(a.pool[0]);
      return launch_pdl(pages_copy_kernel<N>, dim3(grid), dim3(kCopyThreads), 0, s, a);
    }));
  };
  for (int p0 = 0; p0 < pools->n_pools; p0 += kMaxPools) {
    const int n = std::min(kMaxPools, pools->n_pools - p0);
    st = n <= kFewPools ? go(CopyArgs<kFewPools>(), p0, n) : go(CopyArgs<kMaxPools>(), p0, n);
    if (st != FUSE_OK) return st;
  }
  return FUSE_OK;
}

}  // extern "C"
