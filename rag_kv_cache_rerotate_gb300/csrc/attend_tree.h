// How the attention of trees is cut, shared by its kernels.
//
// A unit is one sequence, KV head and group of its query vectors (new token,
// query head); its keys, held tokens and new ones, are cut into tiles.  The units'
// tiles in a row, unit by unit, are dealt to the workers (warps or CTAs) in
// runs of `per` tiles, so that all get the same number whatever the lengths
// are, which only the device knows.  A worker that takes a unit alone writes
// its outputs; otherwise each leaves the softmax of its keys unnormalised, with
// its maximum and sum, in one of its two slots (0: a unit begun by a worker
// before it, 1: one that goes on behind it), and the joining kernel adds up
//   O = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,   M = max_i m_i.
// So the workspace depends on the number of workers alone.
#pragma once

#include "cache_seqs.cuh"

namespace fusekv {

struct TreeArgs {
  SeqArgs seq;
  const int32_t* parents;
  const void* Q;
  const void* k_pool;
  const void* v_pool;
  void* O;
  int n_q_heads, n_kv_heads, g;           // g = n_q_heads / n_kv_heads
  int g_log2;
  int vecs;                               // query vectors of a unit
  int tile;                               // keys of a tile
  int workers;
  float scale;                            // log2(e) / sqrt(d)
  int64_t* start;                         // [n_seq + 1]: tiles in front of each sequence (for the join)
  float* part_o;                          // [worker][2][vecs][d]
  float2* part_ml;                        // [worker][2][vecs]: maximum (log2), sum
};

struct TreePlan {
  int vecs, tile, workers;
  size_t start, part_ml, part_o, total;   // workspace regions
};

__device__ __forceinline__ int units_of(const TreeArgs& a, const Seq& q) {
  return a.n_kv_heads * ((q.n * a.g + a.vecs - 1) / a.vecs);
}
__device__ __forceinline__ int tiles_of(const TreeArgs& a, const Seq& q) {
  return q.n == 0 ? 0 : (q.len + q.n + a.tile - 1) / a.tile;
}
__device__ __forceinline__ int64_t per_worker(const TreeArgs& a, int64_t tiles) {
  return max((int64_t)1, (tiles + a.workers - 1) / a.workers);
}

// Where a worker stands.
struct TreeAt {
  int s;                                  // sequence
  int64_t first;                          // its first tile
  Seq q;
};

// The tiles of all sequences, and each sequence's first one (written to a.start
// by block 0 of the grid, for the join): by a whole block.  s_warp: 33 words.
template <int kThreads>
__device__ __forceinline__ int64_t count_tiles(const TreeArgs& a, int64_t* s_warp) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  constexpr int kWarps = kThreads / 32;
  const bool keep = blockIdx.x == 0;
  int64_t total = 0;
  for (int s0 = 0; s0 < a.seq.n_seq; s0 += kThreads) {
    Seq q{0, 0, 0};
    if (s0 + tid < a.seq.n_seq) seq_of(a.seq, s0 + tid, &q);
    const int64_t own = (int64_t)units_of(a, q) * tiles_of(a, q);
    int64_t inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += z;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_warp[w];
      all += s_warp[w];
    }
    if (keep && s0 + tid < a.seq.n_seq) a.start[s0 + tid] = total + before + inc - own;
    total += all;
    __syncthreads();
  }
  if (keep && tid == 0) a.start[a.seq.n_seq] = total;
  return total;
}

// The sequence that tile t lies in (by a whole warp).
__device__ __forceinline__ TreeAt find_tile(const TreeArgs& a, int64_t t) {
  const int lane = threadIdx.x % 32;
  TreeAt r{a.seq.n_seq, 0, {0, 0, 0}};
  int64_t before = 0;
  for (int s0 = 0; s0 < a.seq.n_seq; s0 += 32) {
    Seq q{0, 0, 0};
    if (s0 + lane < a.seq.n_seq) seq_of(a.seq, s0 + lane, &q);
    const int64_t own = (int64_t)units_of(a, q) * tiles_of(a, q);
    int64_t inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += z;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + inc > t);
    if (past) {
      const int w = __ffs(past) - 1;
      r.s = s0 + w;
      r.first = before + __shfl_sync(0xffffffffu, inc - own, w);
      r.q.row0 = __shfl_sync(0xffffffffu, q.row0, w);
      r.q.n = __shfl_sync(0xffffffffu, q.n, w);
      r.q.len = __shfl_sync(0xffffffffu, q.len, w);
      return r;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return r;
}

// The new tokens that new token i sees: itself and its ancestors, a bit each.
__device__ __forceinline__ uint64_t seen_by(const int32_t* parents, const Seq& q, int i, uint32_t* err) {
  if (!parents) return ~(uint64_t)0 >> (63 - i);
  uint64_t seen = 0;
  for (int j = i; j >= 0; j = parent_of(parents, q, j, err)) seen |= (uint64_t)1 << j;
  return seen;
}

cudaError_t launch_tree_simt(const fuse_layer_desc_t& d, const TreeArgs& a, cudaStream_t s);

}  // namespace fusekv
