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

// What new tokens see of the new ones, themselves and their ancestors, a bit each:
// a warp's lanes hold the masks of nodes `lane` and `lane + 32`.  Pointer jumping:
// after k rounds a mask holds a node's 2^k nearest.
struct Seen {
  unsigned long long m0, m1;
};
__device__ __forceinline__ Seen seen_of_all(const int32_t* parents, const Seq& q, uint32_t* err) {
  const int lane = threadIdx.x % 32;
  Seen s;
  if (!parents) {
    s.m0 = ~0ull >> (63 - lane);
    s.m1 = ~0ull >> (31 - lane);
    return s;
  }
  s.m0 = 1ull << lane;
  s.m1 = s.m0 << 32;
  // the next ones up
  int u0 = lane < q.n ? parent_of(parents, q, lane, err) : -1;
  int u1 = lane + 32 < q.n ? parent_of(parents, q, lane + 32, err) : -1;
  while (__any_sync(0xffffffffu, u0 >= 0 || u1 >= 0)) {
    const unsigned long long a0 = __shfl_sync(0xffffffffu, s.m0, u0 & 31), a1 = __shfl_sync(0xffffffffu, s.m1, u0 & 31);
    const unsigned long long b0 = __shfl_sync(0xffffffffu, s.m0, u1 & 31), b1 = __shfl_sync(0xffffffffu, s.m1, u1 & 31);
    const int c0 = __shfl_sync(0xffffffffu, u0, u0 & 31), c1 = __shfl_sync(0xffffffffu, u1, u0 & 31);
    const int d0 = __shfl_sync(0xffffffffu, u0, u1 & 31), d1 = __shfl_sync(0xffffffffu, u1, u1 & 31);
    if (u0 >= 0) {
      s.m0 |= u0 < 32 ? a0 : a1;
      u0 = u0 < 32 ? c0 : c1;
    }
    if (u1 >= 0) {
      s.m1 |= u1 < 32 ? b0 : b1;
      u1 = u1 < 32 ? d0 : d1;
    }
  }
  return s;
}
// The mask of the node that a lane asks for (by a whole warp).
__device__ __forceinline__ uint64_t seen_by(const Seen& s, int node) {
  const unsigned long long lo = __shfl_sync(0xffffffffu, s.m0, node & 31), hi = __shfl_sync(0xffffffffu, s.m1, node & 31);
  return node < 32 ? lo : hi;
}

// A worker's way through its tiles, unit by unit.
struct TreeWalk {
  TreeAt at;
  int64_t t, end;
};
struct TreePart {
  int s;
  Seq q;
  int h, vg;                              // KV head, group of vectors
  int n_vec;                              // its vectors
  int j0, j1, nt;                         // tiles taken, of the unit's nt
};
__device__ __forceinline__ bool next_part(const TreeArgs& a, TreeWalk& w, TreePart& p) {
  while (w.t < w.end) {
    const int nt = tiles_of(a, w.at.q), units = units_of(a, w.at.q);
    const int64_t rel = w.t - w.at.first, all = (int64_t)units * nt;
    if (rel >= all) {                     // the next sequence
      w.at.first += all;
      if (++w.at.s >= a.seq.n_seq) return false;
      seq_of(a.seq, w.at.s, &w.at.q);
      continue;
    }
    const int groups = units / a.n_kv_heads;
    const int unit = rel >> 32 ? (int)(rel / nt) : (int)((uint32_t)rel / (uint32_t)nt);
    p.s = w.at.s;
    p.q = w.at.q;
    p.h = unit / groups;
    p.vg = unit - p.h * groups;
    p.n_vec = min(a.vecs, p.q.n * a.g - p.vg * a.vecs);
    p.nt = nt;
    p.j0 = (int)(rel - (int64_t)unit * nt);
    p.j1 = (int)min((int64_t)nt, p.j0 + (w.end - w.t));
    w.t += p.j1 - p.j0;
    return true;
  }
  return false;
}

cudaError_t launch_tree_simt(const fuse_layer_desc_t& d, const TreeArgs& a, cudaStream_t s);
// bf16 layers, on the tensor cores (attend_tree_tc.cu).
constexpr int kTreeTcVecs = 256, kTreeTcTile = 128;
cudaError_t launch_tree_tc(const fuse_layer_desc_t& d, const TreeArgs& a, cudaStream_t s);

}  // namespace fusekv
