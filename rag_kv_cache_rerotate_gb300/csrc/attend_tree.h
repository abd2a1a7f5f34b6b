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
  int vecs, vecs_log2;                    // query vectors of a unit
  int tile, tile_log2;                    // keys of a tile
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
  return a.n_kv_heads * ((q.n * a.g + a.vecs - 1) >> a.vecs_log2);
}
__device__ __forceinline__ int tiles_of(const TreeArgs& a, const Seq& q) {
  return q.n == 0 ? 0 : (int)(((uint32_t)q.len + q.n + a.tile - 1) >> a.tile_log2);
}
__device__ __forceinline__ int64_t per_worker(const TreeArgs& a, int64_t tiles) {
  // (divisions of 64 bits take a few hundred cycles)
  if (tiles <= UINT32_MAX / 2) return max(1u, ((uint32_t)tiles + a.workers - 1) / (uint32_t)a.workers);
  return (tiles + a.workers - 1) / a.workers;
}

// Where a worker stands, and the end of its tiles.
struct TreeWalk {
  int s;                                  // sequence
  Seq q;
  int64_t first;                          // its first tile
  int64_t t, end;                         // the worker's next tile, and its last one's next
};

// 32 kEach sequences from s0 on, kEach a lane: their tiles, and the lane's first tile among them.
template <int kEach> struct TileScan {
  Seq q[kEach];
  int64_t own[kEach];
  int64_t before, all;
};
template <int kEach> __device__ __forceinline__ TileScan<kEach> scan_tiles(const TreeArgs& a, int s0) {
  const int lane = threadIdx.x % 32;
  TileScan<kEach> r;
  int64_t sum = 0;
  // (all reads before the first check, whose report would hold the next ones up)
  const int s1 = s0 + lane * kEach;
  int row[kEach + 1], len[kEach];
#pragma unroll
  for (int i = 0; i <= kEach; ++i) row[i] = a.seq.rows[min(s1 + i, a.seq.n_seq)];
#pragma unroll
  for (int i = 0; i < kEach; ++i) len[i] = a.seq.lens[min(s1 + i, a.seq.n_seq - 1)];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    r.q[i] = Seq{0, 0, 0};
    if (s1 + i < a.seq.n_seq) check_seq(a.seq, s1 + i, row[i], row[i + 1], len[i], &r.q[i]);
    r.own[i] = (int64_t)units_of(a, r.q[i]) * tiles_of(a, r.q[i]);
    sum += r.own[i];
  }
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t z = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += z;
  }
  r.before = inc - sum;
  r.all = __shfl_sync(0xffffffffu, inc, 31);
  return r;
}

// The walk of worker w, by its warp; `keep`: also writes each sequence's first tile,
// for the join.
template <int kEach> __device__ __forceinline__ TreeWalk start_walk_of(const TreeArgs& a, int64_t w, bool keep) {
  const int lane = threadIdx.x % 32;
  TreeWalk r{a.seq.n_seq, {0, 0, 0}, 0, 0, 0};
  TileScan<kEach> x;
  int64_t total = 0;
#pragma unroll 1
  for (int s0 = 0; s0 < a.seq.n_seq; s0 += 32 * kEach) {
    x = scan_tiles<kEach>(a, s0);
    if (keep) {
      int64_t at = total + x.before;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int s = s0 + lane * kEach + i;
        if (s < a.seq.n_seq) a.start[s] = at;
        at += x.own[i];
      }
    }
    total += x.all;
  }
  if (keep && lane == 0) a.start[a.seq.n_seq] = total;
  const int64_t per = per_worker(a, total);
  r.t = min(total, w * per);
  r.end = min(total, r.t + per);
  if (r.t == r.end) return r;
  int64_t before = 0;
#pragma unroll 1
  for (int s0 = 0; s0 < a.seq.n_seq; s0 += 32 * kEach) {
    if (a.seq.n_seq > 32 * kEach) x = scan_tiles<kEach>(a, s0);
    // the last lane whose first tile is not behind it, and the last such sequence of its
    // four (sequences without tiles before it share that tile)
    const unsigned in = __ballot_sync(0xffffffffu, before + x.before <= r.t);
    if (r.t < before + x.all) {
      const int k = 31 - __clz(in);
      int64_t first = before + x.before;
      int s = s0 + lane * kEach;
      Seq q = x.q[0];
#pragma unroll
      for (int i = 0; i + 1 < kEach; ++i)
        if (r.t >= first + x.own[i] && s == s0 + lane * kEach + i) {
          first += x.own[i];
          q = x.q[i + 1];
          ++s;
        }
      r.s = __shfl_sync(0xffffffffu, s, k);
      r.first = __shfl_sync(0xffffffffu, first, k);
      r.q.row0 = __shfl_sync(0xffffffffu, q.row0, k);
      r.q.n = __shfl_sync(0xffffffffu, q.n, k);
      r.q.len = __shfl_sync(0xffffffffu, q.len, k);
      break;
    }
    before += x.all;
  }
  return r;
}
// Up to 32 sequences take a lane each, up to 128 one look at four a lane: a walk's start is
// waited for (one token over 4096: 16.1 us, with four a lane 16.4; 16 trees 65.9 and 66.3).
__device__ __forceinline__ TreeWalk start_walk(const TreeArgs& a, int64_t w, bool keep) {
  return a.seq.n_seq <= 32 ? start_walk_of<1>(a, w, keep) : start_walk_of<4>(a, w, keep);
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

// A worker's share of a unit.
struct TreePart {
  int s;
  Seq q;
  int h, vg;                              // KV head, group of vectors
  int n_vec;                              // its vectors
  int j0, j1, nt;                         // tiles taken, of the unit's nt
};
__device__ __forceinline__ bool next_part(const TreeArgs& a, TreeWalk& w, TreePart& p) {
  while (w.t < w.end) {
    const int nt = tiles_of(a, w.q), units = units_of(a, w.q);
    const int64_t rel = w.t - w.first, all = (int64_t)units * nt;
    if (rel >= all) {                     // the next sequence
      w.first += all;
      if (++w.s >= a.seq.n_seq) return false;
      seq_of(a.seq, w.s, &w.q);
      continue;
    }
    const int groups = (w.q.n * a.g + a.vecs - 1) >> a.vecs_log2;
    const int unit = rel >> 32 ? (int)(rel / nt) : (int)((uint32_t)rel / (uint32_t)nt);
    p.s = w.s;
    p.q = w.q;
    p.h = groups == 1 ? unit : (int)((uint32_t)unit / (uint32_t)groups);
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
