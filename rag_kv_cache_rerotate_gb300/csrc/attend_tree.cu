// Attention of trees of new tokens over a paged cache: the entry points, the
// CUDA-core kernel (fp32 layers) and the kernel that joins the workers' parts.
//
// Every new token sees all held tokens and, of the new ones, itself and its
// ancestors, 64 bits of a row's own.  Held and new tokens lie in the same
// pages, so a unit's keys are one list with the mask at its end.
#include <algorithm>
#include <cmath>

#include "attend_tree.h"
#include "checks.h"
#include "launch.h"
#include "trace.h"

namespace fusekv {

namespace {

constexpr int kWarps = 2;                 // workers of a CTA
constexpr int kVecs = 8;                  // query vectors of a unit
constexpr uint32_t kAll = (1u << kVecs) - 1;
constexpr float kRaise = 16.f;            // a reference is raised by scores 2^16 times as heavy
constexpr int kTile = 32;                 // keys of a tile: one a lane
static_assert(kVecs == 1 << 3 && kTile == 1 << 5 && kTreeTcVecs == 1 << 8 && kTreeTcTile == 1 << 7, "logarithms");

// A warp's units, 32 keys at a time: a lane per key for the scores, then a lane
// per D / 32 channels for the sums.  Keys and values are copied to shared memory a
// tile ahead of their use: while a warp sums one tile's values the next one's keys
// are on their way, and its values during the scores.  A vector's reference is not
// its maximum: scores up to 2^kRaise times as heavy do not raise it, so most tiles go
// without the maximum over the lanes (P and its sum have 24 bits at any size).
//
// A few short sequences (5 of up to 300 keys and 12 new tokens, 4 heads of 64) take
// 10 us of dependent reads, sums and code that is fetched for the first time, with
// the join 13; lanes that read keys and values themselves, a few at a time, took 19
// (22).  Many keys (16 sequences of 1000 to 4000 keys and 4 to 12 new tokens, 32 heads
// of 128 on 8) take 277 to 285 us; that took 462.  Latency bounds them: a warp's 37 KB leave
// 1.3 warps a scheduler, which issue in 37 % of the cycles (HBM is at 42 %), and units of
// eight vectors copy the same keys once each.
template <int D> struct SimtShared {        // of a warp
  float4 k[kTile][D / 4];                   // 16-byte pieces swapped by key: lanes read a column of them
  float4 v[kTile][D / 4];
  float q[kVecs][D];
  float p[kTile][kVecs];
};

// 16 bytes, or as many zeros
__device__ __forceinline__ void copy16(void* to, const void* from, bool zeros) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
               "r"(zeros ? 0 : 16)
               : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all groups but the last one
__device__ __forceinline__ void copies_wait1() {
  asm volatile("cp.async.wait_group 1;" ::: "memory");
  __syncwarp();
}

// d + a b, two at a time (half the instructions)
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 d) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(d)));
  return reinterpret_cast<const float2&>(r);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) tree_simt_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int EL = D / 32, kPieces = D / 4, kRowsOnce = 32 / kPieces;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  SimtShared<D>& S = reinterpret_cast<SimtShared<D>*>(smem)[warp];
  pdl_wait();
  pdl_trigger();
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  TreeWalk walk = start_walk(a, w, w == 0);
  TreePart at;
  while (next_part(a, walk, at)) {
    const int h = at.h, vg = at.vg, n_vec = at.n_vec, n_keys = at.q.len + at.q.n;
    auto row_of = [&](int j) {              // of a lane's key
      const int key = j * kTile + lane;
      return j < at.j1 && key < n_keys ? (int)pool_row(a.seq, at.s, key) : -1;
    };
    // Rows of a tile (a key without one gets zeros), or of none: copies have no order among
    // themselves, so that none may be on its way to a place when the next one to it starts.
    auto copy = [&](const void* pool, int row, bool swap, float4 (*to)[kPieces], bool tile) {
      const int r0 = lane / kPieces, c = lane % kPieces;
      const float4* from = reinterpret_cast<const float4*>(pool) + h * kPieces + c;
#pragma unroll 8
      for (int i = 0; tile && i < kTile; i += kRowsOnce) {
        const int r = i + r0, ri = __shfl_sync(0xffffffffu, row, r);
        copy16(&to[r][swap ? c ^ (r & 7) : c], from + (int64_t)max(ri, 0) * (a.n_kv_heads * kPieces), ri < 0);
      }
      copies_end();
    };
    // Few keys make few tiles, and then latency is all there is: reads come first,
    // the checks and sums that wait for them after.
    int row = row_of(at.j0);
    float x[kVecs][EL];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int vi = vg * kVecs + min(v, n_vec - 1), i = vi >> a.g_log2;
      const float* q = reinterpret_cast<const float*>(a.Q) +
                       ((int64_t)(at.q.row0 + i) * a.n_q_heads + h * a.g + (vi & (a.g - 1))) * D;
#pragma unroll
      for (int e = 0; e < EL; ++e) x[v][e] = q[e * 32 + lane];
    }
    copy(a.k_pool, row, true, S.k, true);
    copy(a.v_pool, row, false, S.v, true);
    uint64_t seen[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) seen[v] = 0;
    if (at.j1 * kTile > at.q.len) {         // (uniform) some are new tokens
      const Seen all = seen_of_all(a.parents, at.q, a.seq.err);
#pragma unroll
      for (int v = 0; v < kVecs; ++v) seen[v] = seen_by(all, (vg * kVecs + min(v, n_vec - 1)) >> a.g_log2);
    }
    float m[kVecs], l[kVecs];
    float2 acc[kVecs / 2][EL];              // of two vectors
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      m[v] = -INFINITY;
      l[v] = 0.f;
#pragma unroll
      for (int e = 0; e < EL; ++e) {
        S.q[v][e * 32 + lane] = x[v][e] * a.scale;
        acc[v / 2][e] = make_float2(0.f, 0.f);
      }
    }
    for (int j = at.j0; j < at.j1; ++j) {
      const int rel = j * kTile + lane - at.q.len;  // of a new token
      const int next = row_of(j + 1);
      copies_wait1();                       // this tile's keys
      float2 s2[kVecs];                     // over even and odd channels
#pragma unroll
      for (int v = 0; v < kVecs; ++v) s2[v] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int c = 0; c < kPieces; ++c) {
        const float4 kx = S.k[lane][c ^ (lane & 7)];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
          const float4 qx = *reinterpret_cast<const float4*>(&S.q[v][c * 4]);
          s2[v] = fma2(make_float2(qx.x, qx.y), make_float2(kx.x, kx.y), s2[v]);
          s2[v] = fma2(make_float2(qx.z, qx.w), make_float2(kx.z, kx.w), s2[v]);
        }
      }
      __syncwarp();
      copy(a.k_pool, next, true, S.k, j + 1 < at.j1);
      uint32_t any = 0;                     // bit v: that vector sees this key
      float s[kVecs];
      bool more = false;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const bool ok = row >= 0 && (rel < 0 || (seen[v] >> rel & 1));
        any |= (uint32_t)ok << v;
        s[v] = ok ? s2[v].x + s2[v].y : -INFINITY;
        more |= s[v] > m[v] + kRaise;
      }
      if (__any_sync(0xffffffffu, more)) {  // raise the references to the maxima
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
          float mn = s[v];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
          mn = fmaxf(m[v], mn);
          const float al = exp2f(m[v] - (mn == -INFINITY ? 0.f : mn));
          m[v] = mn;
          l[v] *= al;
#pragma unroll
          for (int e = 0; e < EL; ++e) (v % 2 ? acc[v / 2][e].y : acc[v / 2][e].x) *= al;
        }
      }
      float4 p4[kVecs / 4];
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const float p = any >> v & 1 ? exp2f(s[v] - (m[v] == -INFINITY ? 0.f : m[v])) : 0.f;
        l[v] += p;
        reinterpret_cast<float*>(p4)[v] = p;
      }
#pragma unroll
      for (int v = 0; v < kVecs; v += 4) *reinterpret_cast<float4*>(&S.p[lane][v]) = p4[v / 4];
      copies_wait1();                       // its values
      auto sum = [&](int i, uint32_t who) {
        float vx[EL];
        if constexpr (EL == 4) {
          const float4 y = S.v[i][lane];
          vx[0] = y.x, vx[1] = y.y, vx[2] = y.z, vx[3] = y.w;
        } else {
          const float2 y = reinterpret_cast<const float2*>(S.v[i])[lane];
          vx[0] = y.x, vx[1] = y.y;
        }
        const float2* px = reinterpret_cast<const float2*>(S.p[i]);
#pragma unroll
        for (int v = 0; v < kVecs / 2; ++v)
#pragma unroll
          for (int e = 0; e < EL; ++e)
            acc[v][e] = fma2(px[v], make_float2(who >> (2 * v) & 1 ? vx[e] : 0.f, who >> (2 * v + 1) & 1 ? vx[e] : 0.f),
                             acc[v][e]);
      };
      if (__all_sync(0xffffffffu, any == kAll)) {
#pragma unroll 4
        for (int i = 0; i < kTile; ++i) sum(i, kAll);
      } else {                              // 0 * V is not 0 for an infinite or NaN V
#pragma unroll 2
        for (int i = 0; i < kTile; ++i) sum(i, __shfl_sync(0xffffffffu, any, i));
      }
      __syncwarp();
      copy(a.v_pool, next, false, S.v, j + 1 < at.j1);
      row = next;
    }
    const bool whole = at.j0 == 0 && at.j1 == at.nt;
    const int64_t slot = (w * 2 + (at.j0 == 0 ? 1 : 0)) * kVecs;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l[v] += __shfl_xor_sync(0xffffffffu, l[v], o);
      const int vi = vg * kVecs + v;
      if (v >= n_vec) continue;
      if (whole) {
        float* out = reinterpret_cast<float*>(a.O) +
                 ((int64_t)(at.q.row0 + vi / a.g) * a.n_q_heads + h * a.g + vi % a.g) * D + lane * EL;
#pragma unroll
        for (int e = 0; e < EL; ++e)
          out[e] = l[v] == 0.f ? 0.f : (v % 2 ? acc[v / 2][e].y : acc[v / 2][e].x) / l[v];     // (nothing has weight: zeros)
      } else {
        if (lane == 0) a.part_ml[slot + v] = make_float2(m[v], l[v]);
#pragma unroll
        for (int e = 0; e < EL; ++e) a.part_o[(slot + v) * D + lane * EL + e] = v % 2 ? acc[v / 2][e].y : acc[v / 2][e].x;
      }
    }
    __syncwarp();
  }
}

// Joins the parts of one new token's query heads of one KV head (blockIdx.y), which
// are vectors of the same unit.  kWarps / g warps take a vector (a warp several, where
// g is more), every one of them a share of its parts, kRows of them in flight.
// Latency bounds it, so what the attention does not write (rows, lengths) is read
// before it is waited for, and the first parts beside their weights.  Many rows have few
// parts each: four warps.  Few rows may have many: sixteen.  (Here and in the other files of
// the step times are those of graphs of a few calls, whose launch adds 1 to 2 us to each.  One token over 4096: 3 us of 16;
// 8 trees of 64 over 33k: about 14 of 405, with 28 MB of parts.)
constexpr int kRows = 4;

template <typename T> __device__ __forceinline__ void store4(T* p, float4 v);
template <> __device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
template <> __device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

template <typename T, int D, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int L = D / 4, kSub = 32 / L;  // lanes of a row, rows of a warp's read
  __shared__ float4 s_o[kJoinWarps * kSub][L];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  pdl_trigger();
  const int row = blockIdx.x, h = blockIdx.y;
  const int s = seq_of_row(a.seq.rows, a.seq.n_seq, row);
  Seq q{0, 0, 0};
  if (s < 0 || s >= a.seq.n_seq || !seq_of(a.seq, s, &q) || row < q.row0 || row >= q.row0 + q.n) {
    pdl_wait();                           // who waits for this kernel waits for the one before it, too
    return;
  }
  const int nt = tiles_of(a, q), groups = (q.n * a.g + a.vecs - 1) >> a.vecs_log2;
  const int per_vec = max(1, kJoinWarps >> a.g_log2), share = warp % per_vec;
  const int sub = lane / L, ch = lane % L * 4, step = per_vec * kSub, mine = share * kSub + sub;
  pdl_wait();
  const int64_t per = per_worker(a, a.start[a.seq.n_seq]);
  const int v0 = (row - q.row0) * a.g, vg = v0 >> a.vecs_log2;
  const int64_t u0 = a.start[s] + (int64_t)(h * groups + vg) * nt;
  const int64_t u1 = u0 + nt - 1;
  const int64_t c0 = u1 >> 32 ? u0 / per : (uint32_t)u0 / (uint32_t)per;
  const int64_t c1 = min(u1 >> 32 ? u1 / per : (int64_t)((uint32_t)u1 / (uint32_t)per), (int64_t)a.workers - 1);
  if (c0 == c1) return;                   // written by its one worker
  const int parts = (int)(c1 - c0) + 1;
  for (int j = warp / per_vec; j < a.g; j += kJoinWarps / per_vec) {
    const int v = (v0 + j) & (a.vecs - 1);
    auto slot = [&](int i) { return ((c0 + i) * 2 + (i == 0 ? 1 : 0)) * a.vecs + v; };
    float4 x[kRows];
    auto read = [&](int i) {
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (i + k * step + mine < parts)
          x[k] = *reinterpret_cast<const float4*>(a.part_o + slot(i + k * step + mine) * D + ch);
    };
    read(0);
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < parts) ml = a.part_ml[slot(lane)];
    float M = ml.x;
    for (int i = lane + 32; i < parts; i += 32) M = fmaxf(M, a.part_ml[slot(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < parts; i += kRows * step) {
      if (i > 0) read(i);
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int at = i + k * step + mine;
        // a lane's weight (of a part that saw no key: none; what is there is not used)
        float2 w = ml;
        if (parts > 32) {                 // uniform
          w = at < parts ? a.part_ml[slot(at)] : make_float2(-INFINITY, 0.f);
        } else {
          w.x = __shfl_sync(0xffffffffu, ml.x, at & 31);
          w.y = __shfl_sync(0xffffffffu, ml.y, at & 31);
        }
        if (at >= parts || (w.x == -INFINITY && w.y == 0.f)) continue;
        const float f = exp2f(w.x - ref);
        l = fmaf(f, w.y, l);
        o.x = fmaf(f, x[k].x, o.x);
        o.y = fmaf(f, x[k].y, o.y);
        o.z = fmaf(f, x[k].z, o.z);
        o.w = fmaf(f, x[k].w, o.w);
      }
    }
    if (step > 1) {                       // the vector's shares (one pass where there are several)
      __shared__ float s_l[kJoinWarps * kSub];
      s_o[warp * kSub + sub][lane % L] = o;
      if (lane % L == 0) s_l[warp * kSub + sub] = l;
      if (per_vec > 1)
        __syncthreads();
      else
        __syncwarp();
      if (mine == 0) {
        for (int k = 1; k < step; ++k) {
          const float4 y = s_o[warp * kSub + k][lane];
          o.x += y.x;
          o.y += y.y;
          o.z += y.z;
          o.w += y.w;
          l += s_l[warp * kSub + k];
        }
      }
      __syncwarp();
    }
    if (l == 0.f) l = 1.f;                  // no part has weight, and o is 0
    if (mine == 0)
      store4(reinterpret_cast<T*>(a.O) + ((int64_t)row * a.n_q_heads + h * a.g + j) * D + ch,
             make_float4(o.x / l, o.y / l, o.z / l, o.w / l));
  }
}

template <typename T, int D>
cudaError_t launch_join_d(const TreeArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.seq.n_rows, a.n_kv_heads);
  if (a.seq.n_rows * a.n_kv_heads <= 304)
    return launch_pdl(tree_join_kernel<T, D, 16>, grid, dim3(16 * 32), 0, s, a);
  return launch_pdl(tree_join_kernel<T, D, 4>, grid, dim3(4 * 32), 0, s, a);
}
template <typename T> cudaError_t launch_join(const TreeArgs& a, int d, cudaStream_t s) {
  return d == 128 ? launch_join_d<T, 128>(a, s) : launch_join_d<T, 64>(a, s);
}

// ---- host side ---------------------------------------------------------------

constexpr int kCtas = 152;                // SMs
// CTAs of an SM (fp32 layers): as many fit where d = 64, three where d = 128.  There, too, more
// and shorter runs are faster, as units differ in length: 285 us with five, 368 with three (one
// token over 3000 to 6000, 4 sequences: 53 and 48; d = 64: 32 and 41).
constexpr int kSimtCtas = 5;

fuse_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? FUSE_OK : FUSE_ERR_CUDA; }

TreePlan plan_tree(const fuse_layer_desc_t& d, int n_seq) {
  TreePlan P;
  const bool tc = d.dtype == FUSE_BF16;
  P.vecs = tc ? kTreeTcVecs : kVecs;
  P.tile = tc ? kTreeTcTile : kTile;
  P.workers = tc ? kCtas : kCtas * kSimtCtas * kWarps;
  P.start = sizeof(WsHeader);
  P.part_ml = align_up(P.start + ((size_t)n_seq + 1) * sizeof(int64_t), 256);
  const size_t rows = (size_t)P.workers * 2 * P.vecs;
  P.part_o = align_up(P.part_ml + rows * sizeof(float2), 256);
  P.total = align_up(P.part_o + rows * d.head_dim * sizeof(float), 256);
  return P;
}

}  // namespace

cudaError_t launch_tree_simt(const fuse_layer_desc_t& d, const TreeArgs& a, cudaStream_t s) {
  auto run = [&](auto kernel, int smem) {
    if (cudaError_t e = set_dyn_smem_once(reinterpret_cast<const void*>(kernel), smem)) return e;
    return launch_pdl(kernel, dim3(a.workers / kWarps), dim3(kWarps * 32), smem, s, a);
  };
  return d.head_dim == 128 ? run(tree_simt_kernel<128>, sizeof(SimtShared<128>) * kWarps)
                           : run(tree_simt_kernel<64>, sizeof(SimtShared<64>) * kWarps);
}

}  // namespace fusekv

using namespace fusekv;

extern "C" {

fuse_status_t fuse_tree_workspace_size(const fuse_layer_desc_t* desc, const fuse_seqs_t* seqs,
                                       size_t* bytes) {
  if (!bytes) return FUSE_ERR_INVALID_ARG;
  fuse_status_t st = check_desc(desc);
  if (st != FUSE_OK) return st;
  if (!seqs || seqs->n_seq < 0) return FUSE_ERR_INVALID_ARG;
  if (seqs->n_seq > 65535) return FUSE_ERR_UNSUPPORTED;
  *bytes = plan_tree(*desc, seqs->n_seq).total;
  return FUSE_OK;
}

fuse_status_t fuse_attend_tree(const fuse_layer_desc_t* desc, const fuse_seqs_t* seqs, int64_t n_rows,
                               const int32_t* parents, const void* Q, const void* k_pool,
                               const void* v_pool, void* O, void* ws, size_t ws_bytes,
                               fuse_stream_t stream) {
  fuse_status_t st = check_desc(desc);
  if (st != FUSE_OK) return st;
  TreeArgs a;
  st = check_seqs(seqs, n_rows, FUSE_TREE_MAX_NEW, &a.seq, ws);
  if (st != FUSE_OK) return st;
  if (n_rows > 0 && (!Q || !k_pool || !v_pool || !O)) return FUSE_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(O)) return FUSE_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(parents) & 3u) return FUSE_ERR_MISALIGNED;
  if (desc->n_kv_heads > 65535) return FUSE_ERR_UNSUPPORTED;
  const TreePlan P = plan_tree(*desc, seqs->n_seq);
  st = check_ws(ws, ws_bytes, P.total);
  if (st != FUSE_OK) return st;
  if (n_rows == 0 || seqs->n_seq == 0) return FUSE_OK;
  auto at = [&](size_t off) { return reinterpret_cast<char*>(ws) + off; };
  a.parents = parents;
  a.Q = Q;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.O = O;
  a.n_q_heads = desc->n_q_heads;
  a.n_kv_heads = desc->n_kv_heads;
  a.g = desc->n_q_heads / desc->n_kv_heads;
  a.g_log2 = a.g == 8 ? 3 : a.g == 4 ? 2 : a.g == 2 ? 1 : 0;
  a.vecs = P.vecs;
  a.vecs_log2 = desc->dtype == FUSE_BF16 ? 8 : 3;
  a.tile = P.tile;
  a.tile_log2 = desc->dtype == FUSE_BF16 ? 7 : 5;
  // no more workers than the tables' rows could give tiles to
  const int64_t cap = ((int64_t)seqs->max_blocks * seqs->block_size + P.tile - 1) / P.tile;
  const int64_t groups = ((int64_t)seqs->max_new * a.g + P.vecs - 1) / P.vecs;
  int64_t most = 1;
  for (const int64_t f : {cap, groups, (int64_t)seqs->n_seq, (int64_t)a.n_kv_heads})
    most = std::min<int64_t>(P.workers, most * f);
  a.workers = desc->dtype == FUSE_BF16 ? (int)most : (int)((most + kWarps - 1) / kWarps * kWarps);
  a.scale = 1.4426950408889634f / std::sqrt((float)desc->head_dim);
  a.start = reinterpret_cast<int64_t*>(at(P.start));
  a.part_ml = reinterpret_cast<float2*>(at(P.part_ml));
  a.part_o = reinterpret_cast<float*>(at(P.part_o));
  cudaStream_t s = (cudaStream_t)stream;
  st = cuda_status(traced("attend_tree", s, [&] {
    return desc->dtype == FUSE_BF16 ? launch_tree_tc(*desc, a, s) : launch_tree_simt(*desc, a, s);
  }));
  if (st != FUSE_OK) return st;
  return cuda_status(traced("attend_tree_join", s, [&] {
    return desc->dtype == FUSE_BF16 ? launch_join<__nv_bfloat16>(a, desc->head_dim, s)
                                    : launch_join<float>(a, desc->head_dim, s);
  }));
}

}  // extern "C"
