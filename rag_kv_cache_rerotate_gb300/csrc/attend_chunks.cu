// Attention of new tokens over chunk caches in their storage form: the entry
// points, the CUDA-core kernel (fp32 layers) and the kernel that joins the items.
//
// QCFuse (section 2.1.2, Eq. 4): a chunk's keys, computed at local positions,
// belong at R^pos K; (section 2.1.3, Eq. 6): selected positions hold
// refreshed entries.  KVBoost (section 4.5, Eq. 7): x = zero + code * scale.
//
// The rotation and the scales move to the query, once per chunk and head:
//   q . R^pos (z + c * s) = (R^-pos q) . z + ((R^-pos q) * s) . c
// (z, s per channel), so that a key costs its codes only.  A value's scale
// and zero are per token: sum_t p_t (z_t + s_t c_t) = sum p_t z_t + sum (p_t
// s_t) c_t.  Keys are split over many items (attend_chunks.h); with an item's
// maximum m_i, sum l_i and unnormalised output o_i,
//   O = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,   M = max_i m_i.
// The new tokens' own keys (at most 8 per request, the only ones that some
// of the new tokens see and others do not) are taken by the joining kernel,
// so items need no causal mask and no row is left without a key.
#include <algorithm>
#include <cmath>
#include <vector>

#include "attend_chunks.h"
#include "checks.h"
#include "launch.h"
#include "trace.h"

namespace fusekv {

namespace {

constexpr int kWarps = kItemWarps;
constexpr int kAtOnce = 8;                // keys whose values it reads at a time

// Eight consecutive stored elements as fp32.
template <int ST> __device__ __forceinline__ void load8(const uint8_t* row, int e, float (&x)[8]) {
  if constexpr (ST == FUSE_F32) {
    Vec8<float>::load(reinterpret_cast<const float*>(row) + e, x);
  } else if constexpr (ST == FUSE_U8_ASYM) {
    const uint2 w = *reinterpret_cast<const uint2*>(row + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = (float)((w.x >> (8 * i)) & 0xFFu);
      x[4 + i] = (float)((w.y >> (8 * i)) & 0xFFu);
    }
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(row + e / 2);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)((w >> (4 * i)) & 15u);
  }
}

// EL = 2 or 4 consecutive stored elements as fp32.
template <int ST, int EL>
__device__ __forceinline__ void load_el(const uint8_t* row, int e, float (&x)[EL]) {
  if constexpr (ST == FUSE_F32) {
#pragma unroll
    for (int i = 0; i < EL; ++i) x[i] = reinterpret_cast<const float*>(row)[e + i];
  } else if constexpr (ST == FUSE_U8_ASYM) {
#pragma unroll
    for (int i = 0; i < EL; ++i) x[i] = (float)row[e + i];
  } else {
#pragma unroll
    for (int i = 0; i < EL; i += 2) {
      const uint32_t b = row[(e + i) / 2];
      x[i] = (float)(b & 15u);
      x[i + 1] = (float)(b >> 4);
    }
  }
}

template <int ST> constexpr bool coded() { return ST == FUSE_U8_ASYM || ST == FUSE_U4_ASYM; }
template <int ST> constexpr int row_bytes(int d) {
  return ST == FUSE_F32 ? 4 * d : ST == FUSE_U8_ASYM ? d : d / 2;
}

// The keys of an item.
struct Keys {
  const uint8_t *k, *v;                   // row 0, head 0
  const __half *vs, *vz;
  const int32_t* table;                   // paged: block ids
  int t0, t1;                             // rows [t0, t1)
  int n_skip;                             // selected positions (chunks), ascending
  const int32_t* skip;
  int pos0;                               // request position of row 0 (chunks)
};

// One warp, one item: 32 keys at a time, a lane per key for the scores, then
// a lane per D / 32 channels for the sums.
// Latency bounds it (2 requests of 3 or 4 chunks of 33 to 64 keys at 4 bits: 10
// us with the join), so several rows are read at a time; with the values read
// one by one it took 13.6.
template <int ST, int D>
__device__ void attend_item(const AttendArgs& a, const Keys& y, const float2* cs, const __half* ks,
                            const __half* kz, int r, int h, int vg, int64_t slot, float (*s_q)[D],
                            float (*s_p)[kVecs]) {
  constexpr int EL = D / 32;
  const int lane = threadIdx.x % 32;
  const int n_vec = min(kVecs, a.g * a.n_new - vg * kVecs);
  float cst[kVecs];
  // the query vectors, turned back by the chunk's offset and scaled
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    const int vi = vg * kVecs + v;
    float z = 0.f;
#pragma unroll
    for (int j = lane; j < D / 2; j += 32) {
      float x0 = 0.f, x1 = 0.f;
      if (v < n_vec) {
        const float* q = reinterpret_cast<const float*>(a.Q) +
                         ((int64_t)(r * a.n_new + vi / a.g) * a.n_q_heads + h * a.g + vi % a.g) * D;
        const float q0 = q[j] * a.scale, q1 = q[j + D / 2] * a.scale;
        const float2 w = cs ? cs[j] : make_float2(1.f, 0.f);
        x0 = q0 * w.x + q1 * w.y;
        x1 = q1 * w.x - q0 * w.y;
        if (coded<ST>() && ks) {
          z += x0 * __half2float(kz[h * D + j]) + x1 * __half2float(kz[h * D + j + D / 2]);
          x0 *= __half2float(ks[h * D + j]);
          x1 *= __half2float(ks[h * D + j + D / 2]);
        }
      }
      s_q[v][j] = x0;
      s_q[v][j + D / 2] = x1;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    cst[v] = z;
  }
  __syncwarp();
  float m[kVecs], l[kVecs], zs[kVecs], acc[kVecs][EL];
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    m[v] = -INFINITY;
    l[v] = zs[v] = 0.f;
#pragma unroll
    for (int e = 0; e < EL; ++e) acc[v][e] = 0.f;
  }
  constexpr int RB = row_bytes<ST>(D);
  const int64_t stride = (int64_t)a.n_kv_heads * RB;
  // the first selected position that is not before the item: 32 probes a round
  int sel = 0;
  for (int len = y.n_skip; len > 0;) {
    const int step = (len + 31) / 32, i = sel + (lane + 1) * step - 1;
    const bool below = i < sel + len && y.skip[i] < y.pos0 + y.t0;
    const int parts = __popc(__ballot_sync(0xffffffffu, below));
    sel += parts * step;
    len = min(step - 1, len - parts * step);
  }
  for (int t = y.t0; t < y.t1; t += 32) {
    const int key = t + lane;
    bool ok = key < y.t1;
    int64_t row = key;
    if (ok && y.table) {
      const int b = y.table[key / a.block_size];
      if (b < 0 || b >= a.n_pool_blocks) {
        report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_ATTEND_BLOCK, (uint32_t)b);
        ok = false;
      } else {
        row = (int64_t)b * a.block_size + key % a.block_size;
      }
    }
    if (y.n_skip > 0) {                    // selected positions: at most 32 entries from `sel` on
      const int p = y.pos0 + t, v = sel + lane < y.n_skip ? y.skip[sel + lane] : INT32_MAX;
      const bool here = v >= p && v < p + 32;
      const uint32_t mask = __reduce_or_sync(0xffffffffu, here ? 1u << (v - p) : 0u);
      ok = ok && !(mask >> lane & 1);
      sel += __popc(__ballot_sync(0xffffffffu, v < p + 32));
    }
    float s[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) s[v] = ok ? cst[v] : -INFINITY;
    if (ok) {
      const uint8_t* kr = y.k + row * stride + h * RB;
#pragma unroll 4
      for (int e = 0; e < D; e += 8) {
        float x[8];
        load8<ST>(kr, e, x);
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[v] = fmaf(s_q[v][e + i], x[i], s[v]);
      }
    }
    float vs = 1.f, vz = 0.f;
    if (coded<ST>() && ok) {
      vs = __half2float(y.vs[row * a.n_kv_heads + h]);
      vz = __half2float(y.vz[row * a.n_kv_heads + h]);
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float mt = s[v];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      const float mn = fmaxf(m[v], mt);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float al = exp2f(m[v] - ref), p = ok ? exp2f(s[v] - ref) : 0.f;
      m[v] = mn;
      l[v] = l[v] * al + p;
      zs[v] = zs[v] * al + p * vz;
      s_p[lane][v] = p * vs;
#pragma unroll
      for (int e = 0; e < EL; ++e) acc[v][e] *= al;
    }
    __syncwarp();
    const int64_t at = ok ? row : -1;
    for (int i = 0; i < 32; i += kAtOnce) {            // reads of several keys in flight
      float x[kAtOnce][EL];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int64_t ri = __shfl_sync(0xffffffffu, at, i + j);
#pragma unroll
        for (int e = 0; e < EL; ++e) x[j][e] = 0.f;    // of a key not seen, whose weight is 0
        if (ri >= 0) load_el<ST, EL>(y.v + ri * stride + h * RB, lane * EL, x[j]);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
          for (int e = 0; e < EL; ++e) acc[v][e] = fmaf(s_p[i + j][v], x[j][e], acc[v][e]);
    }
    __syncwarp();
  }
  const int64_t at = ((slot * a.n_kv_heads + h) * a.nvg + vg) * kVecs;
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      l[v] += __shfl_xor_sync(0xffffffffu, l[v], o);
      zs[v] += __shfl_xor_sync(0xffffffffu, zs[v], o);
    }
    if (lane == 0) a.part_ml[at + v] = make_float2(m[v], l[v]);
#pragma unroll
    for (int e = 0; e < EL; ++e) a.part_o[(at + v) * D + lane * EL + e] = acc[v][e] + zs[v];
  }
}

template <int ST, int D>
__global__ void __launch_bounds__(kWarps * 32)
    attend_simt_kernel(const AttendArgs a, const __grid_constant__ ItemTable tab,
                       const __grid_constant__ RopeFreqs f) {
  __shared__ float s_q[kWarps][kVecs][D];
  __shared__ float s_p[kWarps][32][kVecs];
  __shared__ float2 s_cs[D / 2];
  const int warp = threadIdx.x / 32;
  const ItemPlace at = item_place(a, tab);
  pdl_wait();
  pdl_trigger();                           // the join may read the call's inputs before it waits
  if (at.none) return;
  const int h = at.h, vg = at.vg;
  if (at.side) {
    // side rows: those before the new tokens
    const int r = a.req0 + at.part;
    const fuse_request_t R = a.reqs[r];
    const int n = R.k + R.n_query - a.n_new;
    const int t0 = at.seg * a.sseg;
    if (t0 >= n) {                         // only where the two copies of the table differ
      no_keys(a, at);
      return;
    }
    Keys y;
    constexpr int RB = row_bytes<FUSE_F32>(D);
    y.k = reinterpret_cast<const uint8_t*>(a.Ks) + R.out0 * a.n_kv_heads * RB;
    y.v = reinterpret_cast<const uint8_t*>(a.Vs) + R.out0 * a.n_kv_heads * RB;
    y.vs = y.vz = nullptr;
    y.table = nullptr;
    y.t0 = t0;
    y.t1 = min(n, t0 + a.sseg);
    y.n_skip = 0;
    if (h == 0 && vg == 0) {               // the selection, checked where its rows are read
      for (int t = y.t0 + threadIdx.x % 32; t < min(y.t1, R.k); t += 32) {
        const int v = a.idx[R.sel0 + t];
        if (v < 0 || v >= R.n_ctx || (t > 0 && a.idx[R.sel0 + t - 1] >= v))
          report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_ATTEND_SEL, (uint32_t)t);
      }
    }
    attend_item<FUSE_F32, D>(a, y, nullptr, nullptr, nullptr, r, h, vg, at.slot, s_q[warp], s_p[warp]);
    return;
  }
  const fuse_chunk_t C = a.chunks[a.chunk0 + at.part];
  // the chunk's angles, D / 16 pairs a warp.  The frequencies are launch
  // parameters, which a warp reads fast only at one address at a time.
  if (C.pos != 0) {                        // block-uniform
    constexpr int N = D / 2 / kWarps;
    const int lane = threadIdx.x % 32;
    float hi = 0.f, mid = 0.f, lo = 0.f, c, sn;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float fh = f.hi[warp * N + k], fm = f.mid[warp * N + k], fl = f.lo[warp * N + k];
      if (lane == k) {
        hi = fh;
        mid = fm;
        lo = fl;
      }
    }
    rope_cos_sin(C.pos, hi, mid, lo, c, sn);
    if (lane < N) s_cs[warp * N + lane] = make_float2(c, sn);
  }
  __syncthreads();
  const int t0 = at.seg * a.seg;
  if (t0 >= C.len) {                       // past the chunk's end
    no_keys(a, at);
    return;
  }
  const int r = tab.owner[at.part];
  const fuse_request_t R = a.reqs[r];
  Keys y;
  y.k = reinterpret_cast<const uint8_t*>(C.k);
  y.v = reinterpret_cast<const uint8_t*>(C.v);
  y.vs = reinterpret_cast<const __half*>(C.v_scale);
  y.vz = reinterpret_cast<const __half*>(C.v_zero);
  y.table = a.block_size > 0 ? C.block_table : nullptr;
  y.t0 = t0;
  y.t1 = min(C.len, t0 + a.seg);
  y.n_skip = R.k;
  y.skip = a.idx + R.sel0;
  y.pos0 = (int)(C.dst_row - R.row0);
  attend_item<ST, D>(a, y, C.pos != 0 ? s_cs : nullptr, reinterpret_cast<const __half*>(C.k_scale),
                     reinterpret_cast<const __half*>(C.k_zero), r, h, vg, at.slot, s_q[warp], s_p[warp]);
}

// Joins the items of one query vector (blockIdx.x = new token * Hq + head)
// of one request with the new tokens' own keys, and writes its output row.
// An item's row is read by D / 4 lanes, kRows items a lane in flight.  Latency
// bounds it (two dependent reads), so what does not depend on the items (the
// table entry, the own keys) is read before they are waited for, and the first
// rows beside the weights.  256 threads, so that the blocks of 16 requests fit
// the card at once: with 512 the 16 paged requests took 38 us instead of 36,
// with 128 one request took 12 instead of 11.
constexpr int kJoinThreads = 256;
constexpr int kJoinTile = kJoinThreads;   // items whose weights are held at a time
constexpr int kRows = 4;                  // items' rows of a lane in flight
static_assert(kJoinThreads / 32 >= FUSE_ATTEND_MAX_NEW, "a warp takes a new token's own key");

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ void add4(float4& a, float w, const float4& x) {
  a.x = fmaf(w, x.x, a.x);
  a.y = fmaf(w, x.y, a.y);
  a.z = fmaf(w, x.z, a.z);
  a.w = fmaf(w, x.w, a.w);
}

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
    attend_combine_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ JoinTable tab) {
  constexpr int kWarpsJ = kJoinThreads / 32, L = D / 4, kSub = 32 / L;   // lanes, items of a warp step
  __shared__ float s_w[kJoinTile];
  __shared__ float s_own[FUSE_ATTEND_MAX_NEW];
  __shared__ float s_red[2][kWarpsJ];
  __shared__ float4 s_o[kWarpsJ * kSub][L];
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int r = a.req0 + blockIdx.y;
  const int u = blockIdx.x / a.n_q_heads, hq = blockIdx.x % a.n_q_heads;
  const int h = hq / a.g;
  const int vi = u * a.g + hq % a.g;      // vector of its KV head
  const fuse_request_t R = a.reqs[r];
  const int seg0 = tab.seg[blockIdx.y], side0 = tab.side[blockIdx.y];
  const int n_seg = tab.seg[blockIdx.y + 1] - seg0;
  const int n_side = R.k + R.n_query - a.n_new;           // side rows in items
  const int n = n_seg + tab.side[blockIdx.y + 1] - side0;
  // own keys: warp j takes new token j
  const T* Ks = reinterpret_cast<const T*>(a.Ks);
  const T* Vs = reinterpret_cast<const T*>(a.Vs);
  const int64_t qrow = ((int64_t)(r * a.n_new + u) * a.n_q_heads + hq) * D;
  const int64_t own = ((R.out0 + n_side) * a.n_kv_heads + h) * D, own_step = (int64_t)a.n_kv_heads * D;
  float4 v_own = make_float4(0.f, 0.f, 0.f, 0.f);
  if (warp <= u) {
    float s = 0.f;
    if (lane < L) {
      const float4 q = load4(reinterpret_cast<const T*>(a.Q) + qrow + lane * 4);
      const float4 k = load4(Ks + own + warp * own_step + lane * 4);
      v_own = load4(Vs + own + warp * own_step + lane * 4);
      s = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, q.w * k.w)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) s_own[warp] = s * a.scale;
  }
  pdl_wait();
  // item e's vector: chunk segments, then side segments
  const int64_t step = (int64_t)a.n_kv_heads * a.nvg * kVecs;
  const int64_t mine = ((int64_t)h * a.nvg + vi / kVecs) * kVecs + vi % kVecs;
  const int64_t at_seg = seg0 * step + mine;
  const int64_t at_side = (side0 - n_seg) * step + mine;
  auto part = [&](int e) { return (e < n_seg ? at_seg : at_side) + e * step; };
  const int sub = lane / L, ch = lane % L * 4;
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int e0 = 0; e0 == 0 || e0 < n; e0 += kJoinTile) {
    const int cnt = min(kJoinTile, n - e0);
    float2 ml = make_float2(-INFINITY, 0.f);
    if (tid < cnt) ml = a.part_ml[part(e0 + tid)];
    // the first rows are read beside the weights, not after them; what an item
    // without a key left there (nothing) is not used
    const int e1 = warp * kSub + sub;
    float4 x[kRows];
    auto rows = [&](int e) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int ei = e + i * kWarpsJ * kSub;
        if (ei < cnt) x[i] = *reinterpret_cast<const float4*>(a.part_o + part(e0 + ei) * D + ch);
      }
    };
    rows(e1);
    float t = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
    __syncthreads();                      // s_own written; the last tile's weights are used
    if (lane == 0) s_red[0][warp] = t;
    __syncthreads();
    float mn = M;
    for (int w = 0; w < kWarpsJ; ++w) mn = fmaxf(mn, s_red[0][w]);
    if (e0 == 0)
      for (int j = 0; j <= u; ++j) mn = fmaxf(mn, s_own[j]);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float al = exp2f(M - ref);      // 0 in the first tile
    M = mn;
    const float w = exp2f(ml.x - ref);
    l = l * al + w * ml.y;
    // an item without a key is not read: it may have written nothing
    s_w[tid] = tid < cnt && !(ml.x == -INFINITY && ml.y == 0.f) ? w : -1.f;
    acc.x *= al;
    acc.y *= al;
    acc.z *= al;
    acc.w *= al;
    __syncthreads();
    for (int e = e1; e < cnt; e += kRows * kWarpsJ * kSub) {
      if (e != e1) rows(e);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int ei = e + i * kWarpsJ * kSub;
        const float we = ei < cnt ? s_w[ei] : -1.f;
        if (we != -1.f) add4(acc, we, x[i]);
      }
    }
  }
  if (warp <= u && lane < L) {
    const float p = exp2f(s_own[warp] - (M == -INFINITY ? 0.f : M));
    if (lane == 0) l += p;
    add4(acc, p, v_own);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) s_red[1][warp] = l;
  s_o[warp * kSub + sub][lane % L] = acc;
  __syncthreads();
  if (tid >= L) return;
  l = 0.f;
  for (int w = 0; w < kWarpsJ; ++w) l += s_red[1][w];
  acc = s_o[0][tid];
  for (int w = 1; w < kWarpsJ * kSub; ++w) add4(acc, 1.f, s_o[w][tid]);
  store4(reinterpret_cast<T*>(a.O) + qrow + tid * 4,
         make_float4(acc.x / l, acc.y / l, acc.z / l, acc.w / l));
}

template <int ST, int D>
cudaError_t launch_simt_t(const AttendArgs& a, const ItemTable& t, const RopeFreqs& f, cudaStream_t s) {
  return launch_pdl(attend_simt_kernel<ST, D>, dim3((unsigned)item_ctas(a, t)), dim3(kWarps * 32), 0, s, a,
                    t, f);
}

template <int D>
cudaError_t launch_simt_d(int st, const AttendArgs& a, const ItemTable& t, const RopeFreqs& f,
                          cudaStream_t s) {
  if (st == FUSE_U4_ASYM) return launch_simt_t<FUSE_U4_ASYM, D>(a, t, f, s);
  if (st == FUSE_U8_ASYM) return launch_simt_t<FUSE_U8_ASYM, D>(a, t, f, s);
  return launch_simt_t<FUSE_F32, D>(a, t, f, s);
}

// ---- host side ---------------------------------------------------------------

constexpr int64_t kItems = 152 * 12;      // warps of bf16 layers that 152 SMs hold
constexpr int kMaxKeys = 1024;            // keys of an item (a bit each in 32 words)

int cut(int64_t keys, int64_t items, int step) {     // keys per item, a multiple of step
  const int64_t k = (keys + items - 1) / items;
  return (int)std::min<int64_t>(kMaxKeys, std::max<int64_t>(step, (k + step - 1) / step * step));
}

// Where a call's segments are: owner[c], seg0[c]: request and first segment of
// chunk c; first[r], side0[r]: first chunk and first side segment of request r
// (seg0, first, side0: one entry more than there are chunks or requests).
struct AttendTables {
  std::vector<uint16_t> owner;
  std::vector<int32_t> seg0, first, side0;
};

// Checks everything that needs no tensor, and fills T if it is not null.
fuse_status_t plan_attend(const fuse_layer_desc_t* desc, const fuse_chunks_t* chunks,
                          const fuse_requests_t* reqs, int n_new, bool need_device, ReqInfo* info,
                          AttendPlan* P, AttendTables* T) {
  fuse_status_t st = check_desc(desc);
  if (st != FUSE_OK) return st;
  st = check_reqs(reqs, info, need_device);
  if (st != FUSE_OK) return st;
  if (!chunks || n_new < 1 || n_new > FUSE_ATTEND_MAX_NEW) return FUSE_ERR_INVALID_ARG;
  if (reqs->n_req > 0 && !info->sorted) return FUSE_ERR_INVALID_ARG;
  if (chunks->kv_storage != FUSE_U4_ASYM && chunks->kv_storage != FUSE_U8_ASYM &&
      chunks->kv_storage != desc->dtype)
    return FUSE_ERR_UNSUPPORTED;
  if (chunks->kv_layout == FUSE_KV_PAGED && chunks->block_size > 0 &&
      chunks->n_pool_blocks > INT32_MAX / chunks->block_size)
    return FUSE_ERR_UNSUPPORTED;                       // pool rows are 32-bit numbers
  fuse_chunks_t c = *chunks;
  if (!need_device && !c.d_chunks) c.d_chunks = c.h_chunks;    // only its presence is checked
  int max_len = 0;
  st = check_chunks(*desc, &c, info->tot.n_tok, &max_len);
  if (st != FUSE_OK) return st;
  int64_t n_ctx = 0, n_side = 0;
  int r = 0;
  if (T) T->first[0] = 0;
  const fuse_request_t* R = reqs->h_req;
  int64_t end = 0;
  for (int i = 0; i < chunks->n_chunks; ++i) {
    const fuse_chunk_t& q = chunks->h_chunks[i];
    if (i > 0 && q.dst_row < end) return FUSE_ERR_INVALID_ARG;
    end = q.dst_row + q.len;
    // the request whose context holds the chunk (an empty one goes with the
    // request before it)
    while (r < reqs->n_req && q.dst_row + (q.len > 0) > R[r].row0 + R[r].n_ctx) {
      ++r;
      if (T) T->first[r] = i;
    }
    if (q.len > 0 && (r >= reqs->n_req || q.dst_row < R[r].row0 || end > R[r].row0 + R[r].n_ctx))
      return FUSE_ERR_INVALID_ARG;
    if (T) T->owner[i] = (uint16_t)std::min(r, std::max(0, reqs->n_req - 1));
    n_ctx += q.len;
  }
  if (T)
    for (int k = r + 1; k <= reqs->n_req; ++k) T->first[k] = chunks->n_chunks;
  for (int i = 0; i < reqs->n_req; ++i) {
    if (R[i].n_query < n_new) return FUSE_ERR_INVALID_ARG;
    n_side += (int64_t)R[i].k + R[i].n_query - n_new;
  }
  const int g = desc->n_q_heads / desc->n_kv_heads;
  P->nvg = (g * n_new + kVecs - 1) / kVecs;
  const int64_t per = (int64_t)desc->n_kv_heads * P->nvg;
  // Shorter segments share less of an item's start (its query vectors, the
  // join), longer ones leave warps idle at the end.  bf16 layers, at least 64
  // keys: 8 chunks of 512 take 11 us, with 192 keys 13; 16 requests of 0.5k to
  // 8k tokens at the rule's 256 keys 39 us, at 128 45; 8 of 33k at 1024 keys 92
  // us, at 512 100.  Side rows go to half as many items (92 us; as many: 94, a
  // quarter: 100).  fp32 layers, whose lane takes a key: 10 us with 32 keys an
  // item, 13.5 with 64.
  const int least = desc->dtype == FUSE_BF16 ? 64 : 32;
  const int seg = cut(n_ctx * per, kItems, least);
  // the longest chunk's segments are evened out
  P->seg = cut(std::max(max_len, 1), std::max(1, (max_len + seg - 1) / seg), 32);
  P->sseg = cut(n_side * per, kItems / 2, least);
  // a chunk's segments fill whole CTAs
  const int pad = per % kItemWarps == 0 ? 1 : per % 2 == 0 ? 2 : kItemWarps;
  static_assert(kItemWarps == 4, "pad: what makes pad * per a multiple of kItemWarps");
  int64_t slots = 0;
  for (int i = 0; i < chunks->n_chunks; ++i) {
    if (T) T->seg0[i] = (int32_t)slots;
    const int n = (chunks->h_chunks[i].len + P->seg - 1) / P->seg;
    slots += (n + pad - 1) / pad * pad;
  }
  if (T) T->seg0[chunks->n_chunks] = (int32_t)slots;
  for (int i = 0; i < reqs->n_req; ++i) {
    if (T) T->side0[i] = (int32_t)slots;
    slots += ((int64_t)R[i].k + R[i].n_query - n_new + P->sseg - 1) / P->sseg;
  }
  if (T) T->side0[reqs->n_req] = (int32_t)slots;
  P->slots = slots;
  // an item count past a launch's grid is far past what a card holds
  if (slots > INT32_MAX / per) return FUSE_ERR_UNSUPPORTED;
  const size_t vecs = (size_t)P->slots * per * kVecs;
  P->part_ml = sizeof(WsHeader);
  P->part_o = align_up(P->part_ml + vecs * sizeof(float2), 256);
  P->total = align_up(P->part_o + vecs * desc->head_dim * sizeof(float), 256);
  return FUSE_OK;
}

template <typename T> T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(ws) + off);
}

fuse_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? FUSE_OK : FUSE_ERR_CUDA; }

}  // namespace

cudaError_t launch_attend_simt(const fuse_layer_desc_t& d, int st, const AttendArgs& a,
                               const ItemTable& t, const RopeFreqs& f, cudaStream_t s) {
  return d.head_dim == 128 ? launch_simt_d<128>(st, a, t, f, s) : launch_simt_d<64>(st, a, t, f, s);
}

cudaError_t launch_attend_combine(const fuse_layer_desc_t& d, const AttendArgs& a,
                                  const JoinTable& t, bool early, cudaStream_t s) {
  const dim3 grid(a.n_new * a.n_q_heads, a.n_req);
  auto go = [&](auto kernel) {
    if (early) return launch_pdl(kernel, grid, dim3(kJoinThreads), 0, s, a, t);
    kernel<<<grid, kJoinThreads, 0, s>>>(a, t);
    return cudaGetLastError();
  };
  if (d.dtype == FUSE_BF16)
    return d.head_dim == 128 ? go(attend_combine_kernel<__nv_bfloat16, 128>)
                             : go(attend_combine_kernel<__nv_bfloat16, 64>);
  return d.head_dim == 128 ? go(attend_combine_kernel<float, 128>)
                           : go(attend_combine_kernel<float, 64>);
}

}  // namespace fusekv

using namespace fusekv;

extern "C" {

fuse_status_t fuse_attend_workspace_size(const fuse_layer_desc_t* desc, const fuse_chunks_t* chunks,
                                         const fuse_requests_t* reqs, int32_t n_new,
                                         size_t* bytes) {
  if (!bytes) return FUSE_ERR_INVALID_ARG;
  ReqInfo info;
  AttendPlan P;
  const fuse_status_t st = plan_attend(desc, chunks, reqs, n_new, false, &info, &P, nullptr);
  if (st != FUSE_OK) return st;
  *bytes = P.total;
  return FUSE_OK;
}

fuse_status_t fuse_attend_chunks(const fuse_layer_desc_t* desc, const fuse_chunks_t* chunks,
                                 const fuse_requests_t* reqs, int32_t n_new, const void* Q,
                                 const int32_t* idx, const void* Ks, const void* Vs, void* O,
                                 void* ws, size_t ws_bytes, fuse_stream_t stream) {
  if (!chunks || chunks->n_chunks < 0 || !reqs || reqs->n_req < 0) return FUSE_ERR_INVALID_ARG;
  ReqInfo info;
  AttendPlan P;
  AttendTables T;
  try {
    T.owner.resize(chunks->n_chunks);
    T.seg0.resize((size_t)chunks->n_chunks + 1);
    T.first.resize((size_t)reqs->n_req + 1);
    T.side0.resize((size_t)reqs->n_req + 1);
  } catch (...) {
    return FUSE_ERR_INVALID_ARG;
  }
  fuse_status_t st = plan_attend(desc, chunks, reqs, n_new, true, &info, &P, &T);
  if (st != FUSE_OK) return st;
  if (reqs->n_req > 0 && (!Q || !Ks || !Vs || !O)) return FUSE_ERR_INVALID_ARG;
  if (info.tot.n_sel > 0 && !idx) return FUSE_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(Ks) || !aligned16(Vs) || !aligned16(O)) return FUSE_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(idx) & 3u) return FUSE_ERR_MISALIGNED;
  st = check_ws(ws, ws_bytes, P.total);
  if (st != FUSE_OK) return st;
  if (reqs->n_req == 0) return FUSE_OK;
  const RopeFreqs f = make_freqs(*desc);
  AttendArgs a;
  a.chunks = chunks->d_chunks;
  a.reqs = reqs->d_req;
  a.Q = Q;
  a.idx = idx;
  a.Ks = Ks;
  a.Vs = Vs;
  a.O = O;
  a.part_o = at<float>(ws, P.part_o);
  a.part_ml = at<float2>(ws, P.part_ml);
  a.err = at<uint32_t>(ws, 0);
  a.n_pool_blocks = chunks->n_pool_blocks;
  a.n_q_heads = desc->n_q_heads;
  a.n_kv_heads = desc->n_kv_heads;
  a.g = desc->n_q_heads / desc->n_kv_heads;
  a.n_new = n_new;
  a.nvg = P.nvg;
  a.seg = P.seg;
  a.sseg = P.sseg;
  a.block_size = chunks->kv_layout == FUSE_KV_PAGED ? chunks->block_size : 0;
  a.scale = 1.4426950408889634f / std::sqrt((float)desc->head_dim);
  cudaStream_t s = (cudaStream_t)stream;
  // items: as many chunks, and as many requests' side rows, as a launch takes
  ItemTable t;
  const int per = a.n_kv_heads * a.nvg;
  auto take = [](const std::vector<int32_t>& start, int i, int n, int most, uint16_t* out) {
    int k = 0;
    out[0] = 0;
    while (i + k < n && k < most && start[i + k + 1] - start[i] <= kSegBatch) {
      ++k;
      out[k] = (uint16_t)(start[i + k] - start[i]);
    }
    return k;
  };
  bool items = false;
  for (int c = 0, r = 0; c < chunks->n_chunks || r < reqs->n_req; c += a.n_chunks, r += a.n_req) {
    a.chunk0 = c;
    a.n_chunks = take(T.seg0, c, chunks->n_chunks, kChunkBatch, t.seg);
    a.chunk_slot0 = T.seg0[c];
    a.chunk_ctas = (int)((int64_t)t.seg[a.n_chunks] * per / kItemWarps);
    a.chunk_inv = (float)a.n_chunks / std::max<int>(1, t.seg[a.n_chunks]);
    a.req0 = r;
    a.n_req = take(T.side0, r, reqs->n_req, kSideBatch, t.side);
    a.side_slot0 = T.side0[r];
    a.side_inv = (float)a.n_req / std::max<int>(1, t.side[a.n_req]);
    std::copy(T.owner.begin() + c, T.owner.begin() + c + a.n_chunks, t.owner);
    if (item_ctas(a, t) == 0) continue;
    items = true;
    st = cuda_status(traced("attend_chunks", s, [&] {
      const auto launch = desc->dtype == FUSE_BF16 ? launch_attend_mma : launch_attend_simt;
      return launch(*desc, chunks->kv_storage, a, t, f, s);
    }));
    if (st != FUSE_OK) return st;
  }
  // The join reads the call's inputs before it waits for the kernel before it,
  // which is one of the above, begun after what wrote them had ended.  Without
  // an item there is none, and the first join starts after what came before.
  for (int r0 = 0; r0 < reqs->n_req; r0 += kReqBatch) {
    JoinTable j;
    a.req0 = r0;
    a.n_req = std::min(kReqBatch, reqs->n_req - r0);
    for (int i = 0; i <= a.n_req; ++i) {
      j.seg[i] = T.seg0[T.first[r0 + i]];
      j.side[i] = T.side0[r0 + i];
    }
    st = cuda_status(traced("attend_combine", s, [&] {
      return launch_attend_combine(*desc, a, j, items || r0 > 0, s);
    }));
    if (st != FUSE_OK) return st;
  }
  return FUSE_OK;
}

}  // extern "C"
