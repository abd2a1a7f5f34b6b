// Causal attention of whole prompts packed back to back: the entry point and
// the CUDA-core kernel (fp32 layers).
//
// KVBoost (section 3.1, Eq. 2): softmax(q K^T / sqrt(d)) V over j <= s, for
// every row s of every request.
#include <algorithm>
#include <cmath>
#include <vector>

#include "attend_prompt.h"
#include "checks.h"
#include "launch.h"
#include "trace.h"

namespace fusekv {

namespace {

struct PromptArgs {
  const void *Q, *K, *V;
  void* O;
  int n_q_heads, n_kv_heads, g;
  float scale;                            // log2(e) / sqrt(d)
};

constexpr int kKeys = 32;
constexpr int kThreads = 128;

template <int D, int R> struct Smem {
  float q[16 * R][D + 4];
  float k[kKeys][D + 4];
  float v[kKeys][D];
  float p[16 * R][kKeys + 1];
};

// One CTA per (tile, KV head): the tile's positions with the g query heads of
// the KV head form 16 R rows; keys come 32 at a time through shared memory.  A
// thread forms R x 4 scores (rows R i .., keys j, j + 8, ..) and then R rows x
// D / 8 channels of the sums, everything in fp32.  8 requests of 2000 rows (8 / 2
// heads of 128) run at 34 TFLOP/s, under half of the CUDA cores' FMA rate: a
// thread reads 8 x 16 bytes of shared memory for 64 FMA of its scores, and the
// tile meets at two barriers every 32 keys.  Where the tiles are few, the
// longest tile's chain bounds it.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads)
    prompt_simt_kernel(const PromptArgs a, const __grid_constant__ PromptTable p) {
  extern __shared__ __align__(16) uint8_t raw[];
  Smem<D, R>& sm = *reinterpret_cast<Smem<D, R>*>(raw);
  const int tid = threadIdx.x, tx = tid % 8, ty = tid / 8;
  pdl_trigger();
  pdl_wait();
  const int h = blockIdx.x % a.n_kv_heads;
  int part = 0;
  const PromptTile t = prompt_tile(p, 16 * R / a.g, blockIdx.x / a.n_kv_heads, &part);
  const int n_rows = t.rows * a.g;
  const T* Q = reinterpret_cast<const T*>(a.Q);
  const T* K = reinterpret_cast<const T*>(a.K);
  const T* V = reinterpret_cast<const T*>(a.V);
  for (int i = tid; i < 16 * R * D / 8; i += kThreads) {
    const int m = i / (D / 8), e = i % (D / 8) * 8;
    float x[8] = {};
    if (m < n_rows)
      Vec8<T>::load(Q + ((int64_t)(t.row0 + t.first + m / a.g) * a.n_q_heads + h * a.g + m % a.g) * D + e, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) sm.q[m][e + j] = x[j] * a.scale;
  }
  float mx[R], l[R], acc[R][D / 8];
  int pos[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    mx[i] = -INFINITY;
    l[i] = 0.f;
    pos[i] = t.first + (ty * R + i) / a.g;
#pragma unroll
    for (int e = 0; e < D / 8; ++e) acc[i][e] = 0.f;
  }
  const int n_keys = t.first + t.rows;
  // the thread's 8-element pieces of keys and values: the next ones are read
  // while the current ones are worked on, but for R = 4, whose tiles are many
  // (8 requests of 2000 rows, 8 / 2 heads of 128: 2.0 ms, read ahead 2.2)
  constexpr int kPieces = kKeys * D / 8 / kThreads;
  float x[kPieces][8], y[kPieces][8];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int j = (i * kThreads + tid) / (D / 8), e = (i * kThreads + tid) % (D / 8) * 8;
#pragma unroll
      for (int c = 0; c < 8; ++c) x[i][c] = y[i][c] = 0.f;
      if (k0 + j < n_keys) {
        const int64_t at = ((int64_t)(t.row0 + k0 + j) * a.n_kv_heads + h) * D + e;
        Vec8<T>::load(K + at, x[i]);
        Vec8<T>::load(V + at, y[i]);
      }
    }
  };
  if constexpr (R < 4) fetch(0);
  for (int k0 = 0; k0 < n_keys; k0 += kKeys) {
    if constexpr (R == 4) fetch(k0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int j = (i * kThreads + tid) / (D / 8), e = (i * kThreads + tid) % (D / 8) * 8;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        sm.k[j][e + c] = x[i][c];
        sm.v[j][e + c] = y[i][c];
      }
    }
    __syncthreads();
    if constexpr (R < 4)
      if (k0 + kKeys < n_keys) fetch(k0 + kKeys);
    float s[R][4] = {};
#pragma unroll 4
    for (int e = 0; e < D; e += 4) {
      float4 q[R], k[4];
#pragma unroll
      for (int i = 0; i < R; ++i) q[i] = *reinterpret_cast<const float4*>(&sm.q[ty * R + i][e]);
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(&sm.k[tx + 8 * j][e]);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(q[i].x, k[j].x, fmaf(q[i].y, k[j].y, fmaf(q[i].z, k[j].z, fmaf(q[i].w, k[j].w, s[i][j]))));
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (k0 + tx + 8 * j > pos[i]) s[i][j] = -INFINITY;
        m = fmaxf(m, s[i][j]);
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
      m = fmaxf(m, mx[i]);
      const float ref = m == -INFINITY ? 0.f : m;
      const float al = exp2f(mx[i] - ref);
      mx[i] = m;
      l[i] *= al;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w = exp2f(s[i][j] - ref);
        l[i] += w;
        sm.p[ty * R + i][tx + 8 * j] = w;
      }
#pragma unroll
      for (int e = 0; e < D / 8; ++e) acc[i][e] *= al;
    }
    __syncwarp();                          // rows R ty .. are written and read by one warp
    for (int j = 0; j < kKeys; ++j) {
      float w[R], v[D / 8];
#pragma unroll
      for (int i = 0; i < R; ++i) w[i] = sm.p[ty * R + i][j];
#pragma unroll
      for (int e = 0; e < D / 8; e += 4)
        *reinterpret_cast<float4*>(v + e) = *reinterpret_cast<const float4*>(&sm.v[j][8 * e + 4 * tx]);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        // a key that the row does not see must not reach it, whatever it holds
        if (k0 + j > pos[i]) continue;
#pragma unroll
        for (int e = 0; e < D / 8; ++e) acc[i][e] = fmaf(w[i], v[e], acc[i][e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float sum = l[i];
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
    const int m = ty * R + i;
    if (m >= n_rows) continue;
    T* o = reinterpret_cast<T*>(a.O) +
           ((int64_t)(t.row0 + t.first + m / a.g) * a.n_q_heads + h * a.g + m % a.g) * D;
#pragma unroll
    for (int e = 0; e < D / 8; ++e)
      o[8 * (e & ~3) + 4 * tx + (e & 3)] = (T)(acc[i][e] / sum);
  }
}

template <int D, int R>
cudaError_t launch_prompt_simt_t(const PromptArgs& a, const PromptTable& p, cudaStream_t s) {
  const int smem = (int)sizeof(Smem<D, R>);
  const cudaError_t e =
      set_dyn_smem_once(reinterpret_cast<const void*>(prompt_simt_kernel<float, D, R>), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(prompt_simt_kernel<float, D, R>, dim3(p.n_tiles * a.n_kv_heads), dim3(kThreads),
                    smem, s, a, p);
}

template <int D>
cudaError_t launch_prompt_simt_d(int r, const PromptArgs& a, const PromptTable& p, cudaStream_t s) {
  return r == 4 ? launch_prompt_simt_t<D, 4>(a, p, s)
                : r == 2 ? launch_prompt_simt_t<D, 2>(a, p, s) : launch_prompt_simt_t<D, 1>(a, p, s);
}

// Rows of a thread of the CUDA-core kernel.  Four reuse each key most, but a
// request of n rows is a chain of n / 32 steps of 3-4 us: four where they leave
// two tiles for every SM (8 requests of 700 rows, 4 / 2 heads of 64: 132 us, with
// two 164; 8 of 300: 49 and 43), else two where they leave half a tile (one of 700:
// 93, 65 and, with one, 72), else one (one of 50: 11.8, 8.1 and 7.7).
int simt_rows(const std::vector<std::pair<int32_t, int32_t>>& rows, const fuse_layer_desc_t& d, int sms) {
  const int g = d.n_q_heads / d.n_kv_heads;
  auto tiles = [&](int r) {
    int64_t n = 0;
    for (const auto& q : rows) n += (q.second + 16 * r / g - 1) / (16 * r / g);
    return n * d.n_kv_heads;
  };
  return tiles(4) >= 2 * sms ? 4 : 2 * tiles(2) >= sms ? 2 : 1;
}

// A table of requests (row0, len), longest first.
fuse_status_t make_table(const std::pair<int32_t, int32_t>* r, int n, int rtile, PromptTable* p) {
  p->n_req = n;
  int64_t at = 0;
  for (int j = 0; j < n; ++j) {
    const int32_t mine = (r[j].second + rtile - 1) / rtile;
    const int64_t next = j + 1 < n ? (r[j + 1].second + rtile - 1) / rtile : 0;
    p->req[j] = {(int32_t)at, r[j].first, r[j].second, mine,
                 (uint32_t)((((uint64_t)1 << 32) + j) / (j + 1)), 0};
    at += (mine - next) * (j + 1);
    if (at > kMaxUnits) return FUSE_ERR_UNSUPPORTED;
  }
  p->n_tiles = (int32_t)at;
  p->req[n] = {p->n_tiles, 0, 0, 0, 0, 0};
  return FUSE_OK;
}

fuse_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? FUSE_OK : FUSE_ERR_CUDA; }

}  // namespace

cudaError_t launch_prompt_simt(const fuse_layer_desc_t& d, int r, const PromptTable& p, const void* Q,
                               const void* K, const void* V, void* O, cudaStream_t s) {
  const PromptArgs a{Q, K, V, O, d.n_q_heads, d.n_kv_heads, d.n_q_heads / d.n_kv_heads,
                     1.4426950408889634f / std::sqrt((float)d.head_dim)};
  return d.head_dim == 128 ? launch_prompt_simt_d<128>(r, a, p, s) : launch_prompt_simt_d<64>(r, a, p, s);
}

}  // namespace fusekv

using namespace fusekv;

extern "C" fuse_status_t fuse_attend_prompt(const fuse_layer_desc_t* desc,
                                            const fuse_requests_t* reqs, const void* Q,
                                            const void* K, const void* V, void* O, void* ws,
                                            size_t ws_bytes, fuse_stream_t stream) {
  fuse_status_t st = check_desc(desc);
  if (st != FUSE_OK) return st;
  ReqInfo info;
  st = check_reqs(reqs, &info);
  if (st != FUSE_OK) return st;
  if (reqs->n_req > 0 && !info.sorted) return FUSE_ERR_INVALID_ARG;
  if (info.tot.max_tok > 0 && (!Q || !K || !V || !O)) return FUSE_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return FUSE_ERR_MISALIGNED;
  st = check_ws(ws, ws_bytes, sizeof(WsHeader));
  if (st != FUSE_OK) return st;
  std::vector<std::pair<int32_t, int32_t>> rows;
  try {
    rows.reserve(reqs->n_req);
  } catch (...) {
    return FUSE_ERR_INVALID_ARG;
  }
  for (int i = 0; i < reqs->n_req; ++i) {
    const fuse_request_t& q = reqs->h_req[i];
    if (q.n_ctx + q.n_query > 0) rows.emplace_back((int32_t)q.row0, q.n_ctx + q.n_query);
  }
  std::stable_sort(rows.begin(), rows.end(), [](auto& x, auto& y) { return x.second > y.second; });
  cudaStream_t s = (cudaStream_t)stream;
  if (rows.empty()) return FUSE_OK;
  const bool tc = prompt_tc_supported(*desc);
  if (!tc && desc->dtype != FUSE_F32) return FUSE_ERR_UNSUPPORTED;   // no tensor maps: no driver
  int dev = 0, sms = 1;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int r = tc ? 0 : simt_rows(rows, *desc, sms);
  const int rtile = (tc ? 128 : 16 * r) / (desc->n_q_heads / desc->n_kv_heads);
  for (size_t r0 = 0; r0 < rows.size(); r0 += kPromptBatch) {
    PromptTable p;
    st = make_table(rows.data() + r0, (int)std::min<size_t>(kPromptBatch, rows.size() - r0),
                    rtile, &p);
    if (st != FUSE_OK) return st;
    if ((int64_t)p.n_tiles * desc->n_kv_heads > kMaxUnits) return FUSE_ERR_UNSUPPORTED;
    st = cuda_status(traced(tc ? "attend_prompt_tc" : "attend_prompt_simt", s, [&] {
      return tc ? launch_prompt_tc(*desc, p, info.tot.n_tok, Q, K, V, O,
                                   reinterpret_cast<uint32_t*>(ws), s)
                : launch_prompt_simt(*desc, r, p, Q, K, V, O, s);
    }));
    if (st != FUSE_OK) return st;
  }
  return FUSE_OK;
}
