// Rotating new rows and writing them to their pages (fuse_cache_append), and
// keeping the accepted ones of a tree (fuse_cache_keep).
//
// KVBoost (section 3.1, Eq. 3): pair m of a head at position p turns by the
// angle p theta_m.  A turn's fraction is exact: theta_m / 2 pi is given as a
// 64-bit fraction f, and p f mod 2^64 is the fraction of p theta_m / 2 pi whatever
// p is (positions are whole numbers, so whole turns drop out of the product).
// Its upper 32 bits, as a signed number, give sincospi its argument with an
// error of 2^-25 turns.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "cache_seqs.cuh"
#include "launch.h"
#include "trace.h"

namespace fusekv {

namespace {

struct Turns {
  uint64_t f[kMaxHalfDim];                // theta' / 2 pi as a fraction of 2^64
};

struct AppendArgs {
  SeqArgs seq;
  const int32_t* parents;
  const void *Q, *K, *V;
  int64_t q_stride, k_stride, v_stride;   // elements
  void *Qr, *Kr, *k_pool, *v_pool;
  int n_q_heads, n_kv_heads;              // n_q_heads: 0 without Q
  int rot, interleaved;
  float mscale;
  int rows_cta;                           // rows of a CTA
  int units;                              // units of 16 channels of a row
  uint32_t units_inv;                     // ceil(2^32 / units)
};

constexpr int kThreads = 256;
constexpr int kMaxRows = 8;               // rows of a CTA at most
constexpr int kAhead = 2;                 // units that a thread reads at a time

// 8 consecutive elements: two registers of 16 bytes for fp32, one for bf16.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};
template <> struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = bf16_lo(a.x); x[1] = bf16_hi(a.x); x[2] = bf16_lo(a.y); x[3] = bf16_hi(a.y);
    x[4] = bf16_lo(a.z); x[5] = bf16_hi(a.z); x[6] = bf16_lo(a.w); x[7] = bf16_hi(a.w);
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7]));
  }
};

// What a CTA knows of its rows.
struct RowPlace {
  int64_t pool;                           // pool row, -1: not written
  int row;                                // -1: no sequence's
  int pos;
};

// Position and pool row of new row `row`, by a whole warp.
__device__ __forceinline__ RowPlace place_row(const AppendArgs& a, int row) {
  const int lane = threadIdx.x % 32;
  RowPlace p{-1, -1, 0};
  const int s = seq_of_row(a.seq.rows, a.seq.n_seq, row);
  if (s < 0 || s >= a.seq.n_seq) return p;
  Seq q;
  if (!seq_of(a.seq, s, &q) || row < q.row0 || row >= q.row0 + q.n) return p;
  const int i = row - q.row0;
  int depth = i;
  if (a.parents) {
    // lanes hold the parents of the first 32 new tokens and of the others
    int up0 = -1, up1 = -1;
    if (lane <= i) up0 = parent_of(a.parents, q, lane, a.seq.err);
    if (lane + 32 <= i) up1 = parent_of(a.parents, q, lane + 32, a.seq.err);
    depth = 0;
    for (int j = i;;) {
      const int lo = __shfl_sync(0xffffffffu, up0, j & 31), hi = __shfl_sync(0xffffffffu, up1, j & 31);
      j = j < 32 ? lo : hi;
      if (j < 0) break;
      ++depth;
    }
  }
  p.row = row;
  p.pos = q.len + depth;
  p.pool = pool_row(a.seq, s, q.len + i);
  return p;
}

// One unit: 16 channels of a head, two runs of 8 (apart by half the rotated
// channels in the half layout).  A CTA takes rows_cta rows; memory bounds it on
// prompts, the chain of reads in front of the angles on single tokens, so a
// thread's first units are read before that chain.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ Turns turns) {
  __shared__ RowPlace s_row[kMaxRows];
  __shared__ float2 s_cs[kMaxRows][kMaxHalfDim];
  constexpr int kPer = D / 16;            // units of a head
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int row0 = blockIdx.x * a.rows_cta;
  const int n_rows = (int)min((int64_t)a.rows_cta, a.seq.n_rows - row0);
  const int total = n_rows * a.units;
  pdl_wait();
  pdl_trigger();

  struct Unit {
    const T* src;
    int r, head, e0, e1, m;               // m: first pair, -1: copied
    int kind;                             // 0: Q, 1: K, 2: V
  };
  auto unit = [&](int x) {
    Unit u;
    u.r = __umulhi((uint32_t)x, a.units_inv);
    const int y = x - u.r * a.units;
    const int h = y / kPer, c = y % kPer;
    u.kind = h < a.n_q_heads ? 0 : h < a.n_q_heads + a.n_kv_heads ? 1 : 2;
    u.head = u.kind == 0 ? h : u.kind == 1 ? h - a.n_q_heads : h - a.n_q_heads - a.n_kv_heads;
    const int64_t row = row0 + u.r;
    u.src = u.kind == 0   ? reinterpret_cast<const T*>(a.Q) + row * a.q_stride
            : u.kind == 1 ? reinterpret_cast<const T*>(a.K) + row * a.k_stride
                          : reinterpret_cast<const T*>(a.V) + row * a.v_stride;
    u.src += u.head * D;
    u.e0 = 16 * c;
    u.e1 = u.e0 + 8;
    u.m = -1;
    if (u.kind < 2 && u.e0 < a.rot) {
      u.m = 8 * c;
      if (!a.interleaved) {
        u.e0 = u.m;
        u.e1 = u.m + a.rot / 2;
      }
    }
    return u;
  };
  Raw8<T> x[kAhead][2];
  auto read = [&](int base) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = base + k * kThreads + tid;
      if (i < total) {
        const Unit u = unit(i);
        x[k][0].load(u.src + u.e0);
        x[k][1].load(u.src + u.e1);
      }
    }
  };
  read(0);
  for (int r = warp; r < n_rows; r += kThreads / 32) {
    const RowPlace p = place_row(a, row0 + r);
    if (lane == 0) s_row[r] = p;
    for (int m = lane; m < a.rot / 2; m += 32) {
      const uint64_t t = (uint64_t)(uint32_t)p.pos * turns.f[m];
      float c, sn;
      sincospif((float)(int32_t)(t >> 32) * (1.f / 2147483648.f), &sn, &c);
      s_cs[r][m] = make_float2(c * a.mscale, sn * a.mscale);
    }
  }
  __syncthreads();
  for (int base = 0; base < total; base += kAhead * kThreads) {
    if (base > 0) read(base);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = base + k * kThreads + tid;
      if (i >= total) continue;
      const Unit u = unit(i);
      const RowPlace p = s_row[u.r];
      if (p.row < 0) continue;
      if (u.m >= 0) {
        float y[8], z[8];
        x[k][0].get(y);
        x[k][1].get(z);
        const float2* cs = s_cs[u.r] + u.m;
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 w = cs[e], v = cs[4 + e];
            const float y0 = y[2 * e], z0 = z[2 * e];
            y[2 * e] = y0 * w.x - y[2 * e + 1] * w.y;
            y[2 * e + 1] = y[2 * e + 1] * w.x + y0 * w.y;
            z[2 * e] = z0 * v.x - z[2 * e + 1] * v.y;
            z[2 * e + 1] = z[2 * e + 1] * v.x + z0 * v.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 w = cs[e];
            const float y0 = y[e];
            y[e] = y0 * w.x - z[e] * w.y;
            z[e] = z[e] * w.x + y0 * w.y;
          }
        }
        x[k][0].set(y);
        x[k][1].set(z);
      }
      if (u.kind < 2) {
        T* out = reinterpret_cast<T*>(u.kind == 0 ? a.Qr : a.Kr);
        if (out) {
          out += ((int64_t)p.row * (u.kind == 0 ? a.n_q_heads : a.n_kv_heads) + u.head) * D;
          x[k][0].store(out + u.e0);
          x[k][1].store(out + u.e1);
        }
      }
      if (u.kind > 0 && p.pool >= 0) {
        T* out = reinterpret_cast<T*>(u.kind == 1 ? a.k_pool : a.v_pool) +
                 (p.pool * a.n_kv_heads + u.head) * D;
        x[k][0].store(out + u.e0);
        x[k][1].store(out + u.e1);
      }
    }
  }
}

// ---- keep --------------------------------------------------------------------

constexpr int kMaxPools = 64;             // pools of a launch (parameter space)
constexpr int kKeepThreads = 128;
constexpr int kBatch = 4;                 // rows that a thread reads at a time

struct KeepArgs {
  SeqArgs seq;
  const int32_t* path;
  const int32_t* count;
  int32_t max_path;
  int32_t row_bytes;                      // of a token's K (or V)
  char* pool[2 * kMaxPools];              // k, v of each
};

// A sequence's path: whether it can be kept (by a whole block; s_row receives
// the pool rows of the nodes and of the slots that they go to).
__device__ __forceinline__ int kept(const KeepArgs& a, int s, int64_t (*s_row)[2]) {
  Seq q;
  const bool ok = seq_of(a.seq, s, &q);
  const int n = a.count[s];
  bool bad = !ok || n < 0 || n > a.max_path || n > q.n;
  if (!bad && (int)threadIdx.x < n) {
    const int i = threadIdx.x;
    const int32_t* path = a.path + (int64_t)s * a.max_path;
    const int p = path[i], before = i > 0 ? path[i - 1] : -1;
    bad = p <= before || p < 0 || p >= q.n;
    if (!bad) {
      s_row[i][0] = pool_row(a.seq, s, q.len + p);
      s_row[i][1] = p == i ? s_row[i][0] : pool_row(a.seq, s, q.len + i);
      if (s_row[i][0] < 0 || s_row[i][1] < 0) bad = true;
    }
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && ok) report_error(a.seq.err, FUSE_ERR_DEVICE_BOUNDS, SITE_KEEP_PATH, (uint32_t)s);
    return 0;
  }
  return n;
}

// A CTA: one sequence in one pool's keys or values.  path[i] >= i, so a thread
// that takes a column of 16 bytes through the rows in order reads each before
// it is written over.
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const __grid_constant__ KeepArgs a) {
  __shared__ int64_t s_row[FUSE_TREE_MAX_NEW][2];
  static_assert(FUSE_TREE_MAX_NEW <= kKeepThreads, "a thread a path entry");
  pdl_wait();
  pdl_trigger();
  const int n = kept(a, blockIdx.x, s_row);
  char* pool = a.pool[blockIdx.y];
  for (int c = threadIdx.x * 16; c < a.row_bytes; c += kKeepThreads * 16) {
    for (int i = 0; i < n; i += kBatch) {
      uint4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (i + k < n) x[k] = *reinterpret_cast<const uint4*>(pool + s_row[i + k][0] * a.row_bytes + c);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (i + k < n && s_row[i + k][0] != s_row[i + k][1])
          *reinterpret_cast<uint4*>(pool + s_row[i + k][1] * a.row_bytes + c) = x[k];
    }
  }
}

// The lengths, once every CTA of the copies has read them.
__global__ void __launch_bounds__(FUSE_TREE_MAX_NEW) keep_lens_kernel(const __grid_constant__ KeepArgs a) {
  __shared__ int64_t s_row[FUSE_TREE_MAX_NEW][2];
  pdl_wait();
  pdl_trigger();
  const int n = kept(a, blockIdx.x, s_row);
  if (threadIdx.x == 0 && n > 0) a.seq.lens[blockIdx.x] += n;
}

// ---- host side ---------------------------------------------------------------

fuse_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? FUSE_OK : FUSE_ERR_CUDA; }

fuse_status_t check_rope(const fuse_rope_t* r, int head_dim, int* rot) {
  if (!r) return FUSE_ERR_INVALID_ARG;
  if (r->layout != FUSE_ROPE_HALF && r->layout != FUSE_ROPE_INTERLEAVED) return FUSE_ERR_INVALID_ARG;
  *rot = r->rot_dim == 0 ? head_dim : r->rot_dim;
  if (*rot < 0 || *rot > head_dim) return FUSE_ERR_INVALID_ARG;
  if (*rot % 16 != 0) return FUSE_ERR_UNSUPPORTED;
  if (!(r->mscale > 0.0) || !std::isfinite(r->mscale)) return FUSE_ERR_INVALID_ARG;
  if (r->scaling < FUSE_ROPE_PLAIN || r->scaling > FUSE_ROPE_YARN) return FUSE_ERR_INVALID_ARG;
  if (r->scaling == FUSE_ROPE_PLAIN) return FUSE_OK;
  if (!(r->factor >= 1.0) || !std::isfinite(r->factor)) return FUSE_ERR_INVALID_ARG;
  if (r->scaling == FUSE_ROPE_LINEAR) return FUSE_OK;
  if (r->original_len <= 0 || !(r->low > 0.0) || !(r->high > r->low) || !std::isfinite(r->high))
    return FUSE_ERR_INVALID_ARG;
  return FUSE_OK;
}

// The scaled frequencies as fractions of a turn (kept per thread: a power per pair).
const Turns& make_turns(double base, const fuse_rope_t& r, int rot) {
  static thread_local Turns t;
  static thread_local double of_base = 0.0;
  static thread_local fuse_rope_t of;
  static thread_local int of_rot = -1;
  if (of_base == base && of_rot == rot && of.scaling == r.scaling && of.original_len == r.original_len &&
      of.factor == r.factor && of.low == r.low && of.high == r.high)
    return t;
  of_base = base;
  of = r;
  of_rot = rot;
  std::memset(&t, 0, sizeof(t));
  const double two_pi = 6.283185307179586476925286766559;
  double a = 0.0, b = 1.0;
  if (r.scaling == FUSE_ROPE_YARN) {
    auto at = [&](double x) { return rot * std::log(r.original_len / (x * two_pi)) / (2.0 * std::log(base)); };
    a = std::max(0.0, std::floor(at(r.high)));
    b = std::min(rot - 1.0, std::ceil(at(r.low)));
  }
  for (int m = 0; m < rot / 2; ++m) {
    double theta = std::pow(base, -2.0 * m / (double)rot);
    if (r.scaling == FUSE_ROPE_LINEAR) {
      theta /= r.factor;
    } else if (r.scaling == FUSE_ROPE_LLAMA3) {
      const double c = std::min(1.0, std::max(0.0, (r.original_len * theta / two_pi - r.low) / (r.high - r.low)));
      theta = (1.0 - c) * theta / r.factor + c * theta;
    } else if (r.scaling == FUSE_ROPE_YARN) {
      const double ramp = std::min(1.0, std::max(0.0, (m - a) / std::max(b - a, 0.001)));
      theta = (1.0 - ramp) * theta + ramp * theta / r.factor;
    }
    t.f[m] = (uint64_t)std::ldexp(theta / two_pi, 64);      // theta <= 1: below 2^62
  }
  return t;
}

template <typename T>
cudaError_t launch_append(const AppendArgs& a, const Turns& t, int head_dim, int grid, cudaStream_t s) {
  return head_dim == 128 ? launch_pdl(append_kernel<T, 128>, dim3(grid), dim3(kThreads), 0, s, a, t)
                         : launch_pdl(append_kernel<T, 64>, dim3(grid), dim3(kThreads), 0, s, a, t);
}

}  // namespace

fuse_status_t check_seqs(const fuse_seqs_t* q, int64_t n_rows, int max_new, SeqArgs* a, void* ws) {
  if (!q || q->n_seq < 0 || n_rows < 0) return FUSE_ERR_INVALID_ARG;
  if (q->n_seq > 65535 || n_rows > INT32_MAX) return FUSE_ERR_UNSUPPORTED;
  if (q->block_size <= 0 || q->max_blocks <= 0 || q->max_new <= 0 || q->n_pool_blocks <= 0)
    return FUSE_ERR_INVALID_ARG;
  if (q->max_new > max_new) return FUSE_ERR_UNSUPPORTED;
  // slots and pool rows are 32-bit numbers
  if ((int64_t)q->max_blocks * q->block_size > INT32_MAX || q->n_pool_blocks > INT32_MAX / q->block_size)
    return FUSE_ERR_UNSUPPORTED;
  if (q->n_seq > 0 && (!q->tables || !q->lens || !q->rows)) return FUSE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q->tables) | reinterpret_cast<uintptr_t>(q->lens) |
       reinterpret_cast<uintptr_t>(q->rows)) & 3u)
    return FUSE_ERR_MISALIGNED;
  a->tables = q->tables;
  a->lens = q->lens;
  a->rows = q->rows;
  a->n_seq = q->n_seq;
  a->block_size = q->block_size;
  a->max_blocks = q->max_blocks;
  a->max_new = q->max_new;
  a->block_inv = q->block_size > 1 ? (uint32_t)((((uint64_t)1 << 32) + q->block_size - 1) / q->block_size) : 0;
  a->n_pool_blocks = q->n_pool_blocks;
  a->n_rows = n_rows;
  a->err = reinterpret_cast<uint32_t*>(ws);
  return FUSE_OK;
}

}  // namespace fusekv

using namespace fusekv;

extern "C" {

fuse_status_t fuse_cache_append(const fuse_layer_desc_t* desc, const fuse_rope_t* rope,
                                const fuse_seqs_t* seqs, int64_t n_rows, const int32_t* parents,
                                const fuse_append_t* io, void* ws, size_t ws_bytes,
                                fuse_stream_t stream) {
  fuse_status_t st = check_desc(desc);
  if (st != FUSE_OK) return st;
  int rot = 0;
  st = check_rope(rope, desc->head_dim, &rot);
  if (st != FUSE_OK) return st;
  AppendArgs a;
  st = check_seqs(seqs, n_rows, parents ? FUSE_TREE_MAX_NEW : INT32_MAX, &a.seq, ws);
  if (st != FUSE_OK) return st;
  if (!io) return FUSE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(parents) & 3u) return FUSE_ERR_MISALIGNED;
  if (n_rows > 0 && (!io->K || !io->V || !io->k_pool || !io->v_pool || (io->Q != nullptr) != (io->Qr != nullptr)))
    return FUSE_ERR_INVALID_ARG;
  for (const void* p : {io->Q, io->K, io->V, (const void*)io->Qr, (const void*)io->Kr, (const void*)io->k_pool,
                        (const void*)io->v_pool})
    if (!aligned16(p)) return FUSE_ERR_MISALIGNED;
  const int d = desc->head_dim, per16 = 16 / (int)elem_size(desc->dtype);
  const int64_t kv = (int64_t)desc->n_kv_heads * d;
  if ((io->Q && io->q_stride < (int64_t)desc->n_q_heads * d) || io->k_stride < kv || io->v_stride < kv)
    return FUSE_ERR_INVALID_ARG;
  if ((io->Q && io->q_stride % per16) || io->k_stride % per16 || io->v_stride % per16)
    return FUSE_ERR_MISALIGNED;
  st = check_ws(ws, ws_bytes, FUSE_CACHE_WORKSPACE);
  if (st != FUSE_OK) return st;
  if (n_rows == 0 || seqs->n_seq == 0) return FUSE_OK;
  a.parents = parents;
  a.Q = io->Q;
  a.K = io->K;
  a.V = io->V;
  a.q_stride = io->q_stride;
  a.k_stride = io->k_stride;
  a.v_stride = io->v_stride;
  a.Qr = io->Qr;
  a.Kr = io->Kr;
  a.k_pool = io->k_pool;
  a.v_pool = io->v_pool;
  a.n_q_heads = io->Q ? desc->n_q_heads : 0;
  a.n_kv_heads = desc->n_kv_heads;
  a.rot = rot;
  a.interleaved = rope->layout == FUSE_ROPE_INTERLEAVED;
  a.mscale = (float)rope->mscale;
  const int64_t units = ((int64_t)a.n_q_heads + 2 * a.n_kv_heads) * (d / 16);
  if (units > 16384) return FUSE_ERR_UNSUPPORTED;         // units_inv is exact for kMaxRows rows of so many
  a.units = (int)units;
  a.units_inv = (uint32_t)((((uint64_t)1 << 32) + units - 1) / units);
  int dev = 0, sms = 1;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // a CTA takes several rows once the card holds no more CTAs at a time
  a.rows_cta = (int)std::min<int64_t>(kMaxRows, std::max<int64_t>(1, n_rows / (sms * 8)));
  const int grid = (int)((n_rows + a.rows_cta - 1) / a.rows_cta);
  const Turns& t = make_turns(desc->rope_base, *rope, rot);
  cudaStream_t s = (cudaStream_t)stream;
  return cuda_status(traced("cache_append", s, [&] {
    return desc->dtype == FUSE_BF16 ? launch_append<__nv_bfloat16>(a, t, d, grid, s)
                                    : launch_append<float>(a, t, d, grid, s);
  }));
}

fuse_status_t fuse_cache_keep(const fuse_layer_desc_t* desc, const fuse_pools_t* pools,
                              const fuse_seqs_t* seqs, const int32_t* path, int32_t max_path,
                              const int32_t* count, void* ws, size_t ws_bytes,
                              fuse_stream_t stream) {
  fuse_status_t st = check_desc(desc);
  if (st != FUSE_OK) return st;
  KeepArgs a;
  st = check_seqs(seqs, INT32_MAX, FUSE_TREE_MAX_NEW, &a.seq, ws);
  if (st != FUSE_OK) return st;
  if (!pools || pools->n_pools < 0 || pools->reserved != 0) return FUSE_ERR_INVALID_ARG;
  if (pools->kv_storage != desc->dtype) return FUSE_ERR_UNSUPPORTED;
  if (pools->block_size != seqs->block_size || pools->n_blocks != seqs->n_pool_blocks)
    return FUSE_ERR_INVALID_ARG;
  if (pools->n_pools > 0 && !pools->h_pools) return FUSE_ERR_INVALID_ARG;
  for (int i = 0; i < pools->n_pools; ++i) {
    if (!pools->h_pools[i].k || !pools->h_pools[i].v) return FUSE_ERR_INVALID_ARG;
    if (!aligned16(pools->h_pools[i].k) || !aligned16(pools->h_pools[i].v)) return FUSE_ERR_MISALIGNED;
  }
  if (max_path < 1) return FUSE_ERR_INVALID_ARG;
  if (max_path > FUSE_TREE_MAX_NEW) return FUSE_ERR_UNSUPPORTED;
  if (seqs->n_seq > 0 && (!path || !count)) return FUSE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(path) | reinterpret_cast<uintptr_t>(count)) & 3u) return FUSE_ERR_MISALIGNED;
  st = check_ws(ws, ws_bytes, FUSE_CACHE_WORKSPACE);
  if (st != FUSE_OK) return st;
  const int64_t row = (int64_t)desc->n_kv_heads * desc->head_dim * (int64_t)elem_size(desc->dtype);
  if (row > INT32_MAX) return FUSE_ERR_UNSUPPORTED;
  if (seqs->n_seq == 0) return FUSE_OK;
  a.path = path;
  a.count = count;
  a.max_path = max_path;
  a.row_bytes = (int32_t)row;
  cudaStream_t s = (cudaStream_t)stream;
  for (int p0 = 0; p0 < pools->n_pools; p0 += kMaxPools) {
    const int n = std::min(kMaxPools, pools->n_pools - p0);
    for (int i = 0; i < n; ++i) {
      a.pool[2 * i] = reinterpret_cast<char*>(pools->h_pools[p0 + i].k);
      a.pool[2 * i + 1] = reinterpret_cast<char*>(pools->h_pools[p0 + i].v);
    }
    st = cuda_status(traced("cache_keep", s, [&] {
      return launch_pdl(keep_kernel, dim3(seqs->n_seq, 2 * n), dim3(kKeepThreads), 0, s, a);
    }));
    if (st != FUSE_OK) return st;
  }
  st = cuda_status(traced("cache_keep_lens", s, [&] {
    return launch_pdl(keep_lens_kernel, dim3(seqs->n_seq), dim3(FUSE_TREE_MAX_NEW), 0, s, a);
  }));
  if (st != FUSE_OK) return st;
  return FUSE_OK;
}

}  // extern "C"
