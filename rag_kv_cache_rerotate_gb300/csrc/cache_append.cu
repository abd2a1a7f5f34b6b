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
  int parts, parts_log2;                  // warps that share a row, a power of two
};

constexpr int kThreads = 128;
constexpr int kAhead = 3;                 // units that a lane reads at a time

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

// What a warp knows of its row.
struct RowPlace {
  int64_t pool;                           // pool row, -1: not written
  int row;                                // -1: no sequence's
  int pos;
};

// The sequence of new row `row`, by a whole warp; false where it has none.  Up to 128
// sequences are all read at once, four a lane, so that one read's latency finds it
// (64 next tokens: 5.7 us, with a search and then a look at what it found 6.0; a prompt
// of 10368: 44 and 49).  Between them the warps look at every sequence, so that a bad one
// is recorded that no row leads to (w: this warp's number).
__device__ __forceinline__ bool find_seq(const SeqArgs& a, int row, int64_t w, int64_t warps, int* s, Seq* q) {
  if (a.n_seq > 128) {
    for (int64_t i = w * 32 + threadIdx.x % 32; i < a.n_seq; i += warps * 32) seq_of(a, (int)i, q);      // (*q: below)
    *s = seq_of_row(a.rows, a.n_seq, row);
    return *s >= 0 && *s < a.n_seq && seq_of(a, *s, q);
  }
  const int s0 = threadIdx.x % 32 * 4;
  int start[5], len[4];
#pragma unroll
  for (int i = 0; i < 5; ++i) start[i] = a.rows[min(s0 + i, a.n_seq)];
#pragma unroll
  for (int i = 0; i < 4; ++i) len[i] = a.lens[min(s0 + i, a.n_seq - 1)];
  int below = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) below += s0 + i < a.n_seq && start[i] <= row;
  *s = __reduce_add_sync(0xffffffffu, below) - 1;
  if (w == 0) {                           // (all of them are here: the first warp checks them)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (s0 + i < a.n_seq) check_seq(a, s0 + i, start[i], start[i + 1], len[i], q);
  }
  if (*s < 0) return false;
  const int k = *s & 3, from = *s >> 2;
  const int r0 = __shfl_sync(0xffffffffu, k == 0 ? start[0] : k == 1 ? start[1] : k == 2 ? start[2] : start[3], from);
  const int r1 = __shfl_sync(0xffffffffu, k == 0 ? start[1] : k == 1 ? start[2] : k == 2 ? start[3] : start[4], from);
  const int l = __shfl_sync(0xffffffffu, k == 0 ? len[0] : k == 1 ? len[1] : k == 2 ? len[2] : len[3], from);
  return check_seq(a, *s, r0, r1, l, q);
}

// Position and pool row of new row `row`, by a whole warp.
__device__ __forceinline__ RowPlace place_row(const AppendArgs& a, int row, int64_t w) {
  const int lane = threadIdx.x % 32;
  RowPlace p{-1, -1, 0};
  int s;
  Seq q;
  if (!find_seq(a.seq, row, w, a.seq.n_rows << a.parts_log2, &s, &q) || row < q.row0 || row >= q.row0 + q.n) return p;
  const int i = row - q.row0;
  // its page and the parents of the new tokens up to it (lanes hold those of the first
  // 32 and of the others): read before any is looked at
  int in_page, up0 = -1, up1 = -1;
  const int page = a.seq.tables[(int64_t)s * a.seq.max_blocks + page_of(a.seq, q.len + i, &in_page)];
  if (a.parents && lane <= i) up0 = a.parents[q.row0 + lane];
  if (a.parents && lane + 32 <= i) up1 = a.parents[q.row0 + lane + 32];
  int depth = i;
  if (a.parents) {
    up0 = checked_parent(up0, q, lane, a.seq.err);
    up1 = checked_parent(up1, q, lane + 32, a.seq.err);
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
  p.pool = checked_page(a.seq, page, in_page);
  return p;
}

// A warp takes a row, or a share of its heads; D / 16 lanes a head, a lane 16 channels of
// it, two runs of 8 (apart by half the rotated channels in the half layout) and of all
// heads the same ones, so that it reads their angles once.  Memory bounds it on prompts
// (10368 rows of 32 query and 8 KV heads, d = 128: 44 us, 5.8 TB/s; a row's angles shared
// by a block of 256 threads, which waits for them, made 52 of 49), the chain of reads
// in front of the angles on single tokens, so the first units are read before that chain.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ Turns turns) {
  constexpr int kPer = D / 16, kHeads = 32 / kPer;         // lanes of a head, heads at a time
  __shared__ float2 s_cs[kThreads / 32][kMaxHalfDim];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + warp;
  const int64_t row = w >> a.parts_log2;
  const int part = (int)w & (a.parts - 1);
  pdl_wait();
  pdl_trigger();
  if (row >= a.seq.n_rows) return;        // uniform in the warp
  const int c = lane % kPer;
  const bool turned = 16 * c < a.rot;     // (of queries and keys)
  const int e0 = turned && !a.interleaved ? 8 * c : 16 * c;
  const int e1 = turned && !a.interleaved ? e0 + a.rot / 2 : e0 + 8;
  const T* q = reinterpret_cast<const T*>(a.Q) + row * a.q_stride;
  const T* k = reinterpret_cast<const T*>(a.K) + row * a.k_stride;
  const T* v = reinterpret_cast<const T*>(a.V) + row * a.v_stride;
  const int heads = a.n_q_heads + 2 * a.n_kv_heads, step = a.parts * kHeads;
  const int first = part * kHeads + lane / kPer;
  Raw8<T> x[kAhead][2];
  // head h's run at e: a value's channels are copied as they lie
  auto read = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * step;
      if (h < heads) {
        const bool value = h >= a.n_q_heads + a.n_kv_heads;
        const T* src = h < a.n_q_heads ? q + h * D : value ? v + (h - a.n_q_heads - a.n_kv_heads) * D
                                                           : k + (h - a.n_q_heads) * D;
        x[i][0].load(src + (value ? 16 * c : e0));
        x[i][1].load(src + (value ? 16 * c + 8 : e1));
      }
    }
  };
  read(first);
  const RowPlace p = place_row(a, (int)row, w);
  if (p.row < 0) return;                  // uniform
  for (int m = lane; m < a.rot / 2; m += 32) {
    const uint64_t t = (uint64_t)(uint32_t)p.pos * turns.f[m];
    float co, si;
    sincospif((float)(int32_t)(t >> 32) * (1.f / 2147483648.f), &si, &co);
    s_cs[warp][m] = make_float2(co * a.mscale, si * a.mscale);
  }
  __syncwarp();
  float2 cs[8];                           // of the lane's pairs
#pragma unroll
  for (int e = 0; e < 8; ++e) cs[e] = turned ? s_cs[warp][8 * c + e] : make_float2(1.f, 0.f);
  T* qr = reinterpret_cast<T*>(a.Qr) + row * a.n_q_heads * D;
  T* kr = a.Kr ? reinterpret_cast<T*>(a.Kr) + row * a.n_kv_heads * D : nullptr;
  T* kp = reinterpret_cast<T*>(a.k_pool) + p.pool * a.n_kv_heads * D;
  T* vp = reinterpret_cast<T*>(a.v_pool) + p.pool * a.n_kv_heads * D;
  for (int h0 = first; h0 < heads; h0 += kAhead * step) {
    if (h0 != first) read(h0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * step;
      if (h >= heads) continue;
      const int hk = h - a.n_q_heads, hv = hk - a.n_kv_heads;
      if (hv >= 0) {
        if (p.pool >= 0) {
          x[i][0].store(vp + hv * D + 16 * c);
          x[i][1].store(vp + hv * D + 16 * c + 8);
        }
        continue;
      }
      if (turned) {
        float y[8], z[8];
        x[i][0].get(y);
        x[i][1].get(z);
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = cs[e], g = cs[4 + e];
            const float y0 = y[2 * e], z0 = z[2 * e];
            y[2 * e] = y0 * f.x - y[2 * e + 1] * f.y;
            y[2 * e + 1] = y[2 * e + 1] * f.x + y0 * f.y;
            z[2 * e] = z0 * g.x - z[2 * e + 1] * g.y;
            z[2 * e + 1] = z[2 * e + 1] * g.x + z0 * g.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float y0 = y[e];
            y[e] = y0 * cs[e].x - z[e] * cs[e].y;
            z[e] = z[e] * cs[e].x + y0 * cs[e].y;
          }
        }
        x[i][0].set(y);
        x[i][1].set(z);
      }
      T* out = hk < 0 ? qr + h * D : kr ? kr + hk * D : nullptr;
      if (out) {
        x[i][0].store(out + e0);
        x[i][1].store(out + e1);
      }
      if (hk >= 0 && p.pool >= 0) {
        x[i][0].store(kp + hk * D + e0);
        x[i][1].store(kp + hk * D + e1);
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
  // (all reads before the first check)
  const int n = a.count[s], i = threadIdx.x;
  const int32_t* path = a.path + (int64_t)s * a.max_path;
  const int p = i < a.max_path ? path[i] : -1, before = i > 0 && i < a.max_path ? path[i - 1] : -1;
  Seq q;
  const bool ok = seq_of(a.seq, s, &q);
  bool bad = !ok || n < 0 || n > a.max_path || n > q.n;
  if (!bad && i < n) {
    bad = p <= before || p < 0 || p >= q.n;
    if (!bad) {
      int at0, at1;
      const int page0 = a.seq.tables[(int64_t)s * a.seq.max_blocks + page_of(a.seq, q.len + p, &at0)];
      const int page1 = a.seq.tables[(int64_t)s * a.seq.max_blocks + page_of(a.seq, q.len + i, &at1)];
      s_row[i][0] = checked_page(a.seq, page0, at0);
      s_row[i][1] = checked_page(a.seq, page1, at1);
      bad = s_row[i][0] < 0 || s_row[i][1] < 0;
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
// it is written over.  Latency bounds it: with the lengths 4 to 5 us behind the copy of a few
// bytes, on one sequence of 32 layers as on 96 of 8.
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

// The lengths, once every CTA of the copies has read them.  (One kernel for both, a cluster a
// sequence, saves 0.2 us on 8 sequences of one layer and takes 3 more on one of 32, 8 on 3 of 80.)
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
  // (a float on the device)
  if (!((float)r->mscale > 0.f) || !std::isfinite((float)r->mscale)) return FUSE_ERR_INVALID_ARG;
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
  // slots and pool rows are 32-bit numbers, up to the end of their tile
  constexpr int64_t kMost = INT32_MAX - 256;
  if ((int64_t)q->max_blocks * q->block_size > kMost || q->n_pool_blocks > kMost / q->block_size)
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
  const int64_t heads = (int64_t)a.n_q_heads + 2 * a.n_kv_heads;
  if (heads > 65535) return FUSE_ERR_UNSUPPORTED;
  int dev = 0, sms = 1;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // a row is shared while the card holds more warps and they have heads to take
  a.parts = 1;
  a.parts_log2 = 0;
  while (n_rows * a.parts < (int64_t)sms * 16 && a.parts * (512 / d) < heads) {
    a.parts *= 2;
    ++a.parts_log2;
  }
  const int64_t ctas = (n_rows * a.parts + kThreads / 32 - 1) / (kThreads / 32);
  const int grid = (int)ctas;
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
    // rows are moved in place: twice is once too often
    bool again = pools->h_pools[i].k == pools->h_pools[i].v;
    for (int j = 0; j < i; ++j)
      again |= pools->h_pools[j].k == pools->h_pools[i].k || pools->h_pools[j].v == pools->h_pools[i].v ||
               pools->h_pools[j].k == pools->h_pools[i].v || pools->h_pools[j].v == pools->h_pools[i].k;
    if (again) return FUSE_ERR_INVALID_ARG;
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
