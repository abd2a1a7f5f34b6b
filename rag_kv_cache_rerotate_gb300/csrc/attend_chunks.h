// Plan and device tables of the attention over chunk caches, shared by its
// CUDA-core and matrix-instruction kernels.
#pragma once

#include "common.cuh"

namespace fusekv {

constexpr int kVecs = 8;                  // query vectors (new token, query head) of an item
constexpr int kItemWarps = 4;             // items of a CTA, a warp each
constexpr int kReqBatch = 128;            // requests of a join's launch (parameter space)
constexpr int kChunkBatch = 512;          // chunks of an items' launch
constexpr int kSideBatch = 256;           // requests whose side rows it takes
constexpr int kSegBatch = 65535;          // segments of either (16-bit starts; one chunk or request has at most 2^24 / 1024 + 3)

// How the keys of a call are cut.  A chunk's tokens are cut into segments of
// seg tokens, a request's side rows into segments of sseg rows, each of them
// into as many as it needs; an item is one segment, KV head and group of kVecs
// query vectors.  Each item leaves the softmax of its keys unnormalised, with
// its maximum and sum, in the partial slot (segment, head, group); segments are
// counted over the chunks, then over the requests.
struct AttendPlan {
  int seg, sseg;
  int nvg;                                // groups of kVecs query vectors per KV head
  int64_t slots;                          // segments in all
  size_t part_o, part_ml, total;          // workspace regions
};

struct AttendArgs {
  const fuse_chunk_t* chunks;
  const fuse_request_t* reqs;
  const void* Q;
  const int32_t* idx;
  const void* Ks;
  const void* Vs;
  void* O;
  float* part_o;                          // [slot][head][group][vector][d], fp32
  float2* part_ml;                        // [slot][head][group][vector]: maximum (log2), sum
  uint32_t* err;
  int64_t n_pool_blocks;
  int n_q_heads, n_kv_heads, g;           // g = n_q_heads / n_kv_heads
  int n_new, nvg;
  int seg, sseg;
  int block_size;                         // 0: contiguous chunks
  float scale;                            // log2(e) / sqrt(d)
  int chunk0, n_chunks;                   // an items' launch: its chunks
  int chunk_slot0, chunk_ctas;            // their first segment, their CTAs
  int req0, n_req;                        // the requests whose side rows it takes; a join's requests
  int side_slot0;                         // their first segment
  float chunk_inv, side_inv;              // chunks (requests) per segment
};

// An items' launch, by value: reading it costs no trip to HBM.  The request of
// each chunk, and the first segment of each chunk and of each request's side
// rows, counted from the launch's first (the last: their number).
struct ItemTable {
  uint16_t owner[kChunkBatch];
  uint16_t seg[kChunkBatch + 1];
  uint16_t side[kSideBatch + 1];
};
// First segment of the chunks and of the side rows of each request of a join
// (and of the one after the last).
struct JoinTable {
  int32_t seg[kReqBatch + 1];
  int32_t side[kReqBatch + 1];
};

// The part of n that segment x < start[n] lies in; inv = n / start[n], with which
// parts of about the same length are found at the first look.
__device__ __forceinline__ int part_of(const uint16_t* start, int n, float inv, int x) {
  int i = min(n - 1, (int)((x + 0.5f) * inv));
  if (start[i] <= x && x < start[i + 1]) return i;
  int end = n;
  i = 0;
  while (end - i > 1) {                   // start[i] <= x < start[end]
    const int m = (i + end) / 2;
    if (start[m] <= x)
      i = m;
    else
      end = m;
  }
  return i;
}

// Where the calling warp's item is, its keys apart.  A chunk's segments fill
// whole CTAs (empty ones after its end if need be), so the warps of a CTA
// share the chunk.
struct ItemPlace {
  bool side, none;                        // none: a warp past the launch's last side item
  int part;                               // chunk or request, counted from the launch's first
  int seg;                                // segment within it
  int h, vg;
  int slot;                               // segment of the call
};
__device__ __forceinline__ ItemPlace item_place(const AttendArgs& a, const ItemTable& t) {
  ItemPlace p;
  const int per_seg = a.n_kv_heads * a.nvg;
  const int b = (int)blockIdx.x - a.chunk_ctas;
  p.side = b >= 0;
  const int i = (p.side ? b : (int)blockIdx.x) * kItemWarps + (int)threadIdx.x / 32;
  const int seg = i / per_seg;
  p.h = i % per_seg / a.nvg;
  p.vg = i % a.nvg;
  p.none = p.side && seg >= t.side[a.n_req];
  p.part = p.seg = 0;
  if (!p.side) {
    p.part = part_of(t.seg, a.n_chunks, a.chunk_inv, seg);
    p.seg = seg - t.seg[p.part];
  } else if (!p.none) {
    p.part = part_of(t.side, a.n_req, a.side_inv, seg);
    p.seg = seg - t.side[p.part];
  }
  p.slot = (p.side ? a.side_slot0 : a.chunk_slot0) + seg;
  return p;
}
// An item without a key: the join passes it over.
__device__ __forceinline__ void no_keys(const AttendArgs& a, const ItemPlace& p) {
  const int lane = threadIdx.x % 32;
  if (lane < kVecs)
    a.part_ml[(((int64_t)p.slot * a.n_kv_heads + p.h) * a.nvg + p.vg) * kVecs + lane] =
        make_float2(-INFINITY, 0.f);
}

// The items' kernels.  fp32 layers.
cudaError_t launch_attend_simt(const fuse_layer_desc_t& d, int kv_storage, const AttendArgs& a,
                               const ItemTable& t, const RopeFreqs& freqs, cudaStream_t s);
// The same for bf16 layers, on matrix instructions (attend_chunks_mma.cu).
cudaError_t launch_attend_mma(const fuse_layer_desc_t& d, int kv_storage, const AttendArgs& a,
                              const ItemTable& t, const RopeFreqs& freqs, cudaStream_t s);
// CTAs of an items' launch.
inline int64_t item_ctas(const AttendArgs& a, const ItemTable& t) {
  const int64_t side = (int64_t)t.side[a.n_req] * a.n_kv_heads * a.nvg;
  return a.chunk_ctas + (side + kItemWarps - 1) / kItemWarps;
}
// early: the kernel before it in the stream is one of the above (or a join).
cudaError_t launch_attend_combine(const fuse_layer_desc_t& d, const AttendArgs& a,
                                  const JoinTable& t, bool early, cudaStream_t s);

}  // namespace fusekv
