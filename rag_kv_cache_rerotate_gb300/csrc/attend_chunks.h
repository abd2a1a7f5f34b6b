// Plan and device tables of the attention over chunk caches, shared by its
// CUDA-core and matrix-instruction kernels.
#pragma once

#include "common.cuh"

namespace fusekv {

constexpr int kVecs = 8;                  // query vectors (new token, query head) of an item
constexpr int kReqBatch = 128;            // requests of one launch (parameter space)
constexpr int kChunkBatch = 512;          // chunks of one launch

// How the keys of a call are cut.  A chunk's tokens are cut into nsub
// segments of seg tokens, a request's side rows into nside segments of sseg
// rows; an item is one segment, KV head and group of kVecs query vectors.
// Each item leaves the softmax of its keys unnormalised, with its maximum
// and sum, in the partial slot (segment, head, group).
struct AttendPlan {
  int seg, nsub;
  int sseg, nside;
  int nvg;                                // groups of kVecs query vectors per KV head
  int64_t chunk_slots, slots;             // segments: of chunks, in all
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
  int64_t chunk_slots;
  int n_q_heads, n_kv_heads, g;           // g = n_q_heads / n_kv_heads
  int n_new, nvg;
  int seg, nsub, sseg, nside;
  int block_size;                         // 0: contiguous chunks
  float scale;                            // log2(e) / sqrt(d)
  int req0, n_req;                        // requests of this launch
  int chunk0, n_chunks;                   // chunks of this launch
};

// Request of each chunk of a launch, by value: reading it costs no trip to HBM.
struct ChunkOwners {
  uint16_t req[kChunkBatch];
};
// First chunk of each request of a launch (and of the one after the last).
struct RequestChunks {
  int32_t first[kReqBatch + 1];
};

// The items' kernels; side rows of all requests of the launch come with the
// first batch of chunks (side_reqs requests, 0: none).  fp32 layers.
cudaError_t launch_attend_simt(const fuse_layer_desc_t& d, int kv_storage, const AttendArgs& a,
                               const ChunkOwners& owners, const RopeFreqs& freqs, int side_reqs,
                               cudaStream_t s);
// The same for bf16 layers, on matrix instructions (attend_chunks_mma.cu).
cudaError_t launch_attend_mma(const fuse_layer_desc_t& d, int kv_storage, const AttendArgs& a,
                              const ChunkOwners& owners, const RopeFreqs& freqs, int side_reqs,
                              cudaStream_t s);
// early: the kernel before it in the stream is one of the above (or a join).
cudaError_t launch_attend_combine(const fuse_layer_desc_t& d, const AttendArgs& a,
                                  const RequestChunks& rc, bool early, cudaStream_t s);

}  // namespace fusekv
