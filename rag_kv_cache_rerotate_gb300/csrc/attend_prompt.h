// The work of the packed-prompt attention, by value: which tile of which
// request a unit of work is, without a device table.
#pragma once

#include "common.cuh"

namespace fusekv {

constexpr int kPromptBatch = 256;         // requests of one launch (parameter space)

// Requests of one launch, longest first.  A tile is rtile consecutive rows of
// a request.  Tiles are taken from the highest tile index down, at one index
// over all requests that have it: heaviest first.  Between the tile counts of
// consecutive requests the number of requests that have a tile index is
// constant, so tile `t` (in that order) is found from the order's starts:
// tiles [start[j], start[j + 1]) are those of indexes [tiles[j + 1],
// tiles[j]), taken over requests 0 .. j.
struct PromptTable {
  int32_t n_req;
  int32_t n_tiles;                        // in all
  int32_t row0[kPromptBatch];             // first packed row
  int32_t len[kPromptBatch];              // rows, descending, > 0
  int32_t start[kPromptBatch + 1];
};

struct PromptTile {
  int row0;                               // the request's first packed row
  int len;                                // the request's rows
  int first;                              // the tile's first row in the request
  int rows;                               // its rows
};

__host__ __device__ inline PromptTile prompt_tile(const PromptTable& p, int rtile, int t) {
  int lo = 0, hi = p.n_req - 1;           // last j with start[j] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int u = t - p.start[lo], n = lo + 1;
  const int r = u % n;
  const int index = (p.len[lo] + rtile - 1) / rtile - 1 - u / n;
  PromptTile x;
  x.row0 = p.row0[r];
  x.len = p.len[r];
  x.first = index * rtile;
  x.rows = x.len - x.first < rtile ? x.len - x.first : rtile;
  return x;
}

cudaError_t launch_prompt_simt(const fuse_layer_desc_t& d, const PromptTable& p, const void* Q,
                               const void* K, const void* V, void* O, cudaStream_t s);

// bf16 layers: tcgen05 tensor cores (attend_prompt_tc.cu).
bool prompt_tc_supported(const fuse_layer_desc_t& d);
cudaError_t launch_prompt_tc(const fuse_layer_desc_t& d, const PromptTable& p, int64_t n_tok,
                             const void* Q, const void* K, const void* V, void* O, uint32_t* err,
                             cudaStream_t s);

}  // namespace fusekv
