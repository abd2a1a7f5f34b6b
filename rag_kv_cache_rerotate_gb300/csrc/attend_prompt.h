// The work of the packed-prompt attention, by value: which tile of which
// request a unit of work is, without a device table.
#pragma once

#include "common.cuh"

namespace fusekv {

constexpr int kPromptBatch = 64;          // requests of one launch (parameter space)
constexpr int kMaxUnits = 1 << 24;        // (tile, KV head) units of one launch

// Requests of one launch, longest first.  A tile is rtile consecutive rows of
// a request.  Tiles are taken from the highest tile index down, at one index
// over all requests that have it: heaviest first.  Between the tile counts of
// consecutive requests the number of requests that have a tile index is
// constant, so tile `t` (in that order) is found from the order's starts:
// tiles [req[j].start, req[j + 1].start) are those of indexes [tiles of j + 1,
// tiles of j), taken over requests 0 .. j.
struct __align__(8) PromptRequest {
  int32_t start;                          // first tile of the order's part j
  int32_t row0;                           // first packed row
  int32_t len;                            // rows, descending, > 0
  int32_t tiles;
  uint32_t inv;                           // ceil(2^32 / (j + 1)): x / (j + 1) = umulhi(x, inv), x < 2^24
  int32_t pad;
};
struct PromptTable {
  int32_t n_req;
  int32_t n_tiles;                        // in all
  PromptRequest req[kPromptBatch + 1];    // the last: start = n_tiles
};

struct PromptTile {
  int row0;                               // the request's first packed row
  int len;                                // the request's rows
  int first;                              // the tile's first row in the request
  int rows;                               // its rows
};

// Tile t; *part: the order's part that it is in, at most that on entry (tiles
// asked for in ascending order: pass the same variable, at first 0).
__device__ __forceinline__ PromptTile prompt_tile(const PromptTable& p, int rtile, int t, int* part) {
  int j = *part;
  while (p.req[j + 1].start <= t) ++j;    // ends: the last start is past every tile
  *part = j;
  const PromptRequest o = p.req[j];
  const int u = t - o.start, n = j + 1;
  int r = 0, index = o.tiles - 1 - u;
  if (n > 1) {
    const int q = (int)__umulhi((uint32_t)u, o.inv);
    r = u - q * n;
    index = o.tiles - 1 - q;
  }
  const PromptRequest q = p.req[r];
  PromptTile x;
  x.row0 = q.row0;
  x.len = q.len;
  x.first = index * rtile;
  x.rows = x.len - x.first < rtile ? x.len - x.first : rtile;
  return x;
}

// fp32 layers, CUDA cores; the tiles hold 16 r / g rows (r = 1, 2, 4).
cudaError_t launch_prompt_simt(const fuse_layer_desc_t& d, int r, const PromptTable& p, const void* Q,
                               const void* K, const void* V, void* O, cudaStream_t s);

// bf16 layers: tcgen05 tensor cores (attend_prompt_tc.cu).
bool prompt_tc_supported(const fuse_layer_desc_t& d);
cudaError_t launch_prompt_tc(const fuse_layer_desc_t& d, const PromptTable& p, int64_t n_tok,
                             const void* Q, const void* K, const void* V, void* O, uint32_t* err,
                             cudaStream_t s);

}  // namespace fusekv
