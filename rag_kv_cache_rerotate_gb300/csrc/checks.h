// What the files of entry points share: argument checks (defined in api.cu) and
// the cache operators' error sites.
#pragma once

#include "common.cuh"

namespace fusekv {

// Sites of the cache operators, behind those of ErrSite.
enum CacheErrSite : uint32_t {
  SITE_PAGE_ENTRY = 11,      // table entry outside the pool, or naming a page without a reference
  SITE_PAGE_FREE = 12,       // too few free pages
  SITE_PAGE_MOVES = 13,      // move list count or page id out of range
  SITE_ATTEND_BLOCK = 14,    // paged block id outside the pool (attend_chunks)
  SITE_ATTEND_SEL = 15,      // selected index out of range or order (attend_chunks)
  SITE_PROMPT_TIMEOUT = 16,  // prompt-attention pipeline wait gave up
  SITE_PAGE_COUNT = 17,      // negative reference count
  SITE_SEQ_ROWS = 18,        // a sequence's rows, length or table row (fuse_seqs_t)
  SITE_SEQ_PARENT = 19,      // parent out of range
  SITE_SEQ_PAGE = 20,        // page outside the pool
  SITE_TREE_TIMEOUT = 21,    // tree-attention pipeline wait gave up
  SITE_VERIFY_TOKEN = 22,    // drafted token outside the vocabulary
  SITE_VERIFY_PROB = 23,     // probability negative, infinite or NaN
  SITE_KEEP_PATH = 24,       // path or count out of range or order
};

struct ReqInfo {
  fuse_totals_t tot;   // extents implied by the offsets (max over requests)
  int n_req;
  bool sorted;         // row0 ascending, request row ranges disjoint
  int64_t n_qrows;     // sum of n_query: the packed query rows of the scorer
  int32_t max_query;   // max n_query
};

bool aligned16(const void* p);
size_t elem_size(int dtype);   // bytes of an F32 / BF16 element, 1 for codes
fuse_status_t check_desc(const fuse_layer_desc_t* d);
fuse_status_t check_reqs(const fuse_requests_t* r, ReqInfo* info, bool need_device = true);
fuse_status_t check_chunks(const fuse_layer_desc_t& d, const fuse_chunks_t* c, int64_t fused_rows,
                           int* max_len);
fuse_status_t check_ws(void* ws, size_t ws_bytes, size_t need);
RopeFreqs make_freqs(const fuse_layer_desc_t& d);

}  // namespace fusekv
