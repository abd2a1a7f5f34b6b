// Sequences held in pages with their state on the device (fuse_seqs_t): what
// the kernels of a speculative step share.
#pragma once

#include "checks.h"
#include "common.cuh"

namespace fusekv {

struct SeqArgs {
  const int32_t* tables;
  int32_t* lens;
  const int32_t* rows;
  int32_t n_seq, block_size, max_blocks, max_new;
  uint32_t block_inv;                     // ceil(2^32 / block_size), 0 for pages of one token
  int64_t n_pool_blocks, n_rows;
  uint32_t* err;
};

// The page of a slot, and the slot's place in it.  The product with the rounded-up
// inverse gives the quotient or one more.
__device__ __forceinline__ int page_of(const SeqArgs& a, int slot, int* in_page) {
  int b = a.block_inv ? (int)__umulhi((uint32_t)slot, a.block_inv) : slot;
  int r = (int)((uint32_t)slot - (uint32_t)b * (uint32_t)a.block_size);
  if (r < 0) {
    --b;
    r += a.block_size;
  }
  *in_page = r;
  return b;
}

// A sequence in a call: its rows [row0, row0 + n), its held tokens.
struct Seq {
  int row0, n, len;
};

// Whether sequence s, whose row starts and length these are, can be used as it stands (else
// it is recorded, and has no rows).
__device__ __forceinline__ bool check_seq(const SeqArgs& a, int s, int r0, int r1, int len, Seq* q) {
  q->row0 = r0;
  q->len = len;
  q->n = (int)((uint32_t)r1 - (uint32_t)r0);
  if (r0 < 0 || r1 < r0 || r1 > a.n_rows || q->n > a.max_new || len < 0 ||
      (int64_t)len + q->n > (int64_t)a.max_blocks * a.block_size) {
    report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_SEQ_ROWS, (uint32_t)s);
    q->n = 0;
    return false;
  }
  return true;
}
__device__ __forceinline__ bool seq_of(const SeqArgs& a, int s, Seq* q) {
  const int r0 = a.rows[s], r1 = a.rows[s + 1], len = a.lens[s];
  return check_seq(a, s, r0, r1, len, q);
}

// The parent of new token i (-1: none); one out of range is recorded.
__device__ __forceinline__ int checked_parent(int p, const Seq& q, int i, uint32_t* err) {
  if (p >= -1 && p < i) return p;
  report_error(err, FUSE_ERR_DEVICE_BOUNDS, SITE_SEQ_PARENT, (uint32_t)(q.row0 + i));
  return -1;
}
__device__ __forceinline__ int parent_of(const int32_t* parents, const Seq& q, int i, uint32_t* err) {
  if (!parents) return i - 1;
  return checked_parent(parents[q.row0 + i], q, i, err);
}

// The pool row of a slot; -1 where its page is outside the pool (recorded).
__device__ __forceinline__ int64_t checked_page(const SeqArgs& a, int page, int in_page) {
  if (page < 0 || page >= a.n_pool_blocks) {
    report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_SEQ_PAGE, (uint32_t)page);
    return -1;
  }
  return (int64_t)page * a.block_size + in_page;
}
__device__ __forceinline__ int64_t pool_row(const SeqArgs& a, int s, int slot) {
  int in_page;
  const int page = a.tables[(int64_t)s * a.max_blocks + page_of(a, slot, &in_page)];
  return checked_page(a, page, in_page);
}

// The sequence whose rows hold `row`: the last s with rows[s] <= row (by a whole
// warp, 32 probes a round; -1 in front of the first).  Ascending starts of
// sequences without rows are passed over.
__device__ __forceinline__ int seq_of_row(const int32_t* rows, int n_seq, int row) {
  const int lane = threadIdx.x % 32;
  int lo = 0, len = n_seq + 1;             // rows[lo - 1] <= row, or lo == 0
  while (len > 0) {
    const int step = (len + 31) / 32, i = lo + (lane + 1) * step - 1;
    const bool below = i < lo + len && rows[i] <= row;
    const int parts = __popc(__ballot_sync(0xffffffffu, below));
    lo += parts * step;
    len = min(step - 1, len - parts * step);
  }
  return lo - 1;
}

// ---- host side ---------------------------------------------------------------

// Everything of a call's sequences that needs no device memory.
fuse_status_t check_seqs(const fuse_seqs_t* q, int64_t n_rows, int max_new, SeqArgs* a, void* ws);

}  // namespace fusekv
