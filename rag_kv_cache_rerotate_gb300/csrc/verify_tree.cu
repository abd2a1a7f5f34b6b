// Verification of drafted tokens against the target's probabilities
// (fuse_verify_tree).
//
// A draft x drawn from q is kept with probability min(1, r(x) / (S q(x))); after
// a refusal the target's remainder is max(r - S q, 0), unnormalised, S its sum.
// As q >= 0, an entry that has reached 0 stays there, so that after k refusals
//   r = max(p - A q, 0),   A = S_0 + .. + S_(k-1),  S_0 = 1:
// nothing of the vocabulary's size is stored.  Only a refusal and the draw of
// the next token pass over a row; what the walk looks at besides (p and q at the
// drafted tokens) is read for all nodes at once.
//
// The next token is the first x whose running sum passes u' S.  A rounding of
// the sums to fp32 would move that border over several tokens of a large
// vocabulary, so entries, sums and the tests of acceptance are in pairs of floats (48
// bits).  fp64 would be simpler, but an fp64 instruction of sixteen warps keeps an SM busy for
// some 250 cycles: one chain of 8 over 32000 took 27 us with fp64 in the sums and 14 with pairs
// (7.0 now).  64 sampled trees over 150001 tokens take 38.5 us, a star of 63 refusals over
// 32000 155, over 150001 393 (2.5 to 6.2 us a pass).
//
// One cluster per sequence, the vocabulary split over its CTAs, which lie on SMs of their own
// (of 64 clusters of 8 each does); every warp writes its sum into all of them (distributed
// shared memory).  Latency bounds it: a chain of
// reads (parents and tokens, probabilities of the drafts, a row, the part of it
// with the border).
#include <cooperative_groups.h>

#include <algorithm>

#include "cache_seqs.cuh"
#include "launch.h"
#include "trace.h"

namespace fusekv {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kNodes = FUSE_TREE_MAX_NEW;
constexpr int kAhead = 4;                 // groups of four entries that a thread reads at a time

struct VerifyArgs {
  const int32_t* rows;
  const int32_t* parents;
  const int32_t* tokens;
  const float* P;
  const float* Q;                         // null: drafts that were not drawn
  const float* u;
  const float* u_next;
  int32_t *path, *count, *next;
  int64_t p_stride, q_stride, n_rows;
  int32_t vocab, max_path;
  uint32_t* err;
};

// x + y as a pair: s + e exactly.
__device__ __forceinline__ void two_sum(float x, float y, float& s, float& e) {
  s = x + y;
  const float b = s - x;
  e = (x - (s - b)) + (y - b);
}
// A number as the sum of two floats, the second below half a step of the first.  A product whose
// rounding error is formed beside it is a __fmul_rn: the compiler may draw another one into the
// sum behind it, where the error would count twice (24 bits instead of 48).
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  float s, e;
  two_sum(a.h, b.h, s, e);
  e += a.l + b.l;
  Pair r;
  r.h = s + e;
  r.l = e - (r.h - s);
  return r;
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  Pair r;
  const float h = __fmul_rn(a.h, b.h);
  const float l = fmaf(a.h, b.h, -h) + (a.h * b.l + a.l * b.h);
  r.h = h + l;
  r.l = l - (r.h - h);
  return r;
}
__device__ __forceinline__ bool greater(Pair a, Pair b) {
  float s, e;
  two_sum(a.h, -b.h, s, e);
  return s + (e + (a.l - b.l)) > 0.f;
}
__device__ __forceinline__ Pair shfl_xor(Pair a, int o) {
  return Pair{__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)};
}
// Sum over the lanes before this one and this one.
__device__ __forceinline__ Pair scan(Pair a) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair z{__shfl_up_sync(0xffffffffu, a.h, o), __shfl_up_sync(0xffffffffu, a.l, o)};
    if (lane >= o) a = add(z, a);
  }
  return a;
}

// max(p - A q, 0) as a sum of two floats.  Where p is the rounding of A q the first of them is 0 and
// the second all there is, so that its sign is that of both (`positive`): pairs whose first float
// has it, formed where entries are looked at, took 39.9 us instead of 38.6 on 64 sampled trees.
__device__ __forceinline__ Pair remainder_of(float p, float q, Pair A) {
  const float m = __fmul_rn(A.h, q);
  const float me = fmaf(A.h, q, -m);
  float s, e;
  two_sum(p, -m, s, e);
  e = fmaf(-A.l, q, e - me);
  return s + e > 0.f ? Pair{s, e} : Pair{0.f, 0.f};
}

__device__ __forceinline__ bool positive(Pair a) { return a.h + a.l > 0.f; }

// What a pass over a row forms its entries from.  Rows of a large vocabulary need not
// be aligned: `lead` entries are missing in front of a row's first aligned group of
// four.  wide: whole groups are read at once (p and q lie alike; else entry by entry: 74 us
// instead of 38 on 64 sampled trees).
struct Pass {
  const float* p;
  const float* q;                         // null: p alone
  Pair A;
  int lead, vocab;
  bool wide;
  int n_gone;                             // refused tokens whose entry is 0 (without q)
};

// Entries [4 i - lead, 4 i - lead + 4) of a row, those outside the row as 0.
__device__ __forceinline__ float4 read4(const float* row, const Pass& y, int i) {
  const int e = 4 * i - y.lead;
  if (y.wide && e >= 0 && e + 4 <= y.vocab) return __ldg(reinterpret_cast<const float4*>(row + e));
  float x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = e + k >= 0 && e + k < y.vocab ? __ldg(row + e + k) : 0.f;
  return make_float4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ float usable(float x, bool& bad) {
  const bool ok = x >= 0.f && x <= 3.402823466e38f;
  bad |= !ok;
  return ok ? x : 0.f;
}

// The four entries of group i.  Out of line: where entries may not be usable or tokens are
// refused, and for the part that is looked through.
struct Four {
  Pair r[4];
};
__device__ __noinline__ Four entries(const Pass& y, int i, const int* s_gone, uint32_t* err) {
  const float4 pv = read4(y.p, y, i), qv = y.q ? read4(y.q, y, i) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float p[4] = {pv.x, pv.y, pv.z, pv.w}, q[4] = {qv.x, qv.y, qv.z, qv.w};
  Four f;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f.r[k] = Pair{usable(p[k], bad), 0.f};
    if (y.q) f.r[k] = remainder_of(f.r[k].h, usable(q[k], bad), y.A);
  }
  for (int g = 0; g < y.n_gone; ++g) {
    const int at = s_gone[g] - (4 * i - y.lead);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at == k) f.r[k].h = 0.f;
  }
  if (bad) report_error(err, FUSE_ERR_DEVICE_BOUNDS, SITE_VERIFY_PROB, (uint32_t)i);
  return f;
}

__device__ __forceinline__ void tally(Pair& sum, Pair x) {
  float t;
  two_sum(sum.h, x.h, sum.h, t);
  sum.l += t + x.l;
}

// A thread's sum over the groups g0 + its lane, + 32, .. below g1.  Numbers that are not
// usable have a bit pattern past the largest float's; a warp that meets one goes over
// its groups entry by entry, as for rows that are not read in groups.  The row's first
// and last group, where they are not whole, are left out (part_groups).
template <bool kQ>
__device__ __forceinline__ Pair sum_groups(const Pass& y, int g0, int g1, const int* s_gone, uint32_t* err) {
  const int lane = threadIdx.x % 32;
  Pair sum{0.f, 0.f};
  const int first = y.lead > 0, last = (y.vocab + y.lead) / 4;             // whole groups
  const int h0 = max(g0, first), h1 = min(g1, last);
#pragma unroll 1
  for (int g = h0; g < h1; g += 32 * kAhead) {
    float4 p[kAhead], q[kAhead];
    bool plain = y.wide;                  // uniform
    if (plain) {
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = g + 32 * k + lane, e = 4 * i - y.lead;
        p[k] = q[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < h1) {
          p[k] = __ldg(reinterpret_cast<const float4*>(y.p + e));
          if (kQ) q[k] = __ldg(reinterpret_cast<const float4*>(y.q + e));
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        top = max(max(top, __float_as_uint(p[k].x)), __float_as_uint(p[k].y));
        top = max(max(top, __float_as_uint(p[k].z)), __float_as_uint(p[k].w));
        if (kQ) {
          top = max(max(top, __float_as_uint(q[k].x)), __float_as_uint(q[k].y));
          top = max(max(top, __float_as_uint(q[k].z)), __float_as_uint(q[k].w));
        }
      }
      plain = __all_sync(0xffffffffu, top <= 0x7F7FFFFFu);
    }
    if (plain) {
      if (!kQ) {
        for (int n = 0; n < y.n_gone; ++n) {             // refused tokens
          const int at = s_gone[n] + y.lead;
#pragma unroll
          for (int k = 0; k < kAhead; ++k)
            if (at / 4 == g + 32 * k + lane) {
              if (at % 4 == 0) p[k].x = 0.f;
              if (at % 4 == 1) p[k].y = 0.f;
              if (at % 4 == 2) p[k].z = 0.f;
              if (at % 4 == 3) p[k].w = 0.f;
            }
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (g + 32 * k >= h1) break;      // uniform
        const float pe[4] = {p[k].x, p[k].y, p[k].z, p[k].w}, qe[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) tally(sum, kQ ? remainder_of(pe[e], qe[e], y.A) : Pair{pe[e], 0.f});
      }
    } else {
#pragma unroll 1
      for (int i = g + lane; i < min(h1, g + 32 * kAhead); i += 32) {
        const Four f = entries(y, i, s_gone, err);
#pragma unroll
        for (int e = 0; e < 4; ++e) tally(sum, f.r[e]);
      }
    }
  }
  return sum;
}
// The row's first and last group, where they are not whole and this warp's.
__device__ __forceinline__ Pair part_groups(const Pass& y, int g0, int g1, const int* s_gone, uint32_t* err) {
  const int lane = threadIdx.x % 32, last = (y.vocab + y.lead) / 4;
  Pair sum{0.f, 0.f};
  const int i = lane == 0 ? 0 : last;
  const bool there = lane == 0 ? y.lead > 0 : lane == 1 && (y.vocab + y.lead) % 4 != 0 && (last > 0 || y.lead == 0);
  if (there && i >= g0 && i < g1) {
    const Four f = entries(y, i, s_gone, err);
#pragma unroll
    for (int e = 0; e < 4; ++e) tally(sum, f.r[e]);
  }
  return sum;
}

__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const __grid_constant__ VerifyArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  const int n_ctas = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int s = blockIdx.x / n_ctas;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  constexpr int kEach = kMaxCluster * kWarps / 32;         // sums a lane holds
  __shared__ Pair s_sum[2][kMaxCluster * kWarps];          // the cluster's warps' sums, by the pass's parity
  __shared__ Pair s_scan[kWarps];
  __shared__ int s_token[kNodes], s_gone[kNodes], s_path[kNodes];
  __shared__ float s_p[kNodes];
  __shared__ unsigned long long s_child[kNodes];           // a node's children, a bit each
  __shared__ unsigned int s_ok[2];        // nodes that pass the test as it stands
  __shared__ int s_found[2];
  // (a CTA's shared memory may be written once it runs: waited for before the first sums)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  bool begun = false;
  pdl_wait();
  pdl_trigger();
  const int r0 = a.rows[s], r1 = a.rows[s + 1];
  const float un = a.u_next[s];
  int n = (int)((uint32_t)r1 - (uint32_t)r0);
  if (r0 < 0 || r1 < r0 || r1 > a.n_rows || n > a.max_path) {
    if (tid == 0) report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_SEQ_ROWS, (uint32_t)s);
    n = 0;
  }
  // every node's parent, token and probabilities at its parent, a node a thread
  int par = -1, tok = 0;
  float pd = 0.f, qd = 0.f, ud = 0.f;
  if (tid < kNodes) s_child[tid] = 0;
  if (tid < 2) s_ok[tid] = 0;
  if (tid < n) {
    const int row = r0 + tid;
    par = a.parents[row];
    tok = a.tokens[row];
    ud = a.u[row];
    ud = ud < 0.f ? 0.f : ud >= 1.f ? 0.99999994f : ud;              // (NaN stays)
    bool bad = false;
    if (tid > 0) {
      if (par < 0 || par >= tid) {
        report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_SEQ_PARENT, (uint32_t)row);
        par = -1;                         // no node's child
      } else if (tok < 0 || tok >= a.vocab) {
        report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_VERIFY_TOKEN, (uint32_t)row);
        par = -1;
      } else {
        pd = a.P[(int64_t)(r0 + par) * a.p_stride + tok];
        if (a.Q) qd = a.Q[(int64_t)(r0 + par) * a.q_stride + tok];
        pd = usable(pd, bad);
        qd = usable(qd, bad);
      }
    } else {
      par = -1;
    }
    if (bad) report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_VERIFY_PROB, (uint32_t)row);
    s_token[tid] = tok;
    s_p[tid] = pd;
  }
  __syncthreads();
  if (par >= 0) atomicOr(&s_child[par], 1ull << tid);
  // the tests of the nodes in `which` against the remainder A, S: bits in s_ok (call
  // between barriers)
  Pass y;
  y.q = nullptr;
  y.A = Pair{0.f, 0.f};
  y.n_gone = 0;
  y.vocab = a.vocab;
  auto test = [&](unsigned long long which, Pair A, Pair S) {
    if (warp >= kNodes / 32) return;
    bool yes = false;
    if (par >= 0 && (which >> tid & 1)) {
      Pair r{pd, 0.f}, need = mul(Pair{ud, 0.f}, S);
      if (a.Q) {
        r = remainder_of(pd, qd, A);
        need = mul(need, Pair{qd, 0.f});
      } else {
        for (int g = 0; g < y.n_gone; ++g)
          if (s_gone[g] == tok) r.h = 0.f;
      }
      yes = positive(r) && greater(r, need);             // a number that is none: no
    }
    const unsigned int bits = __ballot_sync(0xffffffffu, yes);
    if (lane == 0) s_ok[warp] = bits;
  };
  test(~0ull, y.A, Pair{1.f, 0.f});                  // as first children
  __syncthreads();
  const unsigned long long first_ok = (unsigned long long)s_ok[1] << 32 | s_ok[0];
  const int W = n_ctas * kWarps;
  int groups = 0, seg = 0;                // groups of four of a row, and of a warp's part
  int parity = 0;
  Pair v[kEach];                          // every warp's sum of the last pass: lane L holds those from kEach L on
  // the remainder's sums; returns their total
  auto pass = [&](int node, Pair A) -> Pair {
    y.p = a.P + (int64_t)(r0 + node) * a.p_stride;
    y.q = A.h > 0.f ? a.Q + (int64_t)(r0 + node) * a.q_stride : nullptr;
    y.A = A;
    y.lead = (int)((reinterpret_cast<uintptr_t>(y.p) >> 2) & 3u);
    y.wide = !y.q || (int)((reinterpret_cast<uintptr_t>(y.q) >> 2) & 3u) == y.lead;
    groups = (a.vocab + y.lead + 3) / 4;
    seg = (groups + W - 1) / W;
    const int g0 = (rank * kWarps + warp) * seg, g1 = min(groups, g0 + seg);
    Pair sum = y.q ? sum_groups<true>(y, g0, g1, s_gone, a.err) : sum_groups<false>(y, g0, g1, s_gone, a.err);
    if (g0 == 0 || g1 == groups) sum = add(sum, part_groups(y, g0, g1, s_gone, a.err));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum = add(sum, shfl_xor(sum, o));
    if (!begun) {
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      begun = true;
    }
    if (lane < n_ctas) *cl.map_shared_rank(&s_sum[parity][rank * kWarps + warp], lane) = sum;
    cl.sync();
    Pair all{0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int w = lane * kEach + k;
      v[k] = w < W ? s_sum[parity][w] : Pair{0.f, 0.f};
      all = add(all, v[k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all = add(all, shfl_xor(all, o));
    parity ^= 1;
    return all;
  };

  // the walk, the same in every thread of the cluster
  int cur = 0, kept = n > 0 ? 1 : 0;
  Pair A{0.f, 0.f}, S{1.f, 0.f};
  bool summed = false;                    // v holds the sums of the remainder as it stands
  unsigned long long left = n > 0 ? s_child[0] : 0, ok = first_ok;
  if (tid == 0) s_path[0] = 0;
  while (left) {
    const int c = __ffsll(left) - 1;
    left &= left - 1;
    if (ok >> c & 1) {                    // on to it
      cur = c;
      if (tid == 0) s_path[kept] = c;
      ++kept;
      A = Pair{0.f, 0.f};
      S = Pair{1.f, 0.f};
      y.n_gone = 0;
      summed = false;
      left = s_child[c];
      ok = first_ok;
      continue;
    }
    if (a.Q) {
      A = add(A, S);
      S = pass(cur, A);
      summed = true;
    } else {
      const int x = s_token[c];
      bool again = false;
      for (int g = 0; g < y.n_gone; ++g) again |= s_gone[g] == x;
      __syncthreads();                    // s_gone is read above
      if (!again) {
        S = add(S, Pair{-s_p[c], 0.f});  // what refusals leave of 1
        if (tid == 0) s_gone[y.n_gone] = x;
        ++y.n_gone;
      }
    }
    if (left) {
      __syncthreads();                    // s_gone; s_ok has been read
      test(left, A, S);
      __syncthreads();
      ok = (unsigned long long)s_ok[1] << 32 | s_ok[0];
    }
  }
  __syncthreads();                        // s_gone, s_path
  int token = -1;
  bool mine = rank == 0;                  // this CTA writes the results
  if (n > 0) {
    Pair sum = summed ? S : pass(cur, A);
    if (!(sum.h > 0.f)) {                 // nothing left: the target's own row
      y.n_gone = 0;
      sum = pass(cur, Pair{0.f, 0.f});
    }
    // t = u' sum; the first warp's part whose running sum passes it
    const float uc = un > 0.f ? fminf(un, 0.99999994f) : 0.f;
    Pair t;
    t.h = __fmul_rn(uc, sum.h);
    t.l = fmaf(uc, sum.h, -t.h) + uc * sum.l;
    Pair own{0.f, 0.f};
    int full = -1;                        // the last part that holds anything
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      own = add(own, v[k]);
      if (v[k].h > 0.f) full = lane * kEach + k;
    }
    const Pair inc = scan(own);
    Pair c = Pair{__shfl_up_sync(0xffffffffu, inc.h, 1), __shfl_up_sync(0xffffffffu, inc.l, 1)};
    if (lane == 0) c = Pair{0.f, 0.f};
    int at = INT32_MAX;
    Pair before{0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const Pair next = add(c, v[k]);
      if (at == INT32_MAX && v[k].h > 0.f && greater(next, t)) {
        at = lane * kEach + k;
        before = c;
      }
      c = next;
    }
    int part = (int)__reduce_min_sync(0xffffffffu, (unsigned)at);
    const int last = __reduce_max_sync(0xffffffffu, full);
    const unsigned who = __ballot_sync(0xffffffffu, at == part && part != INT32_MAX);
    const bool end = who == 0;            // t within the sums' rounding of their total: the last entry
    if (end) {
      part = last;
    } else {
      before.h = __shfl_sync(0xffffffffu, before.h, __ffs(who) - 1);
      before.l = __shfl_sync(0xffffffffu, before.l, __ffs(who) - 1);
    }
    mine = part >= 0 ? part / kWarps == rank : rank == 0;
    if (part < 0 && mine && tid == 0)
      report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_VERIFY_PROB, (uint32_t)(r0 + cur));
    if (part >= 0 && mine) {
      // this CTA looks the part through, four entries a thread
      if (tid == 0) {
        s_found[0] = INT32_MAX;
        s_found[1] = -1;
      }
      __syncthreads();
      const int g0 = part * seg, g1 = min(groups, g0 + seg);
      for (int b = g0; b < g1; b += kThreads) {
        const int i = b + tid;
        Pair r[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
        if (i < g1) {
          const Four f = entries(y, i, s_gone, a.err);
#pragma unroll
          for (int k = 0; k < 4; ++k) r[k] = f.r[k];
        }
        const Pair four = add(add(r[0], r[1]), add(r[2], r[3]));
        const Pair upto = scan(four);
        if (lane == 31) s_scan[warp] = upto;
        Pair z = Pair{__shfl_up_sync(0xffffffffu, upto.h, 1), __shfl_up_sync(0xffffffffu, upto.l, 1)};
        if (lane == 0) z = Pair{0.f, 0.f};
        __syncthreads();
        const Pair up = scan(lane < kWarps ? s_scan[lane] : Pair{0.f, 0.f});
        const Pair base{__shfl_sync(0xffffffffu, up.h, (warp + 31) & 31), __shfl_sync(0xffffffffu, up.l, (warp + 31) & 31)};
        const Pair tot = add(before, Pair{__shfl_sync(0xffffffffu, up.h, 31), __shfl_sync(0xffffffffu, up.l, 31)});
        z = add(warp > 0 ? add(before, base) : before, z);
        int first = INT32_MAX, any = -1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z = add(z, r[k]);
          if (positive(r[k])) {
            any = 4 * i - y.lead + k;
            if (first == INT32_MAX && !end && greater(z, t)) first = any;
          }
        }
        if (first != INT32_MAX) atomicMin(&s_found[0], first);
        if (any >= 0) atomicMax(&s_found[1], any);
        before = tot;
        __syncthreads();
        if (s_found[0] != INT32_MAX) break;
      }
      token = s_found[0] != INT32_MAX ? s_found[0] : s_found[1];
    }
  }
  if (mine) {
    if (tid == 0) {
      a.next[s] = token;
      a.count[s] = kept;
    }
    for (int i = tid; i < a.max_path; i += kThreads)
      a.path[(int64_t)s * a.max_path + i] = i < kept ? s_path[i] : -1;
  }
  if (!begun) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

fuse_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? FUSE_OK : FUSE_ERR_CUDA; }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace fusekv

using namespace fusekv;

extern "C" fuse_status_t fuse_verify_tree(int32_t n_seq, int64_t n_rows, int32_t vocab, const int32_t* rows,
                                          const int32_t* parents, const int32_t* tokens, const float* P,
                                          int64_t p_stride, const float* Qd, int64_t q_stride,
                                          const float* u, const float* u_next, int32_t max_path,
                                          int32_t* path, int32_t* count, int32_t* next, void* ws,
                                          size_t ws_bytes, fuse_stream_t stream) {
  if (n_seq < 0 || n_rows < 0 || vocab < 1 || max_path < 1) return FUSE_ERR_INVALID_ARG;
  if (n_seq > 65535 || n_rows > INT32_MAX || vocab > INT32_MAX / 8 || max_path > FUSE_TREE_MAX_NEW)
    return FUSE_ERR_UNSUPPORTED;
  if (n_seq > 0 && (!rows || !u_next || !path || !count || !next)) return FUSE_ERR_INVALID_ARG;
  if (n_rows > 0 && (!parents || !tokens || !P || !u)) return FUSE_ERR_INVALID_ARG;
  if (p_stride < vocab || (Qd && q_stride < vocab)) return FUSE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)rows, (const void*)parents, (const void*)tokens, (const void*)P,
                        (const void*)Qd, (const void*)u, (const void*)u_next, (const void*)path,
                        (const void*)count, (const void*)next})
    if (!aligned4(p)) return FUSE_ERR_MISALIGNED;
  const fuse_status_t st = check_ws(ws, ws_bytes, FUSE_CACHE_WORKSPACE);
  if (st != FUSE_OK) return st;
  if (n_seq == 0) return FUSE_OK;
  VerifyArgs a;
  a.rows = rows;
  a.parents = parents;
  a.tokens = tokens;
  a.P = P;
  a.Q = Qd;
  a.u = u;
  a.u_next = u_next;
  a.path = path;
  a.count = count;
  a.next = next;
  a.p_stride = p_stride;
  a.q_stride = q_stride;
  a.n_rows = n_rows;
  a.vocab = vocab;
  a.max_path = max_path;
  a.err = reinterpret_cast<uint32_t*>(ws);
  cudaStream_t s = (cudaStream_t)stream;
  // As many CTAs a sequence as run at a time, and as have 8 entries a thread: 58 sequences
  // of a vocabulary of 2300 take 11 us with one or two, 17 with eight; 64 of 150 001 take 45
  // with eight, 71 with two; one of 32 000 9 with eight (graphs of a few calls).
  int dev = 0, sms = 1;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int ctas = kMaxCluster;
  while (ctas > 1 && ((int64_t)n_seq * ctas > 4 * (int64_t)sms || vocab < ctas * kThreads * 8)) ctas /= 2;
  return cuda_status(traced("verify_tree", s, [&] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n_seq * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel, a);
  }));
}
