// Attention of trees over a paged cache on tcgen05 tensor cores (bf16 layers).
//
// Work unit: one sequence, KV head and up to 256 query vectors (new token, query
// head of the KV head), as one or two M = 128 tiles; keys stream in tiles of 128
// through a ring in shared memory.  Two streams run side by side, each with a score
// buffer and an accumulator of its own:
//   two M tiles   stream w takes M tile w, both with the same keys
//   one M tile    stream w takes every second key tile; the two softmaxes are
//                 joined when the unit ends
// so that one stream's products run beside the other's softmax.  Per step
//   S = Q K^T     tcgen05.mma into TMEM columns [128 w, 128 w + 128)
//   P = 2^(S - m) eight warps a stream, in registers, bf16, written back over S
//   O += P V      tcgen05.mma with A = P in TMEM, V MN-major in shared memory
// (Two score buffers of 64 keys a stream would hide the hand-overs, but products of
// N = 64 run at half the rate of N = 128: 526 us instead of 412 on 8 trees of 64
// over 33k.  P in two halves, the first one's product beside the second's softmax: 479.)
// With 64 vectors and less a tile of keys and values takes as long as HBM needs for it (16 trees
// over 512 to 8192: 64 us, 6.5 TB/s between the start and the end).  With 256 the chain of a
// stream's step binds it, 2990 cycles: S 610 (its operands come from shared memory), softmax
// 1150, P V 480, hand-overs 750; 8 trees of 64 over 33k take 400 to 420 us, 1.33 to 1.39
// PFLOP/s, and 450 to 475 called back to back, where the power cap holds the clock down.
// The reference m is the first tile's maximum.  A later tile is weighed against it
// as it stands, without its maximum being looked for: only where a thread's sum of
// its weights passes 2^16 (no weight does otherwise) is the row's reference raised, O
// and the running sum rescaled and the tile weighed once more.
//
// Keys and values lie in pages.  With pages of a multiple of 8 tokens a tile is
// copied by TMA boxes of as many rows as always lie in one page, whole heads: a copy
// costs the SM's copy unit about 100 cycles whatever its size, so that boxes of 64
// columns kept pages of 16 tokens at 5.3 TB/s of the 6.6 that pages of 128 reach.  What
// lies behind a sequence's last slot in its page comes along and is masked, its values
// cleared.  With other pages the rows are gathered by 16-byte cp.async (one token over 8 times
// 33k: 4.6 TB/s, with boxes 6.25; single rows as tile::gather4 copies: 2).
// A tile lies in shared memory as [group of 8 rows][64 columns][8 rows], 128-byte swizzled.
//
// What a row does not see must not reach it: its scores are replaced where they
// are masked, and as 0 * V is not 0 for an infinite or NaN V, one warp looks
// the new tokens' values through before their product, clears what is not
// finite, and the rows that do see such an element get it back at the end.
// (Held tokens are seen by every row.)
#include <cudaTypedefs.h>

#include <algorithm>

#include "attend_tree.h"
#include "launch.h"
#include "tc_ptx.cuh"

namespace fusekv {

bool make_map_3d(CUtensorMap* m, const void* base, const uint64_t dims[3], const uint64_t strides[2],
                 const uint32_t box[3]);
bool make_map_groups(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int col_blocks,
                     int row_groups);

namespace {

constexpr int kKB = kTreeTcTile;              // keys per tile
constexpr int kHalf = 128 * 64 * 2;           // 64 columns of a 128-row tile (16 KB)
constexpr int kAtom = 1024;                   // 8 rows of 64 columns
// Two warps load: a copy instruction takes its operands from uniform registers, so
// that a warp's lanes issue theirs one after another.
constexpr int kSoftWarps = 16, kWarpLoad = 16, kLoadWarps = 2, kWarpS = 18, kWarpPV = 19;
constexpr int kThreads = 20 * 32;
constexpr int kParts = 4;                     // parts planned ahead, at most
constexpr int kAhead = 3;                     // tiles whose pages are looked up ahead of their copies
constexpr int kTmemCols = 512;                // S of both streams | O of both
constexpr float kMaxSum = 65536.f;            // of a thread's 32 weights: they keep their relative precision up to there
constexpr float kFar = 1048576.f;             // of a score in log2 units: 2^-4 is its last place
constexpr int kMaxStages = 10;
constexpr int kFix = 8;                       // parts with new tokens that the look may be ahead by, and more

template <int D> struct Ring {
  static constexpr int tile = (D / 64) * kHalf;
  static constexpr int group = (D / 64) * kAtom;         // 8 rows
  static constexpr int stages = D == 128 ? 5 : 10;
};

struct Ctl {
  uint64_t q_full[2], q_empty[2];
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t s_full[2], p_full[2], pv_done[2];             // by stream
  uint64_t x_full, o_empty;
  uint64_t part_full[kParts], part_empty[kParts];
  unsigned long long fix[kFix];               // new tokens with values that are not finite
  uint32_t tmem_base;
  volatile int abort_flag;
  volatile int bad_page;                      // some page of this CTA's units is outside the pool
  float2 ml[2][128];                          // maximum and sum of each stream's rows
  TreePart part[kParts];                      // what the CTA works at, planned ahead by the first load warp
};

constexpr int kCtlBytes = 3 * 1024;           // in front of the tiles, which start at multiples of 1024
static_assert(sizeof(Ctl) <= kCtlBytes, "shared memory");
template <int D> constexpr int smem_bytes() { return kCtlBytes + (2 + Ring<D>::stages) * Ring<D>::tile; }
static_assert(smem_bytes<128>() <= 227 * 1024 && smem_bytes<64>() <= 227 * 1024, "shared memory");

// Which wait gave up: info = wait id << 16 | CTA.
enum TreeWait : uint32_t {
  W_Q_EMPTY = 1, W_EMPTY, W_Q_FULL, W_S_FREE, W_K_FULL, W_P_FULL, W_V_FULL, W_O_EMPTY,
  W_S_FULL, W_PV_DONE, W_O_FULL, W_X_FULL, W_PART_FULL, W_PART_EMPTY
};

__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, Ctl* ctl, uint32_t* err, uint32_t which) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 0; i < tc::kWaitPollLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 63u) == 63u) {
      if (ctl->abort_flag) return false;
      const uint64_t now = tc::global_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > tc::kWaitLimitNs) break;
    }
  }
  if (ctl->abort_flag == 0) {
    ctl->abort_flag = 1;
    report_error(err, FUSE_ERR_TIMEOUT, SITE_TREE_TIMEOUT, which);
  }
  return false;
}
__device__ __forceinline__ bool wait1(uint64_t* bar, uint32_t parity, Ctl* ctl, uint32_t* err, uint32_t which) {
  if (tc::mbar_try_wait(bar, parity & 1)) return true;
  return wait_on(tc::smem_u32(bar), parity & 1, ctl, err, (which << 16) | (blockIdx.x & 0xFFFFu));
}
__device__ __forceinline__ bool wait32(uint64_t* bar, uint32_t parity, Ctl* ctl, uint32_t* err, uint32_t which) {
  return __all_sync(0xffffffffu, wait1(bar, parity, ctl, err, which));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Packed pairs of floats: one instruction does the operation on both halves.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Where piece c (16 bytes) of row m lies in a tile.
template <int D> __device__ __forceinline__ uint32_t piece_at(int m, int c) {
  return (m >> 3) * Ring<D>::group + (c >> 3) * kAtom + (m & 7) * 128 + (((c & 7) ^ (m & 7)) << 4);
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// Arrives on the barrier, whose count provides for it, once this thread's copies so far have landed.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}

// Adds to a row of outputs (or of a part) the elements that are not finite of the values
// of the new tokens in `left`: with them a sum is infinite or NaN whatever it was.
template <typename T>
__device__ __noinline__ void add_nonfinite(T* dst, int n, unsigned long long left, const TreeArgs& a, const TreePart& p,
                                           int e0, int d) {
#pragma unroll 1
  for (; left; left &= left - 1) {
    const int64_t row = pool_row(a.seq, p.s, p.q.len + __ffsll(left) - 1);
    if (row < 0) continue;
    const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(a.v_pool) + (row * a.n_kv_heads + p.h) * d + e0;
#pragma unroll 1
    for (int e = 0; e < n; ++e) {
      const float x = __bfloat162float(v[e]);
      if (!isfinite(x)) dst[e] = (T)((float)dst[e] + x);
    }
  }
}

// A number that the warp's lanes share, as one that the compiler knows them to share:
// the products' operands are formed once, not by lanes.
__device__ __forceinline__ uint64_t uniform64(uint64_t x) {
  return (uint64_t)__shfl_sync(0xffffffffu, (uint32_t)(x >> 32), 0) << 32 | __shfl_sync(0xffffffffu, (uint32_t)x, 0);
}

// The CTA's part i (by a whole warp); false behind the last one.
__device__ __forceinline__ bool take_part(Ctl* ctl, uint32_t& i, TreePart& p, uint32_t* err) {
  const int at = i % kParts;
  if (!wait32(&ctl->part_full[at], i / kParts, ctl, err, W_PART_FULL)) return false;
  p = ctl->part[at];
  __syncwarp();
  if (threadIdx.x % 32 == 0) tc::mbar_arrive(&ctl->part_empty[at]);
  ++i;
  return p.nt > 0;
}

// What every role derives from a part.
struct Steps {
  bool dual;                                  // two M tiles
  int tiles, n;                               // key tiles, steps (of both streams)
  __device__ __forceinline__ explicit Steps(const TreePart& p) {
    dual = p.n_vec > 128;
    tiles = p.j1 - p.j0;
    n = dual ? 2 * tiles : tiles;
  }
  __device__ __forceinline__ int tile(int k) const { return dual ? k >> 1 : k; }
  // Ring items, keys a tile ahead of values: K0 K1 V0 K2 V1 ..
  __device__ __forceinline__ int k_item(int i) const { return i == 0 ? 0 : 2 * i - 1; }
  __device__ __forceinline__ int v_item(int i) const { return i < tiles - 1 ? 2 * i + 2 : 2 * tiles - 1; }
};
// Whether the keys of tile j go past the held tokens.
__device__ __forceinline__ bool has_new(const TreePart& p, int j) { return (j + 1) * kKB > p.q.len; }

// 32 keys' bits of a row: those that it sees, the first of them `rel` past the held tokens.
__device__ __forceinline__ uint32_t seen_word(uint64_t seen, int rel) {
  if (rel <= -32) return 0xffffffffu;
  if (rel < 0) return ((1u << -rel) - 1u) | (uint32_t)(seen << -rel);
  return rel < 64 ? (uint32_t)(seen >> rel) : 0u;
}

// kGather: pages that are not multiples of 8 tokens; else box rows of them are copied at a time.
template <int D, bool kGather>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                   const __grid_constant__ CUtensorMap mapV, const __grid_constant__ TreeArgs a, const int box) {
  constexpr int kTile = Ring<D>::tile, kGroup = Ring<D>::group, kSt = Ring<D>::stages;
  constexpr int kColO = 2 * kKB;
  static_assert(kColO + 2 * D <= kTmemCols, "tensor memory");
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctl* ctl = reinterpret_cast<Ctl*>(smem);
  uint8_t* sQ = smem + kCtlBytes;
  uint8_t* sR = sQ + 2 * kTile;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint32_t* const err = a.seq.err;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&ctl->q_full[i], 1);
      tc::mbar_init(&ctl->q_empty[i], 1);
      tc::mbar_init(&ctl->s_full[i], 1);
      tc::mbar_init(&ctl->p_full[i], kSoftWarps / 2);
      tc::mbar_init(&ctl->pv_done[i], 1);
    }
    for (int i = 0; i < kSt; ++i) {
      tc::mbar_init(&ctl->full[i], kGather ? kLoadWarps * 32 : kLoadWarps);
      tc::mbar_init(&ctl->empty[i], 1);
    }
    tc::mbar_init(&ctl->x_full, kSoftWarps * 32);
    tc::mbar_init(&ctl->o_empty, kSoftWarps * 32);
    for (int i = 0; i < kParts; ++i) {
      tc::mbar_init(&ctl->part_full[i], 1);
      tc::mbar_init(&ctl->part_empty[i], kThreads / 32 - 1);       // every warp but the planning one
    }
    ctl->abort_flag = 0;
    ctl->bad_page = 0;
    tc::fence_barrier_init();
    tc::tma_prefetch_desc(&mapQ);
    tc::tma_prefetch_desc(&mapK);
    tc::tma_prefetch_desc(&mapV);
  }
  if (warp == kWarpS) tc::tmem_alloc(&ctl->tmem_base, kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  pdl_wait();
  pdl_trigger();
  TreePart p{};
  uint32_t part_at = 0;

  if (warp >= kWarpLoad && warp < kWarpLoad + kLoadWarps) {
    // -------------------------------- loads --------------------------------
    const int lw = warp - kWarpLoad;
    uint32_t it = 0, qn0 = 0, qn1 = 0;
    int qb = 0;
    bool ok = true;
    // Boxes: every warp copies every second one, lane i knows its i-th one's page.
    // Gathered rows: every warp takes 64 rows, a lane looks two pages up and copies
    // pieces of all.
    constexpr int kG = kGather ? 2 : 1;
    const int n_box = kKB / box, my_ops = (n_box - lw + kLoadWarps - 1) / kLoadWarps;
    const int none = -1, outside = (int)(a.seq.n_pool_blocks * a.seq.block_size / 8);       // its first group outside the pool
    // the pages of this lane's keys of tile j (-2: no key there), and the slots' places
    auto entries = [&](int j, int (&page)[kG], int (&in_page)[kG]) {
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        const int m = kGather ? lw * 64 + i * 32 + lane : (lane * kLoadWarps + lw) * box, key = j * kKB + m;
        const int b = page_of(a.seq, key, &in_page[i]);
        page[i] = m < kKB && key < p.q.len + p.q.n ? a.seq.tables[(int64_t)p.s * a.seq.max_blocks + b] : -2;
      }
    };
    auto places = [&](const int (&page)[kG], const int (&in_page)[kG], int (&row)[kG]) {
      bool bad = false;
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        const bool there = page[i] >= 0 && page[i] < a.seq.n_pool_blocks;
        row[i] = there ? page[i] * a.seq.block_size + in_page[i] : none;
        bad |= !there && page[i] != -2;
      }
      if (bad) {
        report_error(err, FUSE_ERR_DEVICE_BOUNDS, SITE_SEQ_PAGE, (uint32_t)p.s);
        ctl->bad_page = 1;
      }
    };
    auto issue = [&](const CUtensorMap* map, const void* pool, const int (&row)[kG]) {
      const int st = it % kSt;
      if (!wait32(&ctl->empty[st], (it / kSt) ^ 1, ctl, err, W_EMPTY)) return false;
      uint64_t* bar = &ctl->full[st];
      uint8_t* tile = sR + st * kTile;
      if constexpr (kGather) {
        constexpr int kPieces = D / 8, kRows = 32 / kPieces;       // lanes of a row, rows at a time
        const int c = lane % kPieces, sub = lane / kPieces;
        const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(pool) + (int64_t)p.h * D + c * 8;
        const int64_t step = (int64_t)a.n_kv_heads * D;
        const uint32_t dst = tc::smem_u32(tile);
#pragma unroll
        for (int i = 0; i < kG; ++i)
#pragma unroll
          for (int k0 = 0; k0 < 32 / kRows; k0 += 8) {
            int y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = __shfl_sync(0xffffffffu, row[i], (k0 + k) * kRows + sub);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              cp16(dst + piece_at<D>(lw * 64 + i * 32 + (k0 + k) * kRows + sub, c), src + max(y[k], 0) * step, y[k] >= 0);
          }
        if (ctl->bad_page) {                  // the flag has to be seen by who sees the tile
          asm volatile("cp.async.wait_all;" ::: "memory");
          tc::mbar_arrive(bar);
        } else {
          cp_arrive(bar);
        }
      } else {
        __syncwarp();                         // (bad_page is set before the barrier's phase can end)
        if (lane == 0) tc::mbar_arrive_expect_tx(bar, my_ops * box * D * 2);
        __syncwarp();
        const int group = row[0] >= 0 ? row[0] >> 3 : outside;      // a group outside the pool reads as zeros
#pragma unroll 1
        for (int i = 0; i < my_ops; ++i) {
          const int y = __shfl_sync(0xffffffffu, group, i);
          if (tc::elect_one())
            tc::tma_load_4d(tile + (i * kLoadWarps + lw) * box * D * 2, map, bar, 0, 0, p.h * (D / 64), y);
          __syncwarp();
        }
      }
      ++it;
      return true;
    };
    // the first warp plans: a part while the one before it is being loaded
    TreeWalk walk;
    if (lw == 0) walk = start_walk(a, blockIdx.x, blockIdx.x == 0);
    auto plan = [&] {
      TreePart next;
      if (!next_part(a, walk, next)) next.nt = 0;
      const int at = part_at % kParts;
      if (!wait32(&ctl->part_empty[at], (part_at / kParts) ^ 1, ctl, err, W_PART_EMPTY)) next.nt = 0;
      if (lane == 0) {
        ctl->part[at] = next;
        tc::mbar_arrive(&ctl->part_full[at]);
      }
      ++part_at;
      return next;
    };
    TreePart ahead;
    if (lw == 0) ahead = plan();
    while (ok) {
      if (lw == 0) {
        p = ahead;
        if (p.nt == 0) break;
      } else if (!take_part(ctl, part_at, p, err)) {
        break;
      }
      const Steps u(p);
      int page[kAhead][kG], in_page[kAhead][kG], rc[kG], rn[kG];       // pages ahead; rows of the values' tile, of the keys'
#pragma unroll
      for (int k = 0; k < kAhead; ++k) entries(min(p.j0 + k, p.j1 - 1), page[k], in_page[k]);
      for (int m = 0; lw == 0 && m < (u.dual ? 2 : 1); ++m) {
        const int b = u.dual ? m : qb;
        uint32_t& qn = b ? qn1 : qn0;
        if (!wait32(&ctl->q_empty[b], qn ^ 1, ctl, err, W_Q_EMPTY)) {
          ok = false;
          break;
        }
        ++qn;
        if (lane == 0) {
          // the rows of the next sequences come along: their products are not used
          tc::mbar_arrive_expect_tx(&ctl->q_full[b], kTile);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tc::tma_load_3d(sQ + b * kTile + h * kHalf, &mapQ, &ctl->q_full[b], 64 * h, p.h * a.g,
                            p.q.row0 + ((p.vg * a.vecs + m * 128) >> a.g_log2));
        }
      }
      if (!u.dual) qb ^= 1;
      for (int i = 0; ok && i <= u.tiles; ++i) {
        if (i < u.tiles) {
          places(page[0], in_page[0], rn);
#pragma unroll
          for (int k = 0; k + 1 < kAhead; ++k) {
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              page[k][g] = page[k + 1][g];
              in_page[k][g] = in_page[k + 1][g];
            }
          }
          entries(min(p.j0 + i + kAhead, p.j1 - 1), page[kAhead - 1], in_page[kAhead - 1]);
          ok = issue(&mapK, a.k_pool, rn);
          if (ok && i == 0 && lw == 0) ahead = plan();
        }
        if (ok && i > 0) ok = issue(&mapV, a.v_pool, rc);
#pragma unroll
        for (int k = 0; k < kG; ++k) rc[k] = rn[k];
      }
    }
    if (kGather) asm volatile("cp.async.wait_all;" ::: "memory");
    // copies in flight land before the CTA may end: all have been waited for where no
    // wait gave up
    if (!ok || ctl->abort_flag) {
      for (uint32_t c = it > (uint32_t)kSt ? it - kSt : 0; c < it; ++c) {
        tc::mbar_wait(&ctl->full[c % kSt], (c / kSt) & 1);
      }
      if (qn0 > 0) tc::mbar_wait(&ctl->q_full[0], (qn0 - 1) & 1);
      if (qn1 > 0) tc::mbar_wait(&ctl->q_full[1], (qn1 - 1) & 1);
    }
  } else if (warp == kWarpS) {
    // ------------------------------ S = Q K^T ------------------------------
    constexpr uint32_t idesc = tc::idesc_bf16_f32(128, kKB);
    uint32_t it = 0, c0 = 0, c1 = 0, qn0 = 0, qn1 = 0;
    int qb = 0;
    bool ok = true;
    while (ok && take_part(ctl, part_at, p, err)) {
      const Steps u(p);
      if (u.dual || qb == 0) ok = wait32(&ctl->q_full[0], qn0++, ctl, err, W_Q_FULL);
      if (ok && (u.dual || qb == 1)) ok = wait32(&ctl->q_full[1], qn1++, ctl, err, W_Q_FULL);
      if (!ok) break;
      for (int k = 0; k < u.n; ++k) {
        const int w = k & 1;
        const uint32_t c = w ? c1 : c0;
        // (What was in the ring's slot before has been full: keys of an earlier step, waited for here,
        // or values of a step three before this one or earlier: of the last two steps, which alone
        // need not have been waited for, the values lie at most three places in front.)
        const uint32_t q = it + u.k_item(u.tile(k));
        const int st = q % kSt;
        if (!wait32(&ctl->full[st], q / kSt, ctl, err, W_K_FULL)) {
          ok = false;
          break;
        }
        const uint64_t qd = uniform64(tc::smem_desc_k128(tc::smem_u32(sQ) + (u.dual ? w : qb) * kTile));
        const uint64_t kd = uniform64(tc::smem_desc_k128(tc::smem_u32(sR) + st * kTile, kGroup));
        const uint32_t d = __shfl_sync(0xffffffffu, tmem + w * kKB, 0);
        // the buffer holds P of the stream's step before until that step's P.V is done: waited for
        // last, as it is what the product waits for
        if (c > 0 && !wait32(&ctl->pv_done[w], c - 1, ctl, err, W_S_FREE)) {
          ok = false;
          break;
        }
        if (kGather) tc::fence_proxy_async_smem();         // the copies' writes are the generic proxy's
        tc::tc_fence_after();
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_bf16(d, qd + ((kk >> 2) * kHalf + (kk & 3) * 32) / 16,
                         kd + ((kk >> 2) * kAtom + (kk & 3) * 32) / 16, idesc, kk != 0);
          tc::mma_commit(&ctl->s_full[w]);
          if (!u.dual || w == 1) tc::mma_commit(&ctl->empty[st]);
          if (k == u.n - 1) {
            if (u.dual || qb == 0) tc::mma_commit(&ctl->q_empty[0]);
            if (u.dual || qb == 1) tc::mma_commit(&ctl->q_empty[1]);
          }
        }
        __syncwarp();
        if (w)
          ++c1;
        else
          ++c0;
      }
      if (!u.dual) qb ^= 1;
      it += 2 * u.tiles;
    }
  } else if (warp == kWarpPV) {
    // ------------------------------- O += P V -------------------------------
    constexpr uint32_t idesc = tc::idesc_bf16_f32(128, D, /*b_mn_major=*/true);
    uint32_t it = 0, c0 = 0, c1 = 0, parts = 0, with_new = 0;
    bool ok = true;
    while (ok && take_part(ctl, part_at, p, err)) {
      const Steps u(p);
      unsigned long long found = 0;
      for (int k = 0; k < u.n; ++k) {
        const int w = k & 1, i = u.tile(k);
        const uint32_t q = it + u.v_item(i);
        const int st = q % kSt;
        // (what was in the ring's slot before has been full: it is a value tile of an
        // earlier step, or a key tile whose weights have been waited for)
        if (!wait32(&ctl->full[st], q / kSt, ctl, err, W_V_FULL)) {
          ok = false;
          break;
        }
        if (has_new(p, p.j0 + i) && (!u.dual || w == 0)) {
          // the values of new tokens, and the rows behind them that a box brought along
          constexpr int kPieces = D / 8, kRows = 32 / kPieces;
          const int key0 = (p.j0 + i) * kKB;
          const int n0 = max(p.q.len - key0, 0), n1 = min(kKB, p.q.len + p.q.n - key0);
          const int n2 = kGather ? n1 : (n1 + box - 1) / box * box;
          const int piece = lane % kPieces;
          for (int m = n0 + lane / kPieces; m < n2; m += kRows) {
            uint4* at = reinterpret_cast<uint4*>(sR + st * kTile + piece_at<D>(m, piece));
            uint4 x = make_uint4(0, 0, 0, 0);
            if (m < n1) {
              x = *at;
              if (!(nonfinite2(x.x) || nonfinite2(x.y) || nonfinite2(x.z) || nonfinite2(x.w))) continue;
              x.x = drop_nonfinite(x.x);
              x.y = drop_nonfinite(x.y);
              x.z = drop_nonfinite(x.z);
              x.w = drop_nonfinite(x.w);
              found |= 1ull << (key0 + m - p.q.len);
            }
            *at = x;
          }
          tc::fence_proxy_async_smem();
          found = (unsigned long long)__reduce_or_sync(0xffffffffu, (uint32_t)(found >> 32)) << 32 |
                  __reduce_or_sync(0xffffffffu, (uint32_t)found);
          if (lane == 0) ctl->fix[with_new % kFix] = found;     // read once this product is done
          __syncwarp();
        }
        const uint64_t vd = uniform64(tc::smem_desc_mn128(tc::smem_u32(sR) + st * kTile, kAtom, kGroup));
        const uint32_t d = __shfl_sync(0xffffffffu, tmem + kColO + w * D, 0), ad = __shfl_sync(0xffffffffu, tmem + w * kKB, 0);
        ok = wait32(&ctl->p_full[w], w ? c1 : c0, ctl, err, W_P_FULL);
        // the accumulators were last read at the end of the part before
        if (ok && k == 0) ok = wait32(&ctl->o_empty, parts ^ 1, ctl, err, W_O_EMPTY);
        if (!ok) break;
        if (kGather) tc::fence_proxy_async_smem();
        tc::tc_fence_after();
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kKB / 16; ++kk)
            tc::mma_bf16_ts(d, ad + kk * 8, vd + kk * 2 * kGroup / 16, idesc, (k > 1 || kk != 0) ? 1u : 0u);
          tc::mma_commit(&ctl->pv_done[w]);
          if (!u.dual || w == 1) tc::mma_commit(&ctl->empty[st]);
        }
        __syncwarp();
        if (w)
          ++c1;
        else
          ++c0;
      }
      if (!ok) break;
      ++parts;
      if (has_new(p, p.j1 - 1)) ++with_new;
      it += 2 * u.tiles;
    }
  } else if (warp < kWarpLoad) {
    // ------------------------------- softmax -------------------------------
    // a stream has eight warps: warp i of them TMEM lane quarter i % 4, half i / 4 of
    // it: 16 M rows, a thread two of them with 32 keys each.  (Eight warps for both
    // streams in turn: 440 us instead of 412 on 8 trees of 64 over 33k.)
    const int w = warp >> 3, quarter = warp & 3, half = warp >> 2 & 1;
    const int base = quarter * 32 + half * 16;
    const int c4 = lane & 3;
    const int R0 = base + (lane >> 2), R1 = R0 + 8;
    const float scale = a.scale;
    const uint64_t sc2 = pack2(scale, scale);
    const uint32_t tS = tmem + ((uint32_t)base << 16) + w * kKB;
    uint32_t c = 0, other = 0, parts = 0, with_new = 0;     // steps of this stream and the other one, parts
    while (take_part(ctl, part_at, p, err)) {
      const Steps u(p);
      const bool news = has_new(p, p.j1 - 1);
      Seen all{};
      if (news) all = seen_of_all(a.parents, p.q, err);
      // the rows' references (scores) and this thread's part of their sums; odd: some
      // reference of the warp is -infinity or so large that the rounding of its
      // product would show
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      bool odd = true, ok = true;
      for (int k = w; k < u.n; k += 2, ++c) {
        const int j = p.j0 + u.tile(k);
        if (!wait32(&ctl->s_full[w], c, ctl, err, W_S_FULL)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const bool bad = ctl->bad_page != 0;
        if (__builtin_expect(has_new(p, j) || bad, 0)) {
          // the scores of keys that a row does not see, replaced where they are
          uint64_t seen0 = ~(uint64_t)0, seen1 = seen0;
          if (news) {
            const int v0 = (u.dual ? w * 128 : 0) + R0;
            seen0 = seen_by(all, (p.vg * a.vecs + min(v0, p.n_vec - 1)) >> a.g_log2);
            seen1 = seen_by(all, (p.vg * a.vecs + min(v0 + 8, p.n_vec - 1)) >> a.g_log2);
          }
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            const int rel = j * kKB + 32 * b - p.q.len;
            uint32_t w0 = seen_word(seen0, rel), w1 = seen_word(seen1, rel);
            if (bad) {                        // keys whose page is not in the pool
              const int key = j * kKB + 32 * b + lane;
              int page = 0;
              if (key < p.q.len + p.q.n)
                page = a.seq.tables[(int64_t)p.s * a.seq.max_blocks + key / a.seq.block_size];
              const uint32_t there = __ballot_sync(0xffffffffu, page >= 0 && page < a.seq.n_pool_blocks);
              w0 &= there;
              w1 &= there;
            }
            uint32_t x[16];
            tc::tmem_ld_16x256b_x4(tS + 32 * b, x);
            tc::tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              constexpr uint32_t kMasked = 0xff800000u;    // -infinity
              if (!(w0 >> (8 * q + 2 * c4) & 1)) x[4 * q] = kMasked;
              if (!(w0 >> (8 * q + 2 * c4) & 2)) x[4 * q + 1] = kMasked;
              if (!(w1 >> (8 * q + 2 * c4) & 1)) x[4 * q + 2] = kMasked;
              if (!(w1 >> (8 * q + 2 * c4) & 2)) x[4 * q + 3] = kMasked;
            }
            tc::tmem_st_16x256b_x4(tS + 32 * b, x);
          }
          tc::tmem_st_wait();
        }
        float al0 = 1.f, al1 = 1.f, s0, s1;   // factors of the sums so far; this tile's sums
        // Rows whose reference is set or raised now, and whose was in this step: each row by
        // its own scores alone (the four lanes of a row agree).
        bool want0 = k < 2 || m0 == -INFINITY, want1 = k < 2 || m1 == -INFINITY;
        bool done0 = false, done1 = false;
        bool any_want = odd;                  // uniform; `odd` before the first step
        uint32_t y[32];                       // weights: key pairs of both rows
#pragma unroll 1
        while (true) {
          if (__builtin_expect(any_want, 0)) {
            float a0 = -INFINITY, b0 = -INFINITY;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              uint32_t r[32];
              tc::tmem_ld_16x256b_x8(tS + 64 * h, r);
              tc::tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                a0 = max3(a0, __uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]));
                b0 = max3(b0, __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
              }
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
              a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, o));
              b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, o));
            }
            if (want0) {
              if (k > 1 && m0 != -INFINITY && a0 > m0) al0 = ex2((m0 - a0) * scale);
              m0 = k < 2 ? a0 : fmaxf(m0, a0);
              done0 = true;
            }
            if (want1) {
              if (k > 1 && m1 != -INFINITY && b0 > m1) al1 = ex2((m1 - b0) * scale);
              m1 = k < 2 ? b0 : fmaxf(m1, b0);
              done1 = true;
            }
            odd = __any_sync(0xffffffffu, !(fmaxf(fabsf(m0), fabsf(m1)) * scale < kFar));
          }
          float g0 = -m0 * scale, g1 = -m1 * scale, f0 = 0.f, f1 = 0.f;
          if (__builtin_expect(odd, 0)) {
            // rows whose every score so far is -infinity: weights of 0, not 2^(-inf + inf);
            // rows whose scores are far: the differences first
            f0 = m0 == -INFINITY ? 0.f : m0;
            f1 = m1 == -INFINITY ? 0.f : m1;
            const bool far0 = fabsf(f0) * scale >= kFar, far1 = fabsf(f1) * scale >= kFar;
            g0 = far0 ? 0.f : -f0 * scale;
            g1 = far1 ? 0.f : -f1 * scale;
            if (!far0) f0 = 0.f;
            if (!far1) f1 = 0.f;
          }
          const uint64_t ng0 = pack2(g0, g0), ng1 = pack2(g1, g1);
          uint64_t acc0 = 0, acc1 = 0;        // (even keys, odd keys) of each row
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[32];
            tc::tmem_ld_16x256b_x8(tS + 64 * h, r);
            tc::tmem_ld_wait();
            if (__builtin_expect(odd, 0)) {
#pragma unroll
              for (int q = 0; q < 32; ++q) r[q] = __float_as_uint(__uint_as_float(r[q]) - ((q & 2) ? f1 : f0));
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float2 x01 = unpack2(fma2(pack2(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1])), sc2, ng0));
              const float2 x23 = unpack2(fma2(pack2(__uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3])), sc2, ng1));
              const float e0 = ex2(x01.x), e1 = ex2(x01.y), e2 = ex2(x23.x), e3 = ex2(x23.y);
              acc0 = add2(acc0, pack2(e0, e1));
              acc1 = add2(acc1, pack2(e2, e3));
              y[16 * h + 2 * q] = pack_bf16x2(e0, e1);
              y[16 * h + 2 * q + 1] = pack_bf16x2(e2, e3);
            }
          }
          const float2 z0 = unpack2(acc0), z1 = unpack2(acc1);
          s0 = z0.x + z0.y;
          s1 = z1.x + z1.y;
          // (a sum that is not a number passes it too)
          const bool over0 = !done0 && !(s0 <= kMaxSum), over1 = !done1 && !(s1 <= kMaxSum);
          if (!__any_sync(0xffffffffu, over0 || over1)) break;
          const uint32_t row = 0xFu << (lane & 28);
          want0 = (__ballot_sync(0xffffffffu, over0) & row) != 0;
          want1 = (__ballot_sync(0xffffffffu, over1) & row) != 0;
          any_want = true;
        }
        tc::tmem_st_16x128b_x16(tS, y);
        // the accumulator's rows, by the whole warp when any of them needs it (the
        // factor is 1 for the others), once the stream's step before has been added
        if (__builtin_expect(any_want && __any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f), 0)) {
          if (!wait32(&ctl->pv_done[w], c - 1, ctl, err, W_PV_DONE)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint64_t a0 = pack2(al0, al0), a1 = pack2(al1, al1);
#pragma unroll 1
          for (int e = 0; e < D; e += 64) {
            uint32_t o[32];
            const uint32_t tO = tmem + ((uint32_t)base << 16) + kColO + w * D + e;
            tc::tmem_ld_16x256b_x8(tO, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 32; q += 2) {
              const float2 y = unpack2(mul2(pack2(__uint_as_float(o[q]), __uint_as_float(o[q + 1])), (q & 2) ? a1 : a0));
              o[q] = __float_as_uint(y.x);
              o[q + 1] = __float_as_uint(y.y);
            }
            tc::tmem_st_16x256b_x8(tO, o);
          }
        }
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl->p_full[w]);
        l0 = l0 * al0 + s0;
        l1 = l1 * al1 + s1;
      }
      if (!ok) break;
      other += (u.n + w) / 2;
      // the rows' references and sums to shared memory, in a fixed order
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, o);
        l1 += __shfl_xor_sync(0xffffffffu, l1, o);
      }
      // (of the part before they have been read once its accumulators have)
      if (parts > 0 && !wait32(&ctl->o_empty, parts - 1, ctl, err, W_O_EMPTY)) break;
      if (c4 == 0) {
        ctl->ml[w][R0] = make_float2(m0 * scale, l0);
        ctl->ml[w][R1] = make_float2(m1 * scale, l1);
      }
      tc::mbar_arrive(&ctl->x_full);
      if (!wait32(&ctl->x_full, parts, ctl, err, W_X_FULL)) break;
      if (w < u.n && !wait32(&ctl->pv_done[w], c - 1, ctl, err, W_O_FULL)) break;
      if (1 - w < u.n && !wait32(&ctl->pv_done[1 - w], other - 1, ctl, err, W_O_FULL)) break;
      tc::tc_fence_after();
      // outputs: a thread one M row, with a half of its columns (of two M tiles) or a quarter
      const int row = quarter * 32 + lane;
      const bool whole = p.j0 == 0 && p.j1 == p.nt;
      const bool two = !u.dual && u.n > 1;    // one M tile: the streams' sums are added
      const int64_t slot = ((int64_t)blockIdx.x * 2 + (p.j0 == 0 ? 1 : 0)) * kTreeTcVecs;
      unsigned long long found = 0;
      if (news) {
        found = *(volatile unsigned long long*)&ctl->fix[with_new % kFix];
        ++with_new;
      }
      {
        const int mt = u.dual ? w : 0, cols = u.dual ? D / 2 : D / 4;
        const int e_begin = (u.dual ? half : warp >> 2) * cols;
        const int v = mt * 128 + row;
        const bool valid = v < p.n_vec;
        const int vi = p.vg * a.vecs + min(v, p.n_vec - 1), node = vi >> a.g_log2;
        const float2 x = ctl->ml[mt][row];
        float M = x.x, sum = x.y, f0 = 1.f, f1 = 0.f;
        if (two) {
          const float2 y = ctl->ml[1][row];
          M = fmaxf(x.x, y.x);
          const float ref = M == -INFINITY ? 0.f : M;
          f0 = ex2(x.x - ref);
          f1 = ex2(y.x - ref);
          sum = f0 * x.y + f1 * y.y;
        }
        const unsigned long long fix = found ? found & seen_by(all, node) : 0;
        const bool none = sum == 0.f;         // no key that the row sees has weight: zeros
        const float inv = 1.f / sum;
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.O) +
                             ((int64_t)(p.q.row0 + node) * a.n_q_heads + p.h * a.g + (vi & (a.g - 1))) * D;
        const uint32_t tO = tmem + ((uint32_t)(quarter * 32) << 16) + kColO + mt * D;
        // (a short loop: a part's end runs once, out of a cold instruction cache)
#pragma unroll 1
        for (int e0 = e_begin; e0 < e_begin + cols; e0 += 8) {
          uint32_t o[8], o1[8];
          tc::tmem_ld_32x32b_x8(tO + e0, o);
          if (two) tc::tmem_ld_32x32b_x8(tO + D + e0, o1);
          tc::tmem_ld_wait();
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] = __uint_as_float(o[e]) * f0;
            if (two) y[e] = fmaf(__uint_as_float(o1[e]), f1, y[e]);
          }
          if (valid && whole) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = none ? 0.f : y[e] * inv;
            Vec8<__nv_bfloat16>::store(out + e0, y);
          } else if (valid) {
            Vec8<float>::store(a.part_o + (slot + v) * D + e0, y);
          }
          __syncwarp();
        }
        if (valid && !whole && e_begin == 0) a.part_ml[slot + v] = make_float2(M, sum);
        if (fix && valid) {                   // rare
          if (whole)
            add_nonfinite(out + e_begin, cols, fix, a, p, e_begin, D);
          else
            add_nonfinite(a.part_o + (slot + v) * D + e_begin, cols, fix, a, p, e_begin, D);
        }
        __syncwarp();
      }
      tc::tc_fence_before();
      tc::mbar_arrive(&ctl->o_empty);         // read: the next part's first products may start
      ++parts;
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (ctl->abort_flag) {                      // products in flight get time to end
#pragma unroll 1
    for (int k = 0; k < 1000; ++k) __nanosleep(1000);
    __syncthreads();
  }
  if (warp == kWarpS) tc::tmem_dealloc(tmem, kTmemCols);
}

template <int D, bool kGather>
cudaError_t launch_g(const CUtensorMap& mQ, const CUtensorMap& mK, const CUtensorMap& mV, const TreeArgs& a, int box,
                     cudaStream_t s) {
  const cudaError_t e =
      set_dyn_smem_once(reinterpret_cast<const void*>(tree_tc_kernel<D, kGather>), smem_bytes<D>());
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_tc_kernel<D, kGather>, dim3(a.workers), dim3(kThreads), smem_bytes<D>(), s, mQ, mK, mV, a,
                    box);
}

template <int D> cudaError_t launch_d(const TreeArgs& a, cudaStream_t s) {
  CUtensorMap mQ, mK, mV;
  const uint64_t dq[3] = {(uint64_t)D, (uint64_t)a.n_q_heads, (uint64_t)a.seq.n_rows};
  const uint64_t sq[2] = {(uint64_t)D * 2, (uint64_t)a.n_q_heads * D * 2};
  const uint32_t bq[3] = {64, (uint32_t)a.g, (uint32_t)(128 / a.g)};
  if (!make_map_3d(&mQ, a.Q, dq, sq, bq)) return cudaErrorInvalidValue;
  // the rows of a box: a power of two that divides a page
  const int box = std::min(kKB, a.seq.block_size & -a.seq.block_size);
  if (box < 8) return launch_g<D, true>(mQ, mQ, mQ, a, kKB, s);
  const int64_t rows = a.seq.n_pool_blocks * a.seq.block_size, cols = (int64_t)a.n_kv_heads * D;
  if (!make_map_groups(&mK, a.k_pool, rows, cols, D / 64, box / 8) ||
      !make_map_groups(&mV, a.v_pool, rows, cols, D / 64, box / 8))
    return cudaErrorInvalidValue;
  return launch_g<D, false>(mQ, mK, mV, a, box, s);
}

}  // namespace

cudaError_t launch_tree_tc(const fuse_layer_desc_t& d, const TreeArgs& a, cudaStream_t s) {
  return d.head_dim == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

}  // namespace fusekv
