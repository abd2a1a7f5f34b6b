// Attention of trees over a paged cache on tcgen05 tensor cores (bf16 layers).
//
// Work unit: one sequence, KV head and up to 256 query vectors (new token, query
// head of the KV head), as one or two M = 128 tiles; keys stream in tiles of 128
// through a ring in shared memory.  Two streams alternate, each with a score
// buffer and an accumulator of its own:
//   two M tiles   stream w takes M tile w, both with the same keys
//   one M tile    stream w takes every second key tile; the two softmaxes are
//                 joined when the unit ends
// so that one stream's products run beside the other's softmax.  Per step
//   S = Q K^T     tcgen05.mma into TMEM columns [128 w, 128 w + 128)
//   P = 2^(S - m) eight warps in registers, bf16, written back over S
//   O += P V      tcgen05.mma with A = P in TMEM, V MN-major in shared memory
// The reference m is the first tile's maximum.  A later tile is weighed against it
// as it stands, without its maximum being looked for: only where a thread's sum of
// its weights passes 2^16 (no weight does otherwise) is the reference raised, O and
// the running sum rescaled and the tile weighed once more.
//
// Keys and values lie in pages.  With pages of a multiple of 8 tokens a tile is
// copied by TMA boxes of as many rows as always lie in one page; what lies
// behind a sequence's last slot in its page comes along and is masked, its values
// cleared.  With other pages the rows are gathered four at a time, and a group that is
// not whole (the sequence's end, a page outside the pool) is copied by a lane
// itself.  (Gathering by 16-byte cp.async, four warps, kept the load/store path so
// busy that the softmax's shuffles waited: 550 us instead of @@ on 8 trees of 64 over 33k.)
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
bool make_map_gather(CUtensorMap* m, const void* base, int64_t rows, int64_t cols);

namespace {

constexpr int kKB = kTreeTcTile;              // keys per tile
constexpr int kHalf = 128 * 64 * 2;           // 64 columns of a 128-row tile (16 KB)
// four warps load: a copy instruction takes its operands from uniform registers, so
// that a warp's lanes issue theirs one after another, about 75 cycles each
constexpr int kWarpLoad = 8, kLoadWarps = 4, kWarpS = 12, kWarpPV = 13, kWarpLook = 14;
constexpr int kThreads = 15 * 32;
constexpr int kAhead = 3;                     // tiles whose pages are looked up ahead of their copies
constexpr int kTmemCols = 512;                // S of both streams | O of both
constexpr float kMaxSum = 65536.f;            // of a thread's 32 weights: they keep their relative precision up to there
constexpr float kFar = 1048576.f;             // of a score in log2 units: 2^-4 is its last place
constexpr int kMaxStages = 10;
constexpr int kFix = 8;                       // parts with new tokens that the look may be ahead by, and more

template <int D> struct Ring {
  static constexpr int tile = (D / 64) * kHalf;
  static constexpr int stages = D == 128 ? 5 : 10;
};

struct Ctl {
  uint64_t q_full[2], q_empty[2];
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t look_full[kMaxStages];             // value tiles that are looked through first, by ring slot
  uint64_t s_full[2], p_full[2], pv_done[2];             // by stream
  uint64_t x_full, o_empty;
  unsigned long long fix[kFix];               // new tokens with values that are not finite
  uint32_t tmem_base;
  volatile int abort_flag;
  volatile int bad_page;                      // some page of this CTA's units is outside the pool
  float2 ml[2][128];                          // maximum and sum of each stream's rows
  int64_t s_warp[kThreads / 32];
};

constexpr int kCtlBytes = 3072;               // in front of the tiles, which start at multiples of 1024
static_assert(sizeof(Ctl) <= kCtlBytes, "shared memory");
template <int D> constexpr int smem_bytes() { return kCtlBytes + (2 + Ring<D>::stages) * Ring<D>::tile; }
static_assert(smem_bytes<128>() <= 227 * 1024 && smem_bytes<64>() <= 227 * 1024, "shared memory");

// Which wait gave up: info = wait id << 16 | CTA.
enum TreeWait : uint32_t {
  W_Q_EMPTY = 1, W_EMPTY, W_Q_FULL, W_S_FREE, W_K_FULL, W_P_FULL, W_V_FULL, W_O_EMPTY, W_LOOK_FULL,
  W_S_FULL, W_PV_DONE, W_O_FULL, W_X_FULL
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

__device__ __forceinline__ void arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(tc::smem_u32(bar)), "r"(n) : "memory");
}

// K-step kk (16 columns) of a 128-row K-major tile stored in 64-column halves.
__device__ __forceinline__ uint64_t kmajor_step(uint32_t tile, int kk) {
  return tc::smem_desc_k128(tile + (kk >> 2) * kHalf + (kk & 3) * 32);
}

__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}

// Out of line, as six roles call it once per part.
__device__ __noinline__ bool next_of(const TreeArgs& a, TreeWalk& w, TreePart& p) { return next_part(a, w, p); }

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
  constexpr int kTile = Ring<D>::tile, kSt = Ring<D>::stages;
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
      tc::mbar_init(&ctl->p_full[i], 256);
      tc::mbar_init(&ctl->pv_done[i], 1);
    }
    for (int i = 0; i < kSt; ++i) {
      tc::mbar_init(&ctl->full[i], kLoadWarps);
      tc::mbar_init(&ctl->empty[i], 1);
      tc::mbar_init(&ctl->look_full[i], kLoadWarps);
    }
    tc::mbar_init(&ctl->x_full, 256);
    tc::mbar_init(&ctl->o_empty, 256);
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
  TreeWalk walk = start_walk<kThreads>(a, blockIdx.x, ctl->s_warp);
  const bool work = walk.t < walk.end;        // uniform
  TreePart p{};

  if (!work) {
  } else if (warp >= kWarpLoad && warp < kWarpLoad + kLoadWarps) {
    // -------------------------------- loads --------------------------------
    // a lane copies one box, or gathers a group of four rows
    uint32_t it = 0, qn0 = 0, qn1 = 0;
    int qb = 0;
    bool ok = true;
    constexpr int kG = kGather ? 4 : 1;       // pages that a lane looks up per tile
    const int lw = warp - kWarpLoad;
    const int n_box = kGather ? 32 : kKB / box;
    const int rows = kGather ? 4 : box;       // of a group
    // this lane's copy of a tile: its group (and half of the columns; a gathering lane takes both)
    const int op = lane * kLoadWarps + lw, group = kGather ? op : op % n_box;
    const int ops = kGather ? n_box : n_box * (D / 64);
    const bool mine = op < ops;
    const uint32_t share = (uint32_t)(ops - lw + kLoadWarps - 1) / kLoadWarps * (kTile / ops);       // bytes of the warp's
    const int none = (int)(a.seq.n_pool_blocks * a.seq.block_size);       // a row outside the pool: reads as zeros
    // the pages of this lane's rows of tile j (-2: no key there), and their first slot's place
    auto entries = [&](int j, int (&page)[kG], int& in_page) {
      const int key = j * kKB + group * rows, end = p.q.len + p.q.n;
      const int32_t* table = a.seq.tables + (int64_t)p.s * a.seq.max_blocks;
      int b = page_of(a.seq, key, &in_page), at = in_page;
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        page[i] = mine && key + i < end ? table[b] : -2;
        if (++at == a.seq.block_size) {
          at = 0;
          ++b;
        }
      }
    };
    auto places = [&](const int (&page)[kG], int in_page, int (&row)[kG]) {
      bool bad = false;
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        int at = in_page + i;
        if (kG > 1 && at >= a.seq.block_size) at %= a.seq.block_size;
        const bool there = page[i] >= 0 && page[i] < a.seq.n_pool_blocks;
        row[i] = there ? page[i] * a.seq.block_size + at : none;
        bad |= !there && page[i] != -2;
      }
      if (bad) {
        report_error(err, FUSE_ERR_DEVICE_BOUNDS, SITE_SEQ_PAGE, (uint32_t)p.s);
        ctl->bad_page = 1;
      }
    };
    auto issue = [&](const CUtensorMap* map, const void* pool, const int (&row)[kG], bool look) {
      const int st = it % kSt;
      if (!wait32(&ctl->empty[st], (it / kSt) ^ 1, ctl, err, W_EMPTY)) return false;
      uint64_t* bar = look ? &ctl->look_full[st] : &ctl->full[st];
      uint8_t* tile = sR + st * kTile;
      uint32_t bytes = share;
      bool whole = true;
      if constexpr (kGather) {
        // groups that are not whole: by the lane's own loads and stores
        whole = row[0] != none && row[1] != none && row[2] != none && row[3] != none;
        const unsigned self = __ballot_sync(0xffffffffu, mine && !whole);
        if (self) {
          if (mine && !whole) {
#pragma unroll 1
            for (int i = 0; i < 4 * (D / 8); ++i) {
              const int m = i / (D / 8), c = i % (D / 8);
              const int y = m == 0 ? row[0] : m == 1 ? row[1] : m == 2 ? row[2] : row[3];
              uint4 x = make_uint4(0, 0, 0, 0);
              if (y != none)
                x = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(pool) +
                                                    ((int64_t)y * a.n_kv_heads + p.h) * D + c * 8);
              const int at = group * 4 + m;
              *reinterpret_cast<uint4*>(tile + (c >> 3) * kHalf + at * 128 + (((c & 7) ^ (at & 7)) << 4)) = x;
            }
            tc::fence_proxy_async_smem();
          }
          bytes -= __popc(self) * 4 * D * 2;
          __syncwarp();
        }
      }
      __syncwarp();                           // (bad_page is set before the barrier's phase can end)
      if (lane == 0) tc::mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      if constexpr (kGather) {
        if (mine && whole)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tc::tma_gather4(tile + h * kHalf + group * 512, map, bar, p.h * D + 64 * h, row[0], row[1], row[2], row[3]);
      } else if (mine) {
        const int h = op / n_box;
        tc::tma_load_3d(tile + h * kHalf + group * box * 128, map, bar, 64 * h, p.h, row[0]);
      }
      ++it;
      return true;
    };
    while (ok && next_of(a, walk, p)) {
      const Steps u(p);
      int page[kAhead][kG], in_page[kAhead], rc[kG], rn[kG];       // pages ahead; rows of the values' tile, of the keys'
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
            for (int g = 0; g < kG; ++g) page[k][g] = page[k + 1][g];
            in_page[k] = in_page[k + 1];
          }
          entries(min(p.j0 + i + kAhead, p.j1 - 1), page[kAhead - 1], in_page[kAhead - 1]);
          ok = issue(&mapK, a.k_pool, rn, false);
        }
        if (ok && i > 0) ok = issue(&mapV, a.v_pool, rc, has_new(p, p.j0 + i - 1));
#pragma unroll
        for (int k = 0; k < kG; ++k) rc[k] = rn[k];
      }
    }
    // copies in flight land before the CTA may end: all have been waited for where no
    // wait gave up
    if (!ok || ctl->abort_flag) {
      for (uint32_t c = it > (uint32_t)kSt ? it - kSt : 0; c < it; ++c) {
        tc::mbar_wait(&ctl->full[c % kSt], (c / kSt) & 1);
      }
    }
  } else if (warp == kWarpS) {
    // ------------------------------ S = Q K^T ------------------------------
    constexpr uint32_t idesc = tc::idesc_bf16_f32(128, kKB);
    uint32_t it = 0, c0 = 0, c1 = 0, qn0 = 0, qn1 = 0;
    int qb = 0;
    bool ok = true;
    while (ok && next_of(a, walk, p)) {
      const Steps u(p);
      if (u.dual || qb == 0) ok = wait32(&ctl->q_full[0], qn0++, ctl, err, W_Q_FULL);
      if (ok && (u.dual || qb == 1)) ok = wait32(&ctl->q_full[1], qn1++, ctl, err, W_Q_FULL);
      if (!ok) break;
      for (int k = 0; k < u.n; ++k) {
        const int w = k & 1;
        const uint32_t c = w ? c1 : c0;
        // the buffer holds P of the stream's step before until that step's P.V is done
        // (and with it every ring item up to this one's slot has been full)
        if (c > 0 && !wait32(&ctl->pv_done[w], c - 1, ctl, err, W_S_FREE)) {
          ok = false;
          break;
        }
        const uint32_t q = it + u.k_item(u.tile(k));
        const int st = q % kSt;
        if (!wait32(&ctl->full[st], q / kSt, ctl, err, W_K_FULL)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t qa = tc::smem_u32(sQ) + (u.dual ? w : qb) * kTile, ka = tc::smem_u32(sR) + st * kTile;
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_bf16(tmem + w * kKB, kmajor_step(qa, kk), kmajor_step(ka, kk), idesc, kk != 0);
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
    uint32_t it = 0, c0 = 0, c1 = 0, parts = 0;
    bool ok = true;
    while (ok && next_of(a, walk, p)) {
      const Steps u(p);
      for (int k = 0; k < u.n; ++k) {
        const int w = k & 1, i = u.tile(k);
        const uint32_t q = it + u.v_item(i);
        const int st = q % kSt;
        // P first: the ring's earlier items have been full by then
        ok = wait32(&ctl->p_full[w], w ? c1 : c0, ctl, err, W_P_FULL) &&
             wait32(&ctl->full[st], q / kSt, ctl, err, W_V_FULL);
        // the accumulators were last read at the end of the part before
        if (ok && k == 0) ok = wait32(&ctl->o_empty, parts ^ 1, ctl, err, W_O_EMPTY);
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t va = tc::smem_u32(sR) + st * kTile;
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kKB / 16; ++kk)
            tc::mma_bf16_ts(tmem + kColO + w * D, tmem + w * kKB + kk * 8,
                            tc::smem_desc_mn128(va + kk * 16 * 128, kHalf), idesc, (k > 1 || kk != 0) ? 1u : 0u);
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
      it += 2 * u.tiles;
    }
  } else if (warp == kWarpLook) {
    // ------------------- values of new tokens looked through -------------------
    constexpr int kPieces = D / 8, kRows = 32 / kPieces;
    uint32_t it = 0, look = 0, with_new = 0;
    bool ok = true;
    while (ok && next_of(a, walk, p)) {
      const Steps u(p);
      unsigned long long found = 0;
      bool any = false;
      for (int i = 0; i < u.tiles; ++i) {
        const int j = p.j0 + i;
        if (!has_new(p, j)) continue;
        any = true;
        const int st = (it + u.v_item(i)) % kSt;
        if (!wait32(&ctl->look_full[st], look >> st, ctl, err, W_LOOK_FULL)) {
          ok = false;
          break;
        }
        look ^= 1u << st;
        const int key0 = j * kKB;
        // the new tokens' rows, and those behind them that a box brought along
        const int m0 = max(p.q.len - key0, 0), m1 = min(kKB, p.q.len + p.q.n - key0);
        const int m2 = kGather ? m1 : (m1 + box - 1) / box * box;
        const int piece = lane % kPieces;
        bool changed = false;
        for (int m = m0 + lane / kPieces; m < m2; m += kRows) {
          uint4* at = reinterpret_cast<uint4*>(sR + st * kTile + (piece >> 3) * kHalf + m * 128 +
                                               (((piece & 7) ^ (m & 7)) << 4));
          if (m >= m1) {
            *at = make_uint4(0, 0, 0, 0);
            changed = true;
            continue;
          }
          uint4 x = *at;
          if (nonfinite2(x.x) || nonfinite2(x.y) || nonfinite2(x.z) || nonfinite2(x.w)) {
            x.x = drop_nonfinite(x.x);
            x.y = drop_nonfinite(x.y);
            x.z = drop_nonfinite(x.z);
            x.w = drop_nonfinite(x.w);
            *at = x;
            found |= 1ull << (key0 + m - p.q.len);
            changed = true;
          }
        }
        if (changed) tc::fence_proxy_async_smem();
        found = (unsigned long long)__reduce_or_sync(0xffffffffu, (uint32_t)(found >> 32)) << 32 |
                __reduce_or_sync(0xffffffffu, (uint32_t)found);
        __syncwarp();
        if (lane == 0) {
          ctl->fix[with_new % kFix] = found;
          arrive_n(&ctl->full[st], kLoadWarps);
        }
      }
      with_new += any;
      it += 2 * u.tiles;
    }
  } else if (warp < kWarpLoad) {
    // ------------------------------- softmax -------------------------------
    // warp w: TMEM lane quarter w % 4, half w / 4 of it: 16 M rows, a thread two
    // of them with 32 keys each
    const int quarter = warp & 3, half = warp >> 2;
    const int base = quarter * 32 + half * 16;
    const int c4 = lane & 3;
    const int R0 = base + (lane >> 2), R1 = R0 + 8;
    const float scale = a.scale;
    const uint64_t sc2 = pack2(scale, scale);
    uint32_t c0 = 0, c1 = 0, parts = 0, with_new = 0;       // steps of each stream, parts
    while (next_of(a, walk, p)) {
      const Steps u(p);
      const bool news = has_new(p, p.j1 - 1);
      Seen all{};
      if (news) all = seen_of_all(a.parents, p.q, err);
      // of the stream at hand (m, l) and the other one (n, k): the rows' references
      // (scores) and this thread's part of their sums; odd: some reference of the warp
      // is -infinity or so large that the rounding of its product would show
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      float n0 = -INFINITY, n1 = -INFINITY, k0 = 0.f, k1 = 0.f;
      bool odd = true, odd_n = true;
      bool ok = true;
      for (int k = 0; k < u.n; ++k) {
        const int w = k & 1, j = p.j0 + u.tile(k);
        const uint32_t c = w ? c1 : c0;
        if (!wait32(&ctl->s_full[w], c, ctl, err, W_S_FULL)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t tS = tmem + ((uint32_t)base << 16) + w * kKB;
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
        bool raise = odd || k < 2;            // uniform; a stream's first step sets the references
        uint32_t r[64];
#pragma unroll 1
        while (true) {
          tc::tmem_ld_16x256b_x8(tS, *reinterpret_cast<uint32_t(*)[32]>(r));
          tc::tmem_ld_16x256b_x8(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
          tc::tmem_ld_wait();
          float g0 = -m0 * scale, g1 = -m1 * scale;
          if (__builtin_expect(raise, 0)) {
            float a0 = __uint_as_float(r[0]), a1 = __uint_as_float(r[1]);
            float b0 = __uint_as_float(r[2]), b1 = __uint_as_float(r[3]);
#pragma unroll
            for (int q = 1; q < 15; q += 2) {
              a0 = max3(a0, __uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 4]));
              a1 = max3(a1, __uint_as_float(r[4 * q + 1]), __uint_as_float(r[4 * q + 5]));
              b0 = max3(b0, __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 6]));
              b1 = max3(b1, __uint_as_float(r[4 * q + 3]), __uint_as_float(r[4 * q + 7]));
            }
            a0 = max3(a0, a1, fmaxf(__uint_as_float(r[60]), __uint_as_float(r[61])));
            b0 = max3(b0, b1, fmaxf(__uint_as_float(r[62]), __uint_as_float(r[63])));
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
              a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, o));
              b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, o));
            }
            if (k < 2) {
              m0 = a0;
              m1 = b0;
            } else {
              if (a0 > m0) al0 = ex2((m0 - a0) * scale);
              if (b0 > m1) al1 = ex2((m1 - b0) * scale);
              m0 = fmaxf(m0, a0);
              m1 = fmaxf(m1, b0);
            }
            // (a row whose every score so far is -infinity has weights of 0, not 2^(-inf + inf))
            float f0 = m0 == -INFINITY ? 0.f : m0, f1 = m1 == -INFINITY ? 0.f : m1;
            const bool far = __any_sync(0xffffffffu, fmaxf(fabsf(f0), fabsf(f1)) * scale >= kFar);
            odd = far || __any_sync(0xffffffffu, m0 == -INFINITY || m1 == -INFINITY);
            if (far) {                        // the differences first
#pragma unroll
              for (int q = 0; q < 64; ++q) r[q] = __float_as_uint(__uint_as_float(r[q]) - ((q & 2) ? f1 : f0));
              f0 = f1 = 0.f;
            }
            g0 = -f0 * scale;
            g1 = -f1 * scale;
          }
          const uint64_t ng0 = pack2(g0, g0), ng1 = pack2(g1, g1);
          uint64_t acc0 = 0, acc1 = 0;        // (even keys, odd keys) of each row
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const float2 x01 = unpack2(fma2(pack2(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1])), sc2, ng0));
            const float2 x23 = unpack2(fma2(pack2(__uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3])), sc2, ng1));
            const float e0 = ex2(x01.x), e1 = ex2(x01.y), e2 = ex2(x23.x), e3 = ex2(x23.y);
            acc0 = add2(acc0, pack2(e0, e1));
            acc1 = add2(acc1, pack2(e2, e3));
            r[2 * q] = pack_bf16x2(e0, e1);
            r[2 * q + 1] = pack_bf16x2(e2, e3);
          }
          const float2 y0 = unpack2(acc0), y1 = unpack2(acc1);
          s0 = y0.x + y0.y;
          s1 = y1.x + y1.y;
          if (raise || __all_sync(0xffffffffu, fmaxf(s0, s1) <= kMaxSum && s0 == s0 && s1 == s1)) break;
          raise = true;                       // (a sum that is not a number among them)
        }
        tc::tmem_st_16x128b_x16(tS, *reinterpret_cast<uint32_t(*)[32]>(r));
        // the accumulator's rows, by the whole warp when any of them needs it (the
        // factor is 1 for the others), once the stream's step before has been added
        if (__builtin_expect(raise && __any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f), 0)) {
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
        tc::mbar_arrive(&ctl->p_full[w]);
        l0 = l0 * al0 + s0;
        l1 = l1 * al1 + s1;
        if (w)
          ++c1;
        else
          ++c0;
        // the other stream's turn
        float z;
        z = m0; m0 = n0; n0 = z;
        z = m1; m1 = n1; n1 = z;
        z = l0; l0 = k0; k0 = z;
        z = l1; l1 = k1; k1 = z;
        const bool y = odd;
        odd = odd_n;
        odd_n = y;
      }
      if (!ok) break;
      // the rows' references and sums to shared memory, in a fixed order
      if (u.n & 1) {
        float z;
        z = m0; m0 = n0; n0 = z;
        z = m1; m1 = n1; n1 = z;
        z = l0; l0 = k0; k0 = z;
        z = l1; l1 = k1; k1 = z;
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, o);
        l1 += __shfl_xor_sync(0xffffffffu, l1, o);
        k0 += __shfl_xor_sync(0xffffffffu, k0, o);
        k1 += __shfl_xor_sync(0xffffffffu, k1, o);
      }
      // (of the part before they have been read once its accumulators have)
      if (parts > 0 && !wait32(&ctl->o_empty, parts - 1, ctl, err, W_O_EMPTY)) break;
      if (c4 == 0) {
        ctl->ml[0][R0] = make_float2(m0 * scale, l0);
        ctl->ml[0][R1] = make_float2(m1 * scale, l1);
        ctl->ml[1][R0] = make_float2(n0 * scale, k0);
        ctl->ml[1][R1] = make_float2(n1 * scale, k1);
      }
      tc::mbar_arrive(&ctl->x_full);
      if (!wait32(&ctl->x_full, parts, ctl, err, W_X_FULL)) break;
      if (!wait32(&ctl->pv_done[0], c0 - 1, ctl, err, W_O_FULL)) break;
      if (u.n > 1 && !wait32(&ctl->pv_done[1], c1 - 1, ctl, err, W_O_FULL)) break;
      tc::tc_fence_after();
      // outputs: a thread one M row and half of its columns
      const int row = quarter * 32 + lane;
      const bool whole = p.j0 == 0 && p.j1 == p.nt;
      const bool two = !u.dual && u.n > 1;    // one M tile: the streams' sums are added
      const int64_t slot = ((int64_t)blockIdx.x * 2 + (p.j0 == 0 ? 1 : 0)) * kTreeTcVecs;
      unsigned long long found = 0;
      if (news) {
        found = *(volatile unsigned long long*)&ctl->fix[with_new % kFix];
        ++with_new;
      }
      for (int mt = 0; mt < (u.dual ? 2 : 1); ++mt) {
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
        const float inv = 1.f / sum;
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.O) +
                             ((int64_t)(p.q.row0 + node) * a.n_q_heads + p.h * a.g + (vi & (a.g - 1))) * D;
        const uint32_t tO = tmem + ((uint32_t)(quarter * 32) << 16) + kColO + mt * D;
        // (a short loop: a part's end runs once, out of a cold instruction cache)
#pragma unroll 1
        for (int e0 = half * (D / 2); e0 < (half + 1) * (D / 2); e0 += 8) {
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
            for (int e = 0; e < 8; ++e) y[e] *= inv;
            Vec8<__nv_bfloat16>::store(out + e0, y);
          } else if (valid) {
            Vec8<float>::store(a.part_o + (slot + v) * D + e0, y);
          }
          __syncwarp();
        }
        if (valid && !whole && half == 0) a.part_ml[slot + v] = make_float2(M, sum);
        if (fix && valid) {                   // rare
          const int e0 = half * (D / 2);
          if (whole)
            add_nonfinite(out + e0, D / 2, fix, a, p, e0, D);
          else
            add_nonfinite(a.part_o + (slot + v) * D + e0, D / 2, fix, a, p, e0, D);
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
  const int64_t rows = a.seq.n_pool_blocks * a.seq.block_size;
  // the rows of a box: a power of two that divides a page
  const int box = std::min(kKB, a.seq.block_size & -a.seq.block_size);
  if (box < 8) {
    if (!make_map_gather(&mK, a.k_pool, rows, (int64_t)a.n_kv_heads * D) ||
        !make_map_gather(&mV, a.v_pool, rows, (int64_t)a.n_kv_heads * D))
      return cudaErrorInvalidValue;
    return launch_g<D, true>(mQ, mK, mV, a, box, s);
  }
  const uint64_t dk[3] = {(uint64_t)D, (uint64_t)a.n_kv_heads, (uint64_t)rows};
  const uint64_t sk[2] = {(uint64_t)D * 2, (uint64_t)a.n_kv_heads * D * 2};
  const uint32_t bk[3] = {64, 1, (uint32_t)box};
  if (!make_map_3d(&mK, a.k_pool, dk, sk, bk) || !make_map_3d(&mV, a.v_pool, dk, sk, bk))
    return cudaErrorInvalidValue;
  return launch_g<D, false>(mQ, mK, mV, a, box, s);
}

}  // namespace

cudaError_t launch_tree_tc(const fuse_layer_desc_t& d, const TreeArgs& a, cudaStream_t s) {
  return d.head_dim == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

}  // namespace fusekv
