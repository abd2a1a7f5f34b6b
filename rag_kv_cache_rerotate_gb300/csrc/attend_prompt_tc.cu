// Packed-prompt causal attention on tcgen05 tensor cores (bf16 layers,
// head_dim 64 or 128).
//
// KVBoost (section 3.1, Eq. 2): softmax(q K^T / sqrt(d)) V over j <= s, for
// every row s of every request.
//
// Work unit: one KV head and a tile of 128 / g consecutive rows of one
// request, whose g query heads share that KV head, packed as the M = 128 rows
// of the MMA (row r, head hh -> M row r * g + hh).  Keys stream in blocks of
// 128 from the request's first row up to the tile's last one; as 128 / g
// divides 128, all rows of a tile lie in its last block, which alone needs a
// mask.  Per block b:
//   S = Q K_b^T          tcgen05.mma into TMEM buffer b % 3
//   P = 2^(S - m)        eight warps in registers, bf16, written back over S
//   O += P V_b           tcgen05.mma with A = P in TMEM, V MN-major in shared
//                        memory, O in TMEM columns [384, 384 + d)
// The running maximum m is raised only when a block exceeds it by more than
// 2^16 (then O and the running sum are rescaled).  In the last block both
// products stop at the multiple of 16 keys after the tile's last row.
// Roles, each behind its own mbarriers: warp 0 loads Q (two buffers) and K
// blocks, warp 2 V blocks, warp 1 issues the S MMAs, warp 3 the P.V MMAs,
// warps 4-11 the softmax, warps 12-15 look V through (below) and write O / l
// while the next unit runs.  The softmax warps run up to two units ahead of
// the output, the S buffers permitting.  The kernel is persistent: one CTA per
// SM, units heaviest first, the CTAs visited up and down in turn.
//
// What a row does not see must not reach it.  Scores are replaced where they
// are masked, whatever they were; but 0 * V is not 0 for an infinite or NaN
// V.  So before a unit's last P.V the output warps clear the V rows behind the
// tile's last row, which may be another request's, and any element that is not
// finite in the rows that some rows of the tile see and others do not; later
// they add those elements back to the rows that do see them.
//
// Measured (8 KV heads, g = 4, d = 128): one prompt of 10 368 tokens 538-560 us
// by GPU, 1.6 PFLOP/s, bound by the softmax warps' chain beside a tensor pipe
// that is 69 % active; 16 chunks of 128 to 512 tokens 28 us.  Short units are
// bound by the hand-overs between the roles, whose code does not fit an SM's
// instruction cache: waits and rare paths are out of line (33 -> 28 us), and
// the look through V is not the P.V warp's, which it kept from issuing.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "attend_prompt.h"
#include "checks.h"
#include "launch.h"
#include "tc_ptx.cuh"

namespace fusekv {

bool tma_encode_available();
bool make_map_3d(CUtensorMap* m, const void* base, const uint64_t dims[3], const uint64_t strides[2],
                 const uint32_t box[3]);

namespace {

constexpr int kKB = 128;                      // keys per block
constexpr int kHalf = 128 * 64 * 2;           // 64 columns of a 128-row tile (16 KB)
constexpr int kQBufs = 2;
constexpr int kWarpQK = 0, kWarpS = 1, kWarpV = 2, kWarpPV = 3, kWarpSoft = 4, kWarpOut = 12;
constexpr int kSoftThreads = 256;
constexpr int kThreads = 16 * 32;
constexpr int kTmemCols = 512;                // S buffers | O buffers
// P is rounded to bf16 and summed in fp32 at the same relative precision
// whatever its size: a reference up to 2^16 below the true maximum costs no
// accuracy and saves rescales.
constexpr float kRescaleThreshold = 16.0f;

// Ring depths: what fits beside two Q tiles in 227 KB.  A K block is given up
// after its S, a V block only after the softmax and its P.V.  At d = 128 three K
// and two V buffers take the same time within 1 % on all prompts measured.
template <int D> struct Ring {
  static constexpr int tile = (D / 64) * kHalf;
  static constexpr int K = D == 128 ? 2 : 5;
  static constexpr int V = D == 128 ? 3 : 5;
};
constexpr int kMaxStages = 5;
constexpr int kMaxS = 3, kMaxO = 2;           // S and O buffers, at most
constexpr int kLBufs = 2;                     // row sums: softmax warps run a unit ahead of the output

struct Ctl {
  uint64_t q_full[kQBufs], q_empty[kQBufs];
  uint64_t k_full[kMaxStages], k_empty[kMaxStages];
  uint64_t v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t s_full[kMaxS], p_full[kMaxS], pv_done[kMaxS];      // [block % S buffers]
  uint64_t o_full[kMaxO], o_empty[kMaxO];                     // [unit % O buffers]
  uint64_t l_full[kLBufs], l_empty[kLBufs];                   // [unit % kLBufs]
  // a unit's last V block: landed, looked through [unit % (V stages + 1)]
  uint64_t vl_full[kMaxStages + 1], v_ok[kMaxStages + 1];
  uint32_t tmem_base;
  // the V copies asked for: a bit per stage, v_full was used, and the parity of
  // its next phase; units whose last block was asked for
  uint32_t v_used, v_phase;
  int v_lasts;
  volatile int abort_flag;
  // [unit % (V stages + 1)][output warp] its rows of the unit's last V block
  // held elements that are not finite
  volatile int fix[kMaxStages + 1][4];
  float xl[kLBufs][128];         // [row] softmax row sum of a unit
};

template <int D> constexpr int smem_bytes() {
  return (kQBufs + Ring<D>::K + Ring<D>::V) * Ring<D>::tile + 1024 + (int)sizeof(Ctl);
}
static_assert(smem_bytes<128>() <= 227 * 1024 && smem_bytes<64>() <= 227 * 1024, "shared memory");

struct PromptTcArgs {
  const __nv_bfloat16* V;
  __nv_bfloat16* O;
  int Hq, Hkv, g, rtile;
  int g_log2;
  uint32_t hkv_inv;       // ceil(2^32 / Hkv); 0 past 256 heads
  int n_units;
  float scale_log2;       // log2(e) / sqrt(d)
  uint32_t* err;
  int st32;               // O 32-byte aligned: 256-bit stores
};

// Which wait gave up: info = wait id << 20 | CTA (8 bits) << 12 | key block (12 bits).
enum PromptWait : uint32_t {
  W_Q_EMPTY = 1, W_K_EMPTY, W_V_EMPTY, W_Q_FULL, W_K_FULL, W_S_FREE, W_P_FULL, W_O_EMPTY,
  W_V_FULL, W_S_FULL, W_PV_DONE, W_O_FULL, W_L_FULL, W_L_EMPTY, W_VL_FULL, W_V_OK
};

// What happens when a barrier is not there at the first look.  Out of line:
// the kernel waits in two dozen places, short prompts run through its code
// once per unit, and an SM's instruction cache holds a part of it only.
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
    if ((i & 63u) == 63u) {                // the clock is read late: most waits end before
      if (ctl->abort_flag) return false;
      const uint64_t now = tc::global_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > tc::kWaitLimitNs) break;
    }
  }
  if (ctl->abort_flag == 0) {
    ctl->abort_flag = 1;
    report_error(err, FUSE_ERR_TIMEOUT, SITE_PROMPT_TIMEOUT, which);
  }
  return false;
}

// Waits (bounded) until the V copies asked for have landed: the last phase of
// every barrier, which nothing follows.
__device__ __noinline__ void land_v(Ctl* ctl, int stages) {
  const int lasts = ctl->v_lasts;
#pragma unroll 1
  for (int st = 0; st < stages; ++st)
    if (ctl->v_used >> st & 1) tc::mbar_wait(&ctl->v_full[st], (~ctl->v_phase >> st) & 1);
#pragma unroll 1
  for (int i = lasts > stages + 1 ? lasts - stages - 1 : 0; i < lasts; ++i)
    tc::mbar_wait(&ctl->vl_full[i % (stages + 1)], (i / (stages + 1)) & 1);
}

__device__ __forceinline__ bool wait1(uint64_t* bar, uint32_t parity, Ctl* ctl, uint32_t* err,
                                      uint32_t which, int j) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  return wait_on(tc::smem_u32(bar), parity, ctl, err,
                 (which << 20) | ((blockIdx.x & 0xFFu) << 12) | ((uint32_t)j & 0xFFFu));
}

// The same by every lane of a warp that goes on to warp-collective instructions.
__device__ __forceinline__ bool wait32(uint64_t* bar, uint32_t parity, Ctl* ctl, uint32_t* err,
                                       uint32_t which, int j) {
  return __all_sync(0xffffffffu, wait1(bar, parity, ctl, err, which, j));
}

// The unit of a CTA's i-th round: rounds visit the CTAs upwards and downwards in turn.
__device__ __forceinline__ int unit_at(int i) {
  const int G = (int)gridDim.x, c = (int)blockIdx.x;
  return i * G + ((i & 1) ? G - 1 - c : c);
}

struct Unit {
  PromptTile t;
  int kvh;
  int nkb;                // key blocks
};

__device__ __forceinline__ Unit unit_rec(const PromptTcArgs& a, const PromptTable& p, int u,
                                         int* part) {
  Unit r;
  const int t = a.hkv_inv ? (int)__umulhi((uint32_t)u, a.hkv_inv) : u / a.Hkv;
  r.kvh = u - t * a.Hkv;
  r.t = prompt_tile(p, a.rtile, t, part);
  r.nkb = (r.t.first + r.t.rows - 1) / kKB + 1;
  return r;
}

// Keys of block j that the tile sees, rounded up to the MMAs' step of 16.
__device__ __forceinline__ int block_keys(const Unit& u, int j) {
  return min(kKB, (u.t.first + u.t.rows - j * kKB + 15) & ~15);
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// K-step kk (16 columns) of a 128-row K-major tile stored in 64-column halves.
__device__ __forceinline__ uint64_t kmajor_step(uint32_t tile, int kk) {
  return tc::smem_desc_k128(tile + (kk >> 2) * kHalf + (kk & 3) * 32);
}

__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}

// Adds to a row's outputs the elements that are not finite of n rows of V
// (`step` elements apart): with them the sum is infinite or NaN whatever it
// was, so it does not matter that the outputs are rounded already.
__device__ __noinline__ void add_nonfinite(__nv_bfloat16* dst, const __nv_bfloat16* v, int n, int64_t step,
                                           int d) {
#pragma unroll 1
  for (int k = 0; k < n; ++k, v += step)
#pragma unroll 1
    for (int e = 0; e < d; ++e) {
      const float x = __bfloat162float(v[e]);
      if (!isfinite(x)) dst[e] = __float2bfloat16_rn(__bfloat162float(dst[e]) + x);
    }
}

template <int D, int kSBufs, int kOBufs>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                     const __grid_constant__ CUtensorMap mapV, const PromptTcArgs a,
                     const __grid_constant__ PromptTable table) {
  constexpr int kTile = Ring<D>::tile, kKS = Ring<D>::K, kVS = Ring<D>::V;
  constexpr int kColO = kSBufs * kKB;
  static_assert(kColO + kOBufs * D <= kTmemCols && kSBufs <= kMaxS && kOBufs <= kMaxO, "tensor memory");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + kQBufs * kTile;
  uint8_t* sV = sK + kKS * kTile;
  Ctl* ctl = reinterpret_cast<Ctl*>(sV + kVS * kTile);
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  pdl_trigger();

  if (threadIdx.x == 0) {
    for (int q = 0; q < kQBufs; ++q) {
      tc::mbar_init(&ctl->q_full[q], 1);
      tc::mbar_init(&ctl->q_empty[q], 1);
    }
    for (int s = 0; s < kKS; ++s) {
      tc::mbar_init(&ctl->k_full[s], 1);
      tc::mbar_init(&ctl->k_empty[s], 1);
    }
    for (int s = 0; s < kVS; ++s) {
      tc::mbar_init(&ctl->v_full[s], 1);
      tc::mbar_init(&ctl->v_empty[s], 1);
    }
    for (int s = 0; s < kSBufs; ++s) {
      tc::mbar_init(&ctl->s_full[s], 1);
      tc::mbar_init(&ctl->p_full[s], kSoftThreads);
      tc::mbar_init(&ctl->pv_done[s], 1);
    }
    for (int q = 0; q < kOBufs; ++q) {
      tc::mbar_init(&ctl->o_full[q], 1);
      tc::mbar_init(&ctl->o_empty[q], 128);
    }
    for (int q = 0; q < kLBufs; ++q) {
      tc::mbar_init(&ctl->l_full[q], kSoftThreads);
      tc::mbar_init(&ctl->l_empty[q], 128);
    }
    for (int q = 0; q <= kVS; ++q) {
      tc::mbar_init(&ctl->vl_full[q], 1);
      tc::mbar_init(&ctl->v_ok[q], 4);
    }
    ctl->abort_flag = 0;
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
  const int n_units = a.n_units;
  pdl_wait();                 // inputs of the previous kernel complete and visible

  if (warp == kWarpQK) {
    // --------------------------- Q and K loads ---------------------------
    if (lane == 0) {
      uint32_t kc = 0;
      int i = 0;
      bool ok = true;
      int part = 0;
      for (; unit_at(i) < n_units && ok; ++i) {
        const Unit cur = unit_rec(a, table, unit_at(i), &part);
        const int qb = i % kQBufs;
        if (!wait1(&ctl->q_empty[qb], ((i / kQBufs) & 1) ^ 1, ctl, a.err, W_Q_EMPTY, 0)) break;
        uint8_t* q = sQ + qb * kTile;
        tc::mbar_arrive_expect_tx(&ctl->q_full[qb], kTile);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tc::tma_load_3d(q + h * kHalf, &mapQ, &ctl->q_full[qb], 64 * h, cur.kvh * a.g,
                          cur.t.row0 + cur.t.first);
        for (int j = 0; j < cur.nkb; ++j, ++kc) {
          const int st = kc % kKS;
          if (!wait1(&ctl->k_empty[st], ((kc / kKS) & 1) ^ 1, ctl, a.err, W_K_EMPTY, j)) {
            ok = false;
            break;
          }
          tc::mbar_arrive_expect_tx(&ctl->k_full[st], kTile);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tc::tma_load_3d(sK + st * kTile + h * kHalf, &mapK, &ctl->k_full[st], 64 * h, cur.kvh,
                            cur.t.row0 + j * kKB);
        }
      }
      // let copies in flight land before the CTA may exit
      for (int k = (i > kQBufs ? i - kQBufs : 0); k < i; ++k)
        tc::mbar_wait(&ctl->q_full[k % kQBufs], (k / kQBufs) & 1);
      for (uint32_t c = (kc > (uint32_t)kKS ? kc - kKS : 0); c < kc; ++c)
        tc::mbar_wait(&ctl->k_full[c % kKS], (c / kKS) & 1);
    }
  } else if (warp == kWarpV) {
    // ------------------------------ V loads ------------------------------
    if (lane == 0) {
      uint32_t vc = 0, vph = 0, used = 0;              // v_full: a parity bit per stage, and whether it was used
      int lasts = 0;                                   // units whose last block was asked for
      bool ok = true;
      int part = 0;
      for (int i = 0; unit_at(i) < n_units && ok; ++i) {
        const Unit cur = unit_rec(a, table, unit_at(i), &part);
        for (int j = 0; j < cur.nkb; ++j, ++vc) {
          const int st = vc % kVS;
          if (!wait1(&ctl->v_empty[st], ((vc / kVS) & 1) ^ 1, ctl, a.err, W_V_EMPTY, j)) {
            ok = false;
            break;
          }
          // the last block has a barrier of its own: the output warps wait for
          // no other, and a waiter must visit every phase of a barrier.  Its
          // next use, kVS + 1 units on, comes after this block's P.V
          const bool last = j == cur.nkb - 1;
          uint64_t* bar = last ? &ctl->vl_full[i % (kVS + 1)] : &ctl->v_full[st];
          if (last) {
            ++lasts;
          } else {
            used |= 1u << st;
            vph ^= 1u << st;
          }
          tc::mbar_arrive_expect_tx(bar, kTile);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tc::tma_load_3d(sV + st * kTile + h * kHalf, &mapV, bar, 64 * h, cur.kvh,
                            cur.t.row0 + j * kKB);
        }
      }
      // every block is waited for before its P.V, and that before the CTA's end,
      // unless a wait gives up
      ctl->v_used = used;
      ctl->v_phase = vph;
      ctl->v_lasts = lasts;
    }
  } else if (warp == kWarpS) {
    // ------------------------------ S = Q K^T ------------------------------
    if (lane == 0) {
      uint32_t kc = 0;
      bool ok = true;
      int part = 0;
      for (int i = 0; unit_at(i) < n_units && ok; ++i) {
        const Unit cur = unit_rec(a, table, unit_at(i), &part);
        const int qb = i % kQBufs;
        if (!wait1(&ctl->q_full[qb], (i / kQBufs) & 1, ctl, a.err, W_Q_FULL, 0)) break;
        const uint32_t q_addr = tc::smem_u32(sQ + qb * kTile);
        for (int j = 0; j < cur.nkb; ++j, ++kc) {
          const int st = kc % kKS;
          if (!wait1(&ctl->k_full[st], (kc / kKS) & 1, ctl, a.err, W_K_FULL, j)) {
            ok = false;
            break;
          }
          // the buffer holds P of kSBufs blocks ago until that block's P.V is done
          const uint32_t sb = kc % kSBufs;
          if (!wait1(&ctl->pv_done[sb], ((kc / kSBufs) & 1) ^ 1, ctl, a.err, W_S_FREE, j)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t idesc_s = tc::idesc_bf16_f32(128, block_keys(cur, j));
          const uint32_t kaddr = tc::smem_u32(sK + st * kTile);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_bf16(tmem + sb * kKB, kmajor_step(q_addr, kk), kmajor_step(kaddr, kk), idesc_s,
                         kk != 0);
          tc::mma_commit(&ctl->s_full[sb]);
          tc::mma_commit(&ctl->k_empty[st]);
        }
        if (!ok) break;
        tc::mma_commit(&ctl->q_empty[qb]);
      }
    }
  } else if (warp == kWarpPV) {
    // ------------------------------ O += P V ------------------------------
    if (lane == 0) {
      const uint32_t idesc_o = tc::idesc_bf16_f32(128, D, /*b_mn_major=*/true);
      uint32_t vc = 0, vph = 0;                        // vph: a parity bit per V stage
      bool ok = true;
      int part = 0;
      for (int i = 0; unit_at(i) < n_units && ok; ++i) {
        const Unit cur = unit_rec(a, table, unit_at(i), &part);
        // O was last read by the output warps for unit i - kOBufs
        const int ob = i % kOBufs;
        const uint32_t o = tmem + kColO + ob * D;
        if (!wait1(&ctl->o_empty[ob], ((i / kOBufs) & 1) ^ 1, ctl, a.err, W_O_EMPTY, 0)) break;
        // P.V of block j, in every step of 16 keys or in the first ones
        auto product = [&](int j, int keys) {
          const int st = vc % kVS;
          const uint32_t sb = vc % kSBufs;
          tc::tc_fence_after();
          const uint32_t vaddr = tc::smem_u32(sV + st * kTile);
          const uint32_t pa = tmem + sb * kKB;
#pragma unroll
          for (int kk = 0; kk < kKB / 16; ++kk)
            if (kk * 16 < keys)
              tc::mma_bf16_ts(o, pa + kk * 8, tc::smem_desc_mn128(vaddr + kk * 16 * 128, kHalf),
                              idesc_o, (j | kk) != 0 ? 1u : 0u);
          tc::mma_commit(&ctl->pv_done[sb]);
          tc::mma_commit(&ctl->v_empty[st]);
          ++vc;
        };
        for (int j = 0; j < cur.nkb - 1; ++j) {
          const int st = vc % kVS;
          ok = wait1(&ctl->p_full[vc % kSBufs], (vc / kSBufs) & 1, ctl, a.err, W_P_FULL, j) &&
               wait1(&ctl->v_full[st], (vph >> st) & 1, ctl, a.err, W_V_FULL, j);
          if (!ok) break;
          vph ^= 1u << st;
          product(j, kKB);
        }
        if (!ok) break;
        const int j = cur.nkb - 1, vs = i % (kVS + 1);
        const uint32_t ph = (i / (kVS + 1)) & 1;
        ok = wait1(&ctl->vl_full[vs], ph, ctl, a.err, W_VL_FULL, j) &&
             wait1(&ctl->v_ok[vs], ph, ctl, a.err, W_V_OK, j) &&
             wait1(&ctl->p_full[vc % kSBufs], (vc / kSBufs) & 1, ctl, a.err, W_P_FULL, j);
        if (!ok) break;
        product(j, block_keys(cur, j));
        tc::mma_commit(&ctl->o_full[ob]);
      }
    }
  } else if (warp < kWarpOut) {
    // ------------------------------- softmax -------------------------------
    // warp w: TMEM lane quarter w % 4, half (w - 4) / 4 of it: 16 M rows
    const int base = (warp & 3) * 32 + ((warp - kWarpSoft) >> 2) * 16;
    const uint32_t lane_off = (uint32_t)base << 16;
    const int c4 = lane & 3;
    const int R0 = base + (lane >> 2), R1 = R0 + 8;    // this thread's two M rows
    const float scale = a.scale_log2;
    uint32_t b = 0;
    int part = 0;
    for (int i = 0; unit_at(i) < n_units; ++i) {
      const Unit cur = unit_rec(a, table, unit_at(i), &part);
      const int p0 = cur.t.first + min(R0 >> a.g_log2, cur.t.rows - 1);
      const int p1 = cur.t.first + min(R1 >> a.g_log2, cur.t.rows - 1);
      const int ob = i % kOBufs;
      const uint32_t tO = tmem + lane_off + kColO + ob * D;
      float mu0 = 0.f, mu1 = 0.f;                      // running maxima (log2 units) once j > 0
      float l0 = 0.f, l1 = 0.f;                        // this thread's part of the row sums
      bool ok = true;
      for (int j = 0; j < cur.nkb; ++j, ++b) {
        const uint32_t sb = b % kSBufs;
        if (!wait32(&ctl->s_full[sb], (b / kSBufs) & 1, ctl, a.err, W_S_FULL, j)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t tS = tmem + lane_off + sb * kKB;
        uint32_t r[64];
        tc::tmem_ld_16x256b_x8(tS, *reinterpret_cast<uint32_t(*)[32]>(r));
        tc::tmem_ld_16x256b_x8(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
        tc::tmem_ld_wait();
        if (j == cur.nkb - 1) {                        // the tile's own rows: mask
          constexpr uint32_t kMasked = 0xff800000u;    // -infinity; every row sees a key of its own
          const int key0 = j * kKB;
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const int k = key0 + 8 * q + 2 * c4;
            if (k > p0) r[4 * q] = kMasked;
            if (k + 1 > p0) r[4 * q + 1] = kMasked;
            if (k > p1) r[4 * q + 2] = kMasked;
            if (k + 1 > p1) r[4 * q + 3] = kMasked;
          }
        }
        float m0, m1;
        {
          float a0 = __uint_as_float(r[0]), a1 = __uint_as_float(r[1]);
          float b0 = __uint_as_float(r[2]), b1 = __uint_as_float(r[3]);
#pragma unroll
          for (int q = 1; q < 15; q += 2) {                // repeats 1 .. 14 in pairs
            a0 = max3(a0, __uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 4]));
            a1 = max3(a1, __uint_as_float(r[4 * q + 1]), __uint_as_float(r[4 * q + 5]));
            b0 = max3(b0, __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 6]));
            b1 = max3(b1, __uint_as_float(r[4 * q + 3]), __uint_as_float(r[4 * q + 7]));
          }
          m0 = max3(a0, a1, fmaxf(__uint_as_float(r[60]), __uint_as_float(r[61])));   // repeat 15
          m1 = max3(b0, b1, fmaxf(__uint_as_float(r[62]), __uint_as_float(r[63])));
          m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, 1));
          m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, 1));
          m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, 2));
          m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, 2));
        }
        const float ms0 = m0 * scale, ms1 = m1 * scale;
        float mn0 = mu0, mn1 = mu1;
        bool rs0 = false, rs1 = false;
        if (j == 0) {
          mn0 = ms0;
          mn1 = ms1;
        } else {
          if (ms0 > mu0 + kRescaleThreshold) { mn0 = ms0; rs0 = true; }
          if (ms1 > mu1 + kRescaleThreshold) { mn1 = ms1; rs1 = true; }
        }
        const float al0 = rs0 ? ex2(mu0 - mn0) : 1.f, al1 = rs1 ? ex2(mu1 - mn1) : 1.f;
        // probabilities: key pairs packed as bf16x2, in place over the scores;
        // the scaling and the row sums work on key pairs (f32x2)
        const uint64_t sc2 = pack2(scale, scale);
        // (a row whose every score so far is -infinity has weights of 0, not 2^(-inf + inf))
        const float rf0 = mn0 == -INFINITY ? 0.f : mn0, rf1 = mn1 == -INFINITY ? 0.f : mn1;
        const uint64_t ng0 = pack2(-rf0, -rf0), ng1 = pack2(-rf1, -rf1);
        uint64_t acc0 = 0, acc1 = 0;                    // (even keys, odd keys) of each row
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
        const float2 a0 = unpack2(acc0), a1 = unpack2(acc1);
        const float s0 = a0.x + a0.y, s1 = a1.x + a1.y;
        tc::tmem_st_16x128b_x16(tS, *reinterpret_cast<uint32_t(*)[32]>(r));
        // tcgen05.ld/st are warp-collective: the whole warp rescales its rows
        // of O when any of them needs it (the factor is 1 for the others); O
        // must hold the previous block's P.V
        if (__any_sync(0xffffffffu, rs0 || rs1)) {
          if (!wait32(&ctl->pv_done[(b - 1) % kSBufs], ((b - 1) / kSBufs) & 1, ctl, a.err, W_PV_DONE, j)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 64) {
            uint32_t o[32];
            tc::tmem_ld_16x256b_x8(tO + c, o);
            tc::tmem_ld_wait();
            const uint64_t f0 = pack2(al0, al0), f1 = pack2(al1, al1);
#pragma unroll
            for (int q = 0; q < 32; q += 2) {
              const float2 v = unpack2(mul2(pack2(__uint_as_float(o[q]), __uint_as_float(o[q + 1])), (q & 2) ? f1 : f0));
              o[q] = __float_as_uint(v.x);
              o[q + 1] = __float_as_uint(v.y);
            }
            tc::tmem_st_16x256b_x8(tO + c, o);
          }
        }
        tc::tmem_st_wait();
        tc::tc_fence_before();
        tc::mbar_arrive(&ctl->p_full[sb]);
        l0 = l0 * al0 + s0;
        l1 = l1 * al1 + s1;
        mu0 = mn0;
        mu1 = mn1;
      }
      if (!ok) break;
      // row sums: the four threads of a row, in a fixed order
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      // the row sums of unit i, once the output warps have read those of unit i - kLBufs
      const int lb = i % kLBufs;
      if (!wait32(&ctl->l_empty[lb], ((i / kLBufs) & 1) ^ 1, ctl, a.err, W_L_EMPTY, cur.nkb)) break;
      if (c4 == 0) {
        ctl->xl[lb][R0] = l0;
        ctl->xl[lb][R1] = l1;
      }
      tc::mbar_arrive(&ctl->l_full[lb]);
    }
  } else {
    // ---------------------------- output O / l ----------------------------
    const int quarter = warp & 3;
    const int m = quarter * 32 + lane;
    const int rl = m >> a.g_log2;
    const int hh = m & (a.g - 1);
    // Looks the values of unit i's last block through, each warp every fourth
    // group of rows, before the P.V of that block.
    uint32_t vc = 0;                                   // V blocks of the units looked through
    auto look = [&](const Unit& u, int i) -> bool {
      const int vs = i % (kVS + 1), j = u.nkb - 1, keys = block_keys(u, j);
      if (!wait32(&ctl->vl_full[vs], (i / (kVS + 1)) & 1, ctl, a.err, W_VL_FULL, j)) return false;
      // a lane takes the same 16-byte piece of every kStep-th row after the
      // tile's first one
      constexpr int kPieces = D / 8, kStep = 4 * 32 / kPieces;
      const int row1 = u.t.first + 1 - j * kKB, seen = u.t.first + u.t.rows - j * kKB;
      const int c = lane % kPieces, n0 = quarter * (32 / kPieces) + lane / kPieces;
      uint8_t* at = sV + (vc + j) % kVS * kTile + c / 8 * kHalf + c % 8 * 16;
      // 0 * x is 0 unless x is infinite or NaN
      const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
      __nv_bfloat162 sum[4] = {zero, zero, zero, zero};
      for (int n = row1 + n0; n < seen; n += 4 * kStep) {
        const uint8_t* p = at + n * 128;
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[k] = make_uint4(0, 0, 0, 0);
          if (n + k * kStep < seen) x[k] = *reinterpret_cast<const uint4*>(p + k * kStep * 128);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sum[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[k].x), zero, sum[0]);
          sum[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[k].y), zero, sum[1]);
          sum[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[k].z), zero, sum[2]);
          sum[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[k].w), zero, sum[3]);
        }
      }
      const float2 t = __bfloat1622float2(__hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3])));
      const bool found = __any_sync(0xffffffffu, !(t.x == 0.f && t.y == 0.f));
      if (found || seen < keys) {                      // rare, or the request's last tile
#pragma unroll 1
        for (int n = row1 + n0; n < keys; n += kStep) {
          uint4* p = reinterpret_cast<uint4*>(at + n * 128);
          uint4 x = make_uint4(0, 0, 0, 0);            // behind the tile's last row
          if (n < seen) {
            if (!found) continue;
            x = *p;
            x.x = drop_nonfinite(x.x);
            x.y = drop_nonfinite(x.y);
            x.z = drop_nonfinite(x.z);
            x.w = drop_nonfinite(x.w);
          }
          *p = x;
        }
        tc::fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) {
        ctl->fix[vs][quarter] = found;
        tc::mbar_arrive(&ctl->v_ok[vs]);
      }
      vc += u.nkb;
      return true;
    };
    int part = 0;
    Unit nxt = unit_rec(a, table, unit_at(0), &part);
    bool looked = false;                               // unit nxt
    for (int i = 0; unit_at(i) < n_units; ++i) {
      const Unit cur = nxt;
      // The next unit's values are looked through before this one's output,
      // unless they wait for it: a last block whose buffer an earlier block of
      // its own unit has to give up first
      const bool more = unit_at(i + 1) < n_units;
      if (more) nxt = unit_rec(a, table, unit_at(i + 1), &part);
      const bool early = more && nxt.nkb <= kVS;
      bool ok = true;
#pragma unroll 1
      for (int k = looked ? i + 1 : i; ok && k <= (early ? i + 1 : i); ++k) ok = look(k == i ? cur : nxt, k);
      if (!ok) break;
      looked = early;
      const int ob = i % kOBufs;
      const uint32_t ph = (i / kOBufs) & 1;
      const uint32_t tO = tmem + ((uint32_t)(quarter * 32) << 16) + kColO + ob * D;
      if (!wait32(&ctl->o_full[ob], ph, ctl, a.err, W_O_FULL, cur.nkb)) break;
      const int lb = i % kLBufs, vs = i % (kVS + 1);
      if (!wait32(&ctl->l_full[lb], (i / kLBufs) & 1, ctl, a.err, W_L_FULL, cur.nkb)) break;
      tc::tc_fence_after();
      const float inv = 1.f / ctl->xl[lb][m];
      const bool fix = (ctl->fix[vs][0] | ctl->fix[vs][1] | ctl->fix[vs][2] | ctl->fix[vs][3]) != 0;
      tc::mbar_arrive(&ctl->l_empty[lb]);
      const bool valid = rl < cur.t.rows;
      const int64_t row = cur.t.row0 + cur.t.first;
      __nv_bfloat16* dst = a.O + ((row + rl) * a.Hq + cur.kvh * a.g + hh) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 64) {
        uint32_t r[64];
        tc::tmem_ld_32x32b_x32(tO + c, *reinterpret_cast<uint32_t(*)[32]>(r));
        tc::tmem_ld_32x32b_x32(tO + c + 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
        tc::tmem_ld_wait();
        if (c + 64 == D) {                             // O is read: the next unit's P.V may start
          tc::tc_fence_before();
          tc::mbar_arrive(&ctl->o_empty[ob]);
        }
#pragma unroll
        for (int e = 0; e < 64; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * inv);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[e] = pack_bf16x2(__uint_as_float(r[16 * q + 2 * e]), __uint_as_float(r[16 * q + 2 * e + 1]));
          if (valid && a.st32) {
            // one 256-bit store per 16 values: the 32 bytes fill one sector
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + c + 16 * q),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                         "r"(w[7])
                         : "memory");
          } else if (valid) {
            uint4* d = reinterpret_cast<uint4*>(dst + c + 16 * q);
            d[0] = make_uint4(w[0], w[1], w[2], w[3]);
            d[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
        __syncwarp();                                  // the loads are warp-collective
      }
      if (fix && valid)                                // of the tile's rows that this one sees
        add_nonfinite(dst, a.V + ((row + 1) * a.Hkv + cur.kvh) * D, rl, (int64_t)a.Hkv * D, D);
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (ctl->abort_flag) {                               // copies land, products in flight get time to end
    if (threadIdx.x == 0) land_v(ctl, kVS);
#pragma unroll 1
    for (int k = 0; k < 1000; ++k) __nanosleep(1000);
    __syncthreads();
  }
  if (warp == kWarpS) tc::tmem_dealloc(tmem, kTmemCols);
}

template <int D, int SB, int OB>
cudaError_t launch_d(const fuse_layer_desc_t& d, const PromptTable& p, int64_t n_tok, const void* Q,
                     const void* K, const void* V, void* O, uint32_t* err, cudaStream_t s) {
  const int g = d.n_q_heads / d.n_kv_heads;
  CUtensorMap mQ, mK, mV;
  const uint64_t dq[3] = {(uint64_t)D, (uint64_t)d.n_q_heads, (uint64_t)n_tok};
  const uint64_t sq[2] = {(uint64_t)D * 2, (uint64_t)d.n_q_heads * D * 2};
  const uint32_t bq[3] = {64, (uint32_t)g, (uint32_t)(128 / g)};
  const uint64_t dk[3] = {(uint64_t)D, (uint64_t)d.n_kv_heads, (uint64_t)n_tok};
  const uint64_t sk[2] = {(uint64_t)D * 2, (uint64_t)d.n_kv_heads * D * 2};
  const uint32_t bk[3] = {64, 1, (uint32_t)kKB};
  if (!make_map_3d(&mQ, Q, dq, sq, bq) || !make_map_3d(&mK, K, dk, sk, bk) ||
      !make_map_3d(&mV, V, dk, sk, bk))
    return cudaErrorInvalidValue;
  PromptTcArgs a;
  a.V = reinterpret_cast<const __nv_bfloat16*>(V);
  a.O = reinterpret_cast<__nv_bfloat16*>(O);
  a.Hq = d.n_q_heads;
  a.Hkv = d.n_kv_heads;
  a.g = g;
  a.rtile = 128 / g;
  a.g_log2 = g == 8 ? 3 : g == 4 ? 2 : g == 2 ? 1 : 0;
  // exact for units below 2^24; one head: the division by 1 below
  a.hkv_inv = a.Hkv > 1 && a.Hkv <= 256 ? (uint32_t)((((uint64_t)1 << 32) + a.Hkv - 1) / a.Hkv) : 0;
  a.n_units = p.n_tiles * d.n_kv_heads;
  a.scale_log2 = 1.4426950408889634f / std::sqrt((float)D);
  a.err = err;
  a.st32 = (reinterpret_cast<uintptr_t>(O) & 31u) == 0;
  cudaError_t e =
      set_dyn_smem_once(reinterpret_cast<const void*>(prompt_tc_kernel<D, SB, OB>), smem_bytes<D>());
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 1;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return launch_pdl(prompt_tc_kernel<D, SB, OB>, dim3(std::min(a.n_units, sms)), dim3(kThreads),
                    smem_bytes<D>(), s, mQ, mK, mV, a, p);
}

}  // namespace

bool prompt_tc_supported(const fuse_layer_desc_t& d) {
  return d.dtype == FUSE_BF16 && tma_encode_available();
}

cudaError_t launch_prompt_tc(const fuse_layer_desc_t& d, const PromptTable& p, int64_t n_tok,
                             const void* Q, const void* K, const void* V, void* O, uint32_t* err,
                             cudaStream_t s) {
  // d = 64 leaves room for a second O beside three S; at d = 128 two S and two
  // O were slower (10368 tokens: 692 us against 562; 16 ragged chunks: 35.0
  // against 34.2)
  return d.head_dim == 128 ? launch_d<128, 3, 1>(d, p, n_tok, Q, K, V, O, err, s)
                           : launch_d<64, 3, 2>(d, p, n_tok, Q, K, V, O, err, s);
}

}  // namespace fusekv
