// Attention over chunk caches, bf16 layers: the items' kernel on warp-level
// matrix instructions (attend_chunks.cu holds the formulas and the join).
//
// Bound: every key costs its codes once (132 bytes per KV head at 4 bits and
// d = 128) and 4 d operations per query vector, of which there are at most 8
// at a time; with so few rows the products fit mma.sync (m16n8k16), whose
// operands are registers, and need no 128-row tcgen05 tile built in shared
// memory.  What decides is the instruction count per code, so codes are used
// as they are: the bits of a code c < 1024 in a 16-bit half are the subnormal
// fp16 number c * 2^-24, exactly, and the same code 4 bits higher is c *
// 2^-20.  Two codes per 32-bit operand register thus cost one AND (and every
// second a shift; values, whose register pairs two tokens of a channel, also
// half a byte permute); the powers of two go into the query and the output.
//
// One warp per item (segment, KV head, group of 8 query vectors), its keys in
// slots of 32 (4 bits), 16 (8 bits) or 8 (bf16): 4 KB at d = 128, three slots
// of shared memory per warp filled by 16-byte cp.async two ahead.  The warps
// of a CTA take neighbouring KV heads of the same tokens, so together they
// read whole rows.  Warps share only the chunk's angles.
//   S^T = Q K^T   A = Q (rows 0-7: the vectors' high parts, 8-15: what is
//                 left of them, 22 bits together), B = codes of 8 keys, the
//                 channels in whatever order the lanes hold them
//   O^T += V^T P  A = codes (rows: channels, 16 keys), B = P: the layout in
//                 which S^T comes out is the one that P goes in
// P carries the values' per-token scale, normalised by the largest so far (a
// power of two), in fp16 (bf16 rows: in two bf16 parts).  The maximum and the
// normaliser are raised lazily.
#include <algorithm>

#include "attend_chunks.h"
#include "launch.h"

namespace fusekv {

namespace {

constexpr int kWarps = 8;
constexpr int kSlots = 3;
constexpr float kRaise = 8.0f;            // log2: P <= 2^8, times a scale <= 2^6 stays in fp16

template <int ST, int D> struct Fmt {
  static constexpr bool coded = ST != FUSE_BF16;
  static constexpr int RB = ST == FUSE_BF16 ? 2 * D : ST == FUSE_U8_ASYM ? D : D / 2;   // row bytes
  static constexpr int RC = RB / 16;                   // 16-byte chunks of a row
  static constexpr int TOK = ST == FUSE_BF16 ? 8 : ST == FUSE_U8_ASYM ? 16 : 32;        // keys a slot
  static constexpr int NT = TOK / 8;
  static constexpr int KSTEP = D / 16;
  static constexpr int MT = D / 16;
};
constexpr int slot_bytes(int d) { return 32 * d; }     // TOK keys and values, in every format

template <int D> struct WarpSmem {
  uint8_t slot[kSlots][slot_bytes(D)];
  uint32_t skip[32];                                   // bit per key: selected, not read here
  uint32_t keep[kSlots];                               // bit per key of the slot: inside, page known
  uint32_t pad;
  uint32_t sz[32];                                     // (scale, zero) of the slot's values, fp16
};

struct Item {
  const uint8_t *k, *v;                                // row 0, head h
  const __half *vs, *vz;                               // row 0, head h
  const int32_t* table;                                // paged: block ids
  const int32_t* skip;                                 // selected positions, ascending
  int n_skip, pos0;                                    // their count, request position of row 0
  int t0, t1;
  int r, h, vg;
  int64_t slot;
};

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

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6},"
      " {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Where 16-byte chunk c of row sits in its row: spread so that the lanes of a
// load fall on different banks.
template <int RC> __device__ __forceinline__ int k_chunk(int row, int c) {
  return RC >= 8 ? c ^ ((row & 1) << 2) : c;
}
// Values: keys 0, 2, 4, 6 of eight come first (the lanes of a load hold every second key).
__device__ __forceinline__ int v_row(int key) {
  return (key & ~7) | ((key & 1) << 2) | ((key & 7) >> 1);
}
template <int RC> __device__ __forceinline__ int v_chunk(int row, int c) {
  return RC >= 8 ? c ^ ((row & 3) << 1) : RC == 4 ? c ^ (row & 2) : c;
}

// Channel that element e (0, 1) of half b of a lane's operand register pair
// holds in K-step kk.
template <int ST, int D> __device__ __forceinline__ int q_channel(int tig, int kk, int b, int e) {
  if constexpr (ST == FUSE_U4_ASYM) return tig * (D / 4) + 8 * (kk >> 1) + 2 * (kk & 1) + b + 4 * e;
  if constexpr (ST == FUSE_U8_ASYM) return ((kk >> 2) * 4 + tig) * 16 + 4 * (kk & 3) + 2 * b + e;
  return ((kk >> 1) * 4 + tig) * 8 + 4 * (kk & 1) + 2 * b + e;
}
// Word of channel ch of vector v in the staged query: banks spread over both.
template <int D> __device__ __forceinline__ int q_word(int v, int ch) {
  return v * D + ((ch & ~31) | ((ch + 4 * v + (ch >> 5)) & 31));
}

// Lower bound of x in a[0, n), by all lanes of the warp, 32 probes at a time.
__device__ __forceinline__ int warp_lower_bound(const int32_t* a, int n, int x) {
  const int lane = threadIdx.x % 32;
  int lo = 0, len = n;                                 // the answer is in [lo, lo + len]
  while (len > 0) {
    const int step = (len + 31) / 32;
    const int i = lo + (lane + 1) * step - 1;          // last element of the lane's part
    const bool below = i < lo + len ? a[i] < x : false;
    const int parts = __popc(__ballot_sync(0xffffffffu, below));
    // parts whose last element is below x are skipped whole
    const int skip = parts * step;
    lo += skip;
    len = min(step - 1, len - skip);
    if (len < 0) len = 0;
  }
  return lo;
}

template <int ST, int D>
__device__ __forceinline__ void attend_mma_item(const AttendArgs& a, const Item& y, const float2* cs,
                                                const __half* ks, const __half* kz,
                                                WarpSmem<D>& sm) {
  using F = Fmt<ST, D>;
  constexpr int RB = F::RB, RC = F::RC, TOK = F::TOK, NT = F::NT, KSTEP = F::KSTEP, MT = F::MT;
  constexpr uint32_t kAll = 0xffffffffu;
  const int lane = threadIdx.x % 32, gid = lane >> 2, tig = lane & 3;
  const int64_t stride = (int64_t)a.n_kv_heads * RB;
  const int n_slots = (y.t1 - y.t0 + TOK - 1) / TOK;

  // ---- selected keys of the item, a bit each -------------------------------
  auto mark_selected = [&]() {
    sm.skip[lane] = 0;
    __syncwarp();
    if (y.n_skip > 0) {
      const int p0 = y.pos0 + y.t0, p1 = y.pos0 + y.t1;
      for (int i = warp_lower_bound(y.skip, y.n_skip, p0);; i += 32) {
        const int v = i + lane < y.n_skip ? y.skip[i + lane] : p1;
        const bool in = v >= p0 && v < p1;
        if (in) atomicOr(&sm.skip[(v - p0) >> 5], 1u << ((v - p0) & 31));
        if (!__all_sync(kAll, in)) break;
      }
    }
    __syncwarp();
  };

  // ---- rows of a slot's keys, one per lane ----------------------------------
  // The page id of the slot loaded next is read one slot ahead and looked at
  // only when it is used, so that its read is not waited for.
  int blk = 0, rem = y.t0 + lane, id = 0, t_next = y.t0 + lane;   // this lane's key of that slot
  const int dq = y.table ? TOK / a.block_size : 0, dr = TOK - dq * a.block_size;
  const int bs = y.table ? a.block_size : INT32_MAX;
  if (y.table) {
    blk = rem / bs;
    rem -= blk * bs;
  }
  auto load_id = [&]() {
    if (y.table && lane < TOK && t_next < y.t1) id = y.table[blk];
  };
  auto next_row = [&]() {                              // its row, -1: none; then the next slot's id
    const bool in = lane < TOK && t_next < y.t1;
    int row = in ? rem : -1;
    if (y.table && in) {
      if (id >= 0 && id < a.n_pool_blocks) {
        row = id * bs + rem;
      } else {
        report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_ATTEND_BLOCK, (uint32_t)id);
        row = -1;
      }
    }
    t_next += TOK;
    blk += dq;
    rem += dr;
    if (rem >= bs) {
      rem -= bs;
      ++blk;
    }
    load_id();
    return row;
  };
  // slot s into its buffer; returns the row of this lane's key, -1: none
  auto issue = [&](int s) {
    int row = next_row();
    if constexpr (!F::coded)                           // what is not seen may hold anything
      if (row >= 0 && (sm.skip[(s * TOK + lane) >> 5] >> ((s * TOK + lane) & 31) & 1)) row = -1;
    const uint32_t ok = __ballot_sync(kAll, row >= 0);
    uint8_t* buf = sm.slot[s % kSlots];
    if (lane == 0) sm.keep[s % kSlots] = ok;
    const uint32_t dk = (uint32_t)__cvta_generic_to_shared(buf), dv = dk + TOK * RB;
    const bool whole = ok == (uint32_t)((1ull << TOK) - 1);
    if (!y.table && whole) {               // warp-uniform: TOK consecutive rows
      const int64_t off = (int64_t)(y.t0 + s * TOK + lane / RC) * stride + lane % RC * 16;
      const uint8_t *pk = y.k + off, *pv = y.v + off;
#pragma unroll
      for (int i = 0; i < TOK * RC / 32; ++i) {
        const int key = (i * 32 + lane) / RC, c = (i * 32 + lane) % RC;
        const int vr = v_row(key);
        cp16(dk + key * RB + k_chunk<RC>(key, c) * 16, pk, true);
        cp16(dv + vr * RB + v_chunk<RC>(vr, c) * 16, pv, true);
        pk += (32 / RC) * stride;
        pv += (32 / RC) * stride;
      }
      return row;
    }
#pragma unroll
    for (int i = 0; i < TOK * RC / 32; ++i) {
      const int key = (i * 32 + lane) / RC, c = (i * 32 + lane) % RC;
      const int kr = __shfl_sync(kAll, row, key);
      const int64_t off = (int64_t)max(kr, 0) * stride + c * 16;
      cp16(dk + key * RB + k_chunk<RC>(key, c) * 16, y.k + off, kr >= 0);
      const int vr = v_row(key);
      cp16(dv + vr * RB + v_chunk<RC>(vr, c) * 16, y.v + off, kr >= 0);
    }
    return row;
  };
  // scale and zero of a slot's values: read two slots ahead, looked at when used
  auto load_sz = [&](int row, uint16_t& vs, uint16_t& vz) {
    vs = vz = 0;
    if (F::coded && row >= 0) {
      const int64_t at = (int64_t)row * a.n_kv_heads;
      vs = reinterpret_cast<const uint16_t*>(y.vs)[at];
      vz = reinterpret_cast<const uint16_t*>(y.vz)[at];
    }
  };

  if constexpr (!F::coded) mark_selected();
  load_id();
  uint16_t sz0[2], sz1[2];                             // even and odd slots
  load_sz(issue(0), sz0[0], sz0[1]);
  cp_commit();
  load_sz(issue(1), sz1[0], sz1[1]);
  cp_commit();

  // ---- the query vectors, turned back and scaled, as A operands --------------
  uint32_t qa[KSTEP][4];
  float sscale, cst;                                   // score = sum * sscale + cst (vector gid)
  {
    // a lane's channel pairs (j, j + D / 2): j = NP lane .. NP lane + NP - 1
    constexpr int NP = D / 64;
    const int n_vec = a.g * a.n_new, j0 = NP * lane;
    auto load_pair = [](const __nv_bfloat16* p, float (&x)[NP]) {
      if constexpr (NP == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
        x[0] = bf16_lo(w);
        x[1] = bf16_hi(w);
      } else {
        x[0] = __bfloat162float(*p);
      }
    };
    auto load_half = [](const __half* p, float (&x)[NP]) {
#pragma unroll
      for (int i = 0; i < NP; ++i) x[i] = __half2float(p[i]);
    };
    float x0[kVecs][NP], x1[kVecs][NP], k0[NP], k1[NP], z0[NP], z1[NP];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int vi = y.vg * kVecs + v;
#pragma unroll
      for (int i = 0; i < NP; ++i) x0[v][i] = x1[v][i] = 0.f;
      if (vi < n_vec) {                                // warp-uniform
        const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.Q) +
                                 ((int64_t)(y.r * a.n_new + vi / a.g) * a.n_q_heads + y.h * a.g + vi % a.g) * D;
        load_pair(q + j0, x0[v]);
        load_pair(q + j0 + D / 2, x1[v]);
      }
    }
    if constexpr (F::coded) {
      load_half(ks + y.h * D + j0, k0);
      load_half(ks + y.h * D + j0 + D / 2, k1);
      load_half(kz + y.h * D + j0, z0);
      load_half(kz + y.h * D + j0 + D / 2, z1);
      mark_selected();                                 // its reads run beside those above
    }
    uint32_t* sq = reinterpret_cast<uint32_t*>(sm.slot[2]);   // not in flight yet
    sscale = 1.f;
    cst = 0.f;
    float z[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      z[v] = 0.f;
      if (y.vg * kVecs + v >= n_vec) {                 // warp-uniform: no such vector
#pragma unroll
        for (int i = 0; i < D / 32; ++i) sq[q_word<D>(v, lane + 32 * i)] = 0;
        continue;
      }
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float q0 = x0[v][i] * a.scale, q1 = x1[v][i] * a.scale;
        float r0 = q0, r1 = q1;
        if (cs) {
          const float2 t = cs[j0 + i];
          r0 = q0 * t.x + q1 * t.y;
          r1 = q1 * t.x - q0 * t.y;
        }
        if constexpr (F::coded) {
          z[v] += r0 * z0[i] + r1 * z1[i];
          r0 *= k0[i];
          r1 *= k1[i];
          mx = fmaxf(mx, fmaxf(fabsf(r0), fabsf(r1)));
        }
        x0[v][i] = r0;
        x1[v][i] = r1;
      }
      float up = 1.f;
      if constexpr (F::coded) {
        // fp16 parts want the largest element near 2^12: a power of two apart
        const uint32_t mb = __reduce_max_sync(kAll, __float_as_uint(mx));
        const int e = min(max((int)(mb >> 23), 27), 230);
        up = __uint_as_float((uint32_t)(266 - e) << 23);
        if (v == gid) sscale = 16777216.f * __uint_as_float((uint32_t)(e - 12) << 23);   // 2^24 / up
      }
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int ch = j0 + i + b * (D / 2);
          float x = (b ? x1[v][i] : x0[v][i]) * up;
          uint32_t w;
          if constexpr (F::coded) {
            if (ST == FUSE_U4_ASYM && (ch & 1)) x *= 0.0625f;   // odd codes sit 4 bits higher
            const __half hi = __float2half_rn(x);
            w = pack_half2(__half2float(hi), x - __half2float(hi));
          } else {
            const __nv_bfloat16 hi = __float2bfloat16_rn(x);
            w = pack_bf16x2(__bfloat162float(hi), x - __bfloat162float(hi));
          }
          sq[q_word<D>(v, ch)] = w;
        }
    }
    if constexpr (F::coded) {
      // the eight sums over the lanes, halving the vectors a lane carries:
      // vector gid ends up in its four lanes
#pragma unroll
      for (int n = 4; n > 0; n >>= 1) {
        const bool upper = lane & (4 * n);
#pragma unroll
        for (int v = 0; v < n; ++v) {
          const float give = upper ? z[v] : z[v + n];
          z[v] = (upper ? z[v + n] : z[v]) + __shfl_xor_sync(kAll, give, 4 * n);
        }
      }
      cst = z[0];
      cst += __shfl_xor_sync(kAll, cst, 1);
      cst += __shfl_xor_sync(kAll, cst, 2);
    }
    __syncwarp();
#pragma unroll
    for (int kk = 0; kk < KSTEP; ++kk)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint32_t w0 = sq[q_word<D>(gid, q_channel<ST, D>(tig, kk, b, 0))];
        const uint32_t w1 = sq[q_word<D>(gid, q_channel<ST, D>(tig, kk, b, 1))];
        qa[kk][2 * b] = __byte_perm(w0, w1, 0x5410);          // row gid: high parts
        qa[kk][2 * b + 1] = __byte_perm(w0, w1, 0x7632);      // row gid + 8: what is left
      }
  }

  // ---- the keys ------------------------------------------------------------
  float m = -INFINITY;                                 // vector gid
  uint64_t l2 = 0, z2 = 0;                             // its sums (this lane's even, odd keys)
  int ve = 0;                                          // exponent field of the largest value scale
  float acc[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;

  auto step = [&](int s, uint16_t (&szr)[2]) {
    cp_wait<1>();                                      // slot s has landed
    __syncwarp();                                      // ... for every lane; slot s - 1 is done with
    const uint32_t sz = (uint32_t)szr[0] | (uint32_t)szr[1] << 16;
    load_sz(issue(s + 2), szr[0], szr[1]);
    cp_commit();
    const uint8_t* kb = sm.slot[s % kSlots];
    const uint8_t* vb = kb + TOK * RB;
    const int bit0 = s * TOK;
    const uint32_t keep = sm.keep[s % kSlots] & ~(sm.skip[bit0 >> 5] >> (bit0 & 31));
    bool raise = false;
    float fe = 1.f;                                    // factor of a raised normaliser
    if constexpr (F::coded) {
      sm.sz[lane] = keep >> lane & 1 ? sz : 0u;        // whatever a key not seen holds
      const uint32_t top = __reduce_max_sync(kAll, (keep >> lane & 1) ? sz & 0x7fffu : 0u);
      const int e = min((int)(top >> 10), 30);
      if (e > ve) {                                    // warp-uniform
        fe = __uint_as_float((uint32_t)max(127 + ve - e, 1) << 23);
        ve = e;
        raise = true;
      }
      __syncwarp();
    }
    // scores: S^T rows gid (+ 8: low parts), keys 2 tig, 2 tig + 1 of each 8
    uint64_t sc[NT];                                   // before sscale and cst
    // eight keys at a time form a chain of D / 16 dependent products; two such
    // groups, each in two chains, run side by side
    constexpr int NP2 = NT < 2 ? NT : 2;
#pragma unroll
    for (int nt0 = 0; nt0 < NT; nt0 += NP2) {
      float c[NP2][2][4];
#pragma unroll
      for (int p = 0; p < NP2; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) c[p][e >> 2][e & 3] = 0.f;
      if constexpr (ST == FUSE_U4_ASYM) {
        uint32_t w[NP2][D / 32];
#pragma unroll
        for (int p = 0; p < NP2; ++p) {
          const uint8_t* kr = kb + ((nt0 + p) * 8 + gid) * RB;
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(kr + tig * 16);
            w[p][0] = x.x; w[p][1] = x.y; w[p][2] = x.z; w[p][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(kr + tig * 8);
            w[p][0] = x.x; w[p][1] = x.y;
          }
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int p = 0; p < NP2; ++p) {
              const uint32_t u = b ? w[p][j] >> 8 : w[p][j];
              mma16<true>(c[p][b], qa[2 * j + b][0], qa[2 * j + b][1], qa[2 * j + b][2],
                          qa[2 * j + b][3], u & 0x000f000fu, u & 0x00f000f0u);
            }
      } else {
        constexpr int CH = RC / 4;                     // 16-byte chunks of a lane
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          uint32_t w[NP2][4];
#pragma unroll
          for (int p = 0; p < NP2; ++p) {
            const int key = (nt0 + p) * 8 + gid;
            const uint4 x = *reinterpret_cast<const uint4*>(kb + key * RB + k_chunk<RC>(key, i * 4 + tig) * 16);
            w[p][0] = x.x; w[p][1] = x.y; w[p][2] = x.z; w[p][3] = x.w;
          }
          if constexpr (ST == FUSE_U8_ASYM) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int p = 0; p < NP2; ++p) {
                const int kk = i * 4 + j;
                mma16<true>(c[p][j & 1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3],
                            __byte_perm(w[p][j], 0, 0x4140), __byte_perm(w[p][j], 0, 0x4342));
              }
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int p = 0; p < NP2; ++p) {
                const int kk = i * 2 + j;
                mma16<false>(c[p][j], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], w[p][2 * j],
                             w[p][2 * j + 1]);
              }
          }
        }
      }
#pragma unroll
      for (int p = 0; p < NP2; ++p)
        sc[nt0 + p] = add2(add2(pack2(c[p][0][0], c[p][0][1]), pack2(c[p][1][0], c[p][1][1])),
                           add2(pack2(c[p][0][2], c[p][0][3]), pack2(c[p][1][2], c[p][1][3])));
    }
    const uint32_t mine = keep >> (2 * tig);           // bits 8 nt, 8 nt + 1: this lane's keys
    if (keep != (uint32_t)((1ull << TOK) - 1)) {       // warp-uniform
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float2 x = unpack2(sc[nt]);
        if (!(mine >> (8 * nt) & 1)) x.x = -INFINITY;
        if (!(mine >> (8 * nt + 1) & 1)) x.y = -INFINITY;
        sc[nt] = pack2(x.x, x.y);
      }
    }
    float mt = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 x = unpack2(sc[nt]);
      mt = fmaxf(mt, fmaxf(x.x, x.y));
    }
    mt = fmaxf(mt, __shfl_xor_sync(kAll, mt, 1));
    mt = fmaxf(mt, __shfl_xor_sync(kAll, mt, 2));
    if constexpr (F::coded) mt = mt == -INFINITY ? mt : fmaf(mt, sscale, cst);
    const bool up = mt > m + kRaise;
    if (__any_sync(kAll, up) || raise) {
      const float al = (up ? ex2(m - mt) : 1.f) * fe;  // 0 at the first key
      if (up) m = mt;
      const uint64_t al2 = pack2(al, al);
      l2 = mul2(l2, al2);
      z2 = mul2(z2, al2);
      const float f0 = __shfl_sync(kAll, al, tig * 8), f1 = __shfl_sync(kAll, al, tig * 8 + 4);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        acc[i][0] *= f0;
        acc[i][1] *= f1;
        acc[i][2] *= f0;
        acc[i][3] *= f1;
      }
    }
    // weights, sums, and what multiplies the values; beside codes all carry
    // the factor 2^(20 - ve), with which a scale stays below 2^6
    const float ref = (m == -INFINITY ? 0.f : m) - (F::coded ? (float)(20 - ve) : 0.f);
    const uint64_t a2 = pack2(sscale, sscale), b2 = pack2(cst - ref, cst - ref);
    uint32_t ph[NT], pl[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 x = unpack2(F::coded ? fma2(sc[nt], a2, b2) : add2(sc[nt], b2));
      const uint64_t p = pack2(ex2(x.x), ex2(x.y));
      l2 = add2(l2, p);
      if constexpr (F::coded) {
        const uint2 w = *reinterpret_cast<const uint2*>(&sm.sz[nt * 8 + 2 * tig]);
        const float2 s0 = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
        const float2 s1 = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
        z2 = fma2(p, pack2(s0.y, s1.y), z2);
        const float2 v = unpack2(mul2(p, pack2(s0.x, s1.x)));
        ph[nt] = pack_half2(v.x, v.y);
      } else {
        const float2 v = unpack2(p);
        ph[nt] = pack_bf16x2(v.x, v.y);
        pl[nt] = pack_bf16x2(v.x - bf16_lo(ph[nt]), v.y - bf16_hi(ph[nt]));
      }
    }
    // O^T += V^T P
    if constexpr (F::coded) {
      constexpr int VB = RB / 8;                       // bytes of a row that a lane takes
#pragma unroll
      for (int g2 = 0; g2 < TOK / 16; ++g2) {
        uint32_t w[4][VB / 4];                         // keys 2 tig, 2 tig + 1, 8 + 2 tig, 9 + 2 tig
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int vr = g2 * 16 + (k >> 1) * 8 + (k & 1) * 4 + tig;
          const uint8_t* p = vb + vr * RB + v_chunk<RC>(vr, gid * VB / 16) * 16 + gid * VB % 16;
          if constexpr (VB == 16) {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            w[k][0] = x.x; w[k][1] = x.y; w[k][2] = x.z; w[k][3] = x.w;
          } else if constexpr (VB == 8) {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[k][0] = x.x; w[k][1] = x.y;
          } else {
            w[k][0] = *reinterpret_cast<const uint32_t*>(p);
          }
        }
#pragma unroll
        for (int j = 0; j < VB / 4; ++j)
#pragma unroll
          for (int hi = 0; hi < 2; ++hi) {
            const uint32_t u = __byte_perm(w[0][j], w[1][j], hi ? 0x7632 : 0x5410);
            const uint32_t v = __byte_perm(w[2][j], w[3][j], hi ? 0x7632 : 0x5410);
            if constexpr (ST == FUSE_U4_ASYM) {
              mma16<true>(acc[j * 4 + hi * 2], u & 0x000f000fu, u & 0x00f000f0u, v & 0x000f000fu,
                          v & 0x00f000f0u, ph[2 * g2], ph[2 * g2 + 1]);
              const uint32_t us = u >> 8, vs = v >> 8;
              mma16<true>(acc[j * 4 + hi * 2 + 1], us & 0x000f000fu, us & 0x00f000f0u, vs & 0x000f000fu,
                          vs & 0x00f000f0u, ph[2 * g2], ph[2 * g2 + 1]);
            } else {
              mma16<true>(acc[j * 2 + hi], u & 0x00ff00ffu, (u >> 8) & 0x00ff00ffu, v & 0x00ff00ffu,
                          (v >> 8) & 0x00ff00ffu, ph[2 * g2], ph[2 * g2 + 1]);
            }
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        uint32_t w[2][4];                              // keys 2 tig, 2 tig + 1
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int vr = k * 4 + tig;
          const uint4 x = *reinterpret_cast<const uint4*>(vb + vr * RB + v_chunk<RC>(vr, i * 8 + gid) * 16);
          w[k][0] = x.x; w[k][1] = x.y; w[k][2] = x.z; w[k][3] = x.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t u = __byte_perm(w[0][j], w[1][j], 0x5410), v = __byte_perm(w[0][j], w[1][j], 0x7632);
          mma8_bf16(acc[i * 4 + j], u, v, ph[0]);
          mma8_bf16(acc[i * 4 + j], u, v, pl[0]);
        }
      }
    }
  };
#pragma unroll 1
  for (int s = 0; s < n_slots; s += 2) {
    step(s, sz0);
    if (s + 1 < n_slots) step(s + 1, sz1);
  }
  cp_wait<0>();                                        // nothing in flight when the buffers go

  // ---- the item's partial ----------------------------------------------------
  const float vu = F::coded ? __uint_as_float((uint32_t)(127 + ve - 20) << 23) : 1.f;
  const float2 lp = unpack2(l2), zp = unpack2(z2);
  float l = (lp.x + lp.y) * vu, zs = (zp.x + zp.y) * vu;
  l += __shfl_xor_sync(kAll, l, 1);
  l += __shfl_xor_sync(kAll, l, 2);
  zs += __shfl_xor_sync(kAll, zs, 1);
  zs += __shfl_xor_sync(kAll, zs, 2);
  const int n_vec = min(kVecs, a.g * a.n_new - y.vg * kVecs);
  const int64_t at = ((y.slot * a.n_kv_heads + y.h) * a.nvg + y.vg) * kVecs;
  if (tig == 0 && gid < n_vec) a.part_ml[at + gid] = make_float2(m, l);
  const float un = F::coded ? __uint_as_float((uint32_t)(127 + 24 - 20 + ve) << 23) : 1.f;
  const float un1 = ST == FUSE_U4_ASYM ? un * 0.0625f : un;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int v = 2 * tig + e;
    const float z = __shfl_sync(kAll, zs, v * 4);
    if (v >= n_vec) continue;
    float* o = a.part_o + (at + v) * D;
#pragma unroll
    for (int i = 0; i < MT; i += 2) {
      const int ch = F::coded ? gid * (D / 8) + 2 * i : ((i >> 2) * 8 + gid) * 8 + 2 * (i & 3);
      *reinterpret_cast<float4*>(o + ch) =
          make_float4(fmaf(acc[i][e], un, z), fmaf(acc[i][2 + e], un1, z), fmaf(acc[i + 1][e], un, z),
                      fmaf(acc[i + 1][2 + e], un1, z));
    }
  }
}

template <int ST, int D>
__global__ void __launch_bounds__(kWarps * 32, 2)
    attend_mma_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ ChunkOwners owners,
                      const __grid_constant__ RopeFreqs f, int side_ctas, int n_side_ctas) {
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ float2 s_cs[D / 2];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  WarpSmem<D>& sm = reinterpret_cast<WarpSmem<D>*>(raw)[warp];
  pdl_wait();
  pdl_trigger();                           // the join may read the call's inputs before it waits
  const int per_seg = a.n_kv_heads * a.nvg;
  Item y;
  if ((int)blockIdx.x < n_side_ctas) {
    // side rows: those before the new tokens
    y.r = a.req0 + blockIdx.x / side_ctas;
    const int i = (blockIdx.x % side_ctas) * kWarps + warp;
    const int seg = i / per_seg;
    y.h = i % per_seg / a.nvg;
    y.vg = i % a.nvg;
    const fuse_request_t R = a.reqs[y.r];
    const int n = R.k + R.n_query - a.n_new;
    y.t0 = seg * a.sseg;
    if (seg >= a.nside || y.t0 >= n) return;
    constexpr int RB = Fmt<FUSE_BF16, D>::RB;
    const int64_t row = R.out0 * a.n_kv_heads + y.h;
    y.k = reinterpret_cast<const uint8_t*>(a.Ks) + row * RB;
    y.v = reinterpret_cast<const uint8_t*>(a.Vs) + row * RB;
    y.vs = y.vz = nullptr;
    y.table = y.skip = nullptr;
    y.t1 = min(n, y.t0 + a.sseg);
    y.n_skip = y.pos0 = 0;
    y.slot = a.chunk_slots + (int64_t)y.r * a.nside + seg;
    if (y.h == 0 && y.vg == 0) {           // the selection, checked where its rows are read
      for (int t = y.t0 + lane; t < min(y.t1, R.k); t += 32) {
        const int v = a.idx[R.sel0 + t];
        if (v < 0 || v >= R.n_ctx || (t > 0 && a.idx[R.sel0 + t - 1] >= v))
          report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_ATTEND_SEL, (uint32_t)t);
      }
    }
    attend_mma_item<FUSE_BF16, D>(a, y, nullptr, nullptr, nullptr, sm);
    return;
  }
  const int ctas = (a.nsub * per_seg + kWarps - 1) / kWarps;
  const int b = blockIdx.x - n_side_ctas;
  const int ci = b / ctas;
  const int i = (b % ctas) * kWarps + warp;
  const int seg = i / per_seg;
  y.h = i % per_seg / a.nvg;
  y.vg = i % a.nvg;
  const fuse_chunk_t C = a.chunks[a.chunk0 + ci];
  y.r = owners.req[ci];
  const fuse_request_t R = a.reqs[y.r];
  // the chunk's angles, D / 16 pairs a warp.  The frequencies are launch
  // parameters, which a warp reads fast only at one address at a time.
  if (C.pos != 0) {                        // block-uniform
    constexpr int N = D / 2 / kWarps;
    float hi = 0.f, mid = 0.f, lo = 0.f, c, sn;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float h = f.hi[warp * N + k], m = f.mid[warp * N + k], l = f.lo[warp * N + k];
      if (lane == k) {
        hi = h;
        mid = m;
        lo = l;
      }
    }
    rope_cos_sin(C.pos, hi, mid, lo, c, sn);
    if (lane < N) s_cs[warp * N + lane] = make_float2(c, sn);
  }
  __syncthreads();
  y.t0 = seg * a.seg;
  if (seg >= a.nsub) return;
  if (y.t0 >= C.len) {                     // past the chunk's end: an item without a key
    if (lane < kVecs)
      a.part_ml[(((int64_t)(a.chunk0 + ci) * a.nsub + seg) * per_seg + i % per_seg) * kVecs + lane] =
          make_float2(-INFINITY, 0.f);
    return;
  }
  constexpr int RB = Fmt<ST, D>::RB;
  y.k = reinterpret_cast<const uint8_t*>(C.k) + y.h * RB;
  y.v = reinterpret_cast<const uint8_t*>(C.v) + y.h * RB;
  y.vs = reinterpret_cast<const __half*>(C.v_scale) + y.h;
  y.vz = reinterpret_cast<const __half*>(C.v_zero) + y.h;
  y.table = a.block_size > 0 ? C.block_table : nullptr;
  y.t1 = min(C.len, y.t0 + a.seg);
  y.n_skip = R.k;
  y.skip = a.idx + R.sel0;
  y.pos0 = (int)(C.dst_row - R.row0);
  y.slot = (int64_t)(a.chunk0 + ci) * a.nsub + seg;
  attend_mma_item<ST, D>(a, y, C.pos != 0 ? s_cs : nullptr, reinterpret_cast<const __half*>(C.k_scale),
                         reinterpret_cast<const __half*>(C.k_zero), sm);
}

template <int ST, int D>
cudaError_t launch_mma_t(const AttendArgs& a, const ChunkOwners& o, const RopeFreqs& f,
                         int side_reqs, cudaStream_t s) {
  const int smem = kWarps * (int)sizeof(WarpSmem<D>);
  const cudaError_t e = set_dyn_smem_once(reinterpret_cast<const void*>(attend_mma_kernel<ST, D>), smem);
  if (e != cudaSuccess) return e;
  const int per_seg = a.n_kv_heads * a.nvg;
  const int side = (a.nside * per_seg + kWarps - 1) / kWarps;
  const int ctas = (a.nsub * per_seg + kWarps - 1) / kWarps;
  const int64_t grid = (int64_t)side * side_reqs + (int64_t)ctas * a.n_chunks;
  if (grid == 0) return cudaSuccess;
  return launch_pdl(attend_mma_kernel<ST, D>, dim3((unsigned)grid), dim3(kWarps * 32), smem, s, a, o,
                    f, std::max(side, 1), side * side_reqs);
}

template <int D>
cudaError_t launch_mma_d(int st, const AttendArgs& a, const ChunkOwners& o, const RopeFreqs& f,
                         int side_reqs, cudaStream_t s) {
  if (st == FUSE_U4_ASYM) return launch_mma_t<FUSE_U4_ASYM, D>(a, o, f, side_reqs, s);
  if (st == FUSE_U8_ASYM) return launch_mma_t<FUSE_U8_ASYM, D>(a, o, f, side_reqs, s);
  return launch_mma_t<FUSE_BF16, D>(a, o, f, side_reqs, s);
}

}  // namespace

cudaError_t launch_attend_mma(const fuse_layer_desc_t& d, int st, const AttendArgs& a,
                              const ChunkOwners& o, const RopeFreqs& f, int side_reqs,
                              cudaStream_t s) {
  return d.head_dim == 128 ? launch_mma_d<128>(st, a, o, f, side_reqs, s)
                           : launch_mma_d<64>(st, a, o, f, side_reqs, s);
}

}  // namespace fusekv
