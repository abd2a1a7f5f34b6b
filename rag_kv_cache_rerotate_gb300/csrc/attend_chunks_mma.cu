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
// slots of 64 (4 bits), 32 (8 bits) or 16 (bf16): 8 KB at d = 128, two slots
// of shared memory per warp, filled by 16-byte cp.async one ahead; 12 warps an
// SM.  The warps of a CTA take neighbouring KV heads of the same tokens, so
// together they read whole rows.  Warps share only the chunk's angles.
// P carries the values' per-token scale, normalised by the largest so far (a
// power of two), in fp16 (bf16 rows: in two bf16 parts).  The maximum and the
// normaliser are raised lazily.
//
// Measured with the join (4 bits, 8 KV heads, d = 128, 64 query heads): 8
// requests of 33k tokens 90 us, 4.1 TB/s, where the bytes alone would take
// 54; issue slots are two fifths full and a warp waits for its own results, not
// for HBM.  16 paged requests of 0.5k to 8k tokens 36 us, 8 chunks of 512
// tokens 11 us (latency).  An item runs its start once, so instruction fetches
// count: the vectors are formed in a loop (96 -> 92 us).  Chunks go before side
// rows, whose items are shorter and fill the end (105 -> 96 us).  Slots of half
// the keys in three buffers: 4 % slower; rows of all heads brought by bulk
// copies of 2 KB to 16 warps an SM, 32 keys at a time: 132 us when this was
// 112 (twice the instructions); a warp of its own for bulk copies of single
// head rows 200 us.
#include <algorithm>

#include "attend_chunks.h"
#include "checks.h"
#include "launch.h"

namespace fusekv {

namespace {

constexpr int kWarps = kItemWarps;
constexpr int kSlots = 2;
constexpr float kRaise = 8.0f;            // log2: P <= 2^8, times a scale <= 2^6 stays in fp16
constexpr float kTiny = 1.17549435e-38f;  // 2^-126

template <int ST, int D> struct Fmt {
  static constexpr bool coded = ST != FUSE_BF16;
  static constexpr int RB = ST == FUSE_BF16 ? 2 * D : ST == FUSE_U8_ASYM ? D : D / 2;   // row bytes
  static constexpr int RC = RB / 16;                   // 16-byte chunks of a row
  static constexpr int TOK = ST == FUSE_BF16 ? 16 : ST == FUSE_U8_ASYM ? 32 : 64;       // keys a slot
  static constexpr int ROWS = TOK > 32 ? TOK / 32 : 1;                                  // of a lane
  static constexpr uint32_t kFull = TOK >= 32 ? 0xffffffffu : (1u << TOK) - 1;          // per 32 keys
};
constexpr int slot_bytes(int d) { return 64 * d; }     // TOK keys and values, in every format

template <int D> struct WarpSmem {
  uint8_t slot[kSlots][slot_bytes(D)];
  uint32_t skip[32];                                   // bit per key: selected, not read here
  uint32_t keep[kSlots][2];                            // bit per key of the slot: to be seen
  uint32_t sz[64];                                     // (scale, zero) of the slot's values, fp16
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
// c: the accumulators as (row gid, row gid + 8) pairs of columns.
__device__ __forceinline__ void mma16p(uint64_t (&c)[2], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  const float2 x = unpack2(c[0]), y = unpack2(c[1]);
  float d[4] = {x.x, x.y, y.x, y.y};
  mma16<true>(d, a0, a1, a2, a3, b0, b1);
  c[0] = pack2(d[0], d[1]);
  c[1] = pack2(d[2], d[3]);
}
// Transposes an 8 x 8 matrix of 16-bit elements held two a lane (row gid,
// columns 2 tig and 2 tig + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

// A place in ascending a[0, n) at most 64 before the first element >= x, by
// all lanes of the warp, 256 probes a round (one round up to 16 384 elements).
__device__ __forceinline__ int warp_search(const int32_t* a, int n, int x) {
  const int lane = threadIdx.x % 32;
  int lo = 0, len = n;                                 // the answer is in [lo, lo + len]
  while (len > 64) {
    const int step = (len + 255) / 256;
    bool below[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {                      // last elements of 256 parts
      const int i = lo + (j * 32 + lane + 1) * step - 1;
      below[j] = i < lo + len ? a[i] < x : false;
    }
    int parts = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) parts += __popc(__ballot_sync(0xffffffffu, below[j]));
    // parts whose last element is below x are skipped whole
    lo += parts * step;
    len = min(step - 1, len - parts * step);
  }
  return lo;
}

// The angles by which a chunk's items turn their queries back, shared by the
// CTA: each warp forms D / 16 pairs, and load_query waits for all of them.
// Side rows have none.
struct Angles {
  float2* at;                                          // (cos, sin) of each channel pair
  int pos;                                             // the chunk's offset
  bool chunk;                                          // block-uniform
};
template <int D> __device__ __forceinline__ void form_angles(const Angles& cs, const RopeFreqs& f) {
  if (cs.pos == 0) return;                             // block-uniform
  constexpr int N = D / 2 / kWarps;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // the frequencies are launch parameters, which a warp reads fast only at
  // one address at a time
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
  rope_cos_sin(cs.pos, hi, mid, lo, c, sn);
  if (lane < N) cs.at[warp * N + lane] = make_float2(c, sn);
}

// The query vectors of an item as they are: the lane's channel pairs
// (j, j + D / 2), j = NP lane .. NP lane + NP - 1, NP = D / 64 to a register.
struct RawQuery {
  uint32_t lo[kVecs], hi[kVecs];
};
template <int D>
__device__ __forceinline__ void read_query(const AttendArgs& a, int r, int h, int vg, RawQuery& x) {
  constexpr int NP = D / 64;
  const int lane = threadIdx.x % 32, n_vec = a.g * a.n_new, gl = __ffs(a.g) - 1;   // g = 1, 2, 4, 8
  const __nv_bfloat16* q0 = reinterpret_cast<const __nv_bfloat16*>(a.Q) + NP * lane +
                            ((int64_t)r * a.n_new * a.n_q_heads + h * a.g) * D;
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    const int vi = vg * kVecs + v;
    x.lo[v] = x.hi[v] = 0;
    if (vi < n_vec) {                                  // warp-uniform
      const __nv_bfloat16* q = q0 + ((vi >> gl) * a.n_q_heads + (vi & (a.g - 1))) * D;
      if constexpr (NP == 2) {
        x.lo[v] = *reinterpret_cast<const uint32_t*>(q);
        x.hi[v] = *reinterpret_cast<const uint32_t*>(q + D / 2);
      } else {
        x.lo[v] = *reinterpret_cast<const uint16_t*>(q);
        x.hi[v] = *reinterpret_cast<const uint16_t*>(q + D / 2);
      }
    }
  }
}

// The keys of an item on their way to shared memory: slots of TOK keys in two
// buffers in turn.
template <int ST, int D> struct Feed {
  using F = Fmt<ST, D>;
  static constexpr int RB = F::RB, RC = F::RC, TOK = F::TOK;
  static constexpr uint32_t kAll = 0xffffffffu;
  const AttendArgs& a;
  const Item& y;
  WarpSmem<D>& sm;
  const int lane;
  const int64_t stride;                                // bytes between rows
  const int dq, dr, bs;                                // TOK in pages and rows
  int blk[F::ROWS], rem[F::ROWS], id[F::ROWS];         // this lane's keys of the slot copied next
  int row[F::ROWS];                                    // rows of those of the slot copied last, -1: none
  int slot, buf;                                       // the slot copied next, and its buffer

  __device__ __forceinline__ Feed(const AttendArgs& a_, const Item& y_, WarpSmem<D>& sm_)
      : a(a_), y(y_), sm(sm_), lane(threadIdx.x % 32), stride((int64_t)a_.n_kv_heads * RB),
        dq(y_.table ? TOK / a_.block_size : 0), dr(TOK - dq * (y_.table ? a_.block_size : 0)),
        bs(y_.table ? a_.block_size : INT32_MAX), slot(0), buf(0) {
#pragma unroll
    for (int r = 0; r < F::ROWS; ++r) {
      rem[r] = y.t0 + r * 32 + lane;
      blk[r] = id[r] = 0;
      if (y.table) {
        blk[r] = rem[r] / bs;
        rem[r] -= blk[r] * bs;
      }
    }
    load_id();
  }
  __device__ __forceinline__ bool inside(int r) const {
    const int k = r * 32 + lane;
    return (TOK >= 32 || k < TOK) && y.t0 + slot * TOK + k < y.t1;
  }
  // The page id of the slot copied next is read one slot ahead and looked at
  // only when it is used, so that its read is not waited for.
  __device__ __forceinline__ void load_id() {
#pragma unroll
    for (int r = 0; r < F::ROWS; ++r)
      if (y.table && inside(r)) id[r] = y.table[blk[r]];
  }
  // Copies the next slot.  marked: the selected keys are known.
  __device__ __forceinline__ void copy(bool marked) {
    bool whole = !y.table;
#pragma unroll
    for (int r = 0; r < F::ROWS; ++r) {
      row[r] = inside(r) ? rem[r] : -1;
      if (y.table && row[r] >= 0) {
        if (id[r] >= 0 && id[r] < a.n_pool_blocks) {
          row[r] += id[r] * bs;
        } else {
          report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_ATTEND_BLOCK, (uint32_t)id[r]);
          row[r] = -1;
        }
      }
      const int k = slot * TOK + r * 32;
      uint32_t skip = marked ? sm.skip[k >> 5] : 0u;
      if constexpr (TOK < 32) skip >>= k & 31;
      if constexpr (!F::coded)                         // what is not seen may hold anything
        if (skip >> lane & 1) row[r] = -1;
      const uint32_t ok = __ballot_sync(kAll, row[r] >= 0);
      if (lane == 0) sm.keep[buf][r] = ok & ~skip;
      whole = whole && ok == F::kFull;
      rem[r] += dr;
      blk[r] += dq;
      if (rem[r] >= bs) {
        rem[r] -= bs;
        ++blk[r];
      }
    }
    const uint32_t dk = (uint32_t)__cvta_generic_to_shared(sm.slot[buf]), dv = dk + TOK * RB;
    // four 16-byte pieces of K and of V a lane and turn; the order within rows
    // repeats every 8 keys, so a turn (8 keys or a multiple) only moves on
    constexpr int kTurns = TOK * RC / 128;
    // pages: a loop where its code counts (24.5 -> 23.5 us on 4 drafted tokens
    // at 8 bits); at 4 bits it costs registers that the products need (92 -> 104
    // us on 8 requests of 33k tokens)
    constexpr int kUnroll = F::ROWS == 1 ? 1 : kTurns;
    if (whole) {                                       // warp-uniform: TOK consecutive rows
      const int64_t off = (int64_t)(y.t0 + slot * TOK + lane / RC) * stride + lane % RC * 16;
      const uint8_t *pk = y.k + off, *pv = y.v + off;
#pragma unroll
      for (int o = 0; o < kTurns; ++o)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = (i * 32 + lane) / RC, c = (i * 32 + lane) % RC, vr = v_row(key);
          cp16(dk + o * 2048 + key * RB + k_chunk<RC>(key, c) * 16, pk, true);
          cp16(dv + o * 2048 + vr * RB + v_chunk<RC>(vr, c) * 16, pv, true);
          pk += (32 / RC) * stride;
          pv += (32 / RC) * stride;
        }
    } else {
#pragma unroll kUnroll
      for (int o = 0; o < kTurns; ++o)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = (i * 32 + lane) / RC, c = (i * 32 + lane) % RC, vr = v_row(key);
          // rows are held by 32 keys: a turn's number or a constant says which
          const int of = F::ROWS == 1 ? row[0] : 128 / RC == 32 ? (o ? row[F::ROWS - 1] : row[0]) : row[i * 32 / RC / 32];
          const int kr = __shfl_sync(kAll, of, (o * (128 / RC) + key) & 31);
          const int64_t off = (int64_t)max(kr, 0) * stride + c * 16;
          cp16(dk + o * 2048 + key * RB + k_chunk<RC>(key, c) * 16, y.k + off, kr >= 0);
          cp16(dv + o * 2048 + vr * RB + v_chunk<RC>(vr, c) * 16, y.v + off, kr >= 0);
        }
    }
    cp_commit();
    ++slot;
    buf ^= 1;
    load_id();
  }
  // Marks the selected keys of the item, a bit each, and corrects the words of
  // keys to be seen of slot 0 where it is on its way.
  __device__ __forceinline__ void mark_selected() {
    sm.skip[lane] = 0;
    __syncwarp();
    if (y.n_skip > 0) {
      const int p0 = y.pos0 + y.t0, p1 = y.pos0 + y.t1;
      for (int i = warp_search(y.skip, y.n_skip, p0);; i += 128) {
        int v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = i + j * 32 + lane;
          v[j] = k < y.n_skip ? y.skip[k] : INT32_MAX;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (v[j] >= p0 && v[j] < p1) atomicOr(&sm.skip[(v[j] - p0) >> 5], 1u << ((v[j] - p0) & 31));
        if (__any_sync(kAll, v[3] >= p1)) break;
      }
      __syncwarp();
      if (lane < F::ROWS && slot == 1) sm.keep[0][lane] &= ~sm.skip[lane];
    }
    __syncwarp();
  }
};

// The item's query vectors, turned back by the chunk's angles (position 0: not
// turned) and scaled, as operand registers: qo[kk][b] holds the channel pair
// of half b of K-step kk of vector gid, its high parts, and qo[kk][2 + b] what
// is left of them.  Beside codes: score = sum * sscale + cst (vector gid).
// Staged in the second buffer, which is not in flight yet.
template <int ST, int D>
__device__ __forceinline__ void load_query(const AttendArgs& a, const Item& y, const RawQuery& raw,
                                           const Angles& cs, const __half* ks, const __half* kz,
                                           Feed<ST, D>& feed, uint32_t (&qo)[D / 16][4],
                                           float& sscale, float& cst) {
  using F = Fmt<ST, D>;
  constexpr uint32_t kAll = 0xffffffffu;
  constexpr int NP = D / 64;
  const int lane = threadIdx.x % 32, gid = lane >> 2, tig = lane & 3;
  const int j0 = NP * lane;
  float k0[NP], k1[NP], z0[NP], z1[NP];
  if constexpr (F::coded) {
    ks += y.h * D + j0;
    kz += y.h * D + j0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      k0[i] = __half2float(ks[i]);
      k1[i] = __half2float(ks[i + D / 2]);
      z0[i] = __half2float(kz[i]);
      z1[i] = __half2float(kz[i + D / 2]);
    }
    feed.mark_selected();                              // its reads run beside those above
  }
  if (cs.chunk) __syncthreads();                       // every warp's angles
  // a loop over the vectors, not eight copies of its body: an item runs
  // through this once, and fetching the instructions took longer than they do
  uint32_t* sq = reinterpret_cast<uint32_t*>(feed.sm.slot[1]);
  uint2* own = reinterpret_cast<uint2*>(sq + kVecs * D) + lane;   // [vector][lane]: its channels, then its sum
  sscale = 1.f;
  cst = 0.f;
#pragma unroll
  for (int v = 0; v < kVecs; ++v) own[v * 32] = make_uint2(raw.lo[v], raw.hi[v]);
#pragma unroll 2
  for (int v = 0; v < kVecs; ++v) {
    const uint2 w = own[v * 32];                       // 0: no such vector
    float x[NP][2], mx = 0.f, z = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float q0 = (i ? bf16_hi(w.x) : bf16_lo(w.x)) * a.scale;
      const float q1 = (i ? bf16_hi(w.y) : bf16_lo(w.y)) * a.scale;
      x[i][0] = q0;
      x[i][1] = q1;
      if (cs.pos != 0) {
        const float2 t = cs.at[j0 + i];
        x[i][0] = q0 * t.x + q1 * t.y;
        x[i][1] = q1 * t.x - q0 * t.y;
      }
      if constexpr (F::coded) {
        z += x[i][0] * z0[i] + x[i][1] * z1[i];
        x[i][0] *= k0[i];
        x[i][1] *= k1[i];
        mx = fmaxf(mx, fmaxf(fabsf(x[i][0]), fabsf(x[i][1])));
      }
    }
    float up = 1.f;
    if constexpr (F::coded) {
      own[v * 32].x = __float_as_uint(z);
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
        float t = x[i][b] * up;
        uint32_t w;
        if constexpr (F::coded) {
          if (ST == FUSE_U4_ASYM && (ch & 1)) t *= 0.0625f;     // odd codes sit 4 bits higher
          const __half hi = __float2half_rn(t);
          // an infinite scale: no remainder, whose product with a code would be NaN
          w = pack_half2(__half2float(hi), fabsf(t) == INFINITY ? 0.f : t - __half2float(hi));
        } else {
          const __nv_bfloat16 hi = __float2bfloat16_rn(t);
          w = pack_bf16x2(__bfloat162float(hi), t - __bfloat162float(hi));
        }
        sq[q_word<D>(v, ch)] = w;
      }
  }
  __syncwarp();
  if constexpr (F::coded) {
    // the sum over the lanes of vector gid: eight of them a lane
    const float* part = reinterpret_cast<const float*>(own - lane + gid * 32 + tig * 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) cst += part[2 * ((i + gid) & 7)];
    cst += __shfl_xor_sync(kAll, cst, 1);
    cst += __shfl_xor_sync(kAll, cst, 2);
  }
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t w0 = sq[q_word<D>(gid, q_channel<ST, D>(tig, kk, b, 0))];
      const uint32_t w1 = sq[q_word<D>(gid, q_channel<ST, D>(tig, kk, b, 1))];
      qo[kk][b] = __byte_perm(w0, w1, 0x5410);
      qo[kk][2 + b] = __byte_perm(w0, w1, 0x7632);
    }
}

// An item of codes.
//   S = K Q^T     A = codes (rows: 16 keys), B = the vectors' high parts, then
//                 what is left of them
//   O^T += V^T P  A = codes (rows: 16 channels, 16 keys), B = P, which comes
//                 from S by a transposed 8 x 8 move
// so a lane's scores, sums and outputs belong to vectors 2 tig and 2 tig + 1.
template <int ST, int D>
__device__ __forceinline__ void attend_codes(const AttendArgs& a, const Item& y, const RawQuery& raw,
                                             const Angles& cs, const RopeFreqs& f, const __half* ks,
                                             const __half* kz, WarpSmem<D>& sm) {
  using F = Fmt<ST, D>;
  constexpr int RB = F::RB, RC = F::RC, TOK = F::TOK, NT = TOK / 8, MT = D / 16;
  constexpr uint32_t kAll = 0xffffffffu;
  const int lane = threadIdx.x % 32, gid = lane >> 2, tig = lane & 3;
  const int n_slots = (y.t1 - y.t0 + TOK - 1) / TOK;
  Feed<ST, D> feed(a, y, sm);
  // scale and zero of a slot's values: read when it is copied, looked at when used
  uint16_t vs[F::ROWS], vz[F::ROWS];
  auto load_sz = [&]() {
#pragma unroll
    for (int r = 0; r < F::ROWS; ++r) {
      vs[r] = vz[r] = 0;
      if (feed.row[r] >= 0) {
        const int64_t at = (int64_t)feed.row[r] * a.n_kv_heads;
        vs[r] = reinterpret_cast<const uint16_t*>(y.vs)[at];
        vz[r] = reinterpret_cast<const uint16_t*>(y.vz)[at];
      }
    }
  };
  feed.copy(false);
  load_sz();
  form_angles<D>(cs, f);                               // while the first keys are on their way
  uint32_t q[D / 16][4];
  uint64_t ss, sb;                                     // sscale and cst of the lane's two vectors
  {
    float s1, c1;
    load_query<ST, D>(a, y, raw, cs, ks, kz, feed, q, s1, c1);
    ss = pack2(__shfl_sync(kAll, s1, tig * 8), __shfl_sync(kAll, s1, tig * 8 + 4));
    sb = pack2(__shfl_sync(kAll, c1, tig * 8), __shfl_sync(kAll, c1, tig * 8 + 4));
  }

  float m0 = -INFINITY, m1 = -INFINITY;                // running maxima
  uint64_t l2 = 0, z2 = 0;                             // sums over the lane's keys
  int ve = 0;                                          // exponent field of the largest value scale
  uint32_t seen = 0;                                   // bits of keys to be seen, of all slots
  uint64_t acc[MT][2];                                 // channel rows gid and gid + 8
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = 0;

#pragma unroll 1
  for (int s = 0; s < n_slots; ++s) {
    cp_wait<0>();                                      // the slot has landed
    __syncwarp();                                      // ... for every lane; the one before is done with
    uint32_t keep[F::ROWS], top = 0;
    bool full = true;
#pragma unroll
    for (int r = 0; r < F::ROWS; ++r) {
      keep[r] = sm.keep[s & 1][r];
      full = full && keep[r] == F::kFull;
      seen |= keep[r];
      // 0 for a key not seen, whatever it holds
      const uint32_t w = keep[r] >> lane & 1 ? (uint32_t)vs[r] | (uint32_t)vz[r] << 16 : 0u;
      sm.sz[r * 32 + lane] = w;
      top = max(top, w & 0x7fffu);
    }
    if (s + 1 < n_slots) {
      feed.copy(true);
      load_sz();
    }
    top = __reduce_max_sync(kAll, top);
    __syncwarp();
    const uint8_t* kb = sm.slot[s & 1] + gid * RB;
    const uint8_t* vb = sm.slot[s & 1] + TOK * RB;
    float fe = 1.f;                                    // factor of a raised normaliser
    const int e = min((int)(top >> 10), 30);
    const bool raise = e > ve;                         // warp-uniform
    if (raise) {
      fe = __uint_as_float((uint32_t)max(127 + ve - e, 1) << 23);
      ve = e;
    }
    // scores of keys 8 n + gid; 16 keys form two chains (high parts and rest)
    // of D / 16 dependent products
    uint64_t sc[NT];                                   // before sscale and cst
#pragma unroll
    for (int p = 0; p < NT / 2; ++p) {
      float c[2][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i >> 2][i & 3] = 0.f;
      const uint8_t* kr = kb + p * 16 * RB;
      if constexpr (ST == FUSE_U4_ASYM) {
        uint32_t w[2][D / 32];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(kr + r * 8 * RB + tig * 16);
            w[r][0] = x.x; w[r][1] = x.y; w[r][2] = x.z; w[r][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(kr + r * 8 * RB + tig * 8);
            w[r][0] = x.x; w[r][1] = x.y;
          }
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint32_t u = b ? w[0][j] >> 8 : w[0][j], v = b ? w[1][j] >> 8 : w[1][j];
            const uint32_t a0 = u & 0x000f000fu, a1 = v & 0x000f000fu, a2 = u & 0x00f000f0u,
                           a3 = v & 0x00f000f0u;
            mma16<true>(c[0], a0, a1, a2, a3, q[2 * j + b][0], q[2 * j + b][1]);
            mma16<true>(c[1], a0, a1, a2, a3, q[2 * j + b][2], q[2 * j + b][3]);
          }
      } else {
#pragma unroll
        for (int i = 0; i < RC / 4; ++i) {             // 16-byte chunks of a lane
          uint32_t w[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint4 x = *reinterpret_cast<const uint4*>(kr + r * 8 * RB + k_chunk<RC>(gid, i * 4 + tig) * 16);
            w[r][0] = x.x; w[r][1] = x.y; w[r][2] = x.z; w[r][3] = x.w;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = __byte_perm(w[0][j], 0, 0x4140), a1 = __byte_perm(w[1][j], 0, 0x4140),
                           a2 = __byte_perm(w[0][j], 0, 0x4342), a3 = __byte_perm(w[1][j], 0, 0x4342);
            mma16<true>(c[0], a0, a1, a2, a3, q[i * 4 + j][0], q[i * 4 + j][1]);
            mma16<true>(c[1], a0, a1, a2, a3, q[i * 4 + j][2], q[i * 4 + j][3]);
          }
        }
      }
      sc[2 * p] = add2(pack2(c[0][0], c[0][1]), pack2(c[1][0], c[1][1]));
      sc[2 * p + 1] = add2(pack2(c[0][2], c[0][3]), pack2(c[1][2], c[1][3]));
    }
    if (!full) {                                       // warp-uniform
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (!(keep[n / 4] >> (8 * (n & 3) + gid) & 1)) sc[n] = pack2(-INFINITY, -INFINITY);
    }
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float2 t = unpack2(sc[n]);
      x0 = fmaxf(x0, t.x);
      x1 = fmaxf(x1, t.y);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(kAll, x0, o));
      x1 = fmaxf(x1, __shfl_xor_sync(kAll, x1, o));
    }
    {
      const float2 f = unpack2(ss), g = unpack2(sb);
      if (x0 != -INFINITY) x0 = fmaf(x0, f.x, g.x);
      if (x1 != -INFINITY) x1 = fmaf(x1, f.y, g.y);
    }
    const bool up0 = x0 > m0 + kRaise, up1 = x1 > m1 + kRaise;
    if (__any_sync(kAll, up0 || up1) || raise) {
      const uint64_t al = pack2((up0 ? ex2(m0 - x0) : 1.f) * fe, (up1 ? ex2(m1 - x1) : 1.f) * fe);
      if (up0) m0 = x0;                                // (the factor is 0 at the first key)
      if (up1) m1 = x1;
      l2 = mul2(l2, al);
      z2 = mul2(z2, al);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        acc[i][0] = mul2(acc[i][0], al);
        acc[i][1] = mul2(acc[i][1], al);
      }
    }
    // weights, sums, and what multiplies the values; all carry the factor
    // 2^(20 - ve), with which a scale stays below 2^6
    const float lift = (float)(20 - ve);
    const uint64_t b2 =
        add2(sb, pack2(lift - (m0 == -INFINITY ? 0.f : m0), lift - (m1 == -INFINITY ? 0.f : m1)));
    uint32_t ph[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float2 x = unpack2(fma2(sc[n], ss, b2));
      const uint64_t p = pack2(ex2(x.x), ex2(x.y));
      l2 = add2(l2, p);
      const uint32_t w = sm.sz[n * 8 + gid];
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w));
      z2 = fma2(p, pack2(t.y, t.y), z2);
      const float2 v = unpack2(mul2(p, pack2(t.x, t.x)));
      ph[n] = transpose8x8(pack_half2(v.x, v.y));
    }
    // O^T += V^T P
    constexpr int VB = RB / 8;                         // bytes of a row that a lane takes
#pragma unroll
    for (int g2 = 0; g2 < TOK / 16; ++g2) {
      uint32_t w[4][VB / 4];                           // keys 2 tig, 2 tig + 1, 8 + 2 tig, 9 + 2 tig
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
            mma16p(acc[j * 4 + hi * 2], u & 0x000f000fu, u & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u,
                   ph[2 * g2], ph[2 * g2 + 1]);
            const uint32_t us = u >> 8, vs = v >> 8;
            mma16p(acc[j * 4 + hi * 2 + 1], us & 0x000f000fu, us & 0x00f000f0u, vs & 0x000f000fu,
                   vs & 0x00f000f0u, ph[2 * g2], ph[2 * g2 + 1]);
          } else {
            mma16p(acc[j * 2 + hi], u & 0x00ff00ffu, (u >> 8) & 0x00ff00ffu, v & 0x00ff00ffu,
                   (v >> 8) & 0x00ff00ffu, ph[2 * g2], ph[2 * g2 + 1]);
          }
        }
    }
  }

  // ---- the item's partial ----------------------------------------------------
  const float vu = __uint_as_float((uint32_t)(127 + ve - 20) << 23);
  float2 l = unpack2(mul2(l2, pack2(vu, vu))), z = unpack2(mul2(z2, pack2(vu, vu)));
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    l.x += __shfl_xor_sync(kAll, l.x, o);
    l.y += __shfl_xor_sync(kAll, l.y, o);
    z.x += __shfl_xor_sync(kAll, z.x, o);
    z.y += __shfl_xor_sync(kAll, z.y, o);
  }
  // no key to see: an item without one, whatever the chunk's scales and zeros hold
  if (seen == 0) l = make_float2(0.f, 0.f);
  const int n_vec = min(kVecs, a.g * a.n_new - y.vg * kVecs);
  const int64_t at = ((y.slot * a.n_kv_heads + y.h) * a.nvg + y.vg) * kVecs;
  const float un = __uint_as_float((uint32_t)(127 + 24 - 20 + ve) << 23);
  const float un1 = ST == FUSE_U4_ASYM ? un * 0.0625f : un;    // odd codes sit 4 bits higher
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int v = 2 * tig + e;
    if (v >= n_vec) continue;
    const float zv = e ? z.y : z.x;
    if (gid == 0) a.part_ml[at + v] = make_float2(e ? m1 : m0, e ? l.y : l.x);
    float* o = a.part_o + (at + v) * D + gid * (D / 8);
#pragma unroll
    for (int i = 0; i < MT; i += 2) {
      const float2 r0 = unpack2(acc[i][0]), r1 = unpack2(acc[i][1]), r2 = unpack2(acc[i + 1][0]),
                   r3 = unpack2(acc[i + 1][1]);
      *reinterpret_cast<float4*>(o + 2 * i) =
          e ? make_float4(fmaf(r0.y, un, zv), fmaf(r1.y, un1, zv), fmaf(r2.y, un, zv), fmaf(r3.y, un1, zv))
            : make_float4(fmaf(r0.x, un, zv), fmaf(r1.x, un1, zv), fmaf(r2.x, un, zv), fmaf(r3.x, un1, zv));
    }
  }
}

// An item of bf16 rows.
//   S^T = Q K^T   A = Q (rows 0-7: the vectors' high parts, 8-15: what is
//                 left of them), B = 8 keys
//   O^T += V^T P  A = values (rows: 16 channels, 8 keys), B = P in two parts;
//                 the layout in which S^T comes out is the one P goes in
// A lane's scores belong to vector gid, its outputs to 2 tig and 2 tig + 1.
template <int D>
__device__ __forceinline__ void attend_rows(const AttendArgs& a, const Item& y, const RawQuery& raw,
                                            const Angles& cs, const RopeFreqs& f, WarpSmem<D>& sm) {
  constexpr int ST = FUSE_BF16;
  using F = Fmt<ST, D>;
  constexpr int RB = F::RB, RC = F::RC, TOK = F::TOK, MT = D / 16;
  constexpr uint32_t kAll = 0xffffffffu;
  const int lane = threadIdx.x % 32, gid = lane >> 2, tig = lane & 3;
  const int n_slots = (y.t1 - y.t0 + TOK - 1) / TOK;
  Feed<ST, D> feed(a, y, sm);
  feed.mark_selected();
  feed.copy(true);
  form_angles<D>(cs, f);
  uint32_t q[D / 16][4];
  float one, none;
  load_query<ST, D>(a, y, raw, cs, nullptr, nullptr, feed, q, one, none);
  float m = -INFINITY, l = 0.f;                        // vector gid (its sum: this lane's keys)
  float acc[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 1
  for (int s = 0; s < n_slots; ++s) {
    cp_wait<0>();                                      // the slot has landed
    __syncwarp();                                      // ... for every lane; the one before is done with
    const uint32_t keep = sm.keep[s & 1][0];
    if (s + 1 < n_slots) feed.copy(true);
    const uint8_t* kb = sm.slot[s & 1] + gid * RB;
    const uint8_t* vb = sm.slot[s & 1] + TOK * RB;
    float sc[2][2];                                    // keys 8 n + 2 tig, + 1
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      float c[2][4];                                   // two chains of products
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i >> 2][i & 3] = 0.f;
#pragma unroll
      for (int i = 0; i < RC / 4; ++i) {               // 16-byte chunks of a lane
        const uint4 x =
            *reinterpret_cast<const uint4*>(kb + n * 8 * RB + k_chunk<RC>(gid, i * 4 + tig) * 16);
        mma16<false>(c[0], q[2 * i][0], q[2 * i][2], q[2 * i][1], q[2 * i][3], x.x, x.y);
        mma16<false>(c[1], q[2 * i + 1][0], q[2 * i + 1][2], q[2 * i + 1][1], q[2 * i + 1][3], x.z, x.w);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // an infinite key: the vectors' high parts decide, what is left of them is 0 or of either sign
        const float hi = c[0][e] + c[1][e], rest = c[0][2 + e] + c[1][2 + e];
        sc[n][e] = fabsf(hi) == INFINITY ? hi : hi + rest;
        if (!(keep >> (8 * n + 2 * tig + e) & 1)) sc[n][e] = -INFINITY;
      }
    }
    float mt = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
    mt = fmaxf(mt, __shfl_xor_sync(kAll, mt, 1));
    mt = fmaxf(mt, __shfl_xor_sync(kAll, mt, 2));
    const bool up = mt > m + kRaise;
    if (__any_sync(kAll, up)) {
      const float al = up ? ex2(m - mt) : 1.f;         // 0 at the first key
      if (up) m = mt;
      l *= al;
      const float f0 = __shfl_sync(kAll, al, tig * 8), f1 = __shfl_sync(kAll, al, tig * 8 + 4);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        acc[i][0] *= f0;
        acc[i][1] *= f1;
        acc[i][2] *= f0;
        acc[i][3] *= f1;
      }
    }
    const float ref = m == -INFINITY ? 0.f : m;
    uint32_t ph[2], pl[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float p0 = ex2(sc[n][0] - ref), p1 = ex2(sc[n][1] - ref);
      l += p0 + p1;
      // the high part is cut off, not rounded (2^-16 of the weight is lost in
      // all, 2^-17 if it were), and what is left is at least 2^-126: both parts
      // of a weight above 0 are, so that an infinite value stays infinite
      ph[n] = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
      pl[n] = pack_bf16x2(fmaxf(p0 - bf16_lo(ph[n]), fminf(p0, kTiny)),
                          fmaxf(p1 - bf16_hi(ph[n]), fminf(p1, kTiny)));
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      uint32_t w[4][4];                                // keys 2 tig, 2 tig + 1, 8 + 2 tig, 9 + 2 tig
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int vr = (k >> 1) * 8 + (k & 1) * 4 + tig;
        const uint4 x = *reinterpret_cast<const uint4*>(vb + vr * RB + v_chunk<RC>(vr, i * 8 + gid) * 16);
        w[k][0] = x.x; w[k][1] = x.y; w[k][2] = x.z; w[k][3] = x.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a0 = __byte_perm(w[0][j], w[1][j], 0x5410), a1 = __byte_perm(w[0][j], w[1][j], 0x7632),
                       a2 = __byte_perm(w[2][j], w[3][j], 0x5410), a3 = __byte_perm(w[2][j], w[3][j], 0x7632);
        mma16<false>(acc[i * 4 + j], a0, a1, a2, a3, ph[0], ph[1]);
        mma16<false>(acc[i * 4 + j], a0, a1, a2, a3, pl[0], pl[1]);
      }
    }
  }

  l += __shfl_xor_sync(kAll, l, 1);
  l += __shfl_xor_sync(kAll, l, 2);
  const int n_vec = min(kVecs, a.g * a.n_new - y.vg * kVecs);
  const int64_t at = ((y.slot * a.n_kv_heads + y.h) * a.nvg + y.vg) * kVecs;
  if (tig == 0 && gid < n_vec) a.part_ml[at + gid] = make_float2(m, l);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int v = 2 * tig + e;
    if (v >= n_vec) continue;
    float* o = a.part_o + (at + v) * D + gid * 8;
#pragma unroll
    for (int i = 0; i < MT; i += 2)
      *reinterpret_cast<float4*>(o + (i >> 2) * 64 + 2 * (i & 3)) =
          make_float4(acc[i][e], acc[i][2 + e], acc[i + 1][e], acc[i + 1][2 + e]);
  }
}

template <int ST, int D>
__global__ void __launch_bounds__(kWarps * 32, 3)
    attend_mma_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ ItemTable t,
                      const __grid_constant__ RopeFreqs f) {
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ float2 s_cs[D / 2];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  WarpSmem<D>& sm = reinterpret_cast<WarpSmem<D>*>(raw)[warp];
  const ItemPlace at = item_place(a, t);
  pdl_wait();
  pdl_trigger();                           // the join may read the call's inputs before it waits
  if (at.none) return;
  Item y;
  y.h = at.h;
  y.vg = at.vg;
  y.slot = at.slot;
  // the queries are read first: they do not depend on the tables' entries
  y.r = at.side ? a.req0 + at.part : t.owner[at.part];
  RawQuery rq;
  read_query<D>(a, y.r, y.h, y.vg, rq);
  if (at.side) {
    // side rows: those before the new tokens
    const fuse_request_t R = a.reqs[y.r];
    const int n = R.k + R.n_query - a.n_new;
    y.t0 = at.seg * a.sseg;
    if (y.t0 >= n) {                       // only where the two copies of the table differ
      no_keys(a, at);
      return;
    }
    constexpr int RB = Fmt<FUSE_BF16, D>::RB;
    const int64_t row = R.out0 * a.n_kv_heads + y.h;
    y.k = reinterpret_cast<const uint8_t*>(a.Ks) + row * RB;
    y.v = reinterpret_cast<const uint8_t*>(a.Vs) + row * RB;
    y.vs = y.vz = nullptr;
    y.table = y.skip = nullptr;
    y.t1 = min(n, y.t0 + a.sseg);
    y.n_skip = y.pos0 = 0;
    if (y.h == 0 && y.vg == 0) {           // the selection, checked where its rows are read
      for (int t = y.t0 + lane; t < min(y.t1, R.k); t += 32) {
        const int v = a.idx[R.sel0 + t];
        if (v < 0 || v >= R.n_ctx || (t > 0 && a.idx[R.sel0 + t - 1] >= v))
          report_error(a.err, FUSE_ERR_DEVICE_BOUNDS, SITE_ATTEND_SEL, (uint32_t)t);
      }
    }
    attend_rows<D>(a, y, rq, {nullptr, 0, false}, f, sm);
    return;
  }
  const fuse_chunk_t C = a.chunks[a.chunk0 + at.part];
  const fuse_request_t R = a.reqs[y.r];
  y.t0 = at.seg * a.seg;
  const Angles cs{s_cs, C.pos, true};
  if (y.t0 >= C.len) {                     // past the chunk's end
    form_angles<D>(cs, f);                 // this warp's part for the others
    __syncthreads();
    no_keys(a, at);
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
  if constexpr (ST == FUSE_BF16)
    attend_rows<D>(a, y, rq, cs, f, sm);
  else
    attend_codes<ST, D>(a, y, rq, cs, f, reinterpret_cast<const __half*>(C.k_scale),
                        reinterpret_cast<const __half*>(C.k_zero), sm);
}

template <int ST, int D>
cudaError_t launch_mma_t(const AttendArgs& a, const ItemTable& t, const RopeFreqs& f, cudaStream_t s) {
  const int smem = kWarps * (int)sizeof(WarpSmem<D>);
  const cudaError_t e = set_dyn_smem_once(reinterpret_cast<const void*>(attend_mma_kernel<ST, D>), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attend_mma_kernel<ST, D>, dim3((unsigned)item_ctas(a, t)), dim3(kWarps * 32), smem, s,
                    a, t, f);
}

template <int D>
cudaError_t launch_mma_d(int st, const AttendArgs& a, const ItemTable& t, const RopeFreqs& f,
                         cudaStream_t s) {
  if (st == FUSE_U4_ASYM) return launch_mma_t<FUSE_U4_ASYM, D>(a, t, f, s);
  if (st == FUSE_U8_ASYM) return launch_mma_t<FUSE_U8_ASYM, D>(a, t, f, s);
  return launch_mma_t<FUSE_BF16, D>(a, t, f, s);
}

}  // namespace

cudaError_t launch_attend_mma(const fuse_layer_desc_t& d, int st, const AttendArgs& a,
                              const ItemTable& t, const RopeFreqs& f, cudaStream_t s) {
  return d.head_dim == 128 ? launch_mma_d<128>(st, a, t, f, s) : launch_mma_d<64>(st, a, t, f, s);
}

}  // namespace fusekv
