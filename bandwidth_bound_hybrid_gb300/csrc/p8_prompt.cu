// Prompt attention over the paged 8-bit KV cache on the tensor cores of sm_103a
// (format: p8_dev.cuh).
//
// A tile is 128 query vectors of one sequence and kv head: 128 / G consecutive
// rows with their G heads.  It goes over the blocks that any of its rows sees,
// BN positions a step, with the running maximum and sum of a softmax:
//   S = (q_hi + q_lo) cK^T,   w = 2^(s sK - m) sV 2^(14 - E),   O = (w_hi + w_lo) cV
// q and w as two fp16 parts (22 bits; w to 2^-39 of 2^E), the codes exact in
// fp16, the blocks' scales FP32 factors of a score and of the weight that meets
// a block of V.  2^E is above the step's largest V scale where the step's are
// within 2^4 of each other.  Where they are not ("wide" steps), a block that a
// row does not see, or hardly weighs, must not decide how finely the others
// enter: there a row takes its own E, with 2^E up to 4 times the largest of its
// products 2^(s sK - m) sV.  The open block's rows are fp16 under a power of two,
// one for all of them or, where they are far apart, one each.
// A step's O is added to the outputs in registers, in FP32: the tensor cores
// truncate what they add to an accumulator, which over a long context would be
// 2^-24 a product, all one way.
//
// Roles of a CTA of 16 warps, one an SM:
//   * 8 row warps: a thread has a row's scores of half a step (tcgen05.ld),
//     the maximum is exchanged with the other half's thread; the weights go
//     back into the scores' columns as the A operand of the second product
//     (16 scores become 8 columns of w_hi and 8 of w_lo); then the step before
//     is added, half the elements of a head a thread;
//   * 1 warp copies the codes of a step's blocks (each contiguous in its page,
//     adjacent ones together) to a ring of shared memory in bulk, another
//     fetches their scales;
//   * 4 warps widen them to fp16 tiles in shared memory, 128-byte swizzle, K as
//     K-major B operand and V, laid out alike, as MN-major;
//   * 1 thread issues tcgen05.mma: S of step k + 1 before O of step k, so that
//     the row warps' softmax runs beside the tensor cores; 1 warp hands out the
//     pieces (a CTA's steps of a tile).
// Two score and (hd <= 128) two output accumulators in TMEM: 512 columns.
//
// Work split: the steps of all tiles form one list, of which CTA c takes an
// equal span.  A tile that several CTAs share leaves partials (outputs, maximum,
// sum) in the workspace, joined by a second small kernel.
//
// Bound by a chain, the widening of K and V: 2048 rows of 4 x 128 with 16 heads at
// position 4096 take 200 us, 429 TFLOP/s of the two products (twice that is
// executed, 44% of the measured bf16 rate); of 2 x 256 397 us (432), of 4 x 64
// 150 (286: half the products, but as many scores).  A step of 128 x 128 takes
// 5450 cycles, of which the products need 2048 and the widening 4800 in one warp
// a scheduler; a scheduler issues 3050 instructions for it (two row warps 750
// each, a widening warp 630, waits), in 54% of its cycles.  One row over 30k
// positions takes 45.6 us: a step costs what 128 query vectors cost.
// Measured and not kept, against 197 us then: 8 widening warps (198, the row warps
// with 160 registers), tiles of 256 rows that share the widened codes (219), loads
// of the codes in registers instead of the ring (407), a thread's 64 scores
// unrolled (387: the roles' code then misses the instruction cache).
#include <climits>

#include "p8_dev.cuh"
#include "tc05.cuh"

namespace hy {
namespace p8 {
namespace {

constexpr int kThreads = 512, kRowWarps = 8, kWidenWarps = 4;

template <int HD>
struct Tile {
  static constexpr int BM = 128, BN = HD == 256 ? 64 : 128;
  static constexpr int NBLK = BN / kBlock;        // blocks of a step
  static constexpr int NSK = HD == 256 ? 1 : 2;   // widened tiles of K and of V
  static constexpr int NSV = HD == 64 ? 2 : 1;
  static constexpr int NO = HD == 256 ? 1 : 2;    // output accumulators
  static constexpr int kQ = BM * HD * 2;          // one part of the queries
  static constexpr int kKV = BN * HD * 2;
  static constexpr int kSlot = 8192;              // codes of a ring slot
  static constexpr int kSlots = HD == 256 ? 2 : 6;
  static constexpr int NP = kSlot / 16 / 128;     // 16-byte pieces of a slot that a widening thread has
  static constexpr int NS = BN * HD / kSlot;      // slots of a step's K or V
  static constexpr int SB = NBLK / NS;            // blocks of a slot
  static constexpr int kSmem = 2 * kQ + (NSK + NSV) * kKV + kSlots * kSlot;
};

struct Piece {
  int b, g, i0;             // sequence (-1: no more pieces), kv head, the tile's first row
  unsigned tile;            // the tile's first step in the list
  int first;                // the tile's first row in y and o
  int T, n, rows, t0, t1;   // of the sequence: position, rows; of the tile: rows, first and last position
  View view;
  int steps, s0, s1;        // the tile's steps; this CTA's
};
constexpr int kPieces = 4;  // of them at a time

// What the row and widening warps need of a step.
constexpr int kSteps = 8;  // of them at a time
struct Step {
  float fk[8], fv[8];  // scales of K; of V times 2^(14 - E) (wide: as they are)
  int u[8];            // first positions of the blocks; INT_MAX: not there
  int kind[8];         // 0: codes in the ring, 1: nothing (zeros), 2: the open block
  float ev;            // 2^(E - 14)
  int edge;            // some row does not see all of it
  int wide;            // V's scales are so far apart that each row takes its own E
  // What brings the open block's rows below 2^15 (K) and, as codes are, 2^7 (V).  Rows of about one size share one
  // power of two, and its inverses are in fk and fv.  Rows far apart, which must not take bits from one another, have one
  // each: then `open` is the block (else -1, and rk and rv are not read), the step is wide, a row's scale is fk rk for K
  // and rv for V (0: no row, or one of zeros).
  float uk[kBlock], uv[kBlock], rk[kBlock], rv[kBlock];
  int open;
};

struct alignas(16) Small {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pfull[2], ofull[2], oempty[2], mfull[kSteps],
      mempty[kSteps], rfull[6], rempty[6], wfull[kPieces], wempty[kPieces], qfull, done;
  uint32_t tmem;
  int odd[6];  // of a ring slot: some block's codes are not there
  int open_nan;
  Step step[kSteps];
  Piece piece[kPieces];
  float qf[128];
  float mx[2][2][128];
  float top[2][128];  // of a wide step: log2 of the largest product of weight and V scale
  float ls[2][128];
  // the work
  int T[kMaxB], n[kMaxB], first[kMaxB];
  unsigned at[kMaxB + 1];   // steps of one kv head before each sequence
  unsigned begin, end;      // this CTA's steps
  int b, g, i0;             // its first tile
  unsigned tile;            // and that tile's first step
};

// A CTA's first piece, for the join: whether it is the tail of a tile that began in CTA `lo`, through CTA `hi`.
struct Share {
  int joins, lo, hi, b, g, i0;
};

// The blocks that some query of positions t0 .. t1 sees.
__device__ __forceinline__ View view_range(int t0, int t1, int window, int sinks) {
  View v = view_of(t0, window, sinks);
  v.n += t1 / kBlock - t0 / kBlock;
  return v;
}
// Sequences, the list of steps and this CTA's span of it (the whole CTA).
template <int HD, int G>
__device__ __forceinline__ void plan_work(const Params& p, Small& sm, Share* share) {
  constexpr int BQ = Tile<HD>::BM / G;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < p.nb) {
    const int T = p.len[tid], s = p.row_start[tid], e = p.row_start[tid + 1];
    const bool ok = T >= 0 && s >= 0 && e >= s && e <= p.n &&
                    (long long)T + (e - s) <= (long long)p.c.max_pages * p.c.page_tokens;
    if (!ok && blockIdx.x == 0) set_guard(p.guard, kGuardBadPosition);
    sm.T[tid] = T;
    sm.first[tid] = s;
    sm.n[tid] = ok ? e - s : 0;
  }
  __syncthreads();
  // steps of the tile of sequence b's rows i0 .., 0 past its last
  auto steps_at = [&](int b, int i0) {
    const int n = sm.n[b], t0 = sm.T[b] + i0, t1 = t0 + min(n - i0, BQ) - 1;
    if (i0 >= n) return 0u;
    return (unsigned)(view_range(t0, t1, p.window, p.sinks).n + Tile<HD>::NBLK - 1) / Tile<HD>::NBLK;
  };
#pragma unroll 1
  for (int b = warp; b < p.nb; b += kThreads / 32) {
    unsigned s = 0;
#pragma unroll 1
    for (int i0 = lane * BQ; i0 < sm.n[b]; i0 += 32 * BQ) s += steps_at(b, i0);
    s = __reduce_add_sync(0xffffffffu, s);
    if (lane == 0) sm.at[b + 1] = s;
  }
  __syncthreads();
  if (warp == 0) {
    auto scan = [&](unsigned v) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      return v;
    };
    unsigned head = 0;  // steps of a head
#pragma unroll 1
    for (int b0 = 0; b0 < p.nb; b0 += 32) {
      const unsigned incl = scan(b0 + lane < p.nb ? sm.at[b0 + lane + 1] : 0);
      if (b0 + lane < p.nb) sm.at[b0 + lane + 1] = head + incl;
      head += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) sm.at[0] = 0;
    __syncwarp();
    // CTA c of C takes steps c q + min(c, rem) ..
    const unsigned total = head * p.nkv, c = blockIdx.x;
    const unsigned C = max(1u, min(gridDim.x, total)), q = total / C, rem = total - q * C;
    const unsigned begin = c < C ? c * q + min(c, rem) : total, end = c < C ? begin + q + (c < rem) : total;
    Share mine = {0, 0, 0, 0, 0, 0};
    if (begin < end) {
      const int g = (int)(begin / head);
      const unsigned r = begin - g * head;
      int b = 0;  // the first b with r < at[b + 1]
#pragma unroll 1
      for (int k = 0; k < p.nb; k += 32) {
        const unsigned in = __ballot_sync(0xffffffffu, k + lane < p.nb && r < sm.at[min(k + lane, p.nb - 1) + 1]);
        if (in) {
          b = k + __ffs(in) - 1;
          break;
        }
      }
      unsigned at = sm.at[b], steps = 0;
      int i0 = 0;
#pragma unroll 1
      for (int k = 0;; k += 32 * BQ) {  // (its steps end past r)
        const unsigned s = steps_at(b, k + lane * BQ), incl = scan(s);
        const unsigned in = __ballot_sync(0xffffffffu, r < at + incl);
        if (in) {
          const int l = __ffs(in) - 1;
          i0 = k + l * BQ;
          steps = __shfl_sync(0xffffffffu, s, l);
          at += __shfl_sync(0xffffffffu, incl - s, l);
          break;
        }
        at += __shfl_sync(0xffffffffu, incl, 31);
      }
      const unsigned tile = g * head + at, big = rem * (q + 1);
      if (lane == 0) {
        sm.b = b;
        sm.g = g;
        sm.i0 = i0;
        sm.tile = tile;
      }
      auto cta_of = [&](unsigned s) { return (int)(s < big ? s / (q + 1) : rem + (s - big) / q); };
      const int lo = cta_of(tile), hi = cta_of(tile + steps - 1);
      mine = {begin > tile && lo + 1 == (int)c, lo, hi, b, g, i0};
    }
    if (lane == 0) {
      sm.begin = begin;
      sm.end = end;
      share[blockIdx.x] = mine;
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- packed FP32
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// v truncated to fp16's 11 significant bits: v - trunc11(v) is exact
__device__ __forceinline__ float trunc11(float v) { return __uint_as_float(__float_as_uint(v) & 0xffffe000u); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// the least n with 2^n > v, for v from 2^-126; -126 below, 129 for NaN
__device__ __forceinline__ float log2_above(float v) { return (float)((int)(__float_as_uint(v) >> 23 & 255) - 126); }

// ---------------------------------------------------------------- tcgen05 forms
// fp16 operands, FP32 accumulator; trans_b: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool trans_b) {
  return (1u << 4) | (trans_b ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// MN-major operand, 128-byte swizzle: rows of 64 elements, one per k; 8-row groups 1024 bytes apart, the next 64
// elements `chunk` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr, uint32_t chunk) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)((chunk >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)((1024 >> 4) & 0x3FFF) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 16 columns: load with its wait, store.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
template <int R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
// Registers of a thread by role: 8 x 192 + 4 x 64 + 4 x 64 = 2048, the launch's 16 x 128.
constexpr int kRowRegs = 192, kWidenRegs = 64, kOtherRegs = 64;
static_assert(kRowWarps * kRowRegs + kWidenWarps * kWidenRegs + 4 * kOtherRegs <= kThreads / 32 * 128,
              "register split");

// Whether the phase of the given parity is over, after at most 2 us.
__device__ __forceinline__ bool try_bar(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 2000;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
constexpr int kTries = 1 << 20;  // bounds every wait: two seconds at most
// A thread's wait.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < kTries; ++i)
    if (try_bar(bar, parity)) return true;
  return false;
}
// A warp's wait, all lanes' branches alike (a loop that lanes may leave one by one costs a ready wait 400 cycles
// beside the other roles' warps); false, with the guard set, if it gave up.
__device__ __forceinline__ bool wait_all(const Params& p, uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < kTries; ++i)
    if (__all_sync(0xffffffffu, try_bar(bar, parity))) return true;
  set_guard(p.guard, kGuardWaitTimeout);
  return false;
}
// The pieces of this CTA's span, in order, by one warp for all roles.
template <int HD, int G>
__device__ __forceinline__ void piece_role(const Params& p, Small& sm) {
  Piece w = {sm.b, sm.g, sm.i0, sm.tile};
#pragma unroll 1
  for (int np = 0;; ++np) {
    if (np > 0) {
      w.tile += w.steps;
      w.i0 += Tile<HD>::BM / G;
      if (w.tile >= sm.end) {
        w.b = -1;
      } else if (w.i0 >= w.n) {
        w.i0 = 0;
        do {
          if (++w.b == p.nb) {
            w.b = 0;
            ++w.g;
          }
        } while (sm.n[w.b] == 0);  // (there is one with rows: the list has more steps)
      }
    }
    if (w.b >= 0) {
      w.T = sm.T[w.b];
      w.n = sm.n[w.b];
      w.first = sm.first[w.b] + w.i0;
      w.rows = min(w.n - w.i0, Tile<HD>::BM / G);
      w.t0 = w.T + w.i0;
      w.t1 = w.t0 + w.rows - 1;
      w.view = view_range(w.t0, w.t1, p.window, p.sinks);
      w.steps = (unsigned)(w.view.n + Tile<HD>::NBLK - 1) / Tile<HD>::NBLK;
      w.s0 = (int)(max(sm.begin, w.tile) - w.tile);
      w.s1 = (int)(min(sm.end, w.tile + w.steps) - w.tile);
    }
    const int k = np % kPieces;
    if (np >= kPieces && !wait_all(p, &sm.wempty[k], ((np / kPieces) & 1) ^ 1)) return;
    if ((threadIdx.x & 31) == 0) {
      sm.piece[k] = w;
      mbar_arrive(&sm.wfull[k]);
    }
    if (w.b < 0) return;
  }
}
// Piece np for a warp; false after the last, or if the wait gave up.
__device__ __forceinline__ bool next_piece(const Params& p, Small& sm, int np, Piece& w) {
  const int k = np % kPieces;
  if (!wait_all(p, &sm.wfull[k], (np / kPieces) & 1)) return false;
  w = sm.piece[k];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.wempty[k]);
  return w.b >= 0;
}
constexpr int kPieceReaders = kRowWarps + kWidenWarps + 3;

// A row warp's wait.  One that has given up goes on without waiting (its outputs are worthless, the guard says so),
// so that it still meets the other row warps at their barriers.
__device__ __forceinline__ void wait_row(const Params& p, uint64_t* bar, uint32_t parity, bool& ok) {
  if (ok) ok = wait_all(p, bar, parity);
}

// ---------------------------------------------------------------- widening
// The codes of a word's bytes as fp16 pairs, exact: c + 128 under the exponent of 1024, less 1152.
__device__ __forceinline__ void widen(uint32_t w, uint32_t* h) {
  const __half2 k1152 = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  w ^= 0x80808080u;
  const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), k1152);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), k1152);
  h[0] = *reinterpret_cast<const uint32_t*>(&x);
  h[1] = *reinterpret_cast<const uint32_t*>(&y);
}
// 16 elements from 16 c of row r: two 16-byte chunks of a 128-byte row.
template <int BN>
__device__ __forceinline__ void put16(uint8_t* tile, int r, int c, const uint32_t* h) {
  uint8_t* row = tile + (c >> 2) * (BN * 128) + r * 128;
  const int k = (c & 3) * 2;
  *reinterpret_cast<uint4*>(row + ((k ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(row + (((k + 1) ^ (r & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
}

// Bulk copy to shared memory with the L2's usual policy (a tile's neighbours read the same blocks).
__device__ __forceinline__ void copy_bulk(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

// Order in which the tensor cores take K and V of a piece's steps, K a step ahead: K0, K1, V0, K2, V1, ...
__device__ __forceinline__ bool is_v(int i, int steps) { return i > 0 && (i == 2 * steps - 1 || i % 2 == 0); }

// The copies of the codes into the ring (one warp; lane b the step's block b).  Adjacent blocks of a page are one copy.
template <int HD, int G>
__device__ __forceinline__ void load_role(const Params& p, Small& sm, uint8_t* ring) {
  using Ti = Tile<HD>;
  constexpr int NBLK = Ti::NBLK, SB = Ti::SB, kBytes = kBlock * HD;
  const int lane = threadIdx.x & 31;
  Piece w;
  int slot = 0;
  uint32_t use = 0;  // times the ring has been gone through
  bool ok = true;
#pragma unroll 1
  for (int np = 0; ok && next_piece(p, sm, np, w); ++np) {
    const int ob = (w.T + w.n) / kBlock, steps = w.s1 - w.s0;
    const int* table = p.c.table + (long long)w.b * p.c.max_pages;
    // a block's page and place there are looked up a step before they become an address
    int pg = -1, off = 0;
    auto look_up = [&](int s) {
      const int i = s * NBLK + lane;
      pg = -1;
      if (lane < NBLK && i < w.view.n) {
        const int blk = block_at(w.view, i), at = blk / p.c.bpp;
        off = blk - at * p.c.bpp;
        if (blk != ob) pg = __ldg(table + at);  // (the open block is past the closed ones)
      }
    };
    auto address = [&]() {
      return (unsigned)pg < (unsigned)p.c.pool_pages ? code_at(p.c, pg, w.g, off, HD) : -1;
    };
    look_up(w.s0);
    long long cur = -1, nxt = -1, next2 = address();
    look_up(w.s0 + 1);
#pragma unroll 1
    for (int i = 0; i < 2 * steps && ok; ++i) {
      const bool v = is_v(i, steps);
      if (!v) {
        cur = nxt;
        nxt = next2;
        next2 = address();
        look_up(w.s0 + (i + 1) / 2 + 2);
      }
      // (K of step s is nxt; then V of step s - 1 is cur, but for the last V)
      const long long at = v && i != 2 * steps - 1 ? cur : nxt;
      const int8_t* base = v ? p.c.V : p.c.K;
#pragma unroll 1
      for (int j = 0; j < Ti::NS; ++j) {
        const bool mine = lane / SB == j && at >= 0;
        const unsigned all = __ballot_sync(0xffffffffu, mine);
        const long long before = __shfl_up_sync(0xffffffffu, at, 1);
        const bool starts = mine && (lane % SB == 0 || before < 0 || at != before + kBytes);
        const unsigned heads = __ballot_sync(0xffffffffu, starts);
        // blocks from a start to the next start or gap
        const unsigned stop = (heads | ~all) & (lane < 31 ? ~0u << (lane + 1) : 0u);
        const int n = __ffs(stop) - 1 - lane;
        if (use > 0) ok = wait_all(p, &sm.rempty[slot], (use & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          sm.odd[slot] = __popc(all) != SB;
          mbar_arrive_expect_tx(&sm.rfull[slot], __popc(all) * kBytes);
        }
        __syncwarp();
        if (starts) copy_bulk(ring + slot * Ti::kSlot + (lane % SB) * kBytes, base + at, n * kBytes, &sm.rfull[slot]);
        if (++slot == Ti::kSlots) {
          slot = 0;
          ++use;
        }
      }
    }
  }
  // the CTA must not retire while its copies are in flight: the widening warps have waited for all of them, unless
  // they gave up
  for (int i = 0; i < Ti::kSlots; ++i) {
    const uint32_t n = use + (i < slot);  // times that slot i was filled
    if (n > 0) wait_all(p, &sm.rfull[i], (n - 1) & 1);
  }
}

// The steps' scales and what is special about them (one warp; lane b the step's block b).
template <int HD, int G>
__device__ __forceinline__ void scale_role(const Params& p, Small& sm) {
  using Ti = Tile<HD>;
  constexpr int NBLK = Ti::NBLK;
  const int lane = threadIdx.x & 31;
  Piece w;
  int ks = 0;
#pragma unroll 1
  for (int np = 0; next_piece(p, sm, np, w); ++np) {
    const int end = w.T + w.n, ob = end / kBlock;  // the open block, if end % 16
    // The powers of two of the open block's rows (at its step, which this warp comes to steps before the others do).
    // Returns whether the rows are far apart; top and low take their V scales, fk and fv are those of the block.
    auto open_block = [&](Step& m, uint32_t& top, uint32_t& low, float& fk, float& fv) {
      const int row = lane / 2, rows = end % kBlock;  // half a row a lane
      const uint4* tk = reinterpret_cast<const uint4*>(p.c.tail + w.b * p.c.tail_stride +
                                                       ((long long)w.g * kBlock + row) * HD + lane % 2 * (HD / 2));
      const uint4* tv = tk + (long long)p.nkv * kBlock * HD / 8;
      // the largest finite |x| of pairs, low and high halves; others are noted
      uint32_t a = 0, b = 0, none = 0, nan = 0;
      auto take = [](uint32_t& most, uint32_t x, uint32_t& bad) {
        const uint32_t m = x & 0x7fff7fffu, is = __vcmpgtu2(m, 0x7f7f7f7fu);
        bad |= is;
        most = __vmaxu2(most, m & ~is);
      };
#pragma unroll 1
      for (int i0 = 0; i0 < HD / 16 && row < rows; i0 += 2) {
        uint4 x[2], y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x[i] = tk[i0 + i];
          y[i] = tv[i0 + i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          take(a, x[i].x, none);
          take(a, x[i].y, none);
          take(a, x[i].z, none);
          take(a, x[i].w, none);
          take(b, y[i].x, nan);
          take(b, y[i].y, nan);
          take(b, y[i].z, nan);
          take(b, y[i].w, nan);
        }
      }
      __syncwarp();
      if (nan) sm.open_nan = 1;
      a = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));  // K's in the low half, V's in the high one
      a = __vmaxu2(a, __shfl_xor_sync(0xffffffffu, a, 1));
      b = a >> 16;
      a &= 0xffffu;
      // extremes over the rows that are not 0
      const uint32_t hk = __reduce_max_sync(0xffffffffu, a), lk = __reduce_min_sync(0xffffffffu, a ? a : ~0u);
      const uint32_t hv = __reduce_max_sync(0xffffffffu, b), lv = __reduce_min_sync(0xffffffffu, b ? b : ~0u);
      auto factor = [](uint32_t m, int bits) { return min(bits - 1 + 127 - (int)(m >> 7), 100); };  // |bf16 m| to below 2^bits
      const bool apart = (hk && (hk >> 7) - (lk >> 7) > 8) || (hv && (hv >> 7) - (lv >> 7) > 3);
      const int ek = factor(hk, 15), rk = apart ? factor(a, 15) : ek, rv = factor(apart ? b : hv, 7);
      if (lane % 2 == 0) {
        m.uk[row] = pow2(rk);
        m.uv[row] = pow2(rv);
        m.rk[row] = ek - rk < -126 ? 0.f : pow2(ek - rk);
        m.rv[row] = b ? pow2(-rv) : 0.f;
      }
      fk = pow2(-ek);
      fv = hv && !apart ? pow2(-rv) : 0.f;
      if (hv) {
        top = max(top, __float_as_uint(pow2(-factor(hv, 7))));
        low = min(low, __float_as_uint(pow2(-factor(apart ? lv : hv, 7))));
      }
      return apart;
    };
    const int* table = p.c.table + (long long)w.b * p.c.max_pages;
#pragma unroll 1
    for (int s = w.s0; s < w.s1; ++s, ++ks) {
      int u = INT_MAX, kind = 1;
      float fk = 0.f, fv = 0.f;
      const int i = s * NBLK + lane;
      if (lane < NBLK && i < w.view.n) {
        const int blk = block_at(w.view, i), at = blk / p.c.bpp, off = blk - at * p.c.bpp;
        if (blk == ob) {
          u = blk * kBlock;
          kind = 2;
        } else {
          const int pg = __ldg(table + at);
          if ((unsigned)pg < (unsigned)p.c.pool_pages) {
            const long long sc = scale_at(p.c, pg, w.g, off);
            fk = __ldg(p.c.Ks + sc);
            fv = __ldg(p.c.Vs + sc);
            u = blk * kBlock;
            kind = 0;
          } else {
            set_guard(p.guard, kGuardBadIndex);
          }
        }
      }
      const bool full = lane >= NBLK || (u != INT_MAX && u + kBlock - 1 <= w.t0 &&
                                         (p.window <= 0 || u > w.t1 - p.window || u + kBlock <= p.sinks));
      const bool edge = !__all_sync(0xffffffffu, full);
      const int sl = ks % kSteps;
      if (ks >= kSteps && !wait_all(p, &sm.mempty[sl], ((ks / kSteps) & 1) ^ 1)) return;
      Step& m = sm.step[sl];
      uint32_t top = fv == fv ? __float_as_uint(fv) : 0u, low = fv > 0.f ? __float_as_uint(fv) : ~0u;
      // (the open block is the view's last, if the tile comes to it)
      bool apart = false;
      if (s == w.steps - 1 && end % kBlock != 0 && w.t1 / kBlock == ob) {
        float ok, ov = 0.f;
        apart = open_block(m, top, low, ok, ov);
        if (kind == 2) {
          fk = ok;
          fv = ov;
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
      low = __reduce_min_sync(0xffffffffu, low);
      const bool wide = apart || (top && (top >> 23) - (low >> 23) > 3);
      const int E = top && !wide ? (int)(top >> 23) - 126 : wide ? 14 : 0;  // 2^E above the largest
      if (lane < NBLK) {
        m.fk[lane] = fk;
        m.fv[lane] = fv * pow2(14 - E);
        m.u[lane] = u;
        m.kind[lane] = kind;
      }
      if (lane == 0) {
        m.ev = pow2(E - 14);
        m.edge = edge;
        m.wide = wide;
        m.open = apart ? w.view.n - 1 - s * NBLK : -1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.mfull[sl]);
    }
  }
}

template <int HD, int G>
__device__ __forceinline__ void widen_role(const Params& p, Small& sm, const uint8_t* ring, uint8_t* kbuf,
                                           uint8_t* vbuf) {
  using Ti = Tile<HD>;
  constexpr int BN = Ti::BN, NC = HD / 16, SB = Ti::SB;
  const int wt = threadIdx.x - kRowWarps * 32, lane = threadIdx.x & 31;
  // This thread's 16-byte pieces of a slot: piece c of rows r0, r0 + kStep, ...  A pair of rows is taken by 2 NC
  // threads so that 8 consecutive ones load from and store to eight bank groups (of two adjacent rows, one stores to
  // the even chunks of the 128 bytes, the other to the odd ones).
  const int j = wt % (2 * NC), c = j % NC, r0 = wt / (2 * NC) * 2 + ((j / NC) ^ ((c >> 2) & 1));
  constexpr int kStep = 128 / NC;  // rows from one of a thread's pieces to the next
  Piece w;
  int ks = 0, slot = 0;
  uint32_t use = 0;
#pragma unroll 1
  for (int np = 0; next_piece(p, sm, np, w); ++np) {
    const int open_rows = (w.T + w.n) % kBlock;
    const uint16_t* tail = p.c.tail + w.b * p.c.tail_stride + (long long)w.g * kBlock * HD;
    auto tile_of = [&](int v, int step) {
      constexpr int NSK = Ti::NSK, NSV = Ti::NSV;
      const int n = v ? NSV : NSK, st = step % n;
      if (step >= n && !wait_all(p, v ? &sm.vempty[st] : &sm.kempty[st], ((step / n) & 1) ^ 1)) return false;
      uint8_t* tile = (v ? vbuf : kbuf) + st * Ti::kKV;
#pragma unroll 1
      for (int i = 0; i < Ti::NS; ++i) {
        if (!wait_all(p, &sm.rfull[slot], use & 1)) return false;
        const uint8_t* raw = ring + slot * Ti::kSlot + r0 * HD + c * 16;
        const int odd = sm.odd[slot];
        uint4 x[Ti::NP];
#pragma unroll
        for (int u = 0; u < Ti::NP; ++u) x[u] = *reinterpret_cast<const uint4*>(raw + u * kStep * HD);
#pragma unroll
        for (int u = 0; u < Ti::NP; ++u) {
          uint32_t h[8];
          widen(x[u].x, h);
          widen(x[u].y, h + 2);
          widen(x[u].z, h + 4);
          widen(x[u].w, h + 6);
          put16<BN>(tile, i * (SB * kBlock) + r0 + u * kStep, c, h);
        }
        if (odd) {
          if (!wait_all(p, &sm.mfull[step % kSteps], (step / kSteps) & 1)) return false;
          const Step& m = sm.step[step % kSteps];
          const uint16_t* rows = tail + (long long)v * p.nkv * kBlock * HD + c * 16;
#pragma unroll 1
          for (int u = 0; u < Ti::NP; ++u) {
            const int r = i * (SB * kBlock) + r0 + u * kStep, kind = m.kind[r / kBlock];
            if (kind == 0) continue;
            uint4 y[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};  // rows of the tail that are there
            if (kind == 2 && r % kBlock < open_rows) {
              y[0] = reinterpret_cast<const uint4*>(rows + (r % kBlock) * HD)[0];
              y[1] = reinterpret_cast<const uint4*>(rows + (r % kBlock) * HD)[1];
            }
            const uint32_t z[8] = {y[0].x, y[0].y, y[0].z, y[0].w, y[1].x, y[1].y, y[1].z, y[1].w};
            const float up = kind == 2 ? (v ? m.uv : m.uk)[r % kBlock] : 0.f;  // (not written without an open block)
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {  // V's NaN as 0 (see the outputs)
              uint32_t q = z[k];
              if (v && (q & 0x7f80u) == 0x7f80u) q &= 0xffff0000u;
              if (v && (q & 0x7f800000u) == 0x7f800000u) q &= 0xffffu;
              h[k] = half2_bits(bf16_lo(q) * up, bf16_hi(q) * up);
            }
            put16<BN>(tile, r, c, h);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.rempty[slot]);
        if (++slot == Ti::kSlots) {
          slot = 0;
          ++use;
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v ? &sm.vfull[st] : &sm.kfull[st]);
      return true;
    };
    const int steps = w.s1 - w.s0;
#pragma unroll 1
    for (int i = 0; i < 2 * steps; ++i) {
      const int v = is_v(i, steps);
      if (!tile_of(v, ks + (v ? (i - 1) / 2 : (i + 1) / 2))) return;
    }
    ks += steps;
  }
}

// ---------------------------------------------------------------- products
template <int HD, int G>
__device__ __forceinline__ void mma_role(const Params& p, Small& sm, uint32_t q, uint32_t kbuf, uint32_t vbuf) {
  using Ti = Tile<HD>;
  constexpr int BN = Ti::BN, NSK = Ti::NSK, NSV = Ti::NSV, NO = Ti::NO;
  const uint32_t tmem = sm.tmem, out = tmem + 2 * BN;
  constexpr uint32_t id_s = idesc_f16(128, BN, false), id_o = idesc_f16(128, HD, true);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = wait_bar(bar, parity);
    if (!ok) set_guard(p.guard, kGuardWaitTimeout);
    return ok;
  };
  int ks = 0;
  bool ok = true;
#pragma unroll 1
  for (int np = 0; ok; ++np) {
    if (!(ok = wait(&sm.wfull[np % kPieces], (np / kPieces) & 1))) break;
    const Piece& w = sm.piece[np % kPieces];
    const bool more = w.b >= 0;
    const int steps = w.s1 - w.s0;
    mbar_arrive(&sm.wempty[np % kPieces]);
    if (!more) break;
    ok = wait(&sm.qfull, np & 1);
    auto scores = [&](int k) {
      const int st = k % NSK;
      if (!wait(&sm.kfull[st], (k / NSK) & 1)) return false;
      tc::fence_after_sync();
      const uint32_t d = tmem + (k & 1) * BN;
      uint64_t a0 = tc::sdesc_k128(q), a1 = tc::sdesc_k128(q + Ti::kQ), b = tc::sdesc_k128(kbuf + st * Ti::kKV);
#pragma unroll 1
      for (int c = 0; c < HD / 64; ++c) {  // (addresses in 16-byte units; they stay below the field's 2^14)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          tc::mma_bf16(d, a0 + k * 2, b + k * 2, id_s, c + k > 0);
          tc::mma_bf16(d, a1 + k * 2, b + k * 2, id_s, true);
        }
        a0 += 128 * 128 / 16;
        a1 += 128 * 128 / 16;
        b += BN * 128 / 16;
      }
      tc::mma_commit(&sm.kempty[st]);
      tc::mma_commit(&sm.sfull[k & 1]);
      // the step's scales too: their warp's writes, passed on by an arrival of this thread's
      if (!wait(&sm.mfull[k % kSteps], (k / kSteps) & 1)) return false;
      mbar_arrive(&sm.sfull[k & 1]);
      return true;
    };
    if (ok) ok = scores(ks);
    for (int s = 0; ok && s < steps; ++s, ++ks) {
      if (s + 1 < steps && !(ok = scores(ks + 1))) break;
      const int st = ks % NSV, ob = ks % NO;
      ok = wait(&sm.pfull[ks & 1], (ks >> 1) & 1) && wait(&sm.vfull[st], (ks / NSV) & 1) &&
           (ks < NO || wait(&sm.oempty[ob], ((ks / NO) - 1) & 1));
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t d = out + ob * HD, a = tmem + (ks & 1) * BN;
      uint64_t b = sdesc_mn128(vbuf + st * Ti::kKV, BN * 128);
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        mma_ts(d, a + c * 32, b, id_o, c > 0);
        mma_ts(d, a + c * 32 + 8, b, id_o, true);
        mma_ts(d, a + c * 32 + 16, b + 2048 / 16, id_o, true);
        mma_ts(d, a + c * 32 + 24, b + 2048 / 16, id_o, true);
        b += 4096 / 16;
      }
      tc::mma_commit(&sm.vempty[st]);
      tc::mma_commit(&sm.ofull[ob]);
      mbar_arrive(&sm.mempty[ks % kSteps]);  // the row warps have weighted the step, V is widened: its scales are read
    }
  }
  // every issued MMA has completed before TMEM is released
  tc::mma_commit(&sm.done);
  wait(&sm.done, 0);
}

// ---------------------------------------------------------------- rows
__device__ __forceinline__ uint32_t low_mask(int n) { return n <= 0 ? 0u : n >= 16 ? 0xffffu : (1u << n) - 1; }

template <int HD>
__host__ __device__ constexpr int part_floats_of() { return 128 * HD + 256; }  // outputs, maxima, sums

template <int HD, int G>
__device__ __forceinline__ void row_role(const Params& p, Small& sm, uint8_t* q, float* part) {
  using Ti = Tile<HD>;
  constexpr int BN = Ti::BN, NO = Ti::NO, NV = BN / 2, NA = HD / 2;  // scores and outputs of a thread
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp & 3, half = warp >> 2, row = sub * 32 + lane;
  const uint32_t lanes = (uint32_t)(sub * 32) << 16;
  const uint32_t scores = sm.tmem + lanes + half * NV, outs = sm.tmem + lanes + 2 * BN + half * NA;
  Piece w;
  int ks = 0;
  bool ok = true;
#pragma unroll 1
  for (int np = 0;; ++np) {
    // (the row warps meet at barriers: all of them go on, or none)
    if (named_barrier_or(9, kRowWarps * 32, !next_piece(p, sm, np, w))) break;
    // ------------------------------------------------ queries: warp `warp` rows 16 warp ..
    // normalised by 2^e with 2^e max |q| in [2^9, 2^10): as two fp16 parts q keeps 22 bits of the row's largest
    // (8 lanes a row, 4 rows at a time)
    constexpr int PP = HD / 16;  // rotate-half pairs of a lane
    const int l8 = lane & 7;
#pragma unroll 2
    for (int m = warp * 16 + (lane >> 3); m < warp * 16 + 16; m += 4) {
      const int i = min(m / G, w.rows - 1);  // (rows past the tile's read its last one)
      const float* y = p.y + (w.first + i) * p.ld_y + (long long)(w.g * G + m % G) * HD + l8;
      const float2* rope = p.rope + (long long)(w.t0 + i) * (HD / 2) + l8;
      float x[PP][2];
      uint32_t a = 0;
#pragma unroll
      for (int u = 0; u < PP; ++u) {
        rotate(__ldg(y + u * 8), __ldg(y + u * 8 + HD / 2), __ldg(rope + u * 8), &x[u][0], &x[u][1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[u][h] *= p.scale_log2e;
          a = max(a, __float_as_uint(x[u][h]) & 0x7fffffffu);
        }
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
      const int e = min(max(9 + 127 - (int)(a >> 23), -103), 100);
      const float up = pow2(e);
      if (l8 == 0) sm.qf[m] = pow2(-e);
      uint8_t* at = q + m * 128 + l8 * 2;
#pragma unroll
      for (int u = 0; u < PP; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // element 8 c + l8
          const int c = u + h * (HD / 16);
          const float v = x[u][h] * up;
          const __half hi = __float2half_rn(v), lo = __float2half_rn(v - __half2float(hi));
          uint8_t* d = at + (c >> 3) * (128 * 128) + (((c ^ m) & 7) << 4);
          *reinterpret_cast<__half*>(d) = hi;
          *reinterpret_cast<__half*>(d + Ti::kQ) = lo;
        }
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.qfull);
    // the queries' factors are another warp's: wait for the other row warps
    named_barrier(9, kRowWarps * 32);
    const float qf = sm.qf[row];
    const int t = w.t0 + min(row / G, w.rows - 1);

    uint64_t acc[NA / 2];
#pragma unroll
    for (int i = 0; i < NA / 2; ++i) acc[i] = 0;
    float mx = -INFINITY, lsum = 0.f, corr = 1.f, ev = 0.f;
    // the outputs of step k, under the reference that corr moved the running ones to
    auto gather = [&](int k, float cf, float ef) {
      const int ob = k % NO;
      wait_row(p, &sm.ofull[ob], (k / NO) & 1, ok);
      tc::fence_after_sync();
      const bool moved = __any_sync(0xffffffffu, cf != 1.f);
      const uint64_t c2 = pack2(cf, cf), e2 = pack2(ef, ef);
#pragma unroll
      for (int c = 0; c < NA; c += 32) {
        float v[32];
        tc::tmem_ld32(outs + ob * HD + c, v);
        if (moved) {
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[c / 2 + i] = mul2(acc[c / 2 + i], c2);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c / 2 + i] = fma2(pack2(v[2 * i], v[2 * i + 1]), e2, acc[c / 2 + i]);
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.oempty[ob]);
    };
    // step s, then the outputs of the step before it
#pragma unroll 1
    for (int s = w.s0;; ++s, ++ks) {
      float cf = 1.f, step_ev = 0.f;
      if (s < w.s1) {
        const int buf = ks & 1;
        wait_row(p, &sm.sfull[buf], (ks >> 1) & 1, ok);
        tc::fence_after_sync();
        const Step& m = sm.step[ks % kSteps];
        const int j0 = half * (NV / 16);  // the thread's first block
        const int edge = m.edge;
        // A block's factors.  In a step that some row does not see all of, a scale of 0 or NaN goes into the scores,
        // so that it does not meet the -infinity of the positions out of view (a NaN block makes all of a row's
        // outputs NaN, whether it is K's or V's).
        auto factors = [&](int j, float& f, float& fv) {
          f = m.fk[j0 + j] * qf;
          fv = m.fv[j0 + j];
          const float z = f * 0.f + fv * 0.f;  // 0, or NaN
          if (edge && z != z) fv = 0.f;
          if (edge && !(z == z && f != 0.f)) {
            f = 1.f;
            return z;
          }
          return 1.f;
        };
        // the maximum, 32 scores at a time (loops, not unrolled over the step: the roles share the instruction cache);
        // what is out of view goes back as -infinity
        float top = -INFINITY;
        if ((unsigned)(m.open - j0) < NV / 16) {  // rows with scales of their own
          float v[16];
          uint32_t w[16];
          tmem_ld16(scores + buf * BN + (m.open - j0) * 16, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i] * m.rk[i]);
          tmem_st16(scores + buf * BN + (m.open - j0) * 16, w);
          wait_st();
        }
#pragma unroll 1
        for (int c = 0; c < NV; c += 32) {
          float v[32];
          tc::tmem_ld32(scores + buf * BN + c, v);
          float f[2], fv[2];
          const float z0 = factors(c / 16, f[0], fv[0]), z1 = factors(c / 16 + 1, f[1], fv[1]);
          if (edge) {
            uint32_t bits = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int u = m.u[j0 + c / 16 + h];
              uint32_t see = 0;
              if (u != INT_MAX) {
                see = low_mask(t - u + 1);
                if (p.window > 0) see &= ~low_mask(t - p.window - u + 1) | low_mask(p.sinks - u);
              }
              bits |= see << (16 * h);
            }
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float z = i < 16 ? z0 : z1;
              if (z != 1.f) v[i] = z;
              if (!(bits >> i & 1)) v[i] = -INFINITY;
              w[i] = __float_as_uint(v[i]);
            }
            tmem_st32(scores + buf * BN + c, w);
            wait_st();
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float b = v[h * 16];
#pragma unroll
            for (int i = 1; i < 16; ++i) b = fmaxf(b, v[h * 16 + i]);
            top = fmaxf(top, b * f[h]);
          }
        }
        sm.mx[buf][half][row] = top;
        const bool wide = named_barrier_or(1 + sub, 64, m.wide != 0);  // (the same for both halves, whatever m holds)
        top = fmaxf(top, sm.mx[buf][half ^ 1][row]);
        const float mn = fmaxf(mx, top), ref = mn == -INFINITY ? 0.f : mn;
        cf = mx == mn ? 1.f : ex2(mx - mn);
        mx = mn;
        // weights, their sum and their two parts
        uint64_t sum2 = 0;
        const uint64_t nref = pack2(-ref, -ref), minus1 = pack2(-1.f, -1.f);
        // From about 2^25 on a score's rounding in the maximum is worth factors of 2, and an unrounded product less the
        // maximum gives weights above 1 that no longer fit fp16: there, and in wide steps, each product is rounded as the
        // maximum was.  (A loop of its own: a choice within the other one costs 2048 rows of 4 x 128 3%; all steps wide
        // take them 242 us instead of 199.)
        step_ev = m.ev;
        if (wide || __any_sync(0xffffffffu, fabsf(ref) >= 1048576.f)) {
          const int open = m.open - j0;  // the block whose rows have scales of their own, if it is among the thread's
          float up = 1.f;                // 2^(14 - E) of a row in a wide step
          if (wide) {
            float g = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < NV; c += 16) {
              float v[16], f, fv;
              tmem_ld16(scores + buf * BN + c, v);
              factors(c / 16, f, fv);
              if (c / 16 == open) {
#pragma unroll
                for (int i = 0; i < 16; ++i) g = fmaxf(g, __fsub_rn(__fmul_rn(v[i], f), ref) + log2_above(m.rv[i]));
              } else {
                float b = v[0];
#pragma unroll
                for (int i = 1; i < 16; ++i) b = fmaxf(b, v[i]);
                g = fmaxf(g, __fsub_rn(__fmul_rn(b, f), ref) + log2_above(fv));
              }
            }
            sm.top[half][row] = g;
            named_barrier(1 + sub, 64);
            const int e = (int)ceilf(fmaxf(fmaxf(g, sm.top[half ^ 1][row]), -110.f));
            up = pow2(14 - e);
            step_ev = pow2(e - 14);
          }
#pragma unroll 1
          for (int c = 0; c < NV; c += 16) {
            float v[16], f, fv;
            tmem_ld16(scores + buf * BN + c, v);
            factors(c / 16, f, fv);
            // (bounded for blocks out of view, whose weights are 0; in view what it bounds has weights below 2^-86)
            auto bounded = [](float x) { return x > 0x1p100f ? 0x1p100f : x; };  // NaN stays
            fv = bounded(fv * up);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = ex2(__fsub_rn(__fmul_rn(v[i], f), ref));  // (a packed pair is contracted)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum2 = add2(sum2, pack2(v[2 * i], v[2 * i + 1]));
            if (c / 16 == open) {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] *= bounded(m.rv[i] * up);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) unpack2(mul2(pack2(v[2 * i], v[2 * i + 1]), pack2(fv, fv)), v[2 * i], v[2 * i + 1]);
            }
            uint32_t pr[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float h0 = trunc11(v[2 * i]), h1 = trunc11(v[2 * i + 1]);
              pr[i] = half2_bits(h0, h1);
              pr[8 + i] = half2_bits(v[2 * i] - h0, v[2 * i + 1] - h1);
            }
            tmem_st16(scores + buf * BN + c, pr);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < NV; c += 16) {  // a block's 16 scores become 8 columns of high and 8 of low parts
            float v[16], f, fv;
            tmem_ld16(scores + buf * BN + c, v);
            factors(c / 16, f, fv);
            const uint64_t f2 = pack2(f, f), fv2 = pack2(fv, fv);
            uint32_t pr[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float p0, p1, w0, w1, l0, l1;
              unpack2(fma2(pack2(v[2 * i], v[2 * i + 1]), f2, nref), p0, p1);
              const uint64_t pp = pack2(ex2(p0), ex2(p1));
              sum2 = add2(sum2, pp);
              unpack2(mul2(pp, fv2), w0, w1);
              const float h0 = trunc11(w0), h1 = trunc11(w1);
              unpack2(fma2(pack2(h0, h1), minus1, pack2(w0, w1)), l0, l1);  // w - h, exact
              pr[i] = half2_bits(h0, h1);
              pr[8 + i] = half2_bits(l0, l1);
            }
            tmem_st16(scores + buf * BN + c, pr);
          }
        }
        wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pfull[buf]);
        float s0, s1;
        unpack2(sum2, s0, s1);
        lsum = fmaf(lsum, cf, s0 + s1);
      }
      if (s > w.s0) gather(ks - 1, corr, ev);
      if (s == w.s1) break;
      corr = cf;
      ev = step_ev;
    }

    // ------------------------------------------------ outputs
    sm.ls[half][row] = lsum;
    named_barrier(1 + sub, 64);
    const float l = lsum + sm.ls[half ^ 1][row];
    float* o = nullptr;
    float inv = 1.f;
    const bool whole = w.s0 == 0 && w.s1 == w.steps, live = row < w.rows * G;
    if (whole) {
      inv = l == 0.f ? 0.f : 1.0f / l;
      o = p.o + (w.first + row / G) * p.ld_o + (long long)(w.g * G + row % G) * HD + half * NA;
    } else {
      // a tile that begins here leaves the CTA's second partial, one that goes on its first
      float* d = part + (2ll * blockIdx.x + (w.s0 == 0)) * part_floats_of<HD>();
      o = d + row * HD + half * NA;
      if (half == 0) {
        d[128 * HD + row] = mx;
        d[128 * HD + 128 + row] = l;
      }
    }
    // an open row's NaN in V: in the outputs of the rows that see it
    const int end = w.T + w.n, ob = end / kBlock;
    uint32_t see = 0;
    if (sm.open_nan && w.s1 == w.steps && w.t1 / kBlock == ob) {
      see = low_mask(t - ob * kBlock + 1);
      if (p.window > 0) see &= ~low_mask(t - p.window - ob * kBlock + 1) | low_mask(p.sinks - ob * kBlock);
    }
    const uint16_t* tv = p.c.tail + w.b * p.c.tail_stride + ((long long)p.nkv + w.g) * kBlock * HD + half * NA;
    if (live) {
      const bool vec = ((reinterpret_cast<uintptr_t>(o) & 15) == 0);
#pragma unroll
      for (int i = 0; i < NA / 4; ++i) {
        float r[4];
        unpack2(acc[2 * i], r[0], r[1]);
        unpack2(acc[2 * i + 1], r[2], r[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] *= inv;
        if (vec) {
          reinterpret_cast<float4*>(o)[i] = make_float4(r[0], r[1], r[2], r[3]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i * 4 + k] = r[k];
        }
      }
#pragma unroll 1
      for (int m = 0; see >> m; ++m)
#pragma unroll 1
        for (int i = 0; i < NA; ++i)
          if ((see >> m & 1) && (tv[m * HD + i] & 0x7f80u) == 0x7f80u) o[i] = __uint_as_float(0x7fc00000u);
    }
  }
}

template <int HD, int G>
__global__ void __launch_bounds__(kThreads, 1) k_prompt(const __grid_constant__ Params p) {
  using Ti = Tile<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Small& sm = *reinterpret_cast<Small*>(smem + Ti::kSmem);
  Share* share = reinterpret_cast<Share*>(p.part);
  float* part = p.part + 2048;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.kfull[s], kWidenWarps);
      mbar_init(&sm.vfull[s], kWidenWarps);
      mbar_init(&sm.kempty[s], 1);
      mbar_init(&sm.vempty[s], 1);
      mbar_init(&sm.sfull[s], 2);
      mbar_init(&sm.pfull[s], kRowWarps);
      mbar_init(&sm.ofull[s], 1);
      mbar_init(&sm.oempty[s], kRowWarps);
    }
    for (int s = 0; s < kSteps; ++s) {
      mbar_init(&sm.mfull[s], 1);
      mbar_init(&sm.mempty[s], 1);
    }
    for (int s = 0; s < Ti::kSlots; ++s) {
      mbar_init(&sm.rfull[s], 1);
      mbar_init(&sm.rempty[s], kWidenWarps);
    }
    for (int s = 0; s < kPieces; ++s) {
      mbar_init(&sm.wfull[s], 1);
      mbar_init(&sm.wempty[s], kPieceReaders);
    }
    mbar_init(&sm.qfull, kRowWarps);
    mbar_init(&sm.done, 1);
    sm.open_nan = 0;
    fence_mbar_init();
  }
  plan_work<HD, G>(p, sm, share);
  pdl_launch_dependents();         // (the join waits for all of this kernel)
  if (sm.begin >= sm.end) return;  // the whole CTA
  if (warp == kRowWarps + kWidenWarps) tc::tmem_alloc(&sm.tmem, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  uint8_t *q = smem, *kbuf = smem + 2 * Ti::kQ, *vbuf = kbuf + Ti::NSK * Ti::kKV, *ring = vbuf + Ti::NSV * Ti::kKV;
  if (warp < kRowWarps) {
    regs_inc<kRowRegs>();
    row_role<HD, G>(p, sm, q, part);
  } else if (warp < kRowWarps + kWidenWarps) {
    regs_dec<kWidenRegs>();
    widen_role<HD, G>(p, sm, ring, kbuf, vbuf);
  } else {
    regs_dec<kOtherRegs>();
    if (warp == kRowWarps + kWidenWarps && (threadIdx.x & 31) == 0)
      mma_role<HD, G>(p, sm, smem_addr(q), smem_addr(kbuf), smem_addr(vbuf));
    if (warp == kRowWarps + kWidenWarps + 1) load_role<HD, G>(p, sm, ring);
    if (warp == kRowWarps + kWidenWarps + 2) scale_role<HD, G>(p, sm);
    if (warp == kRowWarps + kWidenWarps + 3) piece_role<HD, G>(p, sm);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kRowWarps + kWidenWarps) {
    tc::fence_after_sync();
    tc::tmem_dealloc(sm.tmem, 512);
  }
}

// The tile that CTA blockIdx.x + 1 found begun, if it is the second of its sharers: their partials joined, 16 rows a
// block, a warp per row.
template <int HD, int G>
__global__ void __launch_bounds__(256) k_join(const __grid_constant__ Params p) {
  const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const Share s = reinterpret_cast<const Share*>(p.part)[c];
  if (!s.joins) return;
  const float* part = p.part + 2048;
  const int first = p.row_start[s.b], n = p.row_start[s.b + 1] - first;
  auto part_of = [&](int k) { return part + (2ll * k + (k == s.lo)) * part_floats_of<HD>(); };
  for (int row = blockIdx.y * 16 + warp; row < blockIdx.y * 16 + 16; row += 8) {
    const int i = s.i0 + row / G;
    if (i >= n) return;
    float R = -INFINITY, den = 0.f;
    for (int k = s.lo + lane; k <= s.hi; k += 32) R = fmaxf(R, part_of(k)[128 * HD + row]);
    R = warp_max(R);
    float a[HD / 32];
#pragma unroll
    for (int d = 0; d < HD / 32; ++d) a[d] = 0.f;
    for (int k = s.lo; k <= s.hi; ++k) {
      const float* q = part_of(k);
      const float r = q[128 * HD + row], f = R == -INFINITY ? (r == r ? 1.f : r) : ex2(r - R);
      den = fmaf(f, q[128 * HD + 128 + row], den);
#pragma unroll
      for (int d = 0; d < HD / 32; ++d) a[d] = fmaf(f, q[row * HD + d * 32 + lane], a[d]);
    }
    const float inv = den == 0.f ? 0.f : 1.0f / den;
    float* o = p.o + (first + i) * p.ld_o + (long long)(s.g * G + row % G) * HD;
#pragma unroll
    for (int d = 0; d < HD / 32; ++d) o[d * 32 + lane] = a[d] * inv;
  }
}

struct Pick {
  void (*k)(Params);
  void (*join)(Params);
  size_t smem, part;
};
template <int HD>
Pick pick_g(int G) {
  const size_t smem = Tile<HD>::kSmem + 1024 + sizeof(Small), part = part_floats_of<HD>();
  switch (G) {
    case 1: return {k_prompt<HD, 1>, k_join<HD, 1>, smem, part};
    case 2: return {k_prompt<HD, 2>, k_join<HD, 2>, smem, part};
    case 4: return {k_prompt<HD, 4>, k_join<HD, 4>, smem, part};
    case 8: return {k_prompt<HD, 8>, k_join<HD, 8>, smem, part};
  }
  return {};
}
Pick pick(int hd, int G) {
  return hd == 64 ? pick_g<64>(G) : hd == 128 ? pick_g<128>(G) : hd == 256 ? pick_g<256>(G) : Pick{};
}

}  // namespace

// shares of at most 256 CTAs, then two partials of each
size_t prompt_workspace(int, int, int nq, int nkv, int hd, int nsm) {
  const int C = nsm < kPromptCtas ? nsm : kPromptCtas;
  return 8192 + 2 * (size_t)C * pick(hd, nq / nkv).part * 4;
}

cudaError_t init_prompt() {
  for (int hd : {64, 128, 256})
    for (int G : {1, 2, 4, 8}) {
      const Pick k = pick(hd, G);
      const cudaError_t e =
          cudaFuncSetAttribute((const void*)k.k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem);
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

cudaError_t prompt(const Params& p, int hd, int nsm, cudaStream_t st) {
  const Pick k = pick(hd, p.nq / p.nkv);
  if (!k.k || p.nb < 1 || p.nb > kMaxB) return cudaErrorInvalidValue;
  const int C = nsm < kPromptCtas ? nsm : kPromptCtas;
  cudaError_t e = launch_k(k.k, dim3(C), dim3(kThreads), k.smem, st, false, p);
  if (e != cudaSuccess || C < 2) return e;
  return launch_k(k.join, dim3(C - 1, 8), dim3(256), 0, st, true, p);
}

}  // namespace p8
}  // namespace hy
