// The paged 8-bit KV cache on sm_103a: the append of rows of many sequences
// and the decode attention (format: p8_dev.cuh).
//
// Attention.  For kv head g with its G = nq / nkv query heads and the rows t in
// view of the sequence's new position,
//   s_jt = sK[t / 16] (q_j . cK[t]),   p_jt = softmax_t(s_jt),
//   o_j = sum over blocks of sV[block] sum_{t in block} p_jt cV[t],
// so both products run on the tensor cores on the codes, which fp16 holds
// exactly, and a block's two scales stay FP32 factors outside: of its 16
// scores, and of its product with V as that is added to the running outputs.
// q and p are split into two fp16 parts (22 bits), which fill the 8 columns of
// an MMA (high and low parts of up to 4 heads) or make it two (8 heads).  A
// batch of single queries against a cache that is read once fills 8 of the 128
// rows of a tcgen05 tile and would still need the codes widened into shared
// memory, so this uses mma.sync, whose operands are widened in registers.
//
// The open block (bf16 rows of the tail and the new row) is the last tile of
// its head.  Scaled by a power of two its values are fp16 numbers exactly (below
// 2^-28 of the block's largest they lose bits), so it takes the same products;
// if the new row closes it, it is quantised and used by its codes.
//
// Work split: the blocks in view of every (sequence, kv head) are tiles; in a
// CTA each warp takes every W-th tile of the CTA's range through its own
// cp.async ring with its own running maximum, sum and outputs (no block
// barrier inside a range).  A CTA gets one range of at most m tiles of one
// (sequence, head), m the least for which the CTAs suffice; where that leaves
// much more than an equal share, all tiles form one list and every CTA takes an
// equal span of it, its ends moved to a nearby border between heads.  A
// (sequence, head) that several CTAs share is joined from their partials
//   R = max_i r_i,  o = sum_i 2^(r_i - R) o_i / sum_i 2^(r_i - R) l_i
// without any CTA waiting: the last of each 24 sharers to arrive joins the 24,
// and the last of those joins the rest.
//
// Measured (4 kv heads x 128, 16 query heads): 8 sequences of 120k-131k rows in
// 170 to 180 us, 5.7 to 6.05 TB/s of a measured copy's 6.8, with 63% of the issue
// slots taken (widening: 5 operations for 4 codes); one of 4096 rows in 11.5 us,
// a chain of latencies.  Registers spill: at head dim 256 (255 of them) 172 to
// 200 bytes, 424 with 8 heads a kv head; at 128 (128, for two CTAs an SM) 136 to
// 164; at 64 16 to 24.
#include "p8_dev.cuh"

namespace hy {
namespace p8 {
namespace {

// ------------------------------------------------------------ append
// A warp (hd 256: two) per block, kv head and K or V: its rows in registers as
// bf16 pairs (4 + 4 adjacent values, the rotate-half partners, in a lane), from
// the tail where they are old; one pass, the block's maximum by one reduction.
// Bound by its bytes.  Small CTAs in one wave: 4 x 2048 rows of 4 x 128 in 13.9
// us (5.7 TB/s), 17.5 in CTAs of 8 warps with 80 registers, which make 1.1.
// VEC: y, the table and kv_new are 16-byte aligned with rows of whole 16 bytes.
template <bool VEC>
__device__ __forceinline__ float4 load4(const float* p) {
  return VEC ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], p[1], p[2], p[3]);
}
template <bool VEC>
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  if (VEC) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
  } else {
    p[0] = a;
    p[1] = b;
    p[2] = c;
    p[3] = d;
  }
}

constexpr int kAppendWarps = 4;  // of a CTA
template <int HD, bool VEC>
__global__ void __launch_bounds__(kAppendWarps * 32, 8) k_append(const __grid_constant__ Params p) {
  constexpr int SP = HD == 256 ? 2 : 1;                             // warps of a unit, each a part of the rows
  constexpr int LV = HD / 8, RP = 32 / LV, NP = kBlock / RP / SP;   // lanes of a row, rows of a pass, passes
  __shared__ int at[kMaxB + 1], T0[kMaxB], first[kMaxB], rows[kMaxB];
  __shared__ uint32_t top[2][kAppendWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    int base = 0;
    for (int b0 = 0; b0 < p.nb; b0 += 32) {
      const int b = b0 + lane;
      int incl = 0;
      if (b < p.nb) {
        const int T = p.len[b], s = p.row_start[b], e = p.row_start[b + 1];
        const bool ok = T >= 0 && s >= 0 && e >= s && e <= p.n &&
                        (long long)T + (e - s) <= (long long)p.c.max_pages * p.c.page_tokens;
        if (!ok && blockIdx.x == 0) set_guard(p.guard, kGuardBadPosition);
        if (ok && e > s) {
          const int j0 = T / kBlock, j1 = (T + (e - s)) / kBlock;  // the first block; the open one after the call
          incl = (T + (e - s) - 1) / kBlock - j0 + 1;
          if (T % kBlock != 0 && j1 > j0 && (T + (e - s)) % kBlock != 0) --incl;
        }
        T0[b] = T;
        first[b] = s;
        rows[b] = e - s;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (b < p.nb) at[b + 1] = base + incl;
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) at[0] = 0;
  }
  __syncthreads();
  const int heads = 2 * p.nkv;
  const long long total = (long long)at[p.nb] * heads;
  const int sub = lane / LV, e = (lane % LV) * 4;  // row of a pass; the lane's first element, of the first half
  const int row_off = warp % SP * (kBlock / SP);
  int turn = 0;
  for (long long unit = blockIdx.x * (long long)(kAppendWarps / SP) + warp / SP; unit < total;
       unit += gridDim.x * (long long)(kAppendWarps / SP)) {
    const int bi = (int)(unit / heads), kg = (int)(unit % heads);
    int b = 0;
    for (int step = kMaxB / 2; step > 0; step >>= 1)  // the last b with at[b] <= bi that has blocks
      if (b + step < p.nb && at[b + step] <= bi) b += step;
    const int T = T0[b], n = rows[b], open = (T + n) / kBlock;
    // The first block reads the tail if it has old rows, and the open block writes it: then one warp takes both,
    // in that order (a lane reads and writes the same elements).
    const bool both = bi == at[b] && T % kBlock != 0 && open > T / kBlock && (T + n) % kBlock != 0;
    for (int j = T / kBlock + bi - at[b], more = both; j >= 0; j = more ? open : -1, more = 0) {
      const int lo = max(T - j * kBlock, 0), hi = min(T + n - j * kBlock, kBlock);  // the new rows of the block
      const bool closes = j * kBlock + kBlock <= T + n;
      const int kv = kg >= p.nkv, g = kv ? kg - p.nkv : kg;
      const long long row0 = first[b] + (j * kBlock - T);  // row of y of the block's row 0 (may be before the first)
      const float* y0 = p.y + (long long)(p.nq + kg) * HD + e;
      const float* rope0 = reinterpret_cast<const float*>(p.rope) + ((long long)j * kBlock * (HD / 2) + e) * 2;
      uint16_t* tail = p.c.tail + b * p.c.tail_stride + ((long long)kv * p.nkv + g) * kBlock * HD + e;
      uint32_t v[NP][4];
      uint32_t a = 0;
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int r = row_off + k * RP + sub;
        const int rc = min(max(r, lo), hi - 1);  // (a lane without a new row reads one all the same)
        const float* yr = y0 + (row0 + rc) * p.ld_y;
        const float4 x0 = load4<VEC>(yr), x1 = load4<VEC>(yr + HD / 2);
        float f0[4] = {x0.x, x0.y, x0.z, x0.w}, f1[4] = {x1.x, x1.y, x1.z, x1.w};
        if (!kv) {
          const float4 c0 = load4<VEC>(rope0 + rc * HD), c1 = load4<VEC>(rope0 + rc * HD + 4);
          rotate(f0[0], f1[0], make_float2(c0.x, c0.y), &f0[0], &f1[0]);
          rotate(f0[1], f1[1], make_float2(c0.z, c0.w), &f0[1], &f1[1]);
          rotate(f0[2], f1[2], make_float2(c1.x, c1.y), &f0[2], &f1[2]);
          rotate(f0[3], f1[3], make_float2(c1.z, c1.w), &f0[3], &f1[3]);
        }
        v[k][0] = store_pair(f0[0], f0[1]);
        v[k][1] = store_pair(f0[2], f0[3]);
        v[k][2] = store_pair(f1[0], f1[1]);
        v[k][3] = store_pair(f1[2], f1[3]);
      }
      if (lo > 0 && closes) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const int r = row_off + k * RP + sub;
          if (r < lo) {
            const uint2 t0 = *reinterpret_cast<const uint2*>(tail + r * HD);
            const uint2 t1 = *reinterpret_cast<const uint2*>(tail + r * HD + HD / 2);
            v[k][0] = t0.x;
            v[k][1] = t0.y;
            v[k][2] = t1.x;
            v[k][3] = t1.y;
          }
        }
      }
      float s = 1.f, inv = 0.f;
      int8_t* codes = nullptr;
      if (closes) {
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) a = abs_max(a, v[k][i]);
        a = __reduce_max_sync(0xffffffffu, a);
        if (SP > 1) {  // (the warps of a unit go the same way; two turns' places, so that one barrier a turn does)
          if (lane == 0) top[turn][warp] = a;
          named_barrier(1 + warp / SP, 32 * SP);
          a = max(a, top[turn][warp ^ 1]);
          turn ^= 1;
        }
        s = block_scale(a, &inv);
        const int pg = page_of(p.c, b, j);
        if (pg < 0) {
          if (lane == 0) set_guard(p.guard, kGuardBadIndex);
        } else {
          codes = (kv ? p.c.V : p.c.K) + code_at(p.c, pg, g, j % p.c.bpp, HD) + e;
          if (lane == 0) (kv ? p.c.Vs : p.c.Ks)[scale_at(p.c, pg, g, j % p.c.bpp)] = s;
        }
      }
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int r = row_off + k * RP + sub;
        float val[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          val[2 * i] = bf16_lo(v[k][i]);
          val[2 * i + 1] = bf16_hi(v[k][i]);
        }
        if (closes) {
          uint32_t w[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = block_code(val[i], inv);
            w[i / 4] |= (uint32_t)(c & 255) << (8 * (i & 3));
            val[i] = __fmul_rn(s, (float)c);
          }
          if (codes) {
            *reinterpret_cast<uint32_t*>(codes + r * HD) = w[0];
            *reinterpret_cast<uint32_t*>(codes + r * HD + HD / 2) = w[1];
          }
        } else if (r >= lo && r < hi) {
          *reinterpret_cast<uint2*>(tail + r * HD) = make_uint2(v[k][0], v[k][1]);
          *reinterpret_cast<uint2*>(tail + r * HD + HD / 2) = make_uint2(v[k][2], v[k][3]);
        }
        if (p.kv_new && r >= lo && r < hi) {
          float* d = p.kv_new + ((row0 + r) * 2 * p.nkv + kg) * HD + e;
          store4<VEC>(d, val[0], val[1], val[2], val[3]);
          store4<VEC>(d + HD / 2, val[4], val[5], val[6], val[7]);
        }
      }
    }
  }
}

// ------------------------------------------------------------ attention
// Per head dim: warps of a CTA, CTAs per SM, and the stages of a warp's ring.
template <int HD>
struct Shape {
  static constexpr int W = 8;
  static constexpr int kThreads = W * 32;
  static constexpr int kCtas = HD == 256 ? 1 : 2;   // per SM
  static constexpr int S = HD == 64 ? 4 : 3;
  static constexpr int NC = HD / 16;                // 16-byte pieces of a row
  static constexpr int kTile = kBlock * HD;         // bytes of a block's K or V codes
  static constexpr int kStage = 2 * kTile;
  static constexpr int kWarpRing = S * kStage;
  static constexpr int kRing = W * kWarpRing;
  static constexpr int kQ = NC * 2 * 32 * 8;        // query operand fragments (two of them for 8 heads)
  static constexpr int kOpen = 2 * kBlock * HD * 2; // the open block's K and V as fp16 (or its codes)
};

struct alignas(16) Small {
  uint32_t amax[8][8];             // per head and pair of 16-element halves: largest |q| (bits)
  float qf[8];                     // per head: 2^-e of the query normalisation
  float r[8][8], l[8][8];          // per warp and head
  float os[2];                     // the open block's scales of K and V
  int last;
  // the work
  int at[kMaxB + 1];               // first unit of each sequence: tiles (spans) or ranges
  int per[kMaxB];                  // units of one of its heads
  int T[kMaxB];                    // positions of the new rows (-1: refused)
  int m;                           // most tiles of a range; 0: spans
  int q, rem, near;
  int unit, unit_end;              // this CTA's units
  int b, g, tile0, ntile, next;    // the item and this CTA's range of it
  int c_lo, np, slot0;             // the CTAs that share the item
};

template <int HD>
constexpr size_t smem_bytes() {
  return (size_t)Shape<HD>::kRing + Shape<HD>::kQ + Shape<HD>::kOpen + sizeof(Small);
}

constexpr int kJoin = 24;       // partials joined at a time
constexpr int kCounters = 32;   // of a (sequence, kv head): the last join's, then one per kJoin sharers
// floats of a partial: outputs [G][HD], references [G], sums [G], in 16-byte pieces
__host__ __device__ constexpr int part_size(int G, int HD) { return (G * (HD + 2) + 3) / 4 * 4; }
// floats of a head's outputs in shared memory: padded, so that a quad's heads fall in different banks
__host__ __device__ constexpr int out_pitch(int HD) { return HD + 8; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
// v truncated to fp16's 11 significant bits: v - trunc11(v) is exact
__device__ __forceinline__ float trunc11(float v) { return __uint_as_float(__float_as_uint(v) & 0xffffe000u); }

// The codes of a word's bytes as fp16 pairs: bytes A and B of the word, biased
// to c + 128, under the exponent of 1024, less 1152; exact.
template <int A, int B>
__device__ __forceinline__ uint32_t widen(uint32_t biased) {
  const uint32_t p = __byte_perm(biased, 0x64646464u, A | 4 << 4 | B << 8 | 4 << 12);
  return h2u(__hsub2(u2h(p), u2h(0x64806480u)));
}

__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t* w, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* w, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}
// transpose of an 8 x 8 matrix of halves held as mma fragments
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Place of 16-byte piece c of row r in a tile with NC pieces a row: rows in
// order, the eight places of each 128-byte line permuted so that the same
// piece of 8 consecutive rows (one ldmatrix phase) lies in eight bank groups.
template <int NC>
__device__ __forceinline__ uint32_t place(int r, int c) {
  if (NC >= 8) return (uint32_t)((r * NC + (c & ~7) + ((c ^ r) & 7)) * 16);
  const int id = r * NC + c, line = id >> 3;  // NC = 4: two rows a line
  return (uint32_t)((line * 8 + ((id ^ line) & 3) + (id & 4)) * 16);
}

// ---------------------------------------------------------------- plan
// The work is a list of units: per sequence b (n_b tiles a head, none when its
// position is refused), head by head, ceil(n_b / m) ranges of about equal
// length a head, a CTA each; or (m = 0) the tiles themselves, in spans: CTA c
// begins at tile c q + min(c, rem) (q = total / CTAs, rem = total % CTAs),
// moved to the border of an item that is within `near` tiles (near <= q / 4, so
// that the order of the CTAs stays).  A call with more than 2^30 tiles is
// refused.  These run in warp 0, all lanes alike unless said.
struct Item {
  int b, g, first, end;  // sequence, kv head, its units in the list
};
__device__ __forceinline__ Item item_at(const Params& p, const Small& sm, int t) {
  const int lane = threadIdx.x & 31;
  int b = 0;
  for (int k = 0; k < p.nb; k += 32) {
    const unsigned in = __ballot_sync(0xffffffffu, k + lane < p.nb && t < sm.at[min(k + lane, p.nb - 1) + 1]);
    if (in) {
      b = k + __ffs(in) - 1;
      break;
    }
  }
  const int n = sm.per[b], g = (int)((unsigned)(t - sm.at[b]) / (unsigned)n);
  return {b, g, sm.at[b] + g * n, sm.at[b] + g * n + n};
}
__device__ __forceinline__ int span_first(const Params& p, const Small& sm, unsigned c) {
  if (c == 0) return 0;
  if (c >= gridDim.x) return sm.at[p.nb];
  const int t = (int)(c * sm.q + min(c, (unsigned)sm.rem));
  const Item it = item_at(p, sm, t);
  return it.end - t <= sm.near ? it.end : t - it.first <= sm.near ? it.first : t;
}
// The CTA whose span, before its ends are moved, holds tile t (0 for t < 0).
__device__ __forceinline__ int span_of(const Small& sm, int t) {
  if (t < 0) return 0;
  const unsigned q = sm.q, rem = sm.rem, big = rem * (q + 1);
  return (int)((unsigned)t < big ? t / (q + 1) : rem + (t - big) / q);
}

// Lengths, the list and this CTA's units.
template <int W>
__device__ __forceinline__ void plan_work(const Params& p, Small& sm) {
  const int lane = threadIdx.x & 31, grid = gridDim.x;
  const long long cap = (long long)p.c.max_pages * p.c.page_tokens;
  unsigned total = 0, items = 0, least = 0, most = 0;  // tiles, items, ranges of W tiles, longest item
  for (int b = lane; b < p.nb; b += 32) {
    int T = p.len[b];
    if (T < 0 || T >= cap) {
      if (blockIdx.x == 0) set_guard(p.guard, kGuardBadPosition);
      T = -1;
    }
    sm.T[b] = T;
    const unsigned n = T < 0 ? 0 : view_of(T, p.window, p.sinks).n;
    sm.per[b] = n;
    total += n;
    items += n > 0;
    least += (n + W - 1) / W;
    most = max(most, n);
  }
  total = p.nkv * __reduce_add_sync(0xffffffffu, total);
  items = p.nkv * __reduce_add_sync(0xffffffffu, items);
  least = p.nkv * __reduce_add_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  // m: a tile per warp if the CTAs suffice (or the few more with which one join does: 4096 rows of 4 x 128 13.6 us in
  // ranges of 8 tiles, 33 sharers and two joins), else the least that fits
  unsigned m = 0;
  if (least <= (unsigned)grid) {
    m = W * max(1u, (most + W * kJoin - 1) / (W * kJoin));
  } else if (items < (unsigned)grid) {
    const unsigned lo0 = max((total + grid - 1) / grid, (unsigned)W);
    // ranges of m tiles are fewer than total / m + items: `hi` fits
    unsigned lo = lo0, hi = min(most, total / (grid - items) + 1);
    while (lo < hi) {
      const unsigned mid = (lo + hi) / 2;
      unsigned r = 0;
      for (int b = lane; b < p.nb; b += 32) r += ((unsigned)sm.per[b] + mid - 1) / mid;
      if (p.nkv * __reduce_add_sync(0xffffffffu, r) <= (unsigned)grid)
        hi = mid;
      else
        lo = mid + 1;
    }
    // a second range costs a CTA about what three tiles of every warp do
    m = hi > lo0 + 3 * W ? 0 : hi;
  }
  unsigned base = 0;
  for (int b0 = 0; b0 < p.nb; b0 += 32) {
    const int b = b0 + lane;
    unsigned per = b < p.nb ? sm.per[b] : 0;
    if (m) per = (per + m - 1) / m;
    unsigned incl = p.nkv * per;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (b < p.nb) {
      sm.at[b + 1] = base + incl;
      sm.per[b] = per;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) {
    sm.at[0] = 0;
    sm.m = m;
    if (!m) {
      sm.q = total / (unsigned)grid;
      sm.rem = total - sm.q * grid;
      sm.near = min(sm.q / 4, 2 * W);
    }
  }
  __syncwarp();
  const int c = blockIdx.x, all = base;
  const int u0 = all == 0 ? 0 : m ? min(c, all) : span_first(p, sm, c);
  const int u1 = all == 0 ? 0 : m ? min(c + 1, all) : span_first(p, sm, c + 1);
  if (lane == 0) {
    sm.unit = u0;
    sm.unit_end = u1;
  }
  __syncwarp();
}

// The range of this CTA that begins at unit t < unit_end, and the CTAs that share its item: those of
// the first and last tile that begin in it after moving.
template <int W>
__device__ __forceinline__ void set_range(const Params& p, Small& sm, int t) {
  const Item it = item_at(p, sm, t);
  const int n = view_of(sm.T[it.b], p.window, p.sinks).n, parts = it.end - it.first, k = t - it.first;
  const int end = min(it.end, sm.unit_end);
  int c_lo = it.first, np = parts, slot0 = 0;
  if (!sm.m) {
    // of the unmoved begins, those past `in` go to the item's end, those up to `lo` to or before its first tile
    const int in = it.end - sm.near - 1 >= it.first ? it.end - sm.near - 1 : it.first - 1;
    const int lo = min(it.first + sm.near, in);
    c_lo = span_of(sm, lo);
    np = span_of(sm, in) - c_lo + 1;
    slot0 = span_first(p, sm, c_lo) != it.first;  // the first sharer's span began before the item
  }
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    sm.b = it.b;
    sm.g = it.g;
    if (sm.m) {
      const int len = (unsigned)n / (unsigned)parts, more = n - len * parts;
      sm.tile0 = k * len + min(k, more);
      sm.ntile = len + (k < more);
    } else {
      sm.tile0 = k;
      sm.ntile = end - t;
    }
    sm.next = end;
    sm.c_lo = c_lo;
    sm.np = np;
    sm.slot0 = slot0;
  }
}

__device__ __forceinline__ void put_out(float* o, const float4& a, float f) {  // o has no alignment of its own
  o[0] = a.x * f;
  o[1] = a.y * f;
  o[2] = a.z * f;
  o[3] = a.w * f;
}
__device__ __forceinline__ void add_scaled(float4& a, float f, const float4& x) {
  a.x = fmaf(f, x.x, a.x);
  a.y = fmaf(f, x.y, a.y);
  a.z = fmaf(f, x.z, a.z);
  a.w = fmaf(f, x.w, a.w);
}
// weight of a partial whose reference is r under the joined one, R (-infinity: nothing in view)
__device__ __forceinline__ float weight(float r, float R) { return R == -INFINITY ? 0.f : ex2(r - R); }
__device__ __forceinline__ float inverse(float den) { return den == 0.f ? 0.f : 1.0f / den; }

// ---------------------------------------------------------------- inputs of a range
// The queries of the item as MMA operands: element d of a head, piece c = d /
// 16, i = d % 16 = 4 w + k, meets byte k of word w of the codes' piece: half k
// & 1 of B register k >> 1, in the lane of quad w and its column.
template <int HD, int G, int W>
__device__ __forceinline__ void load_queries(const Params& p, Small& sm, uint32_t* qfrag) {
  constexpr int NB = HD / 32, NH = G == 8 ? 2 : 1;
  constexpr int NU = G * NB, UW = (NU + W - 1) / W;  // units of 16 rotate-half pairs, two of them in a warp's halves
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = sm.b, g = sm.g, T = sm.T[b];
  const float* y = p.y + (long long)b * p.ld_y;
  const float2* rope = p.rope + (long long)T * (HD / 2);
  // unit u: head u / NB, pairs 32 (u % NB) / 2 ..; a lane holds one pair's one value of each half for 16 lanes
  float x[UW][2];
  float2 cs[UW];
#pragma unroll
  for (int k = 0; k < UW; ++k) {  // (a warp without a unit reads unit 0)
    const int u = warp + k * W < NU ? warp + k * W : 0, j = u / NB, c = u % NB;
    const int d = c * 16 + (lane & 15);
    const float* qh = y + (long long)(g * G + j) * HD;
    x[k][0] = qh[d];
    x[k][1] = qh[d + HD / 2];
    cs[k] = rope[d];
  }
#pragma unroll
  for (int k = 0; k < UW; ++k) {
    const int u = warp + k * W;
    rotate(x[k][0], x[k][1], cs[k], &x[k][0], &x[k][1]);
    x[k][0] *= p.scale_log2e;
    x[k][1] *= p.scale_log2e;
    const uint32_t a = __reduce_max_sync(
        0xffffffffu, max(__float_as_uint(x[k][0]) & 0x7fffffffu, __float_as_uint(x[k][1]) & 0x7fffffffu));
    if (u < NU && lane == 0) sm.amax[u / NB][u % NB] = a;
  }
  __syncthreads();
  // normalised by 2^e with 2^e max |q| in [2^9, 2^10): as two fp16 parts q
  // keeps 22 bits of the head's largest value.  Exponent field arithmetic: a
  // subnormal maximum counts as 2^-127; one past 2^112 (infinite, NaN) overflows.
#pragma unroll
  for (int k = 0; k < UW; ++k) {
    const int u = warp + k * W, j = u / NB, c0 = u % NB;
    if (u < NU) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < NB; ++i) a = max(a, sm.amax[j][i]);
      int e = 9 + 127 - (int)(a >> 23);
      e = min(max(e, -103), 100);
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
      if (lane == 0) sm.qf[j] = __uint_as_float((uint32_t)(127 - e) << 23);
      const int hb = lane >> 4, c = c0 + hb * (NB);  // lanes 0..15 the first half's values, the others the second's
      const float v = (hb ? x[k][1] : x[k][0]) * up;
      const __half h = __float2half_rn(v);
      const __half l = __float2half_rn(v - __half2float(h));
      const int w = (lane & 15) >> 2, i = lane & 3;
      __half* f = reinterpret_cast<__half*>(qfrag);
      auto put = [&](int col, int part, __half val) {  // part: second fragment (low parts of 8 heads)
        f[(((c * NH + part) * 32 + col * 4 + w) * 2 + (i >> 1)) * 2 + (i & 1)] = val;
      };
      if (G == 8) {
        const int col = (j & 3) * 2 + (j >> 2);
        put(col, 0, h);
        put(col, 1, l);
      } else {
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (m % G == j) {
            put(2 * m, 0, h);
            put(2 * m + 1, 0, l);
          }
      }
    }
  }
}

// The open block's K (kv = 0) or V by one warp: the tail's rows and the new
// one.  It stays open: the new row to the tail, the rows in view as fp16 under
// a power of two in `open` (element order as ldmatrix hands out the codes'),
// zeros elsewhere.  It closes: codes to `open` and its page, the scale.
template <int HD>
__device__ __forceinline__ void last_block(const Params& p, Small& sm, uint8_t* open, int kv) {
  constexpr int NV = HD / 8, NU = kBlock * NV / 32;  // 8-element pieces of a row; of a lane
  constexpr int NC = HD / 16;
  const int lane = threadIdx.x & 31;
  const int b = sm.b, g = sm.g, T = sm.T[b], last = T % kBlock, j = T / kBlock;
  uint16_t* tail = p.c.tail + b * p.c.tail_stride + ((long long)kv * p.nkv + g) * kBlock * HD;
  const bool closes = last == kBlock - 1;
  open += kv * (closes ? Shape<HD>::kTile : Shape<HD>::kOpen / 2);
  uint4 x[NU];
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int id = u * 32 + lane, r = id / NV;
    x[u] = make_uint4(0, 0, 0, 0);
    if (r < last) x[u] = *reinterpret_cast<const uint4*>(tail + id * 8);
  }
  float n[8];  // the new row's piece of this lane
  const int d0 = (lane % NV) * 8;
  {
    const float* row = p.y + (long long)b * p.ld_y + (long long)(p.nq + kv * p.nkv + g) * HD;
    if (kv) {
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = row[d0 + i];
    } else {
      const int h0 = d0 & (HD / 2 - 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float r0, r1;
        rotate(row[h0 + i], row[h0 + i + HD / 2], p.rope[(long long)T * (HD / 2) + h0 + i], &r0, &r1);
        n[i] = d0 < HD / 2 ? r0 : r1;
      }
    }
  }
  const uint4 nw = make_uint4(store_pair(n[0], n[1]), store_pair(n[2], n[3]), store_pair(n[4], n[5]),
                              store_pair(n[6], n[7]));
  uint32_t a = 0;
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int r = (u * 32 + lane) / NV;
    if (r == last) x[u] = nw;
    if (!closes && !in_view(j * kBlock + r, T, p.window, p.sinks)) x[u] = make_uint4(0, 0, 0, 0);
    a = abs_max(abs_max(abs_max(abs_max(a, x[u].x), x[u].y), x[u].z), x[u].w);
  }
  float* kv_new = p.kv_new ? p.kv_new + (((long long)b * 2 + kv) * p.nkv + g) * HD + d0 : nullptr;
  if (closes) {
    a = __reduce_max_sync(0xffffffffu, a);
    float inv;
    const float s = block_scale(a, &inv);
    const int pg = page_of(p.c, b, j);
    int8_t* codes = nullptr;
    if (lane == 0) sm.os[kv] = s;
    if (pg < 0) {
      if (lane == 0) set_guard(p.guard, kGuardBadIndex);
    } else {
      codes = (kv ? p.c.V : p.c.K) + code_at(p.c, pg, g, j % p.c.bpp, HD);
      if (lane == 0) (kv ? p.c.Vs : p.c.Ks)[scale_at(p.c, pg, g, j % p.c.bpp)] = s;
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int id = u * 32 + lane, r = id / NV, d = (id % NV) * 8;
      const uint32_t q[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = block_code(i & 1 ? bf16_hi(q[i / 2]) : bf16_lo(q[i / 2]), inv);
        w[i / 4] |= (uint32_t)(c & 255) << (8 * (i & 3));
        if (r == last && kv_new) kv_new[i] = __fmul_rn(s, (float)c);
      }
      *reinterpret_cast<uint2*>(open + place<NC>(r, d / 16) + d % 16) = make_uint2(w[0], w[1]);
      if (codes) *reinterpret_cast<uint2*>(codes + r * HD + d) = make_uint2(w[0], w[1]);
    }
  } else {
    if (lane / NV == last % (32 / NV)) *reinterpret_cast<uint4*>(tail + last * HD + d0) = nw;
    if (kv_new && lane / NV == last % (32 / NV)) {
      const uint32_t q[4] = {nw.x, nw.y, nw.z, nw.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) kv_new[i] = i & 1 ? bf16_hi(q[i / 2]) : bf16_lo(q[i / 2]);
    }
    // largest finite exponent: values below 2^15 after scaling
    if (a >= 0x7f80u) {
      a = 0;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const uint32_t q[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if ((q[i] & 0x7fffu) < 0x7f80u) a = max(a, q[i] & 0x7fffu);
          if (((q[i] >> 16) & 0x7fffu) < 0x7f80u) a = max(a, (q[i] >> 16) & 0x7fffu);
        }
      }
    }
    a = __reduce_max_sync(0xffffffffu, a);
    const int e = min(14 + 127 - (int)(a >> 7), 100);
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    if (lane == 0) sm.os[kv] = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int id = u * 32 + lane, r = id / NV, c = (id % NV) / 2, i0 = (id % 2) * 8;  // elements i0 .. of piece c
      const uint32_t q[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = h2u(__floats2half2_rn(bf16_lo(q[i]) * up, bf16_hi(q[i]) * up));
      // two 8-element groups of the piece, 16 bytes each, at places 2 c and 2 c + 1 of a row of 2 NC
      const uint32_t p0 = place<2 * NC>(r, 2 * c), p1 = place<2 * NC>(r, 2 * c + 1);
      if (kv) {  // even elements, then odd ones
        *reinterpret_cast<uint2*>(open + p0 + i0) =
            make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
        *reinterpret_cast<uint2*>(open + p1 + i0) =
            make_uint2(__byte_perm(h[0], h[1], 0x7632), __byte_perm(h[2], h[3], 0x7632));
      } else {  // pair t of the group: elements 4 t, 4 t + 1, then 4 t + 2, 4 t + 3
        *reinterpret_cast<uint2*>(open + p0 + i0) = make_uint2(h[0], h[2]);
        *reinterpret_cast<uint2*>(open + p1 + i0) = make_uint2(h[1], h[3]);
      }
    }
  }
}

// ---------------------------------------------------------------- joins
// Partials first, first + step, ... (n <= 32 of them) of the item joined into
// the outputs (final) or into the first of them, by TG groups of threads, each
// a TG-th of them.  Not inlined: its loads would cost the tile loop registers.
template <int HD, int G>
__device__ __noinline__ void join_parts(const Params& p, Small& sm, uint8_t* smem, int first, int step, int n,
                                        bool final) {
  using Sh = Shape<HD>;
  constexpr int NV = G * HD / 4, VT = (NV + Sh::kThreads - 1) / Sh::kThreads;  // vectors; of a thread
  constexpr int TG = VT == 1 ? Sh::kThreads / NV : 1;
  constexpr int NX = HD == 256 ? 12 : 8;  // partials of a thread on their way at once
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = VT == 1 ? tid / NV : 0, v0 = tid - grp * NV;
  const int c_lo = sm.c_lo, slot0 = sm.slot0;
  auto part_of = [&](int i) { return p.part + (2ll * (c_lo + i) + (i == 0 ? slot0 : 0)) * part_size(G, HD); };
  float* o = p.o + (long long)sm.b * p.ld_o + (long long)sm.g * G * HD;
  float* wt = reinterpret_cast<float*>(smem);  // [32][G] weights, joined reference and sum per head
  float4* sums = reinterpret_cast<float4*>(smem + 2048);  // [TG][NV]
  float4 x[VT][NX];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
      for (int t = 0; t < VT; ++t)
        if (i0 + i * TG + grp < n && v0 + t * Sh::kThreads < NV)
          x[t][i] = __ldcg(reinterpret_cast<const float4*>(part_of(first + (i0 + i * TG + grp) * step)) + v0 +
                           t * Sh::kThreads);
  };
  load(0);
  for (int j = warp; j < G; j += Sh::W) {
    float r = -INFINITY, l = 0.f;
    if (lane < n) {
      const float* q = part_of(first + lane * step) + G * HD;
      r = __ldcg(q + j);
      l = __ldcg(q + G + j);
    }
    const float R = warp_max(r);
    const float f = lane < n ? weight(r, R) : 0.f;
    const float den = warp_sum(f * l);
    wt[lane * G + j] = f;
    if (lane == 0) {
      wt[32 * G + j] = R;
      wt[33 * G + j] = den;
    }
  }
  __syncthreads();
  float* dst = part_of(first);
  float4 a[VT];
#pragma unroll
  for (int t = 0; t < VT; ++t) a[t] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += NX * TG) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
      for (int t = 0; t < VT; ++t)
        if (i0 + i * TG + grp < n && v0 + t * Sh::kThreads < NV)
          add_scaled(a[t], wt[(i0 + i * TG + grp) * G + (v0 + t * Sh::kThreads) * 4 / HD], x[t][i]);
  }
  if (TG > 1) {
    if (grp > 0) sums[tid] = a[0];
    __syncthreads();
#pragma unroll 1
    for (int k = 1; k < TG; ++k)
      if (grp == 0) add_scaled(a[0], 1.f, sums[k * NV + v0]);
  }
#pragma unroll
  for (int t = 0; t < VT; ++t) {
    const int v = v0 + t * Sh::kThreads, j = v * 4 / HD;
    if (v >= NV || grp > 0) break;
    if (final) {
      put_out(o + v * 4, a[t], inverse(wt[33 * G + j]));
    } else {
      reinterpret_cast<float4*>(dst)[v] = a[t];
      if (v * 4 % HD == 0) {
        dst[G * HD + j] = wt[32 * G + j];
        dst[G * HD + G + j] = wt[33 * G + j];
      }
    }
  }
  __syncthreads();
}

// The warps' outputs joined, and those of the CTAs that share the item.
template <int HD, int G>
__device__ __forceinline__ void join_warps(const Params& p, Small& sm, uint8_t* smem, bool first_range) {
  using Sh = Shape<HD>;
  constexpr int W = Sh::W, OP = out_pitch(HD);
  const int tid = threadIdx.x, cta = blockIdx.x;
  const int b = sm.b, g = sm.g, c_lo = sm.c_lo, np = sm.np;
  float* o = p.o + (long long)b * p.ld_o + (long long)g * G * HD;
  constexpr int NV = G * HD / 4;  // 4-vectors of the outputs
  float* part = p.part + (2ll * cta + (first_range ? 0 : 1)) * part_size(G, HD);
  for (int v = tid; v < NV; v += Sh::kThreads) {
    const int j = v * 4 / HD;
    float R = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) R = fmaxf(R, sm.r[w][j]);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = weight(sm.r[w][j], R);
      add_scaled(a, f, *reinterpret_cast<const float4*>(smem + w * Sh::kWarpRing + (j * OP + v * 4 % HD) * 4));
      den = fmaf(f, sm.l[w][j], den);
    }
    if (np == 1) {
      put_out(o + v * 4, a, inverse(den));
    } else {
      reinterpret_cast<float4*>(part)[v] = a;
      if (v * 4 % HD == 0) {
        part[G * HD + j] = R;
        part[G * HD + G + j] = den;
      }
    }
  }
  __syncthreads();
  if (np > 1) {
    // Whether this CTA is the last of n to arrive at the counter, which is left at zero.
    auto last_of = [&](unsigned* ctr, int n) {
      if (tid == 0) {
        __threadfence();
        const int last = atomicAdd(ctr, 1u) == (unsigned)(n - 1);
        if (last) *ctr = 0;
        __threadfence();
        sm.last = last;
      }
      __syncthreads();
      return sm.last != 0;
    };
    const int me = cta - c_lo, grp = me / kJoin, ng = (np + kJoin - 1) / kJoin;
    unsigned* ctr = p.counter + ((long long)b * p.nkv + g) * kCounters;
    const int n1 = np - grp * kJoin < kJoin ? np - grp * kJoin : kJoin;
    if (last_of(ctr + 1 + grp, n1)) {
      join_parts<HD, G>(p, sm, smem, grp * kJoin, 1, n1, ng == 1);
      if (ng > 1 && last_of(ctr, ng)) join_parts<HD, G>(p, sm, smem, 0, kJoin, ng, true);
    }
  }
}

// One token of each sequence.  MMA layouts (lane = 4 * row8 + quad): the codes
// of 16 cached rows are the A operand of the scores (rows row8 and row8 + 8)
// and, read transposed, of the outputs (elements 2 row8 and 2 row8 + 1 of a
// 16-byte piece); the heads are the columns of B, two adjacent columns to a
// quad lane: for up to 4 heads the fp16 high and low part of head `quad`, for 8
// heads two heads, `quad` and quad + 4, whose low parts are a second product
// into the same accumulator.  So a lane's scores, probabilities, maximum, sum
// and outputs all belong to its own head(s), and only the probabilities change
// sides (movmatrix).
template <int HD, int G>
__global__ void __launch_bounds__(Shape<HD>::kThreads, Shape<HD>::kCtas) k_attn(const __grid_constant__ Params p) {
  using Sh = Shape<HD>;
  constexpr int S = Sh::S, W = Sh::W, NC = Sh::NC;
  constexpr int NH = G == 8 ? 2 : 1;  // heads of a lane
  extern __shared__ __align__(128) uint8_t smem[];
  uint32_t* qfrag = reinterpret_cast<uint32_t*>(smem + Sh::kRing);
  uint8_t* open = smem + Sh::kRing + Sh::kQ;
  Small& sm = *reinterpret_cast<Small*>(smem + Sh::kRing + Sh::kQ + Sh::kOpen);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = lane & 3, row8 = lane >> 2;
  uint8_t* ring = smem + warp * Sh::kWarpRing;
  const uint32_t ring_a = smem_addr(ring);

  if (warp == 0) {
    plan_work<W>(p, sm);
    if (sm.unit < sm.unit_end) set_range<W>(p, sm, sm.unit);
  }
  __syncthreads();
  if (sm.unit >= sm.unit_end) return;

  for (bool more = true, first_range = true; more; first_range = false) {
    const int T = sm.T[sm.b], tile0 = sm.tile0, ntile = sm.ntile, head = sm.g;
    const View view = view_of(T, p.window, p.sinks);
    const int mine = ntile > warp ? (ntile - warp + W - 1) / W : 0;  // tiles of this warp
    const int* table = p.c.table + (long long)sm.b * p.c.max_pages;
    const bool has_last = tile0 + ntile == view.n;
    // The pages and scales of 32 of the warp's tiles, a lane each: page -1 where the table has none, -2 for the
    // last block, which does not come through the ring.
    struct Look {
      int pg, off;  // page, block within it
      float ks, vs;
    };
    auto look_up = [&](int i0) {
      Look k = {-2, 0, 0.f, 0.f};
      const int i = i0 + lane, t = tile0 + warp + i * W;
      if (i < mine && t < view.n - 1) {
        const int blk = block_at(view, t), at = blk / p.c.bpp;
        k.off = blk - at * p.c.bpp;
        k.pg = __ldg(table + at);
        if ((unsigned)k.pg >= (unsigned)p.c.pool_pages) {
          set_guard(p.guard, kGuardBadIndex);
          k.pg = -1;
        } else {
          const long long s = scale_at(p.c, k.pg, head, k.off);
          k.ks = __ldg(p.c.Ks + s);
          k.vs = __ldg(p.c.Vs + s);
        }
      }
      return k;
    };
    uint32_t dst = ring_a;  // stage to fetch into
    auto fetch = [&](int i, const Look& k) {  // tile i of the warp, one of k's, into the next ring stage
      const int page = __shfl_sync(0xffffffffu, k.pg, i & 31);
      const int o = __shfl_sync(0xffffffffu, k.off, i & 31);
      if (i < mine && page >= 0) {
        const long long at = code_at(p.c, page, head, o, HD) + lane * 16;
#pragma unroll
        for (int u = 0; u < NC / 2; ++u) {
          const int id = u * 32 + lane;
          const uint32_t d = dst + place<NC>(id / NC, id % NC);
          cp16(d, p.c.K + at + u * 512);
          cp16(d + Sh::kTile, p.c.V + at + u * 512);
        }
      }
      dst = dst == ring_a + (S - 1) * Sh::kStage ? ring_a : dst + Sh::kStage;
      cp_commit();
    };
    Look cur = look_up(0), nxt = cur;
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i, cur);

    load_queries<HD, G, W>(p, sm, qfrag);
    if (has_last && warp >= W - 2) last_block<HD>(p, sm, open, W - 1 - warp);
    __syncthreads();

    // ---------------------------------------------------- the warp's tiles
    float acc[NC][2 * NH];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 2 * NH; ++k) acc[c][k] = 0.f;
    float mx[NH], lsum[NH], qf[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      mx[h] = -INFINITY;
      lsum[h] = 0.f;
      qf[h] = sm.qf[G == 8 ? quad + 4 * h : quad % G];
    }
    uint32_t st = ring_a;  // stage to read
    for (int i = 0; i < mine; ++i) {
      const int page = __shfl_sync(0xffffffffu, cur.pg, i & 31);
      float fk = __shfl_sync(0xffffffffu, cur.ks, i & 31), fv = __shfl_sync(0xffffffffu, cur.vs, i & 31);
      if ((i & 31) == 8 && (i & ~31) + 32 < mine) nxt = look_up((i & ~31) + 32);  // in time for the fetches ahead
      if ((i & 31) + S - 1 < 32)
        fetch(i + S - 1, cur);
      else
        fetch(i + S - 1, nxt);
      if ((i & 31) == 31) cur = nxt;
      cp_wait<S - 1>();
      __syncwarp();
      const int tile = tile0 + warp + i * W;
      const int u0 = block_at(view, tile) * kBlock;
      const bool is_last = page == -2, halves = is_last && T % kBlock != kBlock - 1;
      uint32_t kst = st, vst = st + Sh::kTile;
      if (is_last) {
        kst = smem_addr(open);
        vst = kst + (halves ? Sh::kOpen / 2 : Sh::kTile);
        fk = sm.os[0];
        fv = sm.os[1];
      }
      if (page != -1) {
        // scores of rows row8 and row8 + 8
        float d[2][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) d[0][k] = d[1][k] = 0.f;
        auto product = [&](int c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
          const uint2 q0 = *reinterpret_cast<const uint2*>(qfrag + (c * NH * 32 + lane) * 2);
          mma(d[c & 1], a0, a1, a2, a3, q0.x, q0.y);
          if (G == 8) {
            const uint2 q1 = *reinterpret_cast<const uint2*>(qfrag + ((c * NH + 1) * 32 + lane) * 2);
            mma(d[c & 1], a0, a1, a2, a3, q1.x, q1.y);
          }
        };
        if (!halves) {
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            uint32_t w[4];  // rows 0-7 and 8-15 of piece c, then of piece c + 1
            ldsm4(w, kst + place<NC>(lane & 15, c + (lane >> 4)));
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] ^= 0x80808080u;
            product(c, widen<0, 1>(w[0]), widen<0, 1>(w[1]), widen<2, 3>(w[0]), widen<2, 3>(w[1]));
            product(c + 1, widen<0, 1>(w[2]), widen<0, 1>(w[3]), widen<2, 3>(w[2]), widen<2, 3>(w[3]));
          }
        } else {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            uint32_t w[4];
            ldsm4(w, kst + place<2 * NC>(lane & 15, 2 * c + (lane >> 4)));
            product(c, w[0], w[1], w[2], w[3]);
          }
        }
        float s[2][NH];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          if (G == 8) {
            s[n][0] = d[0][2 * n] + d[1][2 * n];
            s[n][NH - 1] = d[0][2 * n + 1] + d[1][2 * n + 1];
          } else {
            s[n][0] = (d[0][2 * n] + d[1][2 * n]) + (d[0][2 * n + 1] + d[1][2 * n + 1]);
          }
        }
        // (scaled, then masked: a factor of 0, of a block of zeros, would make NaN of -infinity)
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const float f = fk * qf[h];
          s[0][h] *= f;
          s[1][h] *= f;
        }
        if (is_last || (p.window > 0 && u0 <= T - p.window && u0 + kBlock > p.sinks)) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
            if (!in_view(u0 + n * 8 + row8, T, p.window, p.sinks)) {
#pragma unroll
              for (int h = 0; h < NH; ++h) s[n][h] = -INFINITY;
            }
        }
        bool moved = false;
        float mn[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          float tm = fmaxf(s[0][h], s[1][h]);
          tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 4));
          tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 8));
          tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 16));
          mn[h] = fmaxf(mx[h], tm);
          moved |= mn[h] != mx[h];
        }
        if (__any_sync(0xffffffffu, moved)) {
          float corr[NH];
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            corr[h] = ex2(mx[h] - mn[h]);
            lsum[h] *= corr[h];
            mx[h] = mn[h];
          }
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int k = 0; k < 2 * NH; ++k) acc[c][k] *= corr[G == 8 ? (k & 1) * (NH - 1) : 0];
        }
        // weights times 2^14 as two fp16 parts, rows to columns
        uint32_t ph[2], pl[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float v[NH], h[NH];
#pragma unroll
          for (int k = 0; k < NH; ++k) {
            const float w = ex2(s[n][k] - mx[k]);
            lsum[k] += w;
            v[k] = w * 16384.f;
            h[k] = trunc11(v[k]);
          }
          if (G == 8) {
            ph[n] = movmatrix(h2u(__floats2half2_rn(h[0], h[NH - 1])));
            pl[n] = movmatrix(h2u(__floats2half2_rn(v[0] - h[0], v[NH - 1] - h[NH - 1])));
          } else {
            ph[n] = movmatrix(h2u(__floats2half2_rn(h[0], v[0] - h[0])));
            pl[n] = 0;
          }
        }
        // outputs: a block's products on their own, added to the running outputs in FP32 times its scale (the
        // tensor cores truncate what they add to an accumulator, which over a long context would be 2^-24 a
        // product, all one way)
        auto add = [&](int c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
          float e[4] = {0.f, 0.f, 0.f, 0.f};
          mma(e, a0, a1, a2, a3, ph[0], ph[1]);
          if (G == 8) {
            mma(e, a0, a1, a2, a3, pl[0], pl[1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[c][k % (2 * NH)] = fmaf(fv, e[k], acc[c][k % (2 * NH)]);
          } else {
            acc[c][0] = fmaf(fv, e[0] + e[1], acc[c][0]);
            acc[c][1] = fmaf(fv, e[2] + e[3], acc[c][1]);
          }
        };
        if (!halves) {
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            uint32_t w[4];
            ldsm4t(w, vst + place<NC>(lane & 15, c + (lane >> 4)));
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] ^= 0x80808080u;
            add(c, widen<0, 2>(w[0]), widen<1, 3>(w[0]), widen<0, 2>(w[1]), widen<1, 3>(w[1]));
            add(c + 1, widen<0, 2>(w[2]), widen<1, 3>(w[2]), widen<0, 2>(w[3]), widen<1, 3>(w[3]));
          }
        } else {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            uint32_t w[4];  // rows 0-7 of the even elements, rows 8-15, then of the odd ones
            ldsm4t(w, vst + place<2 * NC>(lane & 15, 2 * c + (lane >> 4)));
            add(c, w[0], w[2], w[1], w[3]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage before it is fetched into again
      st = st == ring_a + (S - 1) * Sh::kStage ? ring_a : st + Sh::kStage;
    }
    cp_wait<0>();
    __syncwarp();

    // ---------------------------------------------------- join the warps
    constexpr int OP = out_pitch(HD);
    float* ow = reinterpret_cast<float*>(ring);  // [G][OP] of this warp, in its own ring
    static_assert(G * OP * 4 <= Sh::kWarpRing, "a warp's outputs fit its ring");
    constexpr float unit = 1.0f / 16384.f;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const int j = quad + 4 * h;
      lsum[h] += __shfl_xor_sync(0xffffffffu, lsum[h], 4);
      lsum[h] += __shfl_xor_sync(0xffffffffu, lsum[h], 8);
      lsum[h] += __shfl_xor_sync(0xffffffffu, lsum[h], 16);
      if (j < G) {
        if (row8 == 0) {
          sm.r[warp][j] = mx[h];
          sm.l[warp][j] = lsum[h];
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
          *reinterpret_cast<float2*>(ow + j * OP + c * 16 + row8 * 2) =
              G == 8 ? make_float2(acc[c][h] * unit, acc[c][(2 + h) % (2 * NH)] * unit)
                     : make_float2(acc[c][0] * unit, acc[c][1] * unit);
      }
    }
    __syncthreads();
    join_warps<HD, G>(p, sm, smem, first_range);
    more = sm.next < sm.unit_end;
    __syncthreads();
    if (more) {
      if (warp == 0) set_range<W>(p, sm, sm.next);
      __syncthreads();
    }
  }
}

using Kern = void (*)(Params);
struct Pick {
  Kern k;
  size_t smem;
  int threads, per_sm, warps;
};
template <int HD>
Pick pick_g(int G) {
  using Sh = Shape<HD>;
  Kern k = G == 1 ? k_attn<HD, 1> : G == 2 ? k_attn<HD, 2> : G == 4 ? k_attn<HD, 4> : G == 8 ? k_attn<HD, 8> : nullptr;
  return {k, smem_bytes<HD>(), Sh::kThreads, Sh::kCtas, Sh::W};
}
Pick pick(int hd, int G) {
  return hd == 64 ? pick_g<64>(G) : hd == 128 ? pick_g<128>(G) : hd == 256 ? pick_g<256>(G) : Pick{};
}

}  // namespace

size_t part_floats(int nq, int nkv, int hd, int nsm) {
  const Pick k = pick(hd, nq / nkv);
  return (size_t)2 * nsm * k.per_sm * part_size(nq / nkv, hd);
}
size_t counters(int nb, int nkv) { return (size_t)nb * nkv * kCounters; }

cudaError_t init() {
  for (int hd : {64, 128, 256})
    for (int G : {1, 2, 4, 8}) {
      const Pick k = pick(hd, G);
      const cudaError_t e =
          cudaFuncSetAttribute((const void*)k.k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem);
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

cudaError_t attention(const Params& p, int hd, int nsm, cudaStream_t st) {
  if (p.nb < 1 || p.nb > kMaxB || p.nkv <= 0 || p.nq % p.nkv) return cudaErrorInvalidValue;
  const Pick k = pick(hd, p.nq / p.nkv);
  if (!k.k) return cudaErrorInvalidValue;
  const long long per = most_blocks(p.c, p.window, p.sinks);
  const long long tiles = p.nkv * per * p.nb, chunks = p.nkv * ((per + k.warps - 1) / k.warps) * p.nb;
  if (tiles > kMaxTiles) return cudaErrorInvalidValue;
  long long grid = (long long)nsm * k.per_sm;
  if (grid > (kCounters - 1) * kJoin) grid = (kCounters - 1) * kJoin;  // what the joins can count
  if (grid > chunks) grid = chunks;
  return launch_k(k.k, dim3((unsigned)grid), dim3(k.threads), k.smem, st, false, p);
}

cudaError_t append(const Params& p, int hd, cudaStream_t st) {
  if (p.n <= 0) return cudaSuccess;
  // rows cut into blocks: at most two more than whole ones for each sequence with rows
  const long long blocks = p.n / kBlock + 2ll * (p.nb < p.n ? p.nb : p.n);
  const int units = hd == 256 ? kAppendWarps / 2 : kAppendWarps;  // of a CTA
  long long grid = (blocks * 2 * p.nkv + units - 1) / units;
  if (grid > 1 << 20) grid = 1 << 20;
  auto ok = [](const void* q) { return ((uintptr_t)q & 15) == 0; };
  const bool vec = ok(p.y) && p.ld_y % 4 == 0 && ok(p.rope) && ok(p.kv_new);
  void (*k)(Params) = nullptr;
  switch (hd) {
    case 64: k = vec ? k_append<64, true> : k_append<64, false>; break;
    case 128: k = vec ? k_append<128, true> : k_append<128, false>; break;
    case 256: k = vec ? k_append<256, true> : k_append<256, false>; break;
    default: return cudaErrorInvalidValue;
  }
  k<<<(unsigned)grid, kAppendWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace p8
}  // namespace hy
