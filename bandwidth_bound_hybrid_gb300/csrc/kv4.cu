// The 4-bit KV cache on sm_103a: GQA decode attention over it, and the
// quantising append of prompt rows.
//
// Format: a k or v vector of hd values is hd / 32 blocks; block b holds codes
// c in [-7, 7] (stored as c + 8: element i in the low nibble of byte i, element
// i + 16 in its high nibble, as in the 4-bit weights) and one fp16 scale s,
// value = s c.
//
// Attention.  For kv head g with its G = nq / nkv query heads and L = T + 1
// rows,
//   s_jt = sum_b sK[t][b] (q_j[b] . cK[t][b]),   p_jt = softmax_t(s_jt),
//   o_j[b] = sum_t (p_jt sV[t][b]) cV[t][b],
// so both products run on the tensor cores on the codes themselves, which
// fp16 holds exactly, and the scales stay FP32 factors outside: of a block's
// partial score, and of the probability that meets a block of V.  q and
// p sV are split into two fp16 parts, which err by 2^-22 of the value, or where
// that is below fp16's subnormals by 2^-34 of the head's largest |q| and 2^-38
// of the largest sV that the warp has met.  (So a block of V far below others
// has fewer bits: 2^-16 of a row at a ratio of 2^22.)  A row-by-8-heads (or
// hi-and-lo-of-4-heads) operand carries them in one MMA.
// A batch of small queries against a cache that is read once fills 8 of the
// 128 rows of a tcgen05 tile and would still need the codes widened into
// shared memory, so this uses mma.sync, whose operands are widened in
// registers.
//
// Work split: the cached rows of every (sequence, kv head) are cut into tiles,
// and in a CTA each warp takes every W-th tile of the CTA's range through its
// own cp.async ring and keeps its own running maximum, sum and outputs (no
// block barrier inside a range).  A CTA gets one range of at most m tiles of
// one (sequence, head), m about the least for which the CTAs suffice (the
// least, where the bounds of the search are at most 31 apart); where that
// leaves much more than an equal share (more heads than CTAs, a few long
// contexts each), all tiles form one list instead and every CTA takes an equal
// span of it, its ends moved to a nearby border between heads.
// An (sequence, head) that several CTAs share is joined from their partials
//   R = max_i r_i,  o = sum_i 2^(r_i - R) o_i / sum_i 2^(r_i - R) l_i
// without any CTA waiting: the last of each 24 sharers to arrive joins the 24,
// and the last of those joins the rest.
//
// Measured (4 kv heads x 128, 16 query heads): 8 sequences of 120k-131k rows in
// 112 us, 5190 GB/s, where widening (5 ALU operations for 8 codes, two issue
// cycles each) and 32 MMAs a tile (eight each) fill four fifths of the issue
// time; one of 4096 rows in 9.2 us, a chain of latencies.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "kv4_dev.cuh"
#include "kv4_plan.h"

namespace hy {
namespace kv4 {
namespace {

// Per head dim: warps of a CTA and CTAs per SM, rows of a warp's tile, and the
// stages of its ring.  Registers set the warps: a lane holds hd / 4 output
// accumulators (hd 128, 4 heads, 8 sequences of 120k-131k: 12 warps an SM 112
// us, 16 warps in two CTAs 116, 8 warps 118, 10 warps 130; hd 256, 8 heads, 8
// sequences of 1k-16k: 8 warps 26.7 us, 12 warps 28.2, 10 warps 30.4, all
// before the plan tried every length, which takes 8 warps to 25.6).
template <int HD>
struct Shape {
  static constexpr int W = HD == 128 ? 12 : 8;
  static constexpr int kThreads = W * 32;
  static constexpr int kCtas = HD == 64 ? 2 : 1;     // per SM
  static constexpr int TR = HD == 256 ? 16 : 32;     // rows of a tile
  static constexpr int S = HD == 128 ? 3 : 4;
  static constexpr int NB = HD / 32;                 // blocks of a row
  static constexpr int kCodes = TR * HD / 2;         // bytes of a tile's K or V codes
  static constexpr int kScales = TR * NB * 2;        // and of their scales
  static constexpr int kKV = kCodes + kScales;
  static constexpr int kStage = 2 * kKV;
  static constexpr int kWarpRing = S * kStage;
  static constexpr int kRing = W * kWarpRing;
  static constexpr int kQ = NB * 2 * 32 * 4 * 4;     // query operand fragments (two of them for 8 heads)
};

struct alignas(16) Small {
  float nk[256], nv[256];          // the new row before quantisation
  uint8_t codes[2][128];           // and its codes and scales
  uint16_t scales[2][8];
  uint32_t amax[8][4];             // per head and pair of blocks: largest |q| (bits)
  float qf[8];                     // per head: 2^-e of the query normalisation
  float r[12][8], l[12][8];
  int last;
  // the work (set by warp 0, so that no warp holds it over its tiles)
  int T[kMaxB];                    // positions of the new rows (-1: refused)
  int at[kMaxB + 1];               // first unit of each sequence: tiles (spans) or ranges
  int per[kMaxB];                  // units of one of its heads
  int m;                           // most tiles of a range; 0: spans
  int q, rem, near;
  int unit, unit_end;              // this CTA's units
  int b, g, first, end, tile0, ntile, next;  // the item and this CTA's range of it
  int c_lo, np, slot0;             // the CTAs that share the item
  const uint8_t *Kc, *Vc, *Ksc, *Vsc;        // its cache rows
};

template <int HD>
constexpr size_t smem_bytes() {
  return (size_t)Shape<HD>::kRing + Shape<HD>::kQ + sizeof(Small);
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
__device__ __forceinline__ float lo_f(uint32_t u) { return __low2float(u2h(u)); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __high2float(u2h(u)); }
// (w & mask) | bits in one operation
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
  return r;
}
// The codes n - 8 of a word's nibbles n as fp16 pairs, one of each 16-bit
// half: the low nibbles of the low and of the high bytes, then their high
// nibbles.  1024 + n - 1032 and (1024 + 16 n) / 16 - 72, all exact.  (Leaving n
// in the scores' operand and subtracting 8 sum q afterwards saves the
// subtractions, 108 us for 114 at 8 x 125k rows, but the tensor cores round
// the larger sums: errors of 0.4e-6 to 1.2e-6 of the outputs for 0.1e-6 to
// 0.4e-6.)
__device__ __forceinline__ void codes(uint32_t w, uint32_t* v) {
  const __half2 k1032 = u2h(0x64086408u), k16th = u2h(0x2c002c00u), k72 = u2h(0xd480d480u);
  const uint32_t w8 = w >> 8;
  v[0] = h2u(__hsub2(u2h(and_or(w, 0x000f000fu, 0x64006400u)), k1032));
  v[1] = h2u(__hsub2(u2h(and_or(w8, 0x000f000fu, 0x64006400u)), k1032));
  v[2] = h2u(__hfma2(u2h(and_or(w, 0x00f000f0u, 0x64006400u)), k16th, k72));
  v[3] = h2u(__hfma2(u2h(and_or(w8, 0x00f000f0u, 0x64006400u)), k16th, k72));
}
// v truncated to fp16's 11 significant bits: v - trunc11(v) is exact
__device__ __forceinline__ float trunc11(float v) { return __uint_as_float(__float_as_uint(v) & 0xffffe000u); }

// d = a b + c
__device__ __forceinline__ void mma_c(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1, float c0, float c1, float c2, float c3) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
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
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// 16-byte asynchronous copy of the first `bytes` (0..16) bytes, the rest zero
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Place of 16-byte block c of row r in a tile's codes: rows in order, the
// eight 16-byte places of each 128-byte line permuted by the line number so
// that the same block of 8 consecutive rows (one ldmatrix phase) lies in
// eight different bank groups.
template <int NB>
__device__ __forceinline__ uint32_t place(int r, int c) {
  const int id = r * NB + c, line = id >> 3;
  return (uint32_t)((line * 8 + ((id & 7) ^ (line & (NB - 1)))) * 16);
}

// (x0, x1) of a rotate-half pair, each product and sum rounded on its own, so
// that a code never depends on how the compiler contracts them.
__device__ __forceinline__ void rotate(float x0, float x1, float2 cs, float* r0, float* r1) {
  *r0 = __fsub_rn(__fmul_rn(x0, cs.x), __fmul_rn(x1, cs.y));  // (x0, x1 are copies: r0, r1 may be their origin)
  *r1 = __fadd_rn(__fmul_rn(x1, cs.x), __fmul_rn(x0, cs.y));
}

// ------------------------------------------------------------ attention
// The work is a list of units: per sequence b (n_b = T_b / TR + 1 tiles, none
// when its position is refused), head by head, ceil(n_b / m) ranges of
// about equal length a head, a CTA each; or (m = 0) the tiles themselves, in
// spans: CTA c begins at tile c q + min(c, rem) (q = total / CTAs, rem = total %
// CTAs), moved to the border of an item that is within `near` tiles (near <=
// q / 4, so that the order of the CTAs stays).  The launch refuses caches of
// more than 2^30 tiles.  These run in warp 0, all lanes alike unless said.
struct Item {
  int b, g, first, end;  // sequence, kv head, its units in the list
};
__device__ __forceinline__ Item item_at(const Params& p, const Small& sm, int t) {
  const int lane = threadIdx.x & 31;
  const int b = __ffs(__ballot_sync(0xffffffffu, lane < p.nb && t < sm.at[lane < p.nb ? lane + 1 : 0])) - 1;
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
template <int TR, int W>
__device__ __forceinline__ void plan_work(const Params& p, Small& sm) {
  const int lane = threadIdx.x & 31;
  int T = -1;
  if (lane < p.nb) {  // lengths: written only by the previous step's last kernel
    T = *p.len[lane];
    if (T < 0 || T >= p.cap[lane]) {
      if (blockIdx.x == 0) set_guard(p.guard, kGuardBadPosition);
      T = -1;
    }
    sm.T[lane] = T;
  }
  const int n = T < 0 ? 0 : T / TR + 1;  // tiles of a head of sequence `lane`
  const int total = p.nkv * (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
  const int items = p.nkv * __popc(__ballot_sync(0xffffffffu, n > 0));
  const int grid = gridDim.x;
  // m: a tile per warp if the CTAs suffice, else the least of 32 candidates that fits, a lane each
  int m = 0, per = (n + W - 1) / W;
  if (p.nkv * (int)__reduce_add_sync(0xffffffffu, (unsigned)per) <= grid) {
    m = W;
  } else {
    if (items <= grid) {
      const int lo = (int)shortest_range(total, grid, W);
      const int hi = (int)longest_range(total, grid, items, lo);
      const unsigned mine = range_length(lo, hi, lane);
      unsigned ranges = 0;
      const float inv = 1.0f / (float)mine;
#pragma unroll
      for (int b = 0; b < kMaxB; ++b)  // (n is 0 past the last sequence)
        ranges += ranges_of(__shfl_sync(0xffffffffu, n, b), mine, inv);
      const unsigned fits = __ballot_sync(0xffffffffu, p.nkv * (int)ranges <= grid);
      m = fits ? (int)__shfl_sync(0xffffffffu, mine, __ffs(fits) - 1) : 0;
      // a second range costs a CTA about what three tiles of every warp do
      if (m > lo + 3 * W) m = 0;
    }
    per = m ? (int)((unsigned)(n + m - 1) / (unsigned)m) : n;
  }
  int incl = p.nkv * per;
#pragma unroll
  for (int o = 1; o < kMaxB; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 0) {
    sm.at[0] = 0;
    sm.m = m;
    if (!m) {
      sm.q = (unsigned)total / (unsigned)grid;
      sm.rem = total - sm.q * grid;
      sm.near = min(sm.q / 4, 2 * W);
    }
  }
  if (lane < kMaxB) {
    sm.at[lane + 1] = incl;
    sm.per[lane] = per;
  }
  __syncwarp();
  const int c = blockIdx.x, all = sm.at[p.nb];
  const int u0 = all == 0 ? 0 : m ? min(c, all) : span_first(p, sm, c);
  const int u1 = all == 0 ? 0 : m ? min(c + 1, all) : span_first(p, sm, c + 1);
  if (lane == 0) {
    sm.unit = u0;
    sm.unit_end = u1;
  }
}

// The range of this CTA that begins at unit t < unit_end, and where its rows are.
template <int HD, int TR, int W>
__device__ __forceinline__ void set_range(const Params& p, Small& sm, int t) {
  const Item it = item_at(p, sm, t);
  const int n = sm.T[it.b] / TR + 1, parts = it.end - it.first, k = t - it.first;
  const int end = min(it.end, sm.unit_end);
  if ((threadIdx.x & 31) == 0) {
    sm.b = it.b;
    sm.g = it.g;
    sm.first = it.first;
    sm.end = it.end;
    if (sm.m == W) {
      sm.tile0 = k * W;
      sm.ntile = min(W, n - k * W);
    } else if (sm.m) {
      const int len = (unsigned)n / (unsigned)parts, more = n - len * parts;
      sm.tile0 = k * len + min(k, more);
      sm.ntile = len + (k < more);
    } else {
      sm.tile0 = k;
      sm.ntile = end - t;
    }
    sm.next = end;
    const long long cap = p.cap[it.b], cap_s = (cap + 3) & ~3ll;
    sm.Kc = p.K[it.b] + it.g * cap * (HD / 2);
    sm.Vc = p.V[it.b] + it.g * cap * (HD / 2);
    sm.Ksc = reinterpret_cast<const uint8_t*>(p.Ks[it.b] + it.g * cap_s * (HD / 32));
    sm.Vsc = reinterpret_cast<const uint8_t*>(p.Vs[it.b] + it.g * cap_s * (HD / 32));
  }
}

// The CTAs that share the item: those of the first and last tile that begin in it after moving.
__device__ __forceinline__ void set_sharers(const Params& p, Small& sm) {
  int c_lo = sm.first, np = sm.end - sm.first, slot0 = 0;
  if (!sm.m) {
    // of the unmoved begins, those past `in` go to the item's end, those up to `lo` to or before its first tile
    const int in = sm.end - sm.near - 1 >= sm.first ? sm.end - sm.near - 1 : sm.first - 1;
    const int lo = min(sm.first + sm.near, in);
    c_lo = span_of(sm, lo);
    np = span_of(sm, in) - c_lo + 1;
    slot0 = span_first(p, sm, c_lo) != sm.first;  // the first sharer's span began before the item
  }
  if ((threadIdx.x & 31) == 0) {
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

// The queries of the item as MMA operands, and the new row if the range ends with it.
template <int HD, int G>
__device__ __forceinline__ void prepare(const Params& p, Small& sm, uint32_t* qfrag) {
  using Sh = Shape<HD>;
  constexpr int NB = Sh::NB, TR = Sh::TR, W = Sh::W, NH = G == 8 ? 2 : 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = sm.b, g = sm.g, T = sm.T[b], tile0 = sm.tile0, ntile = sm.ntile;
  const float* y = p.y + (long long)b * p.ld_y;
  const float2* rope = p.rope + (long long)T * (HD / 2);
  const bool has_new = tile0 + ntile == T / TR + 1;
  // queries: a warp takes blocks c and c + NB / 2 of a head (the halves of its rotate-half pairs)
  constexpr int NU = G * NB / 2, UW = (NU + W - 1) / W;
  float x[UW][2];
  float2 cs[UW];
#pragma unroll
  for (int k = 0; k < UW; ++k) {  // (a warp without a unit reads unit 0)
    const int u = warp + k * W < NU ? warp + k * W : 0, j = u / (NB / 2), c = u % (NB / 2);
    const float* qh = y + (long long)(g * G + j) * HD + c * 32 + lane;
    x[k][0] = qh[0];
    x[k][1] = qh[HD / 2];
    cs[k] = rope[c * 32 + lane];
  }
  if (has_new && warp >= W - 4) {  // the new k and v
    const float* kh = y + (long long)(p.nq + g) * HD;
    const float* vh = y + (long long)(p.nq + p.nkv + g) * HD;
    for (int i = tid - (W - 4) * 32; i < HD / 2; i += 128) {
      const float k0 = kh[i], k1 = kh[i + HD / 2], v0 = vh[i], v1 = vh[i + HD / 2];
      rotate(k0, k1, rope[i], &sm.nk[i], &sm.nk[i + HD / 2]);
      sm.nv[i] = v0;
      sm.nv[i + HD / 2] = v1;
    }
  }
#pragma unroll
  for (int k = 0; k < UW; ++k) {
    const int u = warp + k * W;
    rotate(x[k][0], x[k][1], cs[k], &x[k][0], &x[k][1]);
    x[k][0] *= p.scale_log2e;
    x[k][1] *= p.scale_log2e;
    const uint32_t a = __reduce_max_sync(
        0xffffffffu, max(__float_as_uint(x[k][0]) & 0x7fffffffu, __float_as_uint(x[k][1]) & 0x7fffffffu));
    if (u < NU && lane == 0) sm.amax[u / (NB / 2)][u % (NB / 2)] = a;
  }
  if (warp == 0) set_sharers(p, sm);
  __syncthreads();
  // normalised by 2^e with 2^e max |q| in [2^9, 2^10): as two fp16 parts q
  // keeps 22 bits of the head's largest value.  Exponent field arithmetic: a
  // subnormal maximum counts as 2^-127; one past 2^112 (infinite, NaN) overflows.
#pragma unroll
  for (int k = 0; k < UW; ++k) {
    const int u = warp + k * W, j = u / (NB / 2), c0 = u % (NB / 2);
    if (u < NU) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < NB / 2; ++i) a = max(a, sm.amax[j][i]);
      int e = 9 + 127 - (int)(a >> 23);
      e = min(max(e, -103), 100);
      const int k16 = lane >> 4;
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
      if (lane == 0) sm.qf[j] = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {
        const int c = c0 + hb * (NB / 2);
        const float v = x[k][hb] * up;
        const __half h = __float2half_rn(v);
        const float hf = __half2float(h);
        const __half l = __float2half_rn(v - hf);
        // element `lane` of a block: code byte i of word w, low (k16 = 0) or high nibble; it meets
        // half i >> 1 of B register i & 1 of k-step k16, in the lane of quad w and column row8
        const int w = (lane & 15) >> 2, i = lane & 3;
        __half* f = reinterpret_cast<__half*>(qfrag);
        auto put = [&](int col, int part, __half val) {  // part: second fragment (low parts of 8 heads)
          f[((((c * NH + part) * 32 + col * 4 + w) * 4) + k16 * 2 + (i & 1)) * 2 + (i >> 1)] = val;
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
  if (has_new) {
    for (int u = W - 1 - warp; u < 2 * NB; u += W) {  // block u % NB of K (u < NB) or V
      const int kv = u / NB, c = u % NB;
      int code;
      const uint16_t s = quant_block((kv ? sm.nv : sm.nk)[c * 32 + lane], &code);
      store_block(s, code, sm.codes[kv] + c * 16, &sm.scales[kv][c],
                  p.kv_new ? p.kv_new + (((long long)b * 2 + kv) * p.nkv + g) * HD + c * 32 : nullptr, lane);
      __syncwarp();
      uint8_t* gc = const_cast<uint8_t*>(kv ? sm.Vc : sm.Kc) + (long long)T * (HD / 2) + c * 16;
      if (lane < 4)
        reinterpret_cast<uint32_t*>(gc)[lane] = reinterpret_cast<const uint32_t*>(sm.codes[kv] + c * 16)[lane];
      uint16_t* gs = reinterpret_cast<uint16_t*>(const_cast<uint8_t*>(kv ? sm.Vsc : sm.Ksc));
      if (lane == 4) gs[(long long)T * NB + c] = s;
    }
  }
}

// Partials first, first + step, ... (n <= 32 of them) of the item joined into
// the outputs (final) or into the first of them.  The first loads are on
// their way while one warp per head turns the references into weights.  Not
// inlined: its loads would cost the tile loop registers.
template <int HD, int G>
__device__ __noinline__ void join_parts(const Params& p, Small& sm, uint8_t* smem, int first, int step, int n,
                                        bool final) {
  using Sh = Shape<HD>;
  constexpr int NV = G * HD / 4, VT = (NV + Sh::kThreads - 1) / Sh::kThreads;  // vectors; of a thread
  constexpr int NX = VT == 1 ? 8 : 12;                                          // partials on their way at once
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c_lo = sm.c_lo, slot0 = sm.slot0;
  auto part_of = [&](int i) { return p.part + (2ll * (c_lo + i) + (i == 0 ? slot0 : 0)) * part_size(G, HD); };
  float* o = p.o + (long long)sm.b * p.ld_o + (long long)sm.g * G * HD;
  float* wt = reinterpret_cast<float*>(smem);  // [32][G] weights, joined reference and sum per head
  float4 x[VT][NX];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
      for (int t = 0; t < VT; ++t)
        if (i0 + i < n && tid + t * Sh::kThreads < NV)
          x[t][i] = __ldcg(reinterpret_cast<const float4*>(part_of(first + (i0 + i) * step)) + tid + t * Sh::kThreads);
  };
  load(0);
  if (warp < G) {
    const int j = warp;
    float r = -INFINITY, l = 0.f;
    if (lane < n) {
      const float* q = part_of(first + lane * step) + G * HD;
      r = __ldcg(q + j);
      l = __ldcg(q + G + j);
    }
    const float R = warp_max(r);
    const float f = lane < n ? ex2(r - R) : 0.f;
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
  for (int i0 = 0; i0 < n; i0 += NX) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
      for (int t = 0; t < VT; ++t)
        if (i0 + i < n && tid + t * Sh::kThreads < NV)
          add_scaled(a[t], wt[(i0 + i) * G + (tid + t * Sh::kThreads) * 4 / HD], x[t][i]);
  }
#pragma unroll
  for (int t = 0; t < VT; ++t) {
    const int v = tid + t * Sh::kThreads, j = v * 4 / HD;
    if (v >= NV) break;
    if (final) {
      put_out(o + v * 4, a[t], 1.0f / wt[33 * G + j]);
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
      const float f = ex2(sm.r[w][j] - R);
      add_scaled(a, f, *reinterpret_cast<const float4*>(smem + w * Sh::kWarpRing + (j * OP + v * 4 % HD) * 4));
      den = fmaf(f, sm.l[w][j], den);
    }
    if (np == 1) {
      put_out(o + v * 4, a, 1.0f / den);
    } else {
      reinterpret_cast<float4*>(part)[v] = a;
      if (v * 4 % HD == 0) {
        part[G * HD + j] = R;
        part[G * HD + G + j] = den;
      }
    }
  }
  __syncthreads();
  // ---------------------------------------------------- join the CTAs
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
    unsigned* ctr = p.counter + (b * p.nkv + g) * kCounters;
    const int n1 = np - grp * kJoin < kJoin ? np - grp * kJoin : kJoin;
    if (last_of(ctr + 1 + grp, n1)) {
      join_parts<HD, G>(p, sm, smem, grp * kJoin, 1, n1, ng == 1);
      if (ng > 1 && last_of(ctr, ng)) join_parts<HD, G>(p, sm, smem, 0, kJoin, ng, true);
    }
  }
}

// One token of each sequence.  MMA layouts (lane = 4 * row8 + quad): the codes
// of 16 cached rows are the A operand of the scores (rows row8 and row8 + 8)
// and, read transposed, of the outputs (elements row8); the heads are the
// columns of B, two adjacent columns to a quad lane: for up to 4 heads the
// fp16 high and low part of head `quad`, for 8 heads two heads, `quad` and
// quad + 4, whose low parts are a second product into the same accumulator.
// So a lane's scores, probabilities, maximum, sum and outputs all belong to
// its own head(s), and only the probabilities change sides (movmatrix).
template <int HD, int G>
__global__ void __launch_bounds__(Shape<HD>::kThreads, Shape<HD>::kCtas) k_attn(const __grid_constant__ Params p) {
  using Sh = Shape<HD>;
  constexpr int NB = Sh::NB, S = Sh::S, TR = Sh::TR, W = Sh::W, NR = TR / 8;
  constexpr int NH = G == 8 ? 2 : 1;  // heads of a lane
  extern __shared__ __align__(128) uint8_t smem[];
  uint32_t* qfrag = reinterpret_cast<uint32_t*>(smem + Sh::kRing);
  Small& sm = *reinterpret_cast<Small*>(smem + Sh::kRing + Sh::kQ);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = lane & 3, row8 = lane >> 2;
  uint8_t* ring = smem + warp * Sh::kWarpRing;
  const uint32_t ring_a = smem_addr(ring);

  if (warp == 0) {
    plan_work<TR, W>(p, sm);
    __syncwarp();
    if (sm.unit < sm.unit_end) set_range<HD, TR, W>(p, sm, sm.unit);
  }
  __syncthreads();
  if (sm.at[p.nb] == 0) pdl_wait();  // the next kernel counts on this one for all before it
  if (sm.unit >= sm.unit_end) return;

  for (bool more = true, first_range = true; more; first_range = false) {
    const int T = sm.T[sm.b], tile0 = sm.tile0, ntile = sm.ntile;
    const int mine = ntile > warp ? (ntile - warp + W - 1) / W : 0;  // tiles of this warp
    // the cached rows of the warp's next tile into the next ring stage: each lane its 16-byte pieces
    constexpr int NS = Sh::kScales / 16;  // 16-byte pieces of a tile's K or V scales
    static_assert(2 * NS <= 32, "at most one scale piece per lane");
    const int sc_k = lane % NS;
    int left = T - (tile0 + warp) * TR;   // cached rows from the next tile on (0: only the new row)
    int unfetched = mine;
    const uint8_t *kp, *vp, *sp;
    {
      const long long r0 = (long long)(tile0 + warp) * TR;
      kp = sm.Kc + r0 * (HD / 2) + lane * 16;
      vp = sm.Vc + r0 * (HD / 2) + lane * 16;
      sp = (lane < NS ? sm.Ksc : sm.Vsc) + r0 * NB * 2 + sc_k * 16;
    }
    uint32_t dst = ring_a;                // stage to fetch into
    const uint32_t sd = (lane < NS ? 0 : Sh::kKV) + Sh::kCodes + sc_k * 16;
    auto fetch = [&]() {
      if (unfetched > 0) {
        if (left >= TR) {
#pragma unroll
          for (int u = 0; u < TR * NB / 32; ++u) {
            const int id = u * 32 + lane;
            cp16(dst + place<NB>(id / NB, id % NB), kp + u * 512, 16);
            cp16(dst + Sh::kKV + place<NB>(id / NB, id % NB), vp + u * 512, 16);
          }
          if (lane < 2 * NS) cp16(dst + sd, sp, 16);
        } else {  // past the last cached row: zeros (codes -8 under scales 0), nothing read
#pragma unroll
          for (int u = 0; u < TR * NB / 32; ++u) {
            const int id = u * 32 + lane;
            const bool in = id / NB < left;
            cp16(dst + place<NB>(id / NB, id % NB), in ? kp + u * 512 : sm.Kc, in ? 16 : 0);
            cp16(dst + Sh::kKV + place<NB>(id / NB, id % NB), in ? vp + u * 512 : sm.Vc, in ? 16 : 0);
          }
          const int b16 = left * NB * 2 - sc_k * 16;
          const int bytes = b16 <= 0 ? 0 : (b16 < 16 ? b16 : 16);
          if (lane < 2 * NS) cp16(dst + sd, bytes ? sp : sm.Ksc, bytes);
        }
        kp += W * Sh::kCodes;
        vp += W * Sh::kCodes;
        sp += W * Sh::kScales;
        left -= W * TR;
        --unfetched;
        dst = dst == ring_a + (S - 1) * Sh::kStage ? ring_a : dst + Sh::kStage;
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch();

    if (first_range) {
      pdl_wait();
      pdl_launch_dependents();
    }
    prepare<HD, G>(p, sm, qfrag);
    __syncthreads();

    // ---------------------------------------------------- the warp's tiles
    float acc[NB][2][4];
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[c][t][k] = 0.f;
    float mx[NH], lsum[NH], qf[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      mx[h] = -INFINITY;
      lsum[h] = 0.f;
      qf[h] = sm.qf[G == 8 ? quad + 4 * h : quad % G];
    }
    int sh = 29;  // the products with V take 2^sh p, so that p sV fills fp16's range from above
    // ldmatrix row of this lane: 8-row groups of one block, or (16-row tiles) of two
    auto frag = [&](int cp, int half) {
      return NR == 4 ? place<NB>(lane, cp * 2 + half) : place<NB>(lane & 15, cp * 2 + (lane >> 4));
    };

    uint32_t st = ring_a;                     // stage to read
    int valid = T + 1 - (tile0 + warp) * TR;  // rows of the tile that exist
    for (int i = 0; i < mine; ++i) {
      fetch();
      cp_wait<S - 1>();
      __syncwarp();
      const uint32_t vst = st + Sh::kKV;
      if (valid <= TR) {  // the last tile: the new row's codes and scales are its last row
        const int r = valid - 1;
        if (lane < 2 * NB) {
          const int kv = lane / NB, c = lane % NB;
          uint8_t* d = ring + (st - ring_a) + kv * Sh::kKV;
          *reinterpret_cast<uint4*>(d + place<NB>(r, c)) = *reinterpret_cast<const uint4*>(sm.codes[kv] + c * 16);
          *reinterpret_cast<uint16_t*>(d + Sh::kCodes + (r * NB + c) * 2) = sm.scales[kv][c];
        }
        __syncwarp();
      }
      // largest V scale of the tile (as fp16 bits, a sign masked)
      __half2 vm = u2h(lds32(vst + Sh::kCodes + lane * 4) & 0x7fff7fffu);
#pragma unroll
      for (int u = 1; u < Sh::kScales / 128; ++u)
        vm = __hmax2(vm, u2h(lds32(vst + Sh::kCodes + (u * 32 + lane) * 4) & 0x7fff7fffu));
      uint32_t vmax = max(h2u(vm) & 0xffffu, h2u(vm) >> 16);
      vmax = __reduce_max_sync(0xffffffffu, vmax);

      // scores of rows row8 + 8 n, two blocks at a time
      float s[NR][NH];
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int h = 0; h < NH; ++h) s[n][h] = 0.f;
#pragma unroll
      for (int cp = 0; cp < NB / 2; ++cp) {
        uint32_t sc[NR], w[2][NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) sc[n] = lds32(st + Sh::kCodes + ((n * 8 + row8) * NB + cp * 2) * 2);
        ldsm4(&w[0][0], st + frag(cp, 0));
        if (NR == 4) ldsm4(&w[1][0], st + frag(cp, 1));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = cp * 2 + half;
          const uint4 q0 = *reinterpret_cast<const uint4*>(qfrag + (c * NH * 32 + lane) * 4);
          uint4 q1;
          if (G == 8) q1 = *reinterpret_cast<const uint4*>(qfrag + ((c * NH + 1) * 32 + lane) * 4);
          uint32_t h[NR][4];
#pragma unroll
          for (int n = 0; n < NR; ++n) codes(w[half][n], h[n]);
          // 16 rows a product; the products into one accumulator are apart
          float d[NR / 2][4];
#pragma unroll
          for (int m = 0; m < NR / 2; ++m) {
            const uint32_t *x = h[m * 2], *z = h[m * 2 + 1];
            mma_c(d[m], x[0], z[0], x[1], z[1], q0.x, q0.y, 0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
          for (int m = 0; m < NR / 2; ++m) {
            const uint32_t *x = h[m * 2], *z = h[m * 2 + 1];
            mma(d[m], x[2], z[2], x[3], z[3], q0.z, q0.w);
          }
          if (G == 8) {
#pragma unroll
            for (int m = 0; m < NR / 2; ++m) {
              const uint32_t *x = h[m * 2], *z = h[m * 2 + 1];
              mma(d[m], x[0], z[0], x[1], z[1], q1.x, q1.y);
            }
#pragma unroll
            for (int m = 0; m < NR / 2; ++m) {
              const uint32_t *x = h[m * 2], *z = h[m * 2 + 1];
              mma(d[m], x[2], z[2], x[3], z[3], q1.z, q1.w);
            }
          }
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const float f = half ? hi_f(sc[n]) : lo_f(sc[n]);
            const float *dn = d[n / 2] + (n & 1) * 2;
            if (G == 8) {
              s[n][0] = fmaf(f, dn[0], s[n][0]);
              s[n][NH - 1] = fmaf(f, dn[1], s[n][NH - 1]);
            } else {
              s[n][0] = fmaf(f, dn[0] + dn[1], s[n][0]);
            }
          }
        }
      }
      // sV < 2^(E - 14) with E the exponent field of the largest, so 2^sh p sV <= 2^15
      const int fit = min(29 - (int)(vmax >> 10), sh);
      bool moved = fit != sh;
      float mn[NH];
      if (valid < TR) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int h = 0; h < NH; ++h)
            if (n * 8 + row8 >= valid) s[n][h] = -INFINITY;
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float tm = s[0][h];
#pragma unroll
        for (int n = 1; n < NR; ++n) tm = fmaxf(tm, s[n][h]);
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 4));
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 8));
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 16));
        mn[h] = fmaxf(mx[h], tm * qf[h]);
        moved |= mn[h] != mx[h];
      }
      if (__any_sync(0xffffffffu, moved)) {
        float corr[NH];
        const float down = __uint_as_float((uint32_t)(127 + fit - sh) << 23);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          corr[h] = ex2(mx[h] - mn[h]);
          lsum[h] *= corr[h];
          corr[h] *= down;
          mx[h] = mn[h];
        }
        sh = fit;
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[c][t][k] *= corr[G == 8 ? (k & 1) * (NH - 1) : 0];
      }
      const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          // the argument is near 0 where the weight is large: its rounding stays below 2^-24 of the weight
          const float w = ex2(fmaf(s[n][h], qf[h], -mx[h]));
          lsum[h] += w;
          s[n][h] = w * up;
        }
      // outputs, two blocks at a time
#pragma unroll
      for (int cp = 0; cp < NB / 2; ++cp) {
        uint32_t sc[NR], w[2][NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) sc[n] = lds32(vst + Sh::kCodes + ((n * 8 + row8) * NB + cp * 2) * 2);
        ldsm4t(&w[0][0], vst + frag(cp, 0));
        if (NR == 4) ldsm4t(&w[1][0], vst + frag(cp, 1));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = cp * 2 + half;
          uint32_t ph[NR], pl[NR];
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const float sv = half ? hi_f(sc[n]) : lo_f(sc[n]);
            if (G == 8) {
              const float v0 = s[n][0] * sv, v1 = s[n][NH - 1] * sv, h0 = trunc11(v0), h1 = trunc11(v1);
              ph[n] = movmatrix(h2u(__floats2half2_rn(h0, h1)));
              pl[n] = movmatrix(h2u(__floats2half2_rn(v0 - h0, v1 - h1)));
            } else {
              const float v = s[n][0] * sv, h0 = trunc11(v);
              ph[n] = movmatrix(h2u(__floats2half2_rn(h0, v - h0)));
              pl[n] = 0;
            }
          }
          // codes of 8 rows: elements 2 r, 2 r + 1 (v[0], v[1]) and 2 r + 16, 2 r + 17 of the block, r = row8
          uint32_t v[NR][4];
#pragma unroll
          for (int n = 0; n < NR; ++n) codes(w[half][n], v[n]);
          // a tile's products on their own, added to the running outputs in FP32: the tensor cores truncate
          // what they add to an accumulator, which over a long context would be 2^-24 a product, all one way
          float d[2][4];
#pragma unroll
          for (int part = 0; part < NH; ++part) {
            const uint32_t* pp = part ? pl : ph;
#pragma unroll
            for (int n = 0; n < NR; n += 2)
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const uint32_t a0 = v[n][2 * t], a1 = v[n][2 * t + 1], a2 = v[n + 1][2 * t], a3 = v[n + 1][2 * t + 1];
                if (part == 0 && n == 0)
                  mma_c(d[t], a0, a1, a2, a3, pp[n], pp[n + 1], 0.f, 0.f, 0.f, 0.f);
                else
                  mma(d[t], a0, a1, a2, a3, pp[n], pp[n + 1]);
              }
          }
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[c][t][k] += d[t][k];
        }
      }
      __syncwarp();  // every lane has read the stage before it is fetched into again
      st = st == ring_a + (S - 1) * Sh::kStage ? ring_a : st + Sh::kStage;
      valid -= W * TR;
    }
    cp_wait<0>();
    __syncwarp();

    // ---------------------------------------------------- join the warps
    constexpr int OP = out_pitch(HD);
    float* ow = reinterpret_cast<float*>(ring);  // [G][OP] of this warp, in its own ring
    const float unit = __uint_as_float((uint32_t)(127 - sh) << 23);
    static_assert(G * OP * 4 <= Sh::kWarpRing, "a warp's outputs fit its ring");
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
        for (int c = 0; c < NB; ++c)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float* a = acc[c][t];
            *reinterpret_cast<float2*>(ow + j * OP + c * 32 + t * 16 + row8 * 2) =
                G == 8 ? make_float2(a[h] * unit, a[2 + h] * unit)
                       : make_float2((a[0] + a[1]) * unit, (a[2] + a[3]) * unit);
          }
      }
    }
    __syncthreads();
    join_warps<HD, G>(p, sm, smem, first_range);
    more = sm.next < sm.unit_end;
    __syncthreads();
    if (more) {
      if (warp == 0) set_range<HD, TR, W>(p, sm, sm.next);
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------ append
// Rows of n tokens at positions T .. T + n - 1 of one sequence; blockIdx.y is
// the kv head of k, then of v.  A lane holds the 4 + 4 adjacent values that are
// rotate-half pairs of each other, 8 lanes a block, a warp the vectors of 256 /
// hd tokens; the loads of units(hd) of them are on their way together (8192
// rows of 8 heads x 256: 49.5 us with two, 52.8 with one; x 64: 17.9 and 15.9;
// 2048 rows of 4 x 128: 5.4 and 4.65).  Bound by its bytes: one pass, 16-byte
// accesses.  VEC: y, the table and kv_new are 16-byte aligned with rows of
// whole 16 bytes (8192 rows of 8 heads x 256: 49.5 us so, 60.2 us in 4-byte
// loads and stores, against 44.2 us for the bytes).
__host__ __device__ constexpr int units(int hd) { return hd == 256 ? 2 : 1; }

template <bool VEC>
__device__ __forceinline__ float4 load4(const float* p) {
  return VEC ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], p[1], p[2], p[3]);
}

template <int HD, bool VEC>
__global__ void __launch_bounds__(256) k_append(const AppendParams p) {
  constexpr int NB = HD / 32, VW = 256 / HD, LV = 32 / VW;  // blocks; tokens of a warp, lanes of a vector
  constexpr int kUnits = units(HD);
  const int lane = threadIdx.x & 31;
  const int T = p.len ? *p.len : p.t0;
  if (T < 0 || (long long)T + p.n > p.cap) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_guard(p.guard, kGuardBadPosition);
    return;
  }
  const int kg = blockIdx.y, kv = kg >= p.nkv, g = kv ? kg - p.nkv : kg;
  const int e = (lane % LV) * 4;  // the lane's first element, of the first half
  const float* y0 = p.y + (long long)(p.nq + kg) * HD + e;
  const float* rope0 = reinterpret_cast<const float*>(p.rope + (long long)T * (HD / 2) + e);
  const long long row0 = (long long)g * p.cap + T, row0_s = (long long)g * (((long long)p.cap + 3) & ~3ll) + T;
  uint8_t* codes0 = (kv ? p.V : p.K) + row0 * (HD / 2);
  uint16_t* scales0 = (kv ? p.Vs : p.Ks) + row0_s * NB;
  const long long step = (long long)gridDim.x * (blockDim.x >> 5) * VW;
  for (long long i0 = (blockIdx.x * (long long)(blockDim.x >> 5) + (threadIdx.x >> 5)) * VW; i0 < p.n;
       i0 += step * kUnits) {
    float4 x[kUnits][2], c0[kUnits], c1[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {  // (a lane past the last token reads the first one's)
      const long long at = i0 + u * step + lane / LV, i = at < p.n ? at : 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) x[u][h] = load4<VEC>(y0 + i * p.ld_y + h * (HD / 2));
      if (!kv) {
        c0[u] = load4<VEC>(rope0 + i * HD);
        c1[u] = load4<VEC>(rope0 + i * HD + 4);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (i0 + u * step >= p.n) break;  // the whole warp
      const long long i = i0 + u * step + lane / LV;
      const bool in = i < p.n;
      float f[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f[h][0] = x[u][h].x;
        f[h][1] = x[u][h].y;
        f[h][2] = x[u][h].z;
        f[h][3] = x[u][h].w;
      }
      if (!kv) {
        const float2 cs[4] = {{c0[u].x, c0[u].y}, {c0[u].z, c0[u].w}, {c1[u].x, c1[u].y}, {c1[u].z, c1[u].w}};
#pragma unroll
        for (int k = 0; k < 4; ++k) rotate(f[0][k], f[1][k], cs[k], &f[0][k], &f[1][k]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int el = e + h * (HD / 2), blk = el / 32;
        uint32_t a = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) a = max(a, __float_as_uint(f[h][k]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
        float inv;
        const __half sh = block_scale(a, &inv);
        const float sf = __half2float(sh);
        uint32_t n = 0;
        float val[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = quant_code(f[h][k], inv);
          n |= (uint32_t)(c + 8) << (8 * k);
          val[k] = __fmul_rn(sf, (float)c);
        }
        const uint32_t up = __shfl_down_sync(0xffffffffu, n, 4);  // elements 16 .. 31 of the block: lanes 4 .. 7
        if (in) {
          if ((lane & 7) < 4)
            *reinterpret_cast<uint32_t*>(codes0 + i * (HD / 2) + blk * 16 + (lane & 7) * 4) = n | (up << 4);
          if ((lane & 7) == 0) scales0[i * NB + blk] = __half_as_ushort(sh);
          if (p.kv_new) {
            float* d = p.kv_new + (i * 2 * p.nkv + kg) * HD + el;
            if (VEC) {
              *reinterpret_cast<float4*>(d) = make_float4(val[0], val[1], val[2], val[3]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) d[k] = val[k];
            }
          }
        }
      }
    }
  }
}

using Kern = void (*)(Params);
struct Pick {
  Kern k;
  size_t smem;
  int threads, per_sm, tile, warps;
};
template <int HD>
Pick pick_g(int G) {
  using Sh = Shape<HD>;
  Kern k = G == 1 ? k_attn<HD, 1> : G == 2 ? k_attn<HD, 2> : G == 4 ? k_attn<HD, 4> : G == 8 ? k_attn<HD, 8> : nullptr;
  return {k, smem_bytes<HD>(), Sh::kThreads, Sh::kCtas, Sh::TR, Sh::W};
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

cudaError_t launch(const Params& p, int hd, int nsm, cudaStream_t st, bool pdl) {
  if (p.nb < 1 || p.nb > kMaxB || p.nkv <= 0 || p.nq % p.nkv) return cudaErrorInvalidValue;
  const Pick k = pick(hd, p.nq / p.nkv);
  if (!k.k) return cudaErrorInvalidValue;
  long long tiles = 0, chunks = 0;  // the most the caches can hold
  for (int b = 0; b < p.nb; ++b) {
    const long long n = (p.cap[b] - 1) / k.tile + 1;
    tiles += p.nkv * n;
    chunks += p.nkv * ((n + k.warps - 1) / k.warps);
  }
  if (tiles > (1 << 30)) return cudaErrorInvalidValue;
  long long grid = (long long)nsm * k.per_sm;
  if (grid > (kCounters - 1) * kJoin) grid = (kCounters - 1) * kJoin;  // what the joins can count
  if (grid > chunks) grid = chunks;
  return launch_k(k.k, dim3((unsigned)grid), dim3(k.threads), k.smem, st, pdl, p);
}

cudaError_t append(const AppendParams& p, int hd, cudaStream_t st) {
  if (p.n <= 0) return cudaSuccess;
  if (hd != 64 && hd != 128 && hd != 256) return cudaErrorInvalidValue;
  const int per_block = 8 * (256 / hd) * units(hd);  // tokens
  const dim3 blocks((unsigned)((p.n + (long long)per_block - 1) / per_block), (unsigned)(2 * p.nkv));
  auto ok = [](const void* q) { return ((uintptr_t)q & 15) == 0; };
  const bool vec = ok(p.y) && p.ld_y % 4 == 0 && ok(p.rope) && ok(p.kv_new);
  void (*k)(AppendParams) = nullptr;
  switch (hd) {
    case 64: k = vec ? k_append<64, true> : k_append<64, false>; break;
    case 128: k = vec ? k_append<128, true> : k_append<128, false>; break;
    case 256: k = vec ? k_append<256, true> : k_append<256, false>; break;
    default: return cudaErrorInvalidValue;
  }
  k<<<blocks, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace kv4
}  // namespace hy
