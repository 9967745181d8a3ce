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
// p sV are split into two fp16 parts (relative error 2^-22), which a
// row-by-8-heads (or hi-and-lo-of-4-heads) operand carries in one MMA.
// A batch of small queries against a cache that is read once fills 8 of the
// 128 rows of a tcgen05 tile and would still need the codes widened into
// shared memory, so this uses mma.sync, whose operands are widened in
// registers.
//
// Work split: the cached rows of every (sequence, kv head) are cut into tiles
// of 32 rows, all tiles form one list, and every CTA takes an equal
// contiguous span of it, whatever the mix of lengths.  In a CTA each warp
// takes every 8th tile of the span through its own cp.async ring and keeps
// its own running maximum, sum and outputs (no block barrier inside a span).
// An (sequence, head) that several CTAs share is joined from their partials
//   R = max_i r_i,  o = sum_i 2^(r_i - R) o_i / sum_i 2^(r_i - R) l_i
// by the last of them to arrive.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace hy {
namespace kv4 {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;  // rows of a warp's tile

template <int HD>
struct Shape {
  static constexpr int NB = HD / 32;                 // blocks of a row
  static constexpr int kCodes = kTile * HD / 2;      // bytes of a tile's K or V codes
  static constexpr int kScales = kTile * NB * 2;     // and of their scales
  static constexpr int kStage = 2 * (kCodes + kScales);
  static constexpr int S = HD == 64 ? 4 : 2;         // ring stages of a warp
  static constexpr int kMinCtas = HD == 256 ? 1 : 2; // CTAs per SM
  static constexpr int kRing = kWarps * S * kStage;
  static constexpr int kQ = NB * 32 * 8 * 4;         // query operand fragments
};

struct alignas(16) Small {
  float nk[256], nv[256];          // the new row before quantisation
  uint8_t codes[2][128];           // and its codes and scales
  uint16_t scales[2][8];
  float qf[8];                     // per head: 2^-e of the query normalisation
  float qb[8][8];                  // per block and head: start value of the score accumulator
  float r[kWarps][8], l[kWarps][8];
  int last;
};

template <int HD>
constexpr size_t smem_bytes() {
  return (size_t)Shape<HD>::kRing + Shape<HD>::kQ + sizeof(Small);
}

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

__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
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

// ------------------------------------------------------------ quantisation
// One block of 32 values, one per lane of a full warp: its fp16 scale (bits)
// and the lane's code.  s = fp16(min(max |x| * fp32(1 / 7), 65504)), code =
// round-half-even(x * (1 / s)) clamped to [-7, 7]; an infinity or NaN in the
// block makes the scale NaN, so that it shows in whatever reads the block.
__device__ __forceinline__ uint16_t quant_block(float x, int* code) {
  // |x| as bits: the order of finite values, infinities above, NaN above those
  const uint32_t a = __reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7fffffffu);
  float s = NAN;
  if (a < 0x7f800000u) s = fminf(__fmul_rn(__uint_as_float(a), 1.0f / 7.0f), 65504.0f);
  const __half sh = __float2half_rn(s);
  const float sf = __half2float(sh);
  const float inv = sf > 0.f ? __fdiv_rn(1.0f, sf) : 0.f;
  const float r = fminf(fmaxf(rintf(__fmul_rn(x, inv)), -7.f), 7.f);
  *code = (int)r;
  return __half_as_ushort(sh);
}

// Store a quantised block: byte i (lanes 0..15) of the codes, the scale, and
// the values it stands for (nullable).
__device__ __forceinline__ void store_block(uint16_t s, int code, uint8_t* codes, uint16_t* scale, float* values,
                                            int lane) {
  const uint32_t n = (uint32_t)(code + 8);
  const uint32_t up = __shfl_down_sync(0xffffffffu, n, 16);
  if (lane < 16) codes[lane] = (uint8_t)(n | (up << 4));
  if (lane == 0) *scale = s;
  if (values) values[lane] = __fmul_rn(__half2float(__ushort_as_half(s)), (float)code);
}

// (x0, x1) of a rotate-half pair, each product and sum rounded on its own, so
// that a code never depends on how the compiler contracts them.
__device__ __forceinline__ void rotate(float x0, float x1, float2 cs, float* r0, float* r1) {
  *r0 = __fsub_rn(__fmul_rn(x0, cs.x), __fmul_rn(x1, cs.y));
  *r1 = __fadd_rn(__fmul_rn(x1, cs.x), __fmul_rn(x0, cs.y));
}

// ------------------------------------------------------------ attention
struct Item {
  int b, g, T;           // sequence, kv head, position of the new row
  long long first, end;  // its tiles in the list
};

// The tile list: sequence b has nkv * n_b tiles, n_b = T_b / 32 + 1 (0 when its
// position is refused), head by head.
struct List {
  int T[kMaxB];
  long long total;
};

__device__ __forceinline__ List tile_list(const Params& p) {
  List L;
  L.total = 0;
#pragma unroll
  for (int b = 0; b < kMaxB; ++b) {
    int T = -1;
    if (b < p.nb) {
      T = *p.len[b];
      if (T < 0 || T >= p.cap[b]) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_guard(p.guard, kGuardBadPosition);
        T = -1;
      }
    }
    L.T[b] = T;
    L.total += T < 0 ? 0 : (long long)p.nkv * (T / kTile + 1);
  }
  return L;
}

__device__ __forceinline__ Item item_at(const Params& p, const List& L, long long t) {
  Item it;
  it.b = 0;
  it.g = 0;
  it.T = 0;
  it.first = it.end = 0;
  long long at = 0;
#pragma unroll
  for (int b = 0; b < kMaxB; ++b) {
    const long long n = L.T[b] < 0 ? 0 : L.T[b] / kTile + 1;
    const long long next = at + n * p.nkv;
    if (t >= at && t < next) {
      const int g = (int)((t - at) / n);
      it.b = b;
      it.g = g;
      it.T = L.T[b];
      it.first = at + g * n;
      it.end = it.first + n;
    }
    at = next;
  }
  return it;
}

template <int HD, int G>
__global__ void __launch_bounds__(kThreads, Shape<HD>::kMinCtas) k_attn(const Params p) {
  using Sh = Shape<HD>;
  constexpr int NB = Sh::NB, S = Sh::S;
  extern __shared__ __align__(128) uint8_t smem[];
  uint32_t* qfrag = reinterpret_cast<uint32_t*>(smem + Sh::kRing);
  Small& sm = *reinterpret_cast<Small*>(smem + Sh::kRing + Sh::kQ);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = lane & 3, row8 = lane >> 2;
  const int head = (G == 8 ? row8 : (row8 & 3)) % G;  // the query head of this lane's scores
  uint8_t* ring = smem + warp * (S * Sh::kStage);
  const uint32_t ring_a = smem_addr(ring);

  const List L = tile_list(p);  // lengths: written only by the previous step's last kernel
  if (L.total == 0) {
    pdl_wait();  // the next kernel counts on this one for all before it
    return;
  }
  const long long want = (L.total + p.min_tiles - 1) / p.min_tiles;
  const int C = want < (long long)gridDim.x ? (int)want : (int)gridDim.x;
  const int cta = blockIdx.x;
  if (cta >= C) return;
  const long long t0 = cta * L.total / C, t1 = (cta + 1) * L.total / C;

  bool waited = false;
  for (long long seg = t0; seg < t1;) {
    const Item it = item_at(p, L, seg);
    const long long seg_end = it.end < t1 ? it.end : t1;
    const int T = it.T, b = it.b, g = it.g;
    const int tile0 = (int)(seg - it.first), ntile = (int)(seg_end - seg);
    const int mine = ntile > warp ? (ntile - warp + kWarps - 1) / kWarps : 0;  // tiles of this warp
    const long long cap = p.cap[b], cap_s = (cap + 3) & ~3ll;
    const uint8_t* Kc = p.K[b] + (long long)g * cap * (HD / 2);
    const uint8_t* Vc = p.V[b] + (long long)g * cap * (HD / 2);
    const uint8_t* Ksc = reinterpret_cast<const uint8_t*>(p.Ks[b] + (long long)g * cap_s * NB);
    const uint8_t* Vsc = reinterpret_cast<const uint8_t*>(p.Vs[b] + (long long)g * cap_s * NB);

    // rows [32 k, min(32 k + 32, T)) of tile k = tile0 + warp + 8 i into ring stage i % S
    auto fetch = [&](int i) {
      if (i < mine) {
        const int r0 = (tile0 + warp + kWarps * i) * kTile;
        const int rows = T - r0 < kTile ? T - r0 : kTile;  // cached rows of the tile (0: only the new row)
        const uint32_t st = ring_a + (i % S) * Sh::kStage;
#pragma unroll
        for (int u = 0; u < kTile * NB / 32; ++u) {
          const int id = u * 32 + lane, r = id / NB, c = id % NB;
          const bool in = r < rows;
          const long long off = in ? (long long)r0 * (HD / 2) + id * 16 : 0;
          cp16(st + place<NB>(r, c), Kc + off, in ? 16 : 0);
          cp16(st + Sh::kCodes + Sh::kScales + place<NB>(r, c), Vc + off, in ? 16 : 0);
        }
        constexpr int NS = Sh::kScales / 16;
        const int valid = rows * NB * 2;  // bytes
#pragma unroll
        for (int u = 0; u < (2 * NS + 31) / 32; ++u) {
          const int id = u * 32 + lane;
          if (id < 2 * NS) {
            const int kv = id / NS, c = id % NS;
            const int left = valid - c * 16;
            const int bytes = left <= 0 ? 0 : (left < 16 ? left : 16);
            const uint8_t* src = (kv ? Vsc : Ksc) + (bytes ? (long long)r0 * NB * 2 + c * 16 : 0);
            cp16(st + kv * (Sh::kCodes + Sh::kScales) + Sh::kCodes + c * 16, src, bytes);
          }
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);

    if (!waited) {
      pdl_wait();
      pdl_launch_dependents();
      waited = true;
    }
    // ---------------------------------------------------- queries and the new row
    const float* y = p.y + (long long)b * p.ld_y;
    const float2* rope = p.rope + (long long)T * (HD / 2);
    const bool has_new = seg_end == it.end;
    if (warp < G) {  // one warp per head: rotated, normalised to a power of two, split
      const float* qh = y + (long long)(g * G + warp) * HD;
      constexpr int PL = HD / 64;  // pairs per lane
      float x0[PL], x1[PL], amax = 0.f;
#pragma unroll
      for (int u = 0; u < PL; ++u) {
        const int i = u * 32 + lane;
        rotate(qh[i], qh[i + HD / 2], rope[i], &x0[u], &x1[u]);
        x0[u] *= p.scale_log2e;
        x1[u] *= p.scale_log2e;
        amax = fmaxf(amax, fmaxf(fabsf(x0[u]), fabsf(x1[u])));
      }
      amax = warp_max(amax);
      // 2^e amax in [2^9, 2^10): q as two fp16 parts keeps 22 bits of the head's largest value
      int e = 0;
      if (amax > 0.f && amax < INFINITY) e = 9 - ilogbf(amax);
      e = e > 100 ? 100 : e;
      float sum[2 * PL];
#pragma unroll
      for (int u = 0; u < 2 * PL; ++u) {
        const int el = (u < PL ? u : u - PL) * 32 + lane + (u < PL ? 0 : HD / 2);  // element of the head
        const float v = scalbnf(u < PL ? x0[u] : x1[u - PL], e);
        const __half h = __float2half_rn(v);
        const float hf = __half2float(h);
        const __half l = __float2half_rn(v - hf);
        // operand place of element el: block c, word w (4 codes of each half of a block), byte j, half k
        const int c = el >> 5, i = el & 31, k16 = i >> 4, w = (i & 15) >> 2, j = i & 3;
        // code j of a word meets half (j >> 1) of register (j & 1 ? a2 : a0) of k-step k16
        __half* f = reinterpret_cast<__half*>(qfrag);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const int hm = (G == 8 ? m : (m & 3)) % G;
          if (hm != warp) continue;
          const int base = (((c * 2 + k16) * 32 + m * 4 + w) * 4 + (j & 1) * 2) * 2 + (j >> 1);
          f[base] = h;
          f[base + 2] = l;
        }
        // stored codes reach the MMA as code + 24 or (high nibble of an even byte) code + 72
        const float bias = (k16 == 1 && (j & 1) == 0) ? 72.f : 24.f;
        sum[u] = bias * (hf + __half2float(l));
      }
#pragma unroll
      for (int u = 0; u < 2 * PL; ++u) {  // a block is one u: 32 lanes
        const float t = warp_sum(sum[u]);
        const int c = u < PL ? u : u - PL + NB / 2;
        if (lane == 0) sm.qb[c][warp] = -t;
      }
      if (lane == 0) sm.qf[warp] = scalbnf(1.0f, -e);
    }
    if (has_new) {
      const float* kh = y + (long long)(p.nq + g) * HD;
      const float* vh = y + (long long)(p.nq + p.nkv + g) * HD;
      if (tid < HD / 2) rotate(kh[tid], kh[tid + HD / 2], rope[tid], &sm.nk[tid], &sm.nk[tid + HD / 2]);
      if (tid < HD) sm.nv[tid] = vh[tid];
      __syncthreads();
      for (int u = warp; u < 2 * NB; u += kWarps) {  // block u % NB of K (u < NB) or V
        const int kv = u / NB, c = u % NB;
        int code;
        const uint16_t s = quant_block((kv ? sm.nv : sm.nk)[c * 32 + lane], &code);
        store_block(s, code, sm.codes[kv] + c * 16, &sm.scales[kv][c],
                    p.kv_new ? p.kv_new + (((long long)b * 2 + kv) * p.nkv + g) * HD + c * 32 : nullptr, lane);
        __syncwarp();
        uint8_t* gc = (kv ? p.V[b] : p.K[b]) + ((long long)g * cap + T) * (HD / 2) + c * 16;
        if (lane < 4) reinterpret_cast<uint32_t*>(gc)[lane] = reinterpret_cast<const uint32_t*>(sm.codes[kv] + c * 16)[lane];
        if (lane == 4) (kv ? p.Vs[b] : p.Ks[b])[((long long)g * cap_s + T) * NB + c] = s;
      }
    }
    __syncthreads();

    // ---------------------------------------------------- the warp's tiles
    float acc[NB][2][4];
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[c][t][k] = 0.f;
    float mx = -INFINITY, ref = -INFINITY, lsum = 0.f;
    int sh = 29;  // probabilities are held as 2^sh p: p sV then fills fp16's range from above
    const float qf = sm.qf[head];
    float qb[NB];
#pragma unroll
    for (int c = 0; c < NB; ++c) qb[c] = sm.qb[c][head];

    for (int i = 0; i < mine; ++i) {
      fetch(i + S - 1);
      cp_wait<S - 1>();
      __syncwarp();
      const int r0 = (tile0 + warp + kWarps * i) * kTile;
      uint8_t* stp = ring + (i % S) * Sh::kStage;
      const uint32_t st = ring_a + (i % S) * Sh::kStage;
      const uint32_t vst = st + Sh::kCodes + Sh::kScales;
      const int valid = T + 1 - r0;  // rows of the tile that exist
      if (valid <= kTile) {          // the last tile: the new row's codes and scales are its last row
        const int r = valid - 1;
        if (lane < 2 * NB) {
          const int kv = lane / NB, c = lane % NB;
          uint8_t* d = stp + kv * (Sh::kCodes + Sh::kScales);
          *reinterpret_cast<uint4*>(d + place<NB>(r, c)) = *reinterpret_cast<const uint4*>(sm.codes[kv] + c * 16);
          *reinterpret_cast<uint16_t*>(d + Sh::kCodes + (r * NB + c) * 2) = sm.scales[kv][c];
        }
        __syncwarp();
      }
      // largest V scale of the tile (as fp16 bits: scales are not negative, a sign is masked)
      uint32_t vmax = 0;
#pragma unroll
      for (int u = 0; u < NB / 2; ++u) {
        const uint32_t w = lds32(vst + Sh::kCodes + (u * 32 + lane) * 4);
        vmax = max(vmax, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
      }
      vmax = __reduce_max_sync(0xffffffffu, vmax);

      // scores: heads x 8 rows per MMA, two blocks' scales at a time
      float s[4][2];
#pragma unroll
      for (int n = 0; n < 4; ++n) s[n][0] = s[n][1] = 0.f;
#pragma unroll
      for (int cp = 0; cp < NB / 2; ++cp) {
        uint32_t sc[4][2];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) sc[n][k] = lds32(st + Sh::kCodes + ((n * 8 + quad * 2 + k) * NB + cp * 2) * 2);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = cp * 2 + half;
          uint32_t w[4];
          ldsm4(w, st + place<NB>(lane, c));
          const uint4 a0 = *reinterpret_cast<const uint4*>(qfrag + ((c * 2 + 0) * 32 + lane) * 4);
          const uint4 a1 = *reinterpret_cast<const uint4*>(qfrag + ((c * 2 + 1) * 32 + lane) * 4);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            // 16 + n or 64 + n in fp16 from each nibble n = code + 8
            const uint32_t h0 = and_or(w[n] << 6, 0x03c003c0u, 0x4c004c00u);
            const uint32_t h1 = and_or(w[n], 0x00f000f0u, 0x54005400u);
            const uint32_t h2 = and_or(w[n] >> 2, 0x03c003c0u, 0x4c004c00u);
            const uint32_t h3 = and_or(w[n] >> 6, 0x03c003c0u, 0x4c004c00u);
            float d[4] = {qb[c], qb[c], 0.f, 0.f};
            mma(d, a0.x, a0.y, a0.z, a0.w, h0, h2);
            mma(d, a1.x, a1.y, a1.z, a1.w, h1, h3);
            s[n][0] = fmaf(half ? hi_f(sc[n][0]) : lo_f(sc[n][0]), d[0] + d[2], s[n][0]);
            s[n][1] = fmaf(half ? hi_f(sc[n][1]) : lo_f(sc[n][1]), d[1] + d[3], s[n][1]);
          }
        }
      }
      float tm = -INFINITY;
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          s[n][k] *= qf;
          if (n * 8 + quad * 2 + k >= valid) s[n][k] = -INFINITY;
          tm = fmaxf(tm, s[n][k]);
        }
      tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 1));
      tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 2));
      mx = fmaxf(mx, tm);
      // sV < 2^(E - 14) with E the exponent field of the largest, so 2^sh p sV <= 2^15
      const int fit = 29 - (int)(vmax >> 10);
      sh = fit < sh ? fit : sh;
      const float nref = mx - (float)sh;
      if (__any_sync(0xffffffffu, nref != ref)) {
        const float corr = ex2(ref - nref);
        lsum *= corr;
        const float c0 = __shfl_sync(0xffffffffu, corr, quad * 8), c1 = __shfl_sync(0xffffffffu, corr, quad * 8 + 4);
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            acc[c][t][0] *= c0;
            acc[c][t][1] *= c1;
            acc[c][t][2] *= c0;
            acc[c][t][3] *= c1;
          }
        ref = nref;
      }
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          s[n][k] = ex2(s[n][k] - ref);
          lsum += s[n][k];
        }
      // outputs
#pragma unroll
      for (int cp = 0; cp < NB / 2; ++cp) {
        uint32_t sc[4][2];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) sc[n][k] = lds32(vst + Sh::kCodes + ((n * 8 + quad * 2 + k) * NB + cp * 2) * 2);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = cp * 2 + half;
          uint32_t w[4];
          ldsm4t(w, vst + place<NB>(lane, c));
          uint32_t ph[4], pl[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float v0 = s[n][0] * (half ? hi_f(sc[n][0]) : lo_f(sc[n][0]));
            const float v1 = s[n][1] * (half ? hi_f(sc[n][1]) : lo_f(sc[n][1]));
            ph[n] = h2u(__floats2half2_rn(v0, v1));
            pl[n] = h2u(__floats2half2_rn(v0 - lo_f(ph[n]), v1 - hi_f(ph[n])));
            if (G <= 4 && row8 >= 4) ph[n] = pl[n];  // columns 4..7 carry the low parts
          }
          uint32_t v[4][4];  // codes of 8 rows: elements 2 c', 2 c' + 16, 2 c' + 1, 2 c' + 17 of the block
          const __half2 k1032 = u2h(0x64086408u), k16th = u2h(0x2c002c00u), k72 = u2h(0xd480d480u);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const uint32_t w8 = w[n] >> 8;
            v[n][0] = h2u(__hsub2(u2h(and_or(w[n], 0x000f000fu, 0x64006400u)), k1032));
            v[n][1] = h2u(__hfma2(u2h(and_or(w[n], 0x00f000f0u, 0x64006400u)), k16th, k72));
            v[n][2] = h2u(__hsub2(u2h(and_or(w8, 0x000f000fu, 0x64006400u)), k1032));
            v[n][3] = h2u(__hfma2(u2h(and_or(w8, 0x00f000f0u, 0x64006400u)), k16th, k72));
          }
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            const int n = kt * 2;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              mma(acc[c][t], v[n][t], v[n][t + 2], v[n + 1][t], v[n + 1][t + 2], ph[n], ph[n + 1]);
              if (G == 8) mma(acc[c][t], v[n][t], v[n][t + 2], v[n + 1][t], v[n + 1][t + 2], pl[n], pl[n + 1]);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage before it is fetched into again
    }
    cp_wait<0>();
    __syncwarp();

    // ---------------------------------------------------- join the warps
    lsum += __shfl_xor_sync(0xffffffffu, lsum, 1);
    lsum += __shfl_xor_sync(0xffffffffu, lsum, 2);
    if (quad == 0 && row8 < G) {
      sm.r[warp][row8] = ref;
      sm.l[warp][row8] = lsum;
    }
    float* ow = reinterpret_cast<float*>(ring);  // [G][HD] of this warp, in its own ring
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float a[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k] = acc[c][t][k];
          if (G <= 4) a[k] += __shfl_xor_sync(0xffffffffu, a[k], 2);  // low parts: columns 4..7
        }
        const int e = c * 32 + t * 16 + row8 * 2, j = quad * 2;
        if (j < G) *reinterpret_cast<float2*>(ow + j * HD + e) = make_float2(a[0], a[2]);
        if (j + 1 < G) *reinterpret_cast<float2*>(ow + (j + 1) * HD + e) = make_float2(a[1], a[3]);
      }
    __syncthreads();
    const int c_lo = (int)(((it.first + 1) * C - 1) / L.total), c_hi = (int)((it.end * C - 1) / L.total);
    const int np = c_hi - c_lo + 1;  // CTAs that share the item
    float* o = p.o + (long long)b * p.ld_o + (long long)g * G * HD;
    constexpr int PF = G * (HD + 2);
    float* part = p.part + (2ll * cta + (seg == t0 ? 0 : 1)) * PF;
    for (int e = tid; e < G * HD; e += kThreads) {
      const int j = e / HD;
      float R = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) R = fmaxf(R, sm.r[w][j]);
      float num = 0.f, den = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(sm.r[w][j] - R);
        num = fmaf(f, reinterpret_cast<const float*>(smem + w * (S * Sh::kStage))[e], num);
        den = fmaf(f, sm.l[w][j], den);
      }
      if (np == 1) {
        o[e] = num / den;
      } else {
        part[e] = num;
        if (e % HD == 0) {
          part[G * HD + j] = R;
          part[G * HD + G + j] = den;
        }
      }
    }
    __syncthreads();
    // ---------------------------------------------------- join the CTAs
    if (np > 1) {
      if (tid == 0) {
        __threadfence();
        unsigned* ctr = p.counter + b * p.nkv + g;
        const unsigned old = atomicAdd(ctr, 1u);
        const int last = old == (unsigned)(np - 1);
        if (last) *ctr = 0;  // zero between launches
        __threadfence();
        sm.last = last;
      }
      __syncthreads();
      if (sm.last) {
        float* wt = reinterpret_cast<float*>(smem);  // [np][G] weights, then the joined 1 / l per head
        const int slot0 = (c_lo * L.total / C != it.first) ? 1 : 0;  // the first sharer's span began before the item
        auto part_of = [&](int i) { return p.part + (2ll * (c_lo + i) + (i == 0 ? slot0 : 0)) * PF; };
        if (warp < G) {
          const int j = warp;
          float R = -INFINITY, den = 0.f;
          for (int i = lane; i < np; i += 32) R = fmaxf(R, __ldcg(part_of(i) + G * HD + j));
          R = warp_max(R);
          for (int i = lane; i < np; i += 32) {
            const float* q = part_of(i) + G * HD;
            const float f = ex2(__ldcg(q + j) - R);
            wt[i * G + j] = f;
            den = fmaf(f, __ldcg(q + G + j), den);
          }
          den = warp_sum(den);
          if (lane == 0) wt[np * G + j] = 1.0f / den;
        }
        __syncthreads();
        for (int e = tid; e < G * HD; e += kThreads) {
          const int j = e / HD;
          float num = 0.f;
#pragma unroll 8
          for (int i = 0; i < np; ++i) num = fmaf(wt[i * G + j], __ldcg(part_of(i) + e), num);
          o[e] = num * wt[np * G + j];
        }
      }
      __syncthreads();
    }
    seg = seg_end;
  }
}

// ------------------------------------------------------------ append
// Rows of n tokens at positions T .. T + n - 1 of one sequence: a warp takes
// blocks c and c + NB / 2 of one k or v vector (for k they hold the halves of
// the rotate-half pairs), a value of each per lane.
template <int HD>
__global__ void __launch_bounds__(256) k_append(const AppendParams p) {
  constexpr int NB = HD / 32, NH = NB / 2;
  const int lane = threadIdx.x & 31;
  const int T = *p.len;
  if (T < 0 || (long long)T + p.n > p.cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_guard(p.guard, kGuardBadPosition);
    return;
  }
  const long long cap_s = ((long long)p.cap + 3) & ~3ll;
  const long long units = (long long)p.n * 2 * p.nkv * NH;
  const long long step = (long long)gridDim.x * (blockDim.x >> 5);
  for (long long u = blockIdx.x * (long long)(blockDim.x >> 5) + (threadIdx.x >> 5); u < units; u += step) {
    const int c = (int)(u % NH);
    const int g = (int)(u / NH % p.nkv);
    const int kv = (int)(u / NH / p.nkv % 2);
    const long long i = u / NH / p.nkv / 2;
    const float* x = p.y + i * p.ld_y + (long long)(p.nq + kv * p.nkv + g) * HD + c * 32 + lane;
    float x0 = x[0], x1 = x[HD / 2];
    if (kv == 0) {
      const float2 cs = p.rope[(T + i) * (HD / 2) + c * 32 + lane];
      float r0, r1;
      rotate(x0, x1, cs, &r0, &r1);
      x0 = r0;
      x1 = r1;
    }
    uint8_t* codes = (kv ? p.V : p.K) + ((long long)g * p.cap + T + i) * (HD / 2);
    uint16_t* scales = (kv ? p.Vs : p.Ks) + ((long long)g * cap_s + T + i) * NB;
    float* val = p.kv_new ? p.kv_new + ((i * 2 + kv) * p.nkv + g) * HD : nullptr;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int cc = c + h * NH;
      int code;
      const uint16_t s = quant_block(h ? x1 : x0, &code);
      store_block(s, code, codes + cc * 16, scales + cc, val ? val + cc * 32 : nullptr, lane);
    }
  }
}

using Kern = void (*)(Params);

template <int HD>
Kern pick_g(int G) {
  return G == 1 ? k_attn<HD, 1> : G == 2 ? k_attn<HD, 2> : G == 4 ? k_attn<HD, 4> : G == 8 ? k_attn<HD, 8> : nullptr;
}
Kern pick(int hd, int G, size_t* smem, int* per_sm) {
  *smem = hd == 64 ? smem_bytes<64>() : hd == 128 ? smem_bytes<128>() : smem_bytes<256>();
  *per_sm = hd == 64 ? Shape<64>::kMinCtas : hd == 128 ? Shape<128>::kMinCtas : Shape<256>::kMinCtas;
  return hd == 64 ? pick_g<64>(G) : hd == 128 ? pick_g<128>(G) : hd == 256 ? pick_g<256>(G) : nullptr;
}

}  // namespace

int max_ctas(int hd, int nsm) { return nsm * (hd == 256 ? Shape<256>::kMinCtas : Shape<64>::kMinCtas); }

size_t part_floats(int nq, int nkv, int hd, int nsm) { return (size_t)2 * max_ctas(hd, nsm) * (nq / nkv) * (hd + 2); }

cudaError_t init() {
  for (int hd : {64, 128, 256})
    for (int G : {1, 2, 4, 8}) {
      size_t smem = 0;
      int per_sm = 0;
      Kern k = pick(hd, G, &smem, &per_sm);
      const cudaError_t e = cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

cudaError_t launch(const Params& p, int hd, int nsm, cudaStream_t st, bool pdl) {
  if (p.nb < 1 || p.nb > kMaxB || p.nkv <= 0 || p.nq % p.nkv) return cudaErrorInvalidValue;
  size_t smem = 0;
  int per_sm = 0;
  Kern k = pick(hd, p.nq / p.nkv, &smem, &per_sm);
  if (!k) return cudaErrorInvalidValue;
  Params q = p;
  q.min_tiles = kWarps;
  long long tiles = 0;  // the most the list can hold
  for (int b = 0; b < p.nb; ++b) tiles += (long long)p.nkv * ((p.cap[b] - 1) / kTile + 1);
  long long grid = (tiles + q.min_tiles - 1) / q.min_tiles;
  if (grid > max_ctas(hd, nsm)) grid = max_ctas(hd, nsm);
  return launch_k(k, dim3((unsigned)grid), dim3(kThreads), smem, st, pdl, q);
}

cudaError_t append(const AppendParams& p, int hd, cudaStream_t st) {
  if (p.n <= 0) return cudaSuccess;
  const long long units = (long long)p.n * 2 * p.nkv * (hd / 64);
  long long blocks = (units + 7) / 8;
  if (blocks > 4096) blocks = 4096;
  switch (hd) {
    case 64: k_append<64><<<(unsigned)blocks, 256, 0, st>>>(p); break;
    case 128: k_append<128><<<(unsigned)blocks, 256, 0, st>>>(p); break;
    case 256: k_append<256><<<(unsigned)blocks, 256, 0, st>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace kv4
}  // namespace hy
