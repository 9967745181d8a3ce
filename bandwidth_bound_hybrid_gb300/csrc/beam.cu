// Beam search on sm_103a: selection over the beams and the vocabulary, and
// the reordering of the beams' states.
//
// Selection.  Candidate (w, v) of a group of beams scores
//   s(w, v) = score_w + x_wv - lse_w,  lse_w = log sum_v exp(x_wv),
// and the group's best `picks` are wanted, ties to the lowest w V + v.  Within
// a beam the order is that of the logits, so one pass over the logits is
// enough.  A CTA takes a chunk of a beam's row and streams through it with a
// running maximum and sum of exponentials per lane.  The picks-th largest of
// the CTA's 256 running maxima is a bound that `picks` logits are known to
// reach; it is worked out after 1, 4, 16, 64, ... steps (a bitonic network across
// the lanes of each warp, then merges of the 8 lists), so that between two of
// these a few times `picks` logits reach it.  Those few are kept, by each warp
// on its own: 32 at a time are sorted and merged into the warp's best 32, a
// lane each.  So the pass costs an exponential and a comparison a logit, and is
// bound by reading the logits.
//
// The CTA leaves the chunk's maximum, sum and best `picks`; the last CTA of the
// group turns maxima and sums into lse_w (the sums and the log of the mantissa
// in FP32, the rest in FP64, as the scores are: a lane's sum errs by at most
// 2^-21 a step of 16 logits, the rest of lse_w by 2^-17 together) and selects
// among the chunks' lists by the same kind of bound, from the lists' heads.
// Measured: 64 groups of 8 beams x 151936, 16 picks, 40 beams ended, in 58.5 us
// (4.9 TB/s), one group of 4 in 10.6 us.  The filter is made for logits that
// differ: where the bound is a value that most of a row has (a flat row; a mask
// of the type's lowest value, until as many lanes as picks have met an allowed
// token), every logit passes it, and 64 x 8 rows take up to 0.84 ms, one group
// of 4 up to 65 us.  A mask of -infinity costs 10%.
//
// Reordering.  State i of a group becomes what state parent[i] was, in place:
// a thread owns 16-byte columns of all the group's states, reads the sources
// of those that change, and only then writes.  So no second copy of the states
// is kept.  Bound by the bytes of the states that change: 2 x 8 states of 25
// MB, 4 of them moved, in 34.7 us (5.8 TB/s), 7 in 51.4 (6.4), 11 in 73.8 (6.5).
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace hy {
namespace beam {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 4;                 // CTAs of the selection per SM
constexpr int kPer = 16;                 // logits of a lane at a time
constexpr int kStep = kPer * 32;         // and of a warp
constexpr int kFew = 4;                  // words of a thread in the final selection of few lists
constexpr int kQual = 1024;              // lists looked into by the fast final selection
constexpr int kMoves = 64;               // CTAs of the reordering per SM, at most
constexpr int kBest = 2048;              // and their candidates

// Sums of exponentials are held as S = sum 2^(x log2 e - c(M)) with the largest x
// = M and c(M) the FP32 product M log2 e: one fused multiply-add, one ex2 and one
// addition a logit, and the product's rounding is part of the reference and
// cancels.  From 2^30 on the rounding leaves ex2's range; FP32 numbers of that
// size are 64 apart or equal, so S then counts the x that equal M.
constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ bool large(float M) { return !(fabsf(M) < 0x1p30f); }
// what a sum with reference Ma counts for beside Mb >= Ma
__device__ __forceinline__ float carry(float Ma, float Mb) {
  return Ma == Mb ? 1.f : large(Ma) || large(Mb) ? 0.f : ex2(__fmul_rn(Ma, kLog2e) - __fmul_rn(Mb, kLog2e));
}

// A candidate of a chunk in one word: the logit's order key above the
// complement of the token, so that the larger word is the better candidate
// and no two are equal.  0: none.
__device__ __forceinline__ uint64_t word_of(uint32_t key, uint32_t token) {
  return ((uint64_t)key << 32) | (0xffffffffu - token);
}
__device__ __forceinline__ float word_logit(uint64_t c) { return key_value((uint32_t)(c >> 32)); }
__device__ __forceinline__ uint32_t word_token(uint64_t c) { return 0xffffffffu - (uint32_t)c; }

// The lanes' keys sorted across the warp by a bitonic network, largest in lane 0.
__device__ __forceinline__ uint32_t warp_sort32(uint32_t v, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, v, j);
      const bool larger = ((lane & k) == 0) == ((lane & j) == 0);  // what this lane keeps of the pair
      v = larger ? max(v, o) : min(v, o);
    }
  }
  return v;
}
// The n-th largest (n in 1..32) of all the CTA's keys: the warps' sorted lists merged, by every warp for itself (as a
// tree, a chain of 15 exchanges: 0.4 us less than one list after the other).
__device__ __forceinline__ uint32_t cta_nth(uint32_t (*sorted)[32], uint32_t v, int n, int lane, int warp) {
  sorted[warp][lane] = warp_sort32(v, lane);
  __syncthreads();
  // best 32 of lists 2 i and 2 i + 1, of those of two such, ...: the second of a pair the other way round
  uint32_t best[kWarps / 2];
#pragma unroll
  for (int i = 0; i < kWarps / 2; ++i) best[i] = max(sorted[2 * i][lane], sorted[2 * i + 1][31 - lane]);
#pragma unroll
  for (int w = kWarps / 2; w > 0; w >>= 1) {
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) {
#pragma unroll
      for (int i = 0; i < w; ++i) {
        const uint32_t o = __shfl_xor_sync(0xffffffffu, best[i], j);
        best[i] = ((lane & j) == 0) == ((i & 1) == 0) ? max(best[i], o) : min(best[i], o);
      }
    }
#pragma unroll
    for (int i = 0; i < w / 2; ++i) best[i] = max(best[2 * i], best[2 * i + 1]);
  }
  return __shfl_sync(0xffffffffu, best[0], n - 1);
}

// Sorted across the warp, largest in lane 0: a step of a bitonic network, the
// last log2 steps of it (the lanes' words a bitonic sequence), and all of it.
__device__ __forceinline__ uint64_t keep(uint64_t x, int j, bool larger) {
  const uint64_t o = __shfl_xor_sync(0xffffffffu, (unsigned long long)x, j);
  return (o > x) == larger ? o : x;
}
__device__ __forceinline__ uint64_t warp_merge(uint64_t x, int lane) {
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) x = keep(x, j, (lane & j) == 0);
  return x;
}
__device__ __forceinline__ uint64_t warp_sort(uint64_t x, int lane) {
#pragma unroll
  for (int k = 2; k < 32; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) x = keep(x, j, ((lane & k) == 0) == ((lane & j) == 0));
  }
  return warp_merge(x, lane);
}
// The best 32 of two sorted lists, sorted (`other` in reverse: lane 31 its largest).
__device__ __forceinline__ uint64_t warp_join(uint64_t top, uint64_t other, int lane) {
  return warp_merge(top > other ? top : other, lane);
}

// A candidate of the group: its FP64 score as an order key (0: none; integer
// compares, since FP64 ones are slow here) and flat index w V + v.
struct Cand {
  uint64_t key;
  uint32_t i;
};
__device__ __forceinline__ Cand cand_of(double s, uint32_t i) {
  if (!(s >= -(double)FLT_MAX)) return {0, 0xffffffffu};  // the FP32 score is -infinity
  const uint64_t b = (uint64_t)__double_as_longlong(s + 0.0);  // (-0 as +0)
  return {(b >> 63) ? ~b : b | (1ull << 63), i};
}
__device__ __forceinline__ double cand_score(const Cand& c) {
  if (c.key == 0) return -INFINITY;
  return __longlong_as_double((long long)((c.key >> 63) ? c.key & ~(1ull << 63) : ~c.key));
}
__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
  return a.key > b.key || (a.key == b.key && a.i < b.i);
}

struct Shared {
  union {
    struct {
      uint64_t buf[kWarps][64];        // candidates on their way into the warp's best
      uint64_t list[kWarps][32];       // the warps' best
    } w;
    struct {
      uint64_t key[kBest];             // the group's candidates
      uint32_t i[kBest];
      uint32_t qual[kQual];
    } best;
    uint8_t at[kMaxLists];             // one by one: the next candidate of every list
  };
  uint32_t sorted[2][kWarps][32];      // running maxima of the warps' lanes
  float m[kWarps], sum[kWarps];
  double off[kMaxBeams];               // score_w - lse_w, or score_w of a done beam (-infinity: nothing counts)
  int done[kMaxBeams];
  Cand sel[kMaxPicks], top[kWarps];
  int n, nq, last;
};

__global__ void __launch_bounds__(kThreads, kCtas) k_select(const SelectParams p) {
  __shared__ Shared sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nch = p.chunks, row = blockIdx.x / nch, chunk = blockIdx.x % nch, group = row / p.beams;
  const int P = p.picks, V = p.vocab;
  if (!(p.done && p.done[row])) {
    // ------------------------------------------------------ the chunk
    const float* x = p.logits + (long long)row * p.ld;
    const long long first = (long long)chunk * p.span;
    const int end = (int)(first + p.span < V ? first + p.span : V);
    uint64_t* buf = sm.w.buf[warp];
    uint64_t top = 0;  // 0: none
    int nb = 0;        // words in the buffer
    float M = -INFINITY, s = 0.f;
    auto flush = [&]() {  // the buffer's first 32 words into the best, the others to its front
      __syncwarp();
      const uint64_t w = lane < nb ? buf[lane] : 0, rest = buf[32 + lane];
      __syncwarp();
      buf[lane] = rest;
      __syncwarp();
      nb = nb > 32 ? nb - 32 : 0;
      top = warp_join(top, __shfl_sync(0xffffffffu, (unsigned long long)warp_sort(w, lane), 31 - lane), lane);
    };
    float low = -FLT_MAX;  // -infinity is no candidate
    int due = 1, turn = 0;
    const int steps = (int)((end - first + kWarps * kStep - 1) / (kWarps * kStep));
    float v[kPer], next[kPer];  // a step's logits; the next step's are on their way meanwhile
    auto load = [&](int it, float* d) {
      const int i0 = (int)first + (it * kWarps + warp) * kStep;
      const float* q = x + i0 + lane;
      if (i0 + kStep <= end) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) d[k] = __ldcs(q + k * 32);
      } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) d[k] = i0 + k * 32 + lane < end ? __ldcs(q + k * 32) : -INFINITY;
      }
    };
    load(0, next);
    for (int it = 0; it < steps; ++it) {
      const int i0 = (int)first + (it * kWarps + warp) * kStep + lane;
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[k] = next[k];
      if (it + 1 < steps) load(it + 1, next);
      float m = v[0];
#pragma unroll
      for (int k = 1; k < kPer; ++k) m = fmaxf(m, v[k]);
      m = fmaxf(m, -INFINITY);
      const float Mn = fmaxf(M, m), c = __fmul_rn(Mn, kLog2e);
      float add = 0.f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) add += ex2(fmaf(v[k], kLog2e, -c));
      if (!(add <= FLT_MAX) || large(Mn)) {  // a NaN, which counts as -infinity, or large logits
        add = 0.f;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          if (large(Mn))
            add += v[k] == Mn && Mn > -INFINITY ? 1.f : 0.f;
          else
            add += ex2(fmaf(fmaxf(v[k], -INFINITY), kLog2e, -c));
        }
      }
      s = s * carry(M, Mn) + add;
      M = Mn;
      if (it + 1 == due && (it == 0 || due < steps)) {  // 1, 4, 16, ... steps done
        due *= 4;
        low = fmaxf(low, key_value(cta_nth(sm.sorted[turn ^= 1], order_key(M), P, lane, warp)));
      }
      if (__any_sync(0xffffffffu, m >= low)) {
        uint32_t hit = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) hit |= v[k] >= low ? 1u << k : 0u;
        for (unsigned in; (in = __ballot_sync(0xffffffffu, hit != 0)) != 0; hit &= hit - 1) {
          if (hit) {
            const int i = i0 + (__ffs(hit) - 1) * 32;
            buf[nb + __popc(in & ((1u << lane) - 1))] = word_of(order_key(x[i]), i);
          }
          nb += __popc(in);
          if (nb >= 32) flush();
        }
      }
    }
    flush();
    // the warps' lists, maxima and sums
    const float Mw = warp_max(M);
    const float sw = warp_sum(s * carry(M, Mw));
    if (lane == 0) {
      sm.m[warp] = Mw;
      sm.sum[warp] = sw;
    }
    sm.w.list[warp][lane] = top;
#pragma unroll
    for (int half = kWarps / 2; half > 0; half >>= 1) {
      __syncthreads();
      if (warp < half) sm.w.list[warp][lane] = top = warp_join(top, sm.w.list[warp + half][31 - lane], lane);
    }
    const long long slot = (long long)row * nch + chunk;
    if (warp == 0 && lane < P) p.lists[slot * P + lane] = top;
    if (tid == 0) {
      float Mc = sm.m[0], S = 0.f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) Mc = fmaxf(Mc, sm.m[w]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) S += sm.sum[w] * carry(sm.m[w], Mc);
      p.stats[slot] = make_float2(Mc, S);
    }
  }
  // -------------------------------------------------------- the last CTA of the group
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    const int last = atomicAdd(p.counter + group, 1u) == (unsigned)(p.beams * nch) - 1;
    if (last) p.counter[group] = 0;
    __threadfence();
    sm.last = last;
    sm.n = sm.nq = 0;
  }
  __syncthreads();
  if (!sm.last) return;
  const int row0 = group * p.beams, nl = p.beams * nch;
  const unsigned long long* lists = reinterpret_cast<const unsigned long long*>(p.lists) + (long long)row0 * nch * P;
  // up to kFew words a thread: all of the group's lists at once, on their way while lse is worked out
  const bool few = nl * P <= kFew * kThreads;
  uint64_t words[kFew];
#pragma unroll
  for (int k = 0; k < kFew; ++k) words[k] = few && tid + k * kThreads < nl * P ? __ldcg(lists + tid + k * kThreads) : 0;
  for (int w = warp; w < p.beams; w += kWarps) {  // lse and offset of every beam
    const int r = row0 + w;
    const float2* st = p.stats + (long long)r * nch;
    const float2 t0 = lane < nch ? __ldcg(st + lane) : make_float2(-INFINITY, 0.f);
    const int done = p.done ? p.done[r] != 0 : 0;
    double off = (double)p.score[r];
    if (!done) {
      float M = t0.x;
      for (int c = lane + 32; c < nch; c += 32) M = fmaxf(M, __ldcg(st + c).x);
      M = warp_max(M);
      // the sum as S + err, err the exact rest of every addition (FP64 ones are slow here)
      float S = lane < nch ? __fmul_rn(t0.y, carry(t0.x, M)) : 0.f, err = 0.f;
      auto add = [&](float b, float b_err) {
        const float sum = S + b, of_b = sum - S;
        err += b_err + ((S - (sum - of_b)) + (b - of_b));
        S = sum;
      };
      for (int c = lane + 32; c < nch; c += 32) {
        const float2 t = __ldcg(st + c);
        add(__fmul_rn(t.y, carry(t.x, M)), 0.f);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < nch) add(__shfl_xor_sync(0xffffffffu, S, o), __shfl_xor_sync(0xffffffffu, err, o));
      // log of S = 2^e f, f in [0.75, 1.5): the FP32 logarithm of f errs by 2^-25 at most, e log 2 is FP64
      const int e = (int)((__float_as_uint(S) + 0x00400000u) >> 23) - 127;
      const float f = __uint_as_float(__float_as_uint(S) - ((uint32_t)e << 23));
      const double log2 = 0.69314718055994530942;
      double top = (double)M;
      if (!large(M)) {
        // the reference's value; kLog2e = (1 - d) log2 e makes the sums those of exp((1 - d) x), which lacks d times
        // the mean of x (here: the largest)
        top = (double)__fmul_rn(M, kLog2e) * log2 + (1.0 - (double)kLog2e * log2) * (double)M;
      }
      off -= top + (double)e * log2 + (double)(logf(f) + err / S);
    }
    if (lane == 0) {
      sm.off[w] = off - off == 0.0 ? off : -INFINITY;
      sm.done[w] = done;
    }
  }
  __syncthreads();
  // candidate k of list l = (beam, chunk), its word given
  auto cand = [&](int l, int k, uint64_t word) {
    const int w = l / nch;
    const double off = sm.off[w];
    if (sm.done[w])  // a beam that has ended goes on as it is
      return l == w * nch && k == 0 ? cand_of(off, (uint32_t)w * V + p.eos) : Cand{0, 0xffffffffu};
    return word ? cand_of(off + (double)word_logit(word), (uint32_t)w * V + word_token(word)) : Cand{0, 0xffffffffu};
  };
  auto get = [&](int l, int k) { return cand(l, k, sm.done[l / nch] ? 0 : __ldcg(lists + (long long)l * P + k)); };
  auto keep_if = [&](const Cand& a, uint32_t bound) {
    if ((uint32_t)(a.key >> 32) < bound) return;
    const int at = atomicAdd(&sm.n, 1);
    if (at < kBest) {
      sm.best.key[at] = a.key;
      sm.best.i[at] = a.i;
    }
  };
  // a bound on the upper half of the keys that at least P candidates reach: the P-th largest of the threads'
  Cand mine[kFew];
  uint32_t top_key = 0;
  if (few) {
#pragma unroll
    for (int k = 0; k < kFew; ++k) {
      const int at = tid + k * kThreads;
      mine[k] = at < nl * P ? cand(at / P, at % P, words[k]) : Cand{0, 0xffffffffu};
      top_key = max(top_key, (uint32_t)(mine[k].key >> 32));
    }
  } else {
    for (int l = tid; l < nl; l += kThreads) top_key = max(top_key, (uint32_t)(get(l, 0).key >> 32));
  }
  const uint32_t bound = max(cta_nth(sm.sorted[0], top_key, P, lane, warp), 1u);
  if (few) {
#pragma unroll
    for (int k = 0; k < kFew; ++k) keep_if(mine[k], bound);
  } else {
    for (int l = tid; l < nl; l += kThreads)
      if ((uint32_t)(get(l, 0).key >> 32) >= bound) {
        const int q = atomicAdd(&sm.nq, 1);
        if (q < kQual) sm.best.qual[q] = l;
      }
    __syncthreads();
    for (int q = warp; q < min(sm.nq, kQual); q += kWarps)
      if (lane < P) keep_if(get(sm.best.qual[q], lane), bound);
  }
  __syncthreads();
  const int nq = sm.nq;
  int n = sm.n;
  if (nq <= kQual && n <= kThreads / 4) {  // a quad counts the better ones of a candidate
    const int a = tid / 4;
    Cand c = {0, 0xffffffffu};
    int rank = 0;
    if (a < n) {
      c = {sm.best.key[a], sm.best.i[a]};
#pragma unroll 4
      for (int b = tid % 4; b < n; b += 4) rank += better({sm.best.key[b], sm.best.i[b]}, c);
    }
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    rank += __shfl_xor_sync(0xffffffffu, rank, 2);
    if (a < n && tid % 4 == 0 && rank < P) sm.sel[rank] = c;
    if (n > P) n = P;
  } else if (nq <= kQual && n <= kBest) {
    for (int a = tid; a < n; a += kThreads) {
      const Cand c = {sm.best.key[a], sm.best.i[a]};
      int rank = 0;
      for (int b = 0; b < n && rank < P; ++b) rank += better({sm.best.key[b], sm.best.i[b]}, c);
      if (rank < P) sm.sel[rank] = c;
    }
    if (n > P) n = P;
  } else {
    // more near-equal candidates than the arrays hold (a flat row): the best of the lists' heads, one at a time
    __syncthreads();
    for (int l = tid; l < nl; l += kThreads) sm.at[l] = 0;
    for (n = 0; n < P; ++n) {
      Cand best = {0, 0xffffffffu};
      int from = -1;
      for (int l = tid; l < nl; l += kThreads) {
        if (sm.at[l] >= P) continue;
        const Cand a = get(l, sm.at[l]);
        if (better(a, best)) {
          best = a;
          from = l;
        }
      }
      Cand top = best;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const Cand a = {__shfl_xor_sync(0xffffffffu, (unsigned long long)top.key, o),
                        __shfl_xor_sync(0xffffffffu, top.i, o)};
        if (better(a, top)) top = a;
      }
      if (lane == 0) sm.top[warp] = top;
      __syncthreads();
      top = sm.top[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w)
        if (better(sm.top[w], top)) top = sm.top[w];
      if (top.key == 0) break;  // the same for every thread
      if (from >= 0 && best.i == top.i) ++sm.at[from];
      if (tid == 0) sm.sel[n] = top;
      __syncthreads();
    }
  }
  __syncthreads();
  // -------------------------------------------------------- outputs
  if (warp == 0) {
    // Fewer than P candidates have a probability: the others have score
    // -infinity and follow in index order; n of the first P indices at most
    // are taken, so what is left of those suffices.
    bool taken = false;
    for (int k = 0; k < n; ++k) taken |= sm.sel[k].i == (uint32_t)lane;
    const unsigned free = __ballot_sync(0xffffffffu, !taken && lane < P);
    const int before = __popc(free & ((1u << lane) - 1));
    if (!taken && lane < P && n + before < P) sm.sel[n + before] = {0, (uint32_t)lane};
    __syncwarp();
    if (lane < P) {
      const Cand c = sm.sel[lane];
      const int w = (int)(c.i / (uint32_t)V), token = (int)(c.i % (uint32_t)V);
      const long long at = (long long)group * P + lane;
      p.score_out[at] = (float)cand_score(c);
      p.parent[at] = w;
      p.token[at] = token;
      if (p.done_out) p.done_out[at] = (sm.done[w] || token == p.eos) ? 1 : 0;
    }
  }
}

// ------------------------------------------------------------ reordering
// The columns [x, end) (bytes, 16 each) of the n <= NM states that change, U
// columns of a thread at a time, so that about 8 loads are on their way: all
// are read before anything of these columns is written.
template <int NM, int U>
__device__ __forceinline__ void move(uint8_t* const* src, uint8_t* const* dst, int n, long long x, long long end) {
  for (x += threadIdx.x * 16; x < end; x += (long long)U * kThreads * 16) {
    uint4 v[U][NM];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NM; ++i)
        if (i < n && x + u * kThreads * 16 < end)
          v[u][i] = *reinterpret_cast<const uint4*>(src[i] + x + u * kThreads * 16);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NM; ++i)
        if (i < n && x + u * kThreads * 16 < end) *reinterpret_cast<uint4*>(dst[i] + x + u * kThreads * 16) = v[u][i];
  }
}

// A share of the columns of segment y of group z (or, paged, of segment y %
// n_seg in page first_page + y / n_seg).  B: at least as many beams.
template <int B>
__global__ void __launch_bounds__(kThreads) k_reorder(const ReorderParams p) {
  __shared__ uint8_t *s_src[B], *s_dst[B];
  __shared__ int s_n;
  const int tid = threadIdx.x, z = blockIdx.z;
  long long lo = 0, end = p.seg_bytes;
  int seg = blockIdx.y, page = 0;
  if (p.page_bytes) {  // rows [first_row, end_row) of the sequence that lie in this page
    page = p.first_page + seg / p.n_seg;
    seg %= p.n_seg;
    const int r0 = max(p.first_row - page * p.page_rows, 0), r1 = min(p.end_row - page * p.page_rows, p.page_rows);
    lo = (long long)r0 * p.row_bytes;
    end = (long long)r1 * p.row_bytes;
  }
  if (tid < 32) {  // the states that change
    int q = tid;
    if (tid < p.beams) {
      q = p.parent ? p.parent[(long long)z * p.beams + tid] : 0;
      if (q < 0 || q >= p.beams) {  // left as it is
        if (blockIdx.x == 0 && blockIdx.y == 0) set_guard(p.guard, kGuardBadIndex);
        q = tid;
      }
    }
    const unsigned moved = __ballot_sync(0xffffffffu, q != tid);
    if (q != tid) {
      auto at = [&](int i) {
        uint8_t* b = p.base[i] + z * p.group_stride + seg * p.seg_stride[i];
        return p.page_bytes ? b + p.pages[i][page] * p.page_bytes : b;
      };
      const int to = __popc(moved & ((1u << tid) - 1));
      s_src[to] = at(q);
      s_dst[to] = at(tid);
    }
    if (tid == 0) s_n = __popc(moved);
  }
  __syncthreads();
  const int n = s_n;
  long long x = lo + blockIdx.x * p.share;
  const long long x_end = min(x + p.share, end);
  if (p.skip && blockIdx.x == 0) {  // the first piece: its last words, a thread each
    if (tid < 4 && tid * 4 >= p.skip) {
      uint32_t v[B];
#pragma unroll
      for (int i = 0; i < B; ++i)
        if (i < n) v[i] = *reinterpret_cast<const uint32_t*>(s_src[i] + x + tid * 4);
#pragma unroll
      for (int i = 0; i < B; ++i)
        if (i < n) *reinterpret_cast<uint32_t*>(s_dst[i] + x + tid * 4) = v[i];
    }
    x += 16;
  }
  if (n <= 2) {
    if (n) move<2, 4>(s_src, s_dst, n, x, x_end);
  } else if (B == 4 || n <= 4) {
    move<4, 2>(s_src, s_dst, n, x, x_end);
  } else if (B == 8 || n <= 8) {
    move<8, 1>(s_src, s_dst, n, x, x_end);
  } else {
    move<16, 1>(s_src, s_dst, n, x, x_end);
  }
}

}  // namespace

int chunks(int vocab) { return (int)(((long long)vocab + kChunk - 1) / kChunk); }

// The split of a row.  A CTA of t tiles (of kChunk logits) costs about what t +
// 3.3 tiles take; a tile takes longer the more CTAs an SM holds, more steeply
// from two on, where the memory is busy (measured, in us: 0.65, 0.83, 1.12 and
// 1.41 for 1 to 4; rows of 38 tiles: 456 rows whole in 54 us, in four parts in
// 63; 304 rows whole in 42.5, halved in 40.2; 8 rows in 19 parts in 14.6, in 38
// in 17.2).  So: full waves of kCtas an SM and what the last one holds.
void set_span(SelectParams* p, int groups, int nsm) {
  const long long rows = (long long)groups * p->beams, n = chunks(p->vocab), slots = (long long)nsm * kCtas;
  auto tile = [](double k) { return std::max(0.47 + 0.18 * k, 0.25 + 0.29 * k); };
  double best = 0;
  for (long long c = 1; c <= n && c <= 4096; ++c) {
    const long long t = (n + c - 1) / c, parts = (n + t - 1) / t;
    const long long waves = (rows * parts - 1) / slots;  // before the last
    const double k = (double)(rows * parts - waves * slots) / nsm;
    const double cost = ((double)t + 3.3) * ((double)waves * tile(kCtas) + (tile(k) + tile(std::ceil(k))) / 2);
    if (c == 1 || cost < best) {
      best = cost;
      p->chunks = (int)parts;
      p->span = t * kChunk;
    }
  }
}

cudaError_t select(const SelectParams& p, int groups, cudaStream_t st) {
  const long long grid = (long long)groups * p.beams * p.chunks;
  if (grid <= 0 || grid > 0x7fffffffll || p.beams > kMaxBeams || p.picks < 1 || p.picks > kMaxPicks ||
      (long long)p.beams * p.chunks > kMaxLists)
    return cudaErrorInvalidValue;
  k_select<<<(unsigned)grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// A CTA takes one or two rows of kThreads columns, or a multiple of four (whole
// turns of every move<>) where that is more than kMoves CTAs an SM: one row
// each takes 41.5 us for the 4 moved states above, 12 CTAs an SM 81.5 for the 11.
cudaError_t reorder(const ReorderParams& p, int groups, int segs, int nsm, cudaStream_t st) {
  const long long most = p.page_bytes ? (long long)p.page_rows * p.row_bytes : p.seg_bytes;
  if (groups <= 0 || segs <= 0 || most <= 0) return cudaSuccess;
  if (groups > 65535 || segs > 65535 || p.beams < 1 || p.beams > kMaxBeams) return cudaErrorInvalidValue;
  const long long all = (most / 16 + kThreads - 1) / kThreads;  // rows of columns
  const long long fair = std::max((long long)nsm * kMoves / ((long long)groups * segs), 1ll);
  long long per = (all + fair - 1) / fair;
  if (per > 2) per = (per + 3) / 4 * 4;
  ReorderParams q = p;
  q.share = per * kThreads * 16;
  const long long x = (all + per - 1) / per;
  const dim3 grid((unsigned)x, (unsigned)segs, (unsigned)groups);
  if (p.beams <= 4)
    k_reorder<4><<<grid, kThreads, 0, st>>>(q);
  else if (p.beams <= 8)
    k_reorder<8><<<grid, kThreads, 0, st>>>(q);
  else
    k_reorder<16><<<grid, kThreads, 0, st>>>(q);
  return cudaGetLastError();
}

}  // namespace beam
}  // namespace hy
