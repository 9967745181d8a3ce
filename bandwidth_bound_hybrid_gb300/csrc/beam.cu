// Beam search on sm_103a: selection over the beams and the vocabulary, and
// the reordering of the beams' states.
//
// Selection.  Candidate (w, v) of a group of beams scores
//   s(w, v) = score_w + x_wv - lse_w,  lse_w = log sum_v exp(x_wv),
// and the group's best `picks` are wanted, ties to the lowest w V + v.  Within
// a beam the order is that of the logits, so one pass over the logits is
// enough: every CTA takes a chunk of a beam's row into registers and leaves
// the chunk's maximum, its sum of exponentials and its best `picks` logits;
// the last CTA of the group turns the maxima and sums into lse_w (in FP64, as
// the scores are: candidates of different beams differ in their last bits)
// and selects among the chunks' lists.  Bound by reading the logits once.
//
// A chunk's best: the picks-th largest of a warp's 32 lane maxima is a bound
// that at least `picks` values reach, so only the values that reach the best
// such bound of the CTA (a few dozen) are ranked, each counting its betters.
// The group's best are found in the same way from the lists' heads.
//
// Reordering.  State i of a group becomes what state parent[i] was, in place:
// a thread owns one 16-byte column of all the group's states, reads the
// sources of those that change, and only then writes.  So no second copy of
// the states is kept, and a source is read once from memory whatever the
// number of its children.  Bound by the bytes of the states that change.
#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace hy {
namespace beam {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = kChunk / kThreads;  // logits of a thread
constexpr int kQual = 1024;              // lists looked into by the fast final selection
constexpr int kBest = 2048;              // and their candidates

// A candidate of a chunk in one word: the logit's order key above the
// complement of the token, so that the larger word is the better candidate
// and no two are equal.  0: none.
__device__ __forceinline__ uint64_t word_of(uint32_t key, uint32_t token) {
  return ((uint64_t)key << 32) | (0xffffffffu - token);
}
__device__ __forceinline__ float word_logit(uint64_t c) { return key_value((uint32_t)(c >> 32)); }
__device__ __forceinline__ uint32_t word_token(uint64_t c) { return 0xffffffffu - (uint32_t)c; }

// The n-th largest (n in 1..32) of the lanes' keys: a bitonic sort across the warp.
__device__ __forceinline__ uint32_t warp_nth(uint32_t v, int n, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, v, j);
      const bool larger = ((lane & k) == 0) == ((lane & j) == 0);  // what this lane keeps of the pair
      v = larger ? max(v, o) : min(v, o);
    }
  }
  return __shfl_sync(0xffffffffu, v, n - 1);
}

// A candidate of the group: FP64 score and flat index w V + v.
struct Cand {
  double s;
  uint32_t i;
};
__device__ __forceinline__ bool better(const Cand& a, const Cand& b) { return a.s > b.s || (a.s == b.s && a.i < b.i); }

struct Shared {
  union {
    uint64_t list[kChunk];             // a chunk's candidates
    struct {
      double s[kBest];                 // the group's candidates
      uint32_t i[kBest];
      uint32_t qual[kQual];
    } best;
    uint8_t at[kMaxLists];             // one by one: the next candidate of every list
  };
  uint32_t key[kWarps];
  float m[kWarps], sum[kWarps];
  double off[kMaxBeams];               // score_w - lse_w, or score_w of a done beam (-infinity: nothing counts)
  int done[kMaxBeams];
  Cand sel[kMaxPicks], top[kWarps];
  int n, nq, last;
};

__global__ void __launch_bounds__(kThreads) k_select(const SelectParams p) {
  __shared__ Shared sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nch = p.chunks, row = blockIdx.x / nch, chunk = blockIdx.x % nch, group = row / p.beams;
  const int P = p.picks, V = p.vocab;
  if (!(p.done && p.done[row])) {
    // ------------------------------------------------------ the chunk
    const float* x = p.logits + (long long)row * p.ld;
    const int base = chunk * kChunk;
    float v[kPer], m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = base + k * kThreads + tid;
      v[k] = i < V ? __ldcs(x + i) : -INFINITY;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      v[k] = v[k] == v[k] ? v[k] : -INFINITY;  // a NaN counts as -infinity
      m = fmaxf(m, v[k]);
    }
    const uint32_t nth = warp_nth(order_key(m), P, lane);
    const float wm = warp_max(m);
    if (lane == 0) {
      sm.key[warp] = nth;
      sm.m[warp] = wm;
    }
    if (tid == 0) sm.n = 0;
    __syncthreads();
    uint32_t bound = order_key(-INFINITY) + 1;  // -infinity is no candidate
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      bound = max(bound, sm.key[w]);
      M = fmaxf(M, sm.m[w]);
    }
    const float low = key_value(bound);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      s += __expf(v[k] - M);
      if (v[k] >= low) sm.list[atomicAdd(&sm.n, 1)] = word_of(order_key(v[k]), base + k * kThreads + tid);
    }
    s = warp_sum(s);
    if (lane == 0) sm.sum[warp] = s;
    __syncthreads();
    const int n = sm.n;
    const long long slot = (long long)row * nch + chunk;
    uint64_t* out = p.lists + slot * P;
    for (int a = tid; a < n; a += kThreads) {
      const uint64_t c = sm.list[a];
      int rank = 0;
      for (int b = 0; b < n && rank < P; ++b) rank += sm.list[b] > c;
      if (rank < P) out[rank] = c;
    }
    if (tid >= n && tid < P) out[tid] = 0;
    if (tid == 0) {
      float S = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) S += sm.sum[w];
      p.stats[slot] = make_float2(M, S);  // M -infinity: S is NaN and not read
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
  for (int w = warp; w < p.beams; w += kWarps) {  // lse and offset of every beam
    const int r = row0 + w, done = p.done && p.done[r];
    double off = (double)p.score[r];
    if (!done) {
      const float2* st = p.stats + (long long)r * nch;
      float M = -INFINITY;
      for (int c = lane; c < nch; c += 32) M = fmaxf(M, __ldcg(st + c).x);
      M = warp_max(M);
      double S = 0;
      for (int c = lane; c < nch; c += 32) {
        const float2 t = __ldcg(st + c);
        if (t.x > -INFINITY) S += (double)t.y * exp((double)t.x - (double)M);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
      off -= (double)M + log(S);
    }
    if (lane == 0) {
      sm.off[w] = off - off == 0.0 ? off : -INFINITY;
      sm.done[w] = done;
    }
  }
  __syncthreads();
  // candidate k of list l = (beam, chunk); -infinity: none
  auto get = [&](int l, int k) {
    const int w = l / nch, c = l % nch;
    Cand a = {-INFINITY, 0xffffffffu};
    const double off = sm.off[w];
    if (off == -INFINITY) return a;
    if (sm.done[w]) {  // a beam that has ended goes on as it is
      if (c == 0 && k == 0) a = {off, (uint32_t)w * V + p.eos};
      return a;
    }
    const uint64_t word = __ldcg(reinterpret_cast<const unsigned long long*>(p.lists) + ((long long)row0 * nch + l) * P + k);
    if (word) a = {off + (double)word_logit(word), (uint32_t)w * V + word_token(word)};
    if (a.s < -(double)FLT_MAX) a = {-INFINITY, 0xffffffffu};  // the FP32 score is -infinity
    return a;
  };
  // order key of a score rounded down: at least as many candidates reach it as reach the score
  auto key_of = [](double s) { return order_key(__double2float_rd(s)); };
  uint32_t mine = 0;
  for (int l = tid; l < nl; l += kThreads) mine = max(mine, key_of(get(l, 0).s));
  const uint32_t nth = warp_nth(mine, P, lane);
  if (lane == 0) sm.key[warp] = nth;
  __syncthreads();
  uint32_t bound = order_key(-INFINITY) + 1;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) bound = max(bound, sm.key[w]);
  for (int l = tid; l < nl; l += kThreads)
    if (key_of(get(l, 0).s) >= bound) {
      const int q = atomicAdd(&sm.nq, 1);
      if (q < kQual) sm.best.qual[q] = l;
    }
  __syncthreads();
  const int nq = sm.nq;
  if (nq <= kQual) {
    for (int q = warp; q < nq; q += kWarps) {
      const Cand a = lane < P ? get(sm.best.qual[q], lane) : Cand{-INFINITY, 0xffffffffu};
      if (key_of(a.s) >= bound) {
        const int at = atomicAdd(&sm.n, 1);
        if (at < kBest) {
          sm.best.s[at] = a.s;
          sm.best.i[at] = a.i;
        }
      }
    }
  }
  __syncthreads();
  int n = sm.n;
  if (nq <= kQual && n <= kBest) {
    for (int a = tid; a < n; a += kThreads) {
      const Cand c = {sm.best.s[a], sm.best.i[a]};
      int rank = 0;
      for (int b = 0; b < n && rank < P; ++b) rank += better({sm.best.s[b], sm.best.i[b]}, c);
      if (rank < P) sm.sel[rank] = c;
    }
    if (n > P) n = P;
  } else {
    // more near-equal candidates than the arrays hold (a flat row): the best of the lists' heads, one at a time
    __syncthreads();
    for (int l = tid; l < nl; l += kThreads) sm.at[l] = 0;
    for (n = 0; n < P; ++n) {
      Cand best = {-INFINITY, 0xffffffffu};
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
        const Cand a = {__shfl_xor_sync(0xffffffffu, top.s, o), __shfl_xor_sync(0xffffffffu, top.i, o)};
        if (better(a, top)) top = a;
      }
      if (lane == 0) sm.top[warp] = top;
      __syncthreads();
      top = sm.top[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w)
        if (better(sm.top[w], top)) top = sm.top[w];
      if (top.s == -INFINITY) break;  // the same for every thread
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
    if (!taken && lane < P && n + before < P) sm.sel[n + before] = {-INFINITY, (uint32_t)lane};
    __syncwarp();
    if (lane < P) {
      const Cand c = sm.sel[lane];
      const int w = (int)(c.i / (uint32_t)V), token = (int)(c.i % (uint32_t)V);
      const long long at = (long long)group * P + lane;
      p.score_out[at] = (float)c.s;
      p.parent[at] = w;
      p.token[at] = token;
      if (p.done_out) p.done_out[at] = (sm.done[w] || token == p.eos) ? 1 : 0;
    }
  }
}

// ------------------------------------------------------------ reordering
// Column x of segment y of group z (or, paged, of segment y % n_seg in page
// first_page + y / n_seg).
template <int B>
__global__ void __launch_bounds__(kThreads) k_reorder(const ReorderParams p) {
  __shared__ int s_parent[B];
  const int tid = threadIdx.x, z = blockIdx.z;
  if (tid < p.beams) {
    int q = p.parent ? p.parent[(long long)z * p.beams + tid] : 0;
    if (q < 0 || q >= p.beams) {  // left as it is
      if (blockIdx.x == 0 && blockIdx.y == 0) set_guard(p.guard, kGuardBadIndex);
      q = tid;
    }
    s_parent[tid] = q;
  }
  __syncthreads();
  long long lo = 0, bytes = p.seg_bytes;
  int seg = blockIdx.y, page = 0;
  if (p.page_bytes) {  // rows [first_row, end_row) of the sequence that lie in this page
    page = p.first_page + seg / p.n_seg;
    seg %= p.n_seg;
    const int r0 = max(p.first_row - page * p.page_rows, 0), r1 = min(p.end_row - page * p.page_rows, p.page_rows);
    lo = (long long)r0 * p.row_bytes;
    bytes = (long long)r1 * p.row_bytes;
  }
  for (long long x = lo + ((long long)blockIdx.x * kThreads + tid) * 16; x < bytes; x += (long long)gridDim.x * kThreads * 16) {
    auto at = [&](int i) {
      uint8_t* b = p.base[i] + z * p.group_stride + seg * p.seg_stride[i] + x;
      return reinterpret_cast<uint4*>(p.page_bytes ? b + p.pages[i][page] * p.page_bytes : b);
    };
    uint4 v[B];
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (i < p.beams && s_parent[i] != i) v[i] = *at(s_parent[i]);
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (i < p.beams && s_parent[i] != i) *at(i) = v[i];
  }
}

}  // namespace

int chunks(int vocab) { return (int)(((long long)vocab + kChunk - 1) / kChunk); }

cudaError_t select(const SelectParams& p, int groups, cudaStream_t st) {
  const long long grid = (long long)groups * p.beams * p.chunks;
  if (grid <= 0 || grid > 0x7fffffffll || p.beams > kMaxBeams || p.picks < 1 || p.picks > kMaxPicks ||
      (long long)p.beams * p.chunks > kMaxLists)
    return cudaErrorInvalidValue;
  k_select<<<(unsigned)grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t reorder(const ReorderParams& p, int groups, int segs, cudaStream_t st) {
  const long long most = p.page_bytes ? (long long)p.page_rows * p.row_bytes : p.seg_bytes;
  if (groups <= 0 || segs <= 0 || most <= 0) return cudaSuccess;
  if (groups > 65535 || segs > 65535 || p.beams < 1 || p.beams > kMaxBeams) return cudaErrorInvalidValue;
  long long x = (most / 16 + kThreads - 1) / kThreads;
  if (x > 4096) x = 4096;
  const dim3 grid((unsigned)x, (unsigned)segs, (unsigned)groups);
  if (p.beams <= 4)
    k_reorder<4><<<grid, kThreads, 0, st>>>(p);
  else if (p.beams <= 8)
    k_reorder<8><<<grid, kThreads, 0, st>>>(p);
  else
    k_reorder<16><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace beam
}  // namespace hy
