// Prompt attention over the paged 8-bit KV cache: a warp per query row and kv
// head, FP32 throughout.
#include "p8_dev.cuh"

namespace hy {
namespace p8 {
namespace {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int HD, int G>
__global__ void __launch_bounds__(128) k_rows(const Params p) {
  extern __shared__ float smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane & 1, row = lane >> 1;
  const long long unit = blockIdx.x * 4ll + warp;
  const long long i = unit / p.nkv;
  const int g = (int)(unit % p.nkv);
  float* q = smem + warp * G * HD;
  if (i >= p.n) return;
  int b = 0;
  while (b < p.nb && !(p.row_start[b] <= i && i < p.row_start[b + 1])) ++b;
  if (b == p.nb) return;
  const int rs = p.row_start[b], re = p.row_start[b + 1], T = p.len[b];
  const long long cap = (long long)p.c.max_pages * p.c.page_tokens;
  if (T < 0 || rs < 0 || re > p.n || (long long)T + (re - rs) > cap) {
    if (lane == 0) set_guard(p.guard, kGuardBadPosition);
    return;
  }
  const int t = T + (int)(i - rs), end = T + (re - rs);
  const float* y = p.y + i * p.ld_y;
  for (int k = lane; k < G * HD / 2; k += 32) {
    const int j = k / (HD / 2), d = k % (HD / 2);
    float x0 = y[(g * G + j) * HD + d], x1 = y[(g * G + j) * HD + d + HD / 2];
    rotate(x0, x1, p.rope[(long long)t * (HD / 2) + d], &x0, &x1);
    q[j * HD + d] = x0 * p.scale_log2e;
    q[j * HD + d + HD / 2] = x1 * p.scale_log2e;
  }
  __syncwarp();
  const View v = view_of(t, p.window, p.sinks);
  float m[G], l[G], o[G][HD / 32];
#pragma unroll
  for (int j = 0; j < G; ++j) {
    m[j] = -INFINITY;
    l[j] = 0.f;
#pragma unroll
    for (int k = 0; k < HD / 32; ++k) o[j][k] = 0.f;
  }
  for (int n = 0; n < v.n; ++n) {
    const int blk = block_at(v, n);
    const bool open = blk == end / kBlock;
    float s[G];
#pragma unroll
    for (int j = 0; j < G; ++j) s[j] = 0.f;
    const uint16_t* tk = p.c.tail + b * p.c.tail_stride + (long long)g * kBlock * HD;
    const uint16_t* tv = tk + (long long)p.nkv * kBlock * HD;
    const int8_t *kc = nullptr, *vc = nullptr;
    float ks = 1.f, vs = 1.f;
    if (!open) {
      const int pg = page_of(p.c, b, blk);
      if (pg < 0) {
        if (lane == 0) set_guard(p.guard, kGuardBadIndex);
        continue;
      }
      kc = p.c.K + code_at(p.c, pg, g, blk % p.c.bpp, HD);
      vc = p.c.V + code_at(p.c, pg, g, blk % p.c.bpp, HD);
      ks = p.c.Ks[scale_at(p.c, pg, g, blk % p.c.bpp)];
      vs = p.c.Vs[scale_at(p.c, pg, g, blk % p.c.bpp)];
    }
    const int u = blk * kBlock + row;
    const bool seen = in_view(u, t, p.window, p.sinks);
    if (seen)
      for (int d = half * (HD / 2); d < (half + 1) * (HD / 2); ++d) {
        const float x = open ? bf16_to_f32(tk[row * HD + d]) : (float)kc[row * HD + d];
#pragma unroll
        for (int j = 0; j < G; ++j) s[j] = fmaf(x, q[j * HD + d], s[j]);
      }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      s[j] += __shfl_xor_sync(0xffffffffu, s[j], 1);
      s[j] = seen ? s[j] * ks : -INFINITY;
      const float mn = fmaxf(m[j], warp_max(s[j]));
      const float corr = mn == -INFINITY ? 1.f : ex2(m[j] - mn);
      m[j] = mn;
      s[j] = seen ? ex2(s[j] - mn) : 0.f;
      l[j] = l[j] * corr + 0.5f * warp_sum(s[j]);
#pragma unroll
      for (int k = 0; k < HD / 32; ++k) o[j][k] *= corr;
    }
    for (int r = 0; r < kBlock; ++r) {
      if (!in_view(blk * kBlock + r, t, p.window, p.sinks)) continue;
#pragma unroll
      for (int k = 0; k < HD / 32; ++k) {
        const int d = k * 32 + lane;
        const float x = open ? bf16_to_f32(tv[r * HD + d]) : (float)vc[r * HD + d] * vs;
#pragma unroll
        for (int j = 0; j < G; ++j) o[j][k] = fmaf(__shfl_sync(0xffffffffu, s[j], 2 * r), x, o[j][k]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < G; ++j)
#pragma unroll
    for (int k = 0; k < HD / 32; ++k)
      p.o[i * p.ld_o + (g * G + j) * HD + k * 32 + lane] = l[j] == 0.f ? 0.f : o[j][k] / l[j];
}

template <int HD>
void (*pick(int G))(Params) {
  return G == 1 ? k_rows<HD, 1> : G == 2 ? k_rows<HD, 2> : G == 4 ? k_rows<HD, 4> : k_rows<HD, 8>;
}

}  // namespace

size_t prompt_workspace(int, int, int, int, int, int) { return 256; }
cudaError_t init_prompt() { return cudaSuccess; }
cudaError_t prompt(const Params& p, int hd, int, cudaStream_t st) {
  const int G = p.nq / p.nkv;
  auto k = hd == 64 ? pick<64>(G) : hd == 128 ? pick<128>(G) : pick<256>(G);
  const long long units = (long long)p.n * p.nkv;
  k<<<(unsigned)((units + 3) / 4), 128, 4 * G * hd * 4, st>>>(p);
  return cudaGetLastError();
}

}  // namespace p8
}  // namespace hy
