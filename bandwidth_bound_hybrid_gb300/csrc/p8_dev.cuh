// The paged 8-bit KV cache's format on the device.  A block is 16 rows of one
// kv head, rounded to bf16; closed, it is int8 codes c with one FP32 scale s,
// value s c; the rows of a sequence's open block are bf16 in its tail.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace hy {
namespace p8 {

// (x0, x1) of a rotate-half pair, each product and sum rounded on its own, so
// that a code never depends on how the compiler contracts them.
__device__ __forceinline__ void rotate(float x0, float x1, float2 cs, float* r0, float* r1) {
  *r0 = __fsub_rn(__fmul_rn(x0, cs.x), __fmul_rn(x1, cs.y));
  *r1 = __fadd_rn(__fmul_rn(x1, cs.x), __fmul_rn(x0, cs.y));
}

// Two values rounded to bf16 (a in the low half); what is not finite becomes NaN.
__device__ __forceinline__ uint32_t store_pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
  if ((u & 0x7f80u) == 0x7f80u) u = (u & 0xffff0000u) | 0x7fc0u;
  if ((u & 0x7f800000u) == 0x7f800000u) u = (u & 0xffffu) | 0x7fc00000u;
  return u;
}
__device__ __forceinline__ uint32_t abs_max(uint32_t m, uint32_t pair) {
  return max(m, max(pair & 0x7fffu, (pair >> 16) & 0x7fffu));
}

// Scale of a block whose largest |x| has the bf16 bits a (a NaN above all):
// s = a / 127 and the factor of the values, 127 / a; both 0 for a < 2^-100, a
// NaN: s = NaN, factor 0.
__device__ __forceinline__ float block_scale(uint32_t a, float* inv) {
  const float x = __uint_as_float(a << 16);
  *inv = 0.f;
  if (a >= 0x7f80u) return __uint_as_float(0x7fc00000u);
  if (x < 7.888609052210118e-31f) return 0.f;  // 2^-100
  *inv = __fdiv_rn(127.f, x);
  return __fdiv_rn(x, 127.f);
}
// round-half-even(x * (127 / a)) clamped to [-127, 127]; 0 where the factor is
__device__ __forceinline__ int block_code(float x, float inv) {
  return inv == 0.f ? 0 : (int)fminf(fmaxf(rintf(__fmul_rn(x, inv)), -127.f), 127.f);
}

// The page of block j of sequence b, or -1 where the table holds none.
__device__ __forceinline__ int page_of(const Cache& c, int b, int j) {
  const int pg = __ldg(c.table + (long long)b * c.max_pages + j / c.bpp);
  return (unsigned)pg < (unsigned)c.pool_pages ? pg : -1;
}
__device__ __forceinline__ long long code_at(const Cache& c, int pg, int g, int at, int hd) {
  return pg * c.page_stride + (long long)(g * c.page_tokens + at * kBlock) * hd;
}
__device__ __forceinline__ long long scale_at(const Cache& c, int pg, int g, int at) {
  return pg * c.scale_stride + (long long)g * c.bpp + at;
}

// The blocks that a query at position t sees, as a list: those of the first
// `sinks` positions below the window's first block, then the window's.
struct View {
  int ns, wb, n;  // sink blocks, the window's first block, blocks in all
};
__device__ __forceinline__ View view_of(int t, int window, int sinks) {
  View v;
  v.wb = window > 0 && t - window + 1 > 0 ? (unsigned)(t - window + 1) / kBlock : 0;
  v.ns = min(v.wb, (int)(((unsigned)sinks + kBlock - 1) / kBlock));
  v.n = v.ns + (int)((unsigned)t / kBlock) - v.wb + 1;
  return v;
}
__device__ __forceinline__ int block_at(const View& v, int i) { return i < v.ns ? i : i - v.ns + v.wb; }
__device__ __forceinline__ bool in_view(int u, int t, int window, int sinks) {
  return u <= t && (window <= 0 || u < sinks || u > t - window);
}

}  // namespace p8
}  // namespace hy
