// The 4-bit KV cache's format on the device: a vector is blocks of 32 values,
// each with one fp16 scale s and codes c in [-7, 7] stored as c + 8 (element i
// in the low nibble of byte i, element i + 16 in its high nibble).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace hy {
namespace kv4 {

// The scale of a block whose largest |x| has the bits a (the order of finite
// values, infinities above, NaN above those): s = fp16(min(max |x| * fp32(1 /
// 7), 65504)), and what the values are multiplied by, 1 / s (0 for s = 0).  An
// infinity or NaN in the block makes the scale NaN, so that it shows in
// whatever reads the block.
__device__ __forceinline__ __half block_scale(uint32_t a, float* inv) {
  float s = NAN;
  if (a < 0x7f800000u) s = fminf(__fmul_rn(__uint_as_float(a), 1.0f / 7.0f), 65504.0f);
  const __half sh = __float2half_rn(s);
  const float sf = __half2float(sh);
  *inv = sf > 0.f ? __fdiv_rn(1.0f, sf) : 0.f;
  return sh;
}
// code = round-half-even(x * (1 / s)) clamped to [-7, 7]
__device__ __forceinline__ int quant_code(float x, float inv) {
  return (int)fminf(fmaxf(rintf(__fmul_rn(x, inv)), -7.f), 7.f);
}

// One block of 32 values, one per lane of a full warp: its fp16 scale (bits) and the lane's code.
__device__ __forceinline__ uint16_t quant_block(float x, int* code) {
  float inv;
  const __half sh = block_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7fffffffu), &inv);
  *code = quant_code(x, inv);
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

// Values 8 w .. 8 w + 7 of a row's block in the order low nibbles 4 w .. 4 w + 3,
// then 16 + 4 w .. (word w of the block's 16 bytes).
__device__ __forceinline__ void unpack_word(uint32_t word, float s, float* lo, float* hi) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = (float)((int)((word >> (8 * i)) & 15u) - 8) * s;
    hi[i] = (float)((int)((word >> (8 * i + 4)) & 15u) - 8) * s;
  }
}

}  // namespace kv4
}  // namespace hy
