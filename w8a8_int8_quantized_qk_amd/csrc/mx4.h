// Quantisation to microscaled 4-bit blocks (device code only).
//
// gfx950 converts with v_cvt_scalef32_pk_fp4_f32: it divides by the power of
// two in its scale operand's exponent field, rounds to the nearest code, ties to
// the even one, and saturates at 6 (checked over all 65536 bf16 and fp16 values
// and over binary32 around every border, subnormals among them).
#pragma once

#include "quant_math.h"

namespace qk {
namespace mx4 {

// The scale byte of a block whose largest magnitude has these bits as
// binary32: the exponent field of 2^(floor(log2) - 2), at least 0; 255 (NaN) for a
// block with an infinity or NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top_bits) {
  const uint32_t e = top_bits >> 23;
  return e == 255 ? 255 : e > 2 ? e - 2 : 0;
}

// Codes of eight values under a scale byte, the first in the low half of the first byte;
// 0 under NaN.
__device__ __forceinline__ uint32_t codes8(const float* v, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
  return byte == 255 ? 0 : w;
}

__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// A whole block in one lane.
struct Block {
  uint32_t codes[4], scale;
};
__device__ __forceinline__ Block quantised(const float (&v)[32]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) top = qm::max_u32(top, magnitude_bits(v[i]));
  Block b;
  b.scale = scale_byte(top);
#pragma unroll
  for (int i = 0; i < 4; ++i) b.codes[i] = codes8(v + 8 * i, b.scale);
  return b;
}

}  // namespace mx4
}  // namespace qk
