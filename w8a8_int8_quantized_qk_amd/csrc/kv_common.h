// What the kernels of the paged 8-bit cache share: how work items are laid
// over ragged sequences, and the conversion of codes (device code only).
#pragma once

#include "quant_math.h"

namespace qk {
namespace kv {

// 16 and 8 bytes at any alignment the element type allows
template <int ALIGN>
struct __attribute__((packed, aligned(ALIGN))) Raw16 {
  uint32_t w[4];
};
// (and as vectors, for accesses past the caches)
typedef uint32_t Loose16 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t Loose8 __attribute__((ext_vector_type(2), aligned(2)));
template <int ALIGN>
struct __attribute__((packed, aligned(ALIGN))) Raw8 {
  uint32_t w[2];
};
template <int ALIGN>
struct __attribute__((packed, aligned(ALIGN))) Raw4 {
  uint32_t w;
};

// Ragged sequences are cut into items whose number the host knows without
// knowing the lengths: sequence b of rows cu[b] .. cu[b + 1] owns items
// base(b) .. base(b + 1), base(b) = floor(cu[b] * mul / size) + extra * b, and
// uses the first of them.  base(b + 1) - base(b) >= floor(n * mul / size) +
// extra for n rows, which covers the pieces of `size` that n * mul columns
// have (extra = 1), or that n positions touch when they start inside a piece
// (extra = 2).  The number of items is base(seqs).  (The attention's prompt tiles
// have a base of their own, since short sequences have none.)
__host__ __device__ __forceinline__ int64_t item_base(int64_t row, int mul, int size, int extra, int b) {
  return row * mul / size + static_cast<int64_t>(extra) * b;
}

// The sequence that owns `item`, its first row, the next one's, and its entry
// of `each` (start or length): the last sequence whose base(first row, number)
// is at or below the item.  The lanes of a wave look at 64 sequences at a time, each lane with its
// sequence's numbers in hand, so that nothing has to be loaded again for the
// one that is found; the result is uniform.  seq < 0: none.
struct Owner {
  int seq, first, next, value;
};
template <typename Base>
__device__ __forceinline__ Owner find_sequence(int64_t item, const int* cu, const int* each, int seqs, Base base) {
  const int lane = threadIdx.x & 63;
  Owner o{-1, 0, 0, 0};
  for (int b0 = 0; b0 < seqs; b0 += 64) {
    const int b = min(b0 + lane, seqs - 1);
    const int first = cu[b], next = cu[b + 1], value = each[b];
    const bool below = b0 + lane < seqs && base(first, b) <= item;
    const int n = __popcll(__ballot(below));
    if (n == 0) break;
    o.seq = b0 + n - 1;
    o.first = __builtin_amdgcn_readlane(first, n - 1);
    o.next = __builtin_amdgcn_readlane(next, n - 1);
    o.value = __builtin_amdgcn_readlane(value, n - 1);
    if (n < 64) break;
  }
  return o;
}

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

// Four codes as binary16, exactly.  INT8: with its sign bit turned the byte
// is code + 128; put under the exponent of 1024 it reads 1024 + 128 + code,
// and 1152 is subtracted (both exact in 11 bits).  FP8: the hardware's
// conversion.
template <bool FP8>
__device__ __forceinline__ void codes4_to_half(uint32_t w, half2_t& lo, half2_t& hi) {
  if constexpr (FP8) {
    lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
  } else {
    const half2_t off = {static_cast<_Float16>(1152.0f), static_cast<_Float16>(1152.0f)};
    const uint32_t u = w ^ 0x80808080u;
    lo = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - off;
    hi = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - off;
  }
}

template <bool FP8>
__device__ __forceinline__ half8_t codes8_to_half(uint32_t a, uint32_t b) {
  half2_t x, y, z, w;
  codes4_to_half<FP8>(a, x, y);
  codes4_to_half<FP8>(b, z, w);
  return half8_t{x[0], x[1], y[0], y[1], z[0], z[1], w[0], w[1]};
}

// Byte i of a word as the value its code stands for, times no scale.
template <bool FP8>
__device__ __forceinline__ void codes4_to_float(uint32_t w, float (&f)[4]) {
  if constexpr (FP8) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    f[0] = a[0];
    f[1] = a[1];
    f[2] = b[0];
    f[3] = b[1];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  }
}

// Four values in units of a scale s (r = RN(1 / s)) as packed codes: the
// exact quotient, rounded to nearest even.  |x| <= qmax * s up to rounding.
template <bool FP8>
__device__ __forceinline__ uint32_t codes4_of(const float (&x)[4], float s, float r) {
  if constexpr (FP8) {
    return qm::pack4_fp8(qm::fp8_ratio_own(x[0], s, r), qm::fp8_ratio_own(x[1], s, r),
                         qm::fp8_ratio_own(x[2], s, r), qm::fp8_ratio_own(x[3], s, r));
  } else {
    return qm::pack4_low_bytes(qm::code_word_dynamic(x[0], s, r), qm::code_word_dynamic(x[1], s, r),
                               qm::code_word_dynamic(x[2], s, r), qm::code_word_dynamic(x[3], s, r));
  }
}

}  // namespace kv
}  // namespace qk
