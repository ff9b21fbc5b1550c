// Microscaled 4-bit floating point for gfx950: quantisation, plain and of
// silu(gate) * up, and the way back.
//
// A row is cut into blocks of 32 consecutive values with one power of two each
// (the Open Compute Project's Microscaling Formats specification, version 1.0:
// E2M1 elements under an E8M0 scale, and its conversion from scalar values):
//   scale = 2^(floor(log2(max |x|)) - 2), held to at least 2^-127
//   code  = x / scale rounded to 0, 0.5, 1, 1.5, 2, 3, 4 or 6 and its sign,
//           nearest, ties to the even code, at most 6
// x / scale is a shift of the exponent and below 8, so nothing but the rounding
// to 4 bits is inexact.  The scale's byte is its exponent + 127: the exponent
// field of max |x| as binary32, less 2.  A block with an infinity or a NaN has
// the byte 255, which stands for NaN, and codes 0.
//
// Bound by memory: four lanes share a block, eight values (16 or 32 bytes)
// each, so a wave reads 1 KiB of 16-bit rows in one piece and writes 256 bytes
// of codes and 16 of scales.  bf16, 4096 x 14336 there 27.1 us (5.5 TB/s), back 21.6
// (6.9), one after the other 48.8 (6.1); of silu(gate) * up 56 (4.7); 8 x 4096 2.3 us
// either way.  Reading past the caches there gains nothing (27.7).  On the way back the
// 16-bit values of large calls are stored past them (22.5 us without, and 29.8 for 21.6
// where three outputs take turns; 2048 x 4096 3.9 for 4.8), binary32's, of which a lane
// has two pieces, not (88 us for 51).
#include "kv_common.h"
#include "mx4.h"

namespace qk {
namespace {

using kv::Raw16;
using qm::Elem;

constexpr int kBlock = 256;
constexpr int kEach = 8;  // values per lane, a quarter of a block
constexpr int64_t kPastCaches = 8 << 20;  // bytes of 16-bit values that are stored past the caches

// Eight values at any alignment the element type allows.
template <int DT>
__device__ __forceinline__ void load8(const char* p, float (&f)[kEach]) {
  constexpr int B = Elem<DT>::kBytes;
#pragma unroll
  for (int i = 0; i < kEach * B / 16; ++i) {
    const Raw16<B> w = *reinterpret_cast<const Raw16<B>*>(p + 16 * i);
    Elem<DT>::unpack(make_uint4(w.w[0], w.w[1], w.w[2], w.w[3]), f + i * Elem<DT>::kPerUnit);
  }
}

// Lane i of a quad sees the maximum of its four lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = qm::max_u32(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, false)));  // lane ^ 1
  return qm::max_u32(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, false)));  // lane ^ 2
}

// silu(h[:, :k]) * h[:, k:] with SILU.  Item i is a quarter of a block.
template <int DT, bool SILU>
__global__ __launch_bounds__(kBlock) void mx4_quant_kernel(const char* __restrict__ x, int64_t ldx, int64_t items,
                                                           uint32_t per_row, int64_t k_bytes, uint8_t* __restrict__ q,
                                                           uint8_t* __restrict__ scale, int64_t lds) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  if (i >= items) return;  // whole quads
  const uint32_t row = static_cast<uint32_t>(i) / per_row, at = static_cast<uint32_t>(i) - row * per_row;
  const char* const from = x + (row * ldx + static_cast<int64_t>(at) * kEach) * Elem<DT>::kBytes;
  float v[kEach];
  load8<DT>(from, v);
  if constexpr (SILU) {
    float up[kEach];
    load8<DT>(from + k_bytes, up);
#pragma unroll
    for (int e = 0; e < kEach; ++e) v[e] = qm::silu_times<DT != QK_F32>(v[e], up[e]);
  }
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) top = qm::max_u32(top, mx4::magnitude_bits(v[e]));
  const uint32_t byte = mx4::scale_byte(quad_max(top));
  reinterpret_cast<uint32_t*>(q)[i] = mx4::codes8(v, byte);
  if ((at & 3) == 0) scale[row * lds + (at >> 2)] = static_cast<uint8_t>(byte);
}

template <int DT, bool PAST>
__global__ __launch_bounds__(kBlock) void mx4_dequant_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                                             int64_t lds, int64_t items, uint32_t per_row,
                                                             char* __restrict__ x, int64_t ldx) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  if (i >= items) return;
  const uint32_t row = static_cast<uint32_t>(i) / per_row, at = static_cast<uint32_t>(i) - row * per_row;
  const uint32_t w = reinterpret_cast<const uint32_t*>(q)[i], byte = scale[row * lds + (at >> 2)];
  const float s = __uint_as_float(byte << 23);
  float v[kEach];
  typedef float pair_t __attribute__((ext_vector_type(2)));
  const pair_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1),
               c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
  v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
  constexpr int B = Elem<DT>::kBytes, W = kEach * B / 4;  // words
  constexpr uint32_t kNaN = DT == QK_F32 ? 0x7fc00000u : DT == QK_BF16 ? 0x7fc07fc0u : 0x7e007e00u;
  uint32_t out[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (DT == QK_F32)
      out[i] = __float_as_uint(v[i]);
    else
      out[i] = qm::pack2_narrow<DT>(v[2 * i], v[2 * i + 1]);
    out[i] = byte == 255 ? kNaN : out[i];
  }
  kv::Loose16* const to = reinterpret_cast<kv::Loose16*>(x + (row * ldx + static_cast<int64_t>(at) * kEach) * B);
  // (not in a loop: out of one of a single turn the compiler moved the store, and
  // that went through the caches)
  auto put = [&](int h) {
    const kv::Loose16 piece = {out[4 * h], out[4 * h + 1], out[4 * h + 2], out[4 * h + 3]};
    if constexpr (PAST)
      __builtin_nontemporal_store(piece, to + h);
    else
      to[h] = piece;
  };
  put(0);
  if constexpr (W == 8) put(1);
}

dim3 grid_of(int64_t items) { return dim3(static_cast<unsigned>((items + kBlock - 1) / kBlock)); }

template <int DT>
hipError_t quant(const Mx4RowsArgs& a, int64_t items, uint32_t per_row, hipStream_t stream) {
  if (a.silu)
    return launch(mx4_quant_kernel<DT, true>, grid_of(items), dim3(kBlock), 0, stream, static_cast<const char*>(a.x),
                  a.ldx, items, per_row, static_cast<int64_t>(a.k) * Elem<DT>::kBytes, a.q, a.scale, a.lds);
  return launch(mx4_quant_kernel<DT, false>, grid_of(items), dim3(kBlock), 0, stream, static_cast<const char*>(a.x), a.ldx,
                items, per_row, 0, a.q, a.scale, a.lds);
}

template <int DT>
hipError_t dequant(const Mx4RowsArgs& a, int64_t items, uint32_t per_row, hipStream_t stream) {
  char* const x = static_cast<char*>(const_cast<void*>(a.x));
  if constexpr (DT != QK_F32) {
    if (items * kEach * Elem<DT>::kBytes > kPastCaches)
      return launch(mx4_dequant_kernel<DT, true>, grid_of(items), dim3(kBlock), 0, stream, a.q, a.scale, a.lds, items,
                    per_row, x, a.ldx);
  }
  return launch(mx4_dequant_kernel<DT, false>, grid_of(items), dim3(kBlock), 0, stream, a.q, a.scale, a.lds, items, per_row,
                x, a.ldx);
}

}  // namespace

hipError_t launch_mx4_rows(const Mx4RowsArgs& a, bool back, hipStream_t stream) {
  const uint32_t per_row = static_cast<uint32_t>(a.k) / kEach;
  const int64_t items = static_cast<int64_t>(a.m) * per_row;
  if (!grid_fits((items + kBlock - 1) / kBlock, kBlock)) return hipErrorInvalidConfiguration;
  switch (a.dtype) {
    case QK_F32: return back ? dequant<QK_F32>(a, items, per_row, stream) : quant<QK_F32>(a, items, per_row, stream);
    case QK_BF16: return back ? dequant<QK_BF16>(a, items, per_row, stream) : quant<QK_BF16>(a, items, per_row, stream);
    default: return back ? dequant<QK_F16>(a, items, per_row, stream) : quant<QK_F16>(a, items, per_row, stream);
  }
}

}  // namespace qk
