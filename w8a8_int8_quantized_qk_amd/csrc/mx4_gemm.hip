// The product of two microscaled 4-bit operands for gfx950:
//   out[i][j] = output_scale * sum_k A(i, k) B(j, k)
// with A(i, k) = code * 2^(scale byte - 127), a scale per 32 consecutive k.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes both operands as they are stored: a lane
// holds 32 consecutive codes of one row (16 bytes) in four registers, and one
// byte of a fifth is that block's scale, so neither is converted or
// multiplied.  Sums are binary32.
//
// The weight's rows are the first operand: a lane's four sums are then four
// consecutive columns of one output row.
#include "gemm_tile.h"
#include "quant_math.h"

namespace qk {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;       // the instruction's number of the element type
constexpr uint32_t kOne = 127;  // the scale byte of 1

__device__ __forceinline__ v8i operand(const uint4& w) {
  return v8i{static_cast<int>(w.x), static_cast<int>(w.y), static_cast<int>(w.z), static_cast<int>(w.w), 0, 0, 0, 0};
}

// One output value, rounded to its type once.
template <int DT>
__device__ __forceinline__ void put(void* out, int64_t at, float v) {
  if constexpr (DT == QK_F32)
    static_cast<float*>(out)[at] = v;
  else
    static_cast<uint16_t*>(out)[at] = static_cast<uint16_t>(qm::pack2_narrow<DT>(v, 0.0f));
}

// Few rows: bound by the weight's bytes.  A workgroup has 16 columns (rows of
// the weight) and 16 F rows of A, its W waves a part of k each; their sums meet
// in LDS in the order of the waves.  Operands come straight from memory: each
// lane's 16 bytes are what the instruction wants from it.
template <int DT, int F, int W>
__global__ __launch_bounds__(64 * W) void mx4_gemm_rows_kernel(Mx4GemmArgs g, int steps_each) {
  __shared__ v4f sums[W][F][64];
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * F;
  const int blocks = g.k / 32;
  const int64_t row_bytes = g.k / 2;
  const uint8_t* const b = g.b + min(n0 + r, g.n - 1) * row_bytes;
  const uint8_t* const sb = g.scale_b + min(n0 + r, g.n - 1) * g.ldsb;
  const uint8_t* a[F];
  const uint8_t* sa[F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    a[f] = g.a + min(m0 + 16 * f + r, g.m - 1) * row_bytes;
    sa[f] = g.scale_a + min(m0 + 16 * f + r, g.m - 1) * g.ldsa;
  }
  v4f acc[F];
#pragma unroll
  for (int f = 0; f < F; ++f) acc[f] = v4f{0, 0, 0, 0};
  const int first = wave * steps_each, last = min(first + steps_each, (blocks + 3) / 4);
#pragma unroll 4
  for (int s = first; s < last; ++s) {
    const int at = 4 * s + c;  // the lane's block
    const bool in = at < blocks;
    const int here = in ? at : blocks - 1;
    const uint4 w = *reinterpret_cast<const uint4*>(b + 16 * here);
    const uint32_t ws = in ? sb[here] : kOne;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      uint4 x = *reinterpret_cast<const uint4*>(a[f] + 16 * here);
      if (!in) x = make_uint4(0, 0, 0, 0);
      const uint32_t xs = in ? sa[f][here] : kOne;
      acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(x), acc[f], kFp4, kFp4, 0,
                                                               static_cast<int>(ws), 0, static_cast<int>(xs));
    }
  }
#pragma unroll
  for (int f = 0; f < F; ++f) sums[wave][f][lane] = acc[f];
  __syncthreads();
  for (int f = wave; f < F; f += W) {
    v4f v = sums[0][f][lane];
    for (int w = 1; w < W; ++w) v += sums[w][f][lane];
    const int row = m0 + 16 * f + r, col = n0 + 4 * c;
    if (row >= g.m) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < g.n) put<DT>(g.out, static_cast<int64_t>(row) * g.n + col + e, v[e] * g.output_scale);
  }
}

template <int DT, int F, int W>
hipError_t rows(const Mx4GemmArgs& g, hipStream_t stream) {
  const int steps = (g.k / 32 + 3) / 4;
  const dim3 grid(static_cast<unsigned>((g.n + 15) / 16), static_cast<unsigned>((g.m + 16 * F - 1) / (16 * F)));
  return launch(mx4_gemm_rows_kernel<DT, F, W>, grid, dim3(64 * W), 0, stream, g, (steps + W - 1) / W);
}

template <int DT>
hipError_t by_size(const Mx4GemmArgs& g, hipStream_t stream) {
  if (g.m <= 16) return rows<DT, 1, 4>(g, stream);
  return rows<DT, 4, 4>(g, stream);
}

}  // namespace

hipError_t launch_gemm_mx4(const Mx4GemmArgs& g, hipStream_t stream) {
  const int64_t groups = static_cast<int64_t>((g.n + 15) / 16) * ((g.m + 15) / 16);
  if (!grid_fits(groups, 256) || (g.m + 15) / 16 > 65535) return hipErrorInvalidConfiguration;
  switch (g.out_dtype) {
    case QK_F32: return by_size<QK_F32>(g, stream);
    case QK_BF16: return by_size<QK_BF16>(g, stream);
    default: return by_size<QK_F16>(g, stream);
  }
}

}  // namespace qk
