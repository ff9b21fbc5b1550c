// Root-mean-square norm of every head's query and key and the rotation by its
// position, in one pass, for gfx950:
//   y = (x * inv) * w,  inv = 1 / sqrt(mean(x^2) + eps)    (binary32; y = x without w)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
// for the pairs (a, b) = (i, i + r / 2), or (2 i, 2 i + 1), of a head's first r
// elements, at the angle position * freqs[i]; the other elements keep y.
//
// The angle of a far position has many whole turns, so it is formed and its
// turns are taken off in binary64: t = position * (freqs[i] / 2 pi), t - rint(4 t) / 4
// is exact and at most an eighth of a turn, and loses nothing when it is rounded to
// binary32 (t is off by 2^-52 of itself: 2^-25 of a turn at position 2^29).
// Sine and cosine of at most pi / 4 are their Taylor sums in binary32, up to
// x^9 and x^10 (the next terms are below 2^-28 and 2^-33).
#include "kv_common.h"

namespace qk {
namespace {

using qm::Elem;

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / 64;
constexpr int kMostPairs = 128;

struct Turn {
  float cos, sin;
};
__device__ __forceinline__ Turn turn_of(int pos, double freq) {
  const double t = static_cast<double>(pos) * (freq * 0.15915494309189535);
  const double quarter = __builtin_rint(t * 4.0);
  const float x = static_cast<float>((t - quarter * 0.25) * 6.283185307179586);
  const int q = static_cast<int>(static_cast<int64_t>(quarter) & 3);
  const float x2 = x * x;
  float s = __builtin_fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
  s = __builtin_fmaf(x2, s, 8.3333333e-3f);
  s = __builtin_fmaf(x2, s, -1.6666667e-1f);
  s = __builtin_fmaf(x * x2, s, x);
  float c = __builtin_fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);
  c = __builtin_fmaf(x2, c, -1.3888889e-3f);
  c = __builtin_fmaf(x2, c, 4.1666667e-2f);
  c = __builtin_fmaf(x2, c, -0.5f);
  c = __builtin_fmaf(x2, c, 1.0f);
  const float a = q & 1 ? s : c, b = q & 1 ? c : s;
  return Turn{q == 1 || q == 2 ? -a : a, q & 2 ? -b : b};
}

// N values at p, at any alignment the element type allows, and back.
template <int DT, int N>
__device__ __forceinline__ void load(const char* p, float* f) {
  constexpr int B = Elem<DT>::kBytes;
  if constexpr (N * B >= 16) {
#pragma unroll
    for (int i = 0; i < N * B / 16; ++i) {
      const kv::Raw16<B> w = *reinterpret_cast<const kv::Raw16<B>*>(p + 16 * i);
      Elem<DT>::unpack(make_uint4(w.w[0], w.w[1], w.w[2], w.w[3]), f + i * Elem<DT>::kPerUnit);
    }
  } else if constexpr (N * B == 8) {
    const kv::Raw8<B> w = *reinterpret_cast<const kv::Raw8<B>*>(p);
    float all[Elem<DT>::kPerUnit];
    Elem<DT>::unpack(make_uint4(w.w[0], w.w[1], 0, 0), all);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = all[i];
  } else {
    static_assert(N == 1, "8 or 16 bytes, or one value");
    f[0] = Elem<DT>::load(p, 0);
  }
}
template <int DT, int N>
__device__ __forceinline__ void store(char* p, const float* f) {
  constexpr int B = Elem<DT>::kBytes;
  if constexpr (N == 1) {
    if constexpr (DT == QK_F32)
      *reinterpret_cast<float*>(p) = f[0];
    else
      *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(qm::pack2_narrow<DT>(f[0], 0.0f));
  } else {
    constexpr int W = N * B / 4;  // words
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (DT == QK_F32)
        w[i] = __float_as_uint(f[i]);
      else
        w[i] = qm::pack2_narrow<DT>(f[2 * i], f[2 * i + 1]);
    }
    if constexpr (W == 2) {
      *reinterpret_cast<kv::Raw8<B>*>(p) = kv::Raw8<B>{{w[0], w[1]}};
    } else {
#pragma unroll
      for (int i = 0; i < W / 4; ++i)
        *reinterpret_cast<kv::Raw16<B>*>(p + 16 * i) = kv::Raw16<B>{{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]}};
    }
  }
}

// One workgroup per row (token); a head is L lanes of a wave, a lane has P
// pairs of it: two pieces of P elements r / 2 apart, or one of 2 P (pairs side
// by side, and the elements past r).  P = 4 where r is a multiple of 8;
// otherwise P = 1 and a lane takes U pairs, L apart.
template <int DT, int P, int L, int U, bool SIDE>
__global__ __launch_bounds__(kBlock) void norm_rope_kernel(NormRopeArgs a) {
  constexpr int B = Elem<DT>::kBytes;
  constexpr int kHeads = 64 / L;  // heads that a wave has at a time
  __shared__ Turn turns[kMostPairs];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = blockIdx.x;
  int pos;
  if (a.cu) {
    const kv::Owner o = kv::find_sequence(row, a.cu, a.start, a.seqs, [](int first, int) { return first; });
    if (o.seq < 0 || o.first < 0 || row >= o.next) return;  // uniform over the workgroup
    pos = static_cast<int>(static_cast<uint32_t>(o.value) + static_cast<uint32_t>(row - o.first));
  } else {
    pos = a.start[row];
  }
  if (static_cast<int>(threadIdx.x) < a.rotary / 2) turns[threadIdx.x] = turn_of(pos, a.freqs[threadIdx.x]);
  __syncthreads();

  const int within = lane % L, pairs = a.dim / 2, half = a.rotary / 2;
  const int all = a.heads + a.kv_heads;
  for (int h0 = wave * kHeads; h0 < all; h0 += kWaves * kHeads) {
    const int h = h0 + lane / L;
    const bool is_q = h < a.heads, live = h < all;
    const int64_t at = is_q ? row * a.ldq + static_cast<int64_t>(h) * a.dim : row * a.ldk + static_cast<int64_t>(h - a.heads) * a.dim;
    const int64_t to = is_q ? row * a.ldqo + static_cast<int64_t>(h) * a.dim : row * a.ldko + static_cast<int64_t>(h - a.heads) * a.dim;
    const char* const from = static_cast<const char*>(is_q ? a.q : a.k) + at * B;
    char* const dst = static_cast<char*>(is_q ? a.q_out : a.k_out) + to * B;
    const void* const weight = is_q ? a.q_weight : a.k_weight;
    float x[U][2 * P];
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = (within + u * L) * P;  // the first pair
#pragma unroll
      for (int e = 0; e < 2 * P; ++e) x[u][e] = 0.0f;
      if (!live || i >= pairs) continue;
      if (!SIDE && i < half) {
        load<DT, P>(from + i * B, x[u]);
        load<DT, P>(from + (half + i) * B, x[u] + P);
      } else if constexpr (P > 1) {
        load<DT, 2 * P>(from + 2 * i * B, x[u]);
      } else {
        load<DT, 1>(from + 2 * i * B, x[u]);
        load<DT, 1>(from + (2 * i + 1) * B, x[u] + 1);
      }
#pragma unroll
      for (int e = 0; e < 2 * P; ++e) sum = __builtin_fmaf(x[u][e], x[u][e], sum);
    }
    if (weight) {
#pragma unroll
      for (int d = 1; d < L; d <<= 1) sum += __shfl_xor(sum, d);
      const float inv = 1.0f / __builtin_sqrtf(sum / static_cast<float>(a.dim) + a.eps);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = (within + u * L) * P;
        if (i >= pairs) continue;
#pragma unroll
        for (int e = 0; e < 2 * P; ++e) {
          const int d = !SIDE && i < half ? (e < P ? i + e : half + i + e - P) : 2 * i + e;
          const float w = a.weight_f32 ? static_cast<const float*>(weight)[d] : Elem<DT>::load(weight, d);
          x[u][e] = (x[u][e] * inv) * w;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = (within + u * L) * P;
      if (!live || i >= pairs) continue;
      if (i < half) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const Turn t = turns[i + p];
          const int ia = SIDE ? 2 * p : p, ib = SIDE ? 2 * p + 1 : P + p;
          const float ya = x[u][ia], yb = x[u][ib];
          x[u][ia] = __builtin_fmaf(ya, t.cos, -(yb * t.sin));
          x[u][ib] = __builtin_fmaf(yb, t.cos, ya * t.sin);
        }
      }
      if (!SIDE && i < half) {
        store<DT, P>(dst + i * B, x[u]);
        store<DT, P>(dst + (half + i) * B, x[u] + P);
      } else if constexpr (P > 1) {
        store<DT, 2 * P>(dst + 2 * i * B, x[u]);
      } else {
        store<DT, 1>(dst + 2 * i * B, x[u]);
        store<DT, 1>(dst + (2 * i + 1) * B, x[u] + 1);
      }
    }
  }
}

template <int DT, int P, int L, int U>
hipError_t go(const NormRopeArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.tokens)), block(kBlock);
  return a.interleaved ? launch(norm_rope_kernel<DT, P, L, U, true>, grid, block, 0, stream, a)
                       : launch(norm_rope_kernel<DT, P, L, U, false>, grid, block, 0, stream, a);
}

template <int DT>
hipError_t by_size(const NormRopeArgs& a, hipStream_t stream) {
  if (a.rotary % 8 != 0) return go<DT, 1, 64, 2>(a, stream);
  if (a.dim <= 64) return go<DT, 4, 8, 1>(a, stream);
  if (a.dim <= 128) return go<DT, 4, 16, 1>(a, stream);
  return go<DT, 4, 32, 1>(a, stream);
}

}  // namespace

hipError_t launch_norm_rope(const NormRopeArgs& a, hipStream_t stream) {
  if (!grid_fits(a.tokens, kBlock)) return hipErrorInvalidConfiguration;
  switch (a.dtype) {
    case QK_F32: return by_size<QK_F32>(a, stream);
    case QK_BF16: return by_size<QK_BF16>(a, stream);
    default: return by_size<QK_F16>(a, stream);
  }
}

}  // namespace qk
