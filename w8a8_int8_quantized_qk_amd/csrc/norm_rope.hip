// Root-mean-square norm of every head's query and key and the rotation by its
// position, in one pass, for gfx950:
//   y = (x * inv) * w,  inv = 1 / sqrt(mean(x^2) + eps)    (binary32, and the mean in
//                       binary64 where its squares leave that; y = x without w)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
// for the pairs (a, b) = (i, i + r / 2), or (2 i, 2 i + 1), of a head's first r
// elements, at the angle position * freqs[i]; the other elements keep y.
//
// The angle of a far position has many whole turns, so it is formed and its
// turns are taken off in binary64: t = position * (freqs[i] / 2 pi), t - rint(4 t) / 4
// is exact and at most an eighth of a turn, and loses nothing when it is rounded to
// binary32 (t is off by less than 2^-51 of itself, three roundings: 2^-25 of a turn at
// position 2^29).
// Sine and cosine of at most pi / 4 are their Taylor sums in binary32, up to
// x^9 and x^10 (the next terms are below 2^-29 and 2^-33).
#include <algorithm>
#include <type_traits>

#include "kv_common.h"

namespace qk {
namespace {

using qm::Elem;

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / 64;
constexpr int kMostPairs = 128;
constexpr int64_t kFill = 16384;  // waves that keep the memory busy (4096: 29.2 us for 27.3 in the case below)
// Outputs beyond this are stored past the caches, which do not hold them until they
// are read.
constexpr int64_t kPastCaches = 8 << 20;
// A mean (with eps) from here on has lost nothing to squares below binary32's range:
// those of a head of 256 are less than 2^-141 together.
constexpr float kLeastMean = 0x1p-100f;

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
template <int DT, int N, bool PAST>
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
      const kv::Loose8 v = {w[0], w[1]};
      if constexpr (PAST)
        __builtin_nontemporal_store(v, reinterpret_cast<kv::Loose8*>(p));
      else
        *reinterpret_cast<kv::Loose8*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const kv::Loose16 v = {w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
        if constexpr (PAST)
          __builtin_nontemporal_store(v, reinterpret_cast<kv::Loose16*>(p + 16 * i));
        else
          *reinterpret_cast<kv::Loose16*>(p + 16 * i) = v;
      }
    }
  }
}

// A value of the lane that `move` names for each half of its bits: of binary32
// in one exchange, of binary64 in two.
template <typename F>
__device__ __forceinline__ float exchanged(float v, F move) { return __uint_as_float(move(__float_as_uint(v))); }
template <typename F>
__device__ __forceinline__ double exchanged(double v, F move) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
  const uint32_t lo = move(static_cast<uint32_t>(b)), hi = move(static_cast<uint32_t>(b >> 32));
  return __longlong_as_double(static_cast<long long>(static_cast<uint64_t>(hi) << 32 | lo));
}

// Sum over the L neighbouring lanes that hold a head.
template <int L, typename T>
__device__ __forceinline__ T head_sum(T v) {
  auto from = [&](auto ctrl) {
    return exchanged(v, [](uint32_t b) {
      return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(b), decltype(ctrl)::value, 0xF, 0xF, false));
    });
  };
  v += from(std::integral_constant<int, 0xB1>{});                         // lane ^ 1
  v += from(std::integral_constant<int, 0x4E>{});                         // lane ^ 2
  if constexpr (L >= 8) v += from(std::integral_constant<int, 0x141>{});  // the other four of eight
  if constexpr (L >= 16) v += from(std::integral_constant<int, 0x140>{}); // the other eight of 16
  if constexpr (L >= 32) {
    v = exchanged(v, [](uint32_t b) { return __builtin_amdgcn_permlane16_swap(b, b, false, false)[0]; }) +
        exchanged(v, [](uint32_t b) { return __builtin_amdgcn_permlane16_swap(b, b, false, false)[1]; });
  }
  if constexpr (L >= 64) {
    v = exchanged(v, [](uint32_t b) { return __builtin_amdgcn_permlane32_swap(b, b, false, false)[0]; }) +
        exchanged(v, [](uint32_t b) { return __builtin_amdgcn_permlane32_swap(b, b, false, false)[1]; });
  }
  return v;
}

// A wave has a row's position, the sines and cosines of its pairs (a pair or two
// per lane, handed round through LDS of its own) and `groups` of its heads, 64 / L
// of them at a time: L lanes to a head, P pairs to a lane.  Those are one piece of
// 2 P elements where pairs lie side by side, else two pieces of P, r / 2 apart, or,
// past r, half of what is left apart.  A piece is 16 bytes, next to its neighbour's, where r
// allows it (32 bytes per lane in two halves took up to twice as long); where r is no
// multiple of 8 (4 for binary32 side by side) P is 1, and a lane takes U pairs, L apart.
//
// Bound by memory: 7690 rows of 32 + 8 heads of 128, bf16, the outputs of three calls in
// turn, 26.6 us (5.9 TB/s; 34.6 with plain stores; 28.6 with two groups in flight per wave,
// for 27); r = 64 side by side 28.9 (36.0); in place 27 to 30 either way; with P = 1, dim 80
// and r = 20 56.  One row 3.3 us, 64 rows 3.5.  (Eight waves a SIMD are asked for where that costs no
// scratch: without it 27.4 us for 26.3 at r = 64 side by side, one output, and 34.6 for 31.9
// at 4000 rows of 40 heads of 80 where P is 1; with P = 8 values went to scratch, 9.7 us for
// 7.9 at 4000 rows of 40 heads of 64.)
template <int DT, int P, int L, int U, bool SIDE, bool PAST>
__global__ __launch_bounds__(kBlock, SIDE || P == 1 ? 8 : 1) void norm_rope_kernel(NormRopeArgs a, int parts, int groups) {
  constexpr int B = Elem<DT>::kBytes;
  constexpr int kHeads = 64 / L;  // of a group
  __shared__ Turn all_turns[kWaves][kMostPairs];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned item = blockIdx.x * kWaves + wave;
  const unsigned of_row = item / static_cast<unsigned>(parts);
  if (of_row >= static_cast<unsigned>(a.tokens)) return;
  const int row = static_cast<int>(of_row), part = static_cast<int>(item - of_row * parts);
  Turn* const turns = all_turns[wave];
  const int within = lane % L, pairs = a.dim / 2, half = a.rotary / 2;
  // elements of the P pairs from pair i on
  auto first_of = [&](int i) { return SIDE ? 2 * i : i < half ? i : half + i; };
  auto second_of = [&](int i) { return SIDE ? 2 * i + P : i < half ? half + i : pairs + i; };
  const int q_groups = (a.heads + kHeads - 1) / kHeads, last = q_groups + (a.kv_heads + kHeads - 1) / kHeads;
  const int g0 = part * groups, g1 = min(g0 + groups, last);

  bool ready = false;  // the row's turns
  bool mine = true;    // some sequence's row
  auto prepare = [&] {
    if (ready) return;
    ready = true;
    int pos;
    if (a.cu) {
      const kv::Owner o = kv::find_sequence(row, a.cu, a.start, a.seqs, [](int first, int) { return first; });
      mine = o.seq >= 0 && o.first >= 0 && row < o.next;
      pos = static_cast<int>(static_cast<uint32_t>(o.value) + static_cast<uint32_t>(row - o.first));
    } else {
      pos = a.start[row];
    }
    for (int i = lane; i < half; i += 64) turns[i] = turn_of(pos, a.freqs[i]);
    __builtin_amdgcn_wave_barrier();
  };

  // heads of one tensor, groups first .. end of it
  auto side = [&](int first, int end, const void* in, int64_t ld, int heads, const void* weight, void* out, int64_t ldo) {
    if (first >= end) return;
    const char* const from_row = static_cast<const char*>(in) + row * ld * B;
    char* const to_row = static_cast<char*>(out) + row * ldo * B;
    float w[U][2 * P];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 2 * P; ++e) w[u][e] = 1.0f;
    if (weight) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = (within + u * L) * P;
        if (i >= pairs) continue;
        const int at = first_of(i), other = second_of(i);
        if (a.weight_f32) {
          const float* const f = static_cast<const float*>(weight);
#pragma unroll
          for (int e = 0; e < P; ++e) w[u][e] = f[at + e], w[u][P + e] = f[other + e];
        } else {
          const char* const f = static_cast<const char*>(weight);
          if constexpr (SIDE && P > 1) {
            load<DT, 2 * P>(f + at * B, w[u]);
          } else {
            load<DT, P>(f + at * B, w[u]);
            load<DT, P>(f + other * B, w[u] + P);
          }
        }
      }
    }
    for (int group = first; group < end; ++group) {
      const int h = group * kHeads + lane / L;
      const char* const from = from_row + h * a.dim * B;
      float x[U][2 * P];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = (within + u * L) * P;  // the first pair
#pragma unroll
        for (int e = 0; e < 2 * P; ++e) x[u][e] = 0.0f;
        if (h >= heads || i >= pairs) continue;
        if constexpr (SIDE && P > 1) {
          load<DT, 2 * P>(from + first_of(i) * B, x[u]);
        } else {
          load<DT, P>(from + first_of(i) * B, x[u]);
          load<DT, P>(from + second_of(i) * B, x[u] + P);
        }
      }
      prepare();
      if (!mine) return;
      if (weight) {
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < 2 * P; ++e) sum = __builtin_fmaf(x[u][e], x[u][e], sum);
        const float mean = head_sum<L>(sum) / static_cast<float>(a.dim) + a.eps;
        float inv = 1.0f / __builtin_sqrtf(mean);
        // Squares that left binary32's range (beyond it, or too small beside eps): the
        // sum again in binary64, and a power of two in x where the quotient has no
        // binary32 of full precision.  Heads in range keep what they have; binary16's
        // squares are all in range.
        const bool out_of_range = h < heads && !(mean >= kLeastMean && mean < __builtin_inff());
        if (DT != QK_F16 && __any(out_of_range)) [[unlikely]] {
          double wide = 0.0;
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 2 * P; ++e) {
              const double d = static_cast<double>(x[u][e]);
              wide = __builtin_fma(d, d, wide);
            }
          wide = 1.0 / sqrt(head_sum<L>(wide) / static_cast<double>(a.dim) + static_cast<double>(a.eps));
          const float raise = !out_of_range ? 1.0f : wide > 0x1p126 ? 0x1p32f : wide < 0x1p-126 ? 0x1p-8f : 1.0f;
          if (out_of_range) inv = static_cast<float>(wide / static_cast<double>(raise));
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 2 * P; ++e) x[u][e] *= raise;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < 2 * P; ++e) x[u][e] = (x[u][e] * inv) * w[u][e];
      }
      char* const to = to_row + h * a.dim * B;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = (within + u * L) * P;
        if (h >= heads || i >= pairs) continue;
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
        if constexpr (SIDE && P > 1) {
          store<DT, 2 * P, PAST>(to + first_of(i) * B, x[u]);
        } else {
          store<DT, P, PAST>(to + first_of(i) * B, x[u]);
          store<DT, P, PAST>(to + second_of(i) * B, x[u] + P);
        }
      }
    }
  };
  side(g0, min(g1, q_groups), a.q, a.ldq, a.heads, a.q_weight, a.q_out, a.ldqo);
  side(max(g0, q_groups) - q_groups, g1 - q_groups, a.k, a.ldk, a.kv_heads, a.k_weight, a.k_out, a.ldko);
}

template <int DT, int P, int L, int U, bool SIDE>
hipError_t go(const NormRopeArgs& a, hipStream_t stream) {
  constexpr int kHeads = 64 / L;
  const int groups = (a.heads + kHeads - 1) / kHeads + (a.kv_heads + kHeads - 1) / kHeads;
  // a wave per row where there are enough rows, else as many as there are groups
  const int wanted = static_cast<int>(std::min<int64_t>(groups, std::max<int64_t>(1, kFill / a.tokens)));
  const int each = (groups + wanted - 1) / wanted, parts = (groups + each - 1) / each;
  const int64_t blocks = (static_cast<int64_t>(a.tokens) * parts + kWaves - 1) / kWaves;
  if (!grid_fits(blocks, kBlock)) return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks)), block(kBlock);
  if constexpr (P > 1) {
    const int64_t bytes = static_cast<int64_t>(a.tokens) * (a.heads + a.kv_heads) * a.dim * Elem<DT>::kBytes;
    if (bytes > kPastCaches) return launch(norm_rope_kernel<DT, P, L, U, SIDE, true>, grid, block, 0, stream, a, parts, each);
  }
  return launch(norm_rope_kernel<DT, P, L, U, SIDE, false>, grid, block, 0, stream, a, parts, each);
}

template <int DT, int P, bool SIDE>
hipError_t by_dim(const NormRopeArgs& a, hipStream_t stream) {
  if (a.dim <= 64) return go<DT, P, 32 / P, 1, SIDE>(a, stream);
  if (a.dim <= 128) return go<DT, P, 64 / P, 1, SIDE>(a, stream);
  return go<DT, P, 128 / P, 1, SIDE>(a, stream);
}

template <int DT>
hipError_t by_size(const NormRopeArgs& a, hipStream_t stream) {
  constexpr int kSide = Elem<DT>::kPerUnit / 2;  // pairs in 16 bytes
  if (a.interleaved) {
    if (a.rotary % (2 * kSide) == 0) return by_dim<DT, kSide, true>(a, stream);
    return go<DT, 1, 64, 2, true>(a, stream);
  }
  if constexpr (DT != QK_F32) {
    if (a.rotary % 16 == 0) return by_dim<DT, 8, false>(a, stream);
  }
  if (a.rotary % 8 == 0) return by_dim<DT, 4, false>(a, stream);
  return go<DT, 1, 64, 2, false>(a, stream);
}

}  // namespace

hipError_t launch_norm_rope(const NormRopeArgs& a, hipStream_t stream) {
  if (a.tokens >= 1 << 24) return hipErrorInvalidConfiguration;
  switch (a.dtype) {
    case QK_F32: return by_size<QK_F32>(a, stream);
    case QK_BF16: return by_size<QK_BF16>(a, stream);
    default: return by_size<QK_F16>(a, stream);
  }
}

}  // namespace qk
