// Writing new tokens into a paged 8-bit key/value cache, and reading them
// back, for gfx950.
//
// The cache holds, for each block of P positions and each head, the keys'
// codes as [P][dim], the values' codes as [dim][P] and one binary32 scale for
// either.  Values lie transposed because the product P V wants consecutive
// positions in a lane; the write turns them in registers, once per token.
//
// A write gives a block the scale
//   need = max(max |x| over the call's new tokens in it, 1e-12) / qmax
//   s    = max(s_old, need)   if positions before the new ones hold tokens of
//                             the same sequence, need otherwise,
// codes its new tokens as round(x / s) and, where s > s_old, moves the earlier
// codes c to round(c * s_old / s).  A scale only grows while a block fills, so
// an earlier token is rounded again at most once per growth.  Positions past
// the sequence's new end keep what they held.  A non-finite scale (an infinity
// or a NaN among the block's tokens) gives codes 0, so the block reads as NaN.
//
// One wave holds 16 positions of one (block, head, K or V) in registers; the
// waves of a larger block exchange their maxima through LDS.  Each task is the
// only writer of its tile and its scale, so there are no atomics and the
// result does not depend on the order of execution.  Bound by HBM for prompts
// (3 bytes a value for 16-bit inputs), by latency for single tokens.  8 heads of
// dim 128: eight prompts of 300 to 2048 tokens in 15 us (63 MB, 4.2 TB/s), one
// token of each of 64 sequences in 5.4 us; read back, 100003 positions in 119 us
// (614 MB, 5.2 TB/s), four prefixes of up to 1500 in 6.5 us.
#include "kv_common.h"

namespace qk {
namespace {

using kv::Raw16;
using kv::Raw4;
using kv::Raw8;
using qm::Elem;

struct Params {
  KvCacheView c;
  KvRowsArgs a;
  int64_t items;
  int magic;  // u * magic >> 16 = u / (dim / 8) for u < 512
};

struct Task {
  bool live;
  int seq;
  int sub;      // which 16 positions of the block
  int lo, hi;   // the call's positions within the block
  int64_t row;  // the source row of position 0 of the block (may be below the sequence's first)
  int head;
  bool value;
  int64_t tile;  // block * heads + head
};

// The piece of work of this wave.  Every index that comes from device memory
// (rows, lengths, block numbers) is checked against what the host passed, and
// the piece is dropped when it points outside.
__device__ __forceinline__ Task find_task(const Params& p) {
  Task t{};
  const int waves = p.c.block >> 4;  // per task
  const int64_t wave = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 6) +
                       __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t task = wave / waves;
  t.sub = static_cast<int>(wave - task * waves);
  t.value = task & 1;
  const int64_t ih = task >> 1;
  const int64_t item = ih / p.c.heads;
  t.head = static_cast<int>(ih - item * p.c.heads);
  if (item >= p.items) return t;
  const kv::Owner o = kv::find_sequence(item, p.a.cu, p.a.start, p.a.seqs, [&](int row, int seq) {
    return kv::item_base(row, 1, p.c.block, 2, seq);
  });
  const int b = o.seq, first = o.first, n = o.next - o.first, start = o.value;
  if (b < 0 || first < 0 || n <= 0 || n > p.a.tokens - first || start < 0 || start > 0x7fffffff - n) return t;
  const int64_t at = start / p.c.block + (item - kv::item_base(first, 1, p.c.block, 2, b));
  const int64_t pos0 = at * p.c.block;
  if (pos0 >= static_cast<int64_t>(start) + n || at >= p.c.width) return t;
  const int page = p.c.table[b * p.c.ldt + at];
  if (page < 0 || page >= p.c.blocks) return t;
  t.lo = pos0 < start ? static_cast<int>(start - pos0) : 0;
  t.hi = static_cast<int>(min(static_cast<int64_t>(p.c.block), start + static_cast<int64_t>(n) - pos0));
  t.row = first + pos0 - start;
  t.tile = static_cast<int64_t>(page) * p.c.heads + t.head;
  t.seq = b;
  t.live = true;
  return t;
}

// 8 consecutive values of a row
template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t i, float (&f)[8]) {
  using E = Elem<DT>;
  const char* p = static_cast<const char*>(base) + i * E::kBytes;
#pragma unroll
  for (int h = 0; h < 8 / E::kPerUnit; ++h) {
    const auto w = reinterpret_cast<const Raw16<E::kBytes>*>(p)[h];
    float part[E::kPerUnit];
    E::unpack(make_uint4(w.w[0], w.w[1], w.w[2], w.w[3]), part);
#pragma unroll
    for (int e = 0; e < E::kPerUnit; ++e) f[h * E::kPerUnit + e] = part[e];
  }
}
// 2 consecutive values of a row
template <int DT>
__device__ __forceinline__ void load2(const void* base, int64_t i, float& a, float& b) {
  const char* p = static_cast<const char*>(base) + i * Elem<DT>::kBytes;
  if constexpr (DT == QK_F32) {
    const auto w = *reinterpret_cast<const Raw8<4>*>(p);
    a = __uint_as_float(w.w[0]);
    b = __uint_as_float(w.w[1]);
  } else {
    const uint32_t w = reinterpret_cast<const Raw4<2>*>(p)->w;
    if constexpr (DT == QK_BF16) {
      a = qm::bf16_lo(w);
      b = qm::bf16_hi(w);
    } else {
      a = qm::f16_bits(w & 0xffffu);
      b = qm::f16_bits(w >> 16);
    }
  }
}

// Four earlier codes moved from scale s0 to s.  The quotient is clamped, unlike
// a new token's: a code of -128, or a negative s0 larger than s, exceeds the
// range.  FP8 NaN codes stay NaN.
template <bool FP8>
__device__ __forceinline__ uint32_t moved4(uint32_t w, float s0, float s, float r) {
  float f[4];
  kv::codes4_to_float<FP8>(w, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] *= s0;
  if constexpr (FP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f[i] != f[i] ? f[i] : qm::fp8_ratio(f[i], s, r);
    return qm::pack4_fp8(f[0], f[1], f[2], f[3]);
  } else {
    return qm::pack4_low_bytes(qm::code_word_bounded(f[0], s, r), qm::code_word_bounded(f[1], s, r),
                               qm::code_word_bounded(f[2], s, r), qm::code_word_bounded(f[3], s, r));
  }
}

// DP: dim rounded up to 64, 128 or 256.
template <int DT, bool FP8, int DP>
__global__ __launch_bounds__(512) void kv_write_kernel(Params p) {
  constexpr int NU = DP / 32;               // 8-value units per lane of 16 rows of keys
  constexpr int NC = DP > 128 ? 2 : 1;      // pairs of columns per lane of 16 rows of values
  __shared__ uint32_t tops[8];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Task t = find_task(p);
  const int dim = p.c.dim, P = p.c.block;
  const int p0 = t.sub * 16;  // this wave's first position within the block
  const int64_t head0 = static_cast<int64_t>(t.head) * dim;
  // keys: [unit][8 columns]; values: [4 pair + quarter][4 positions of either column]
  float x[NU > NC * 4 ? NU : NC * 4][8];

  // Loads are unconditional, from the nearest row or column that there is, and
  // what lies outside is masked afterwards: a load under a condition would be
  // waited for on the spot.
  uint32_t top = 0;
  if (t.live) {
    if (!t.value) {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int u = min(lane + 64 * i, 2 * dim - 1), r = (u * p.magic) >> 16;
        const int d = (u - r * (dim / 8)) * 8, pos = min(max(p0 + r, t.lo), t.hi - 1);
        load8<DT>(p.a.k, (t.row + pos) * p.a.ldk + head0 + d, x[i]);
      }
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int u = min(lane + 64 * i, 2 * dim - 1), pos = p0 + ((u * p.magic) >> 16);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = qm::max_u32(m, __float_as_uint(x[i][e]) & 0x7fffffffu);
        top = qm::max_u32(top, pos >= t.lo && pos < t.hi ? m : 0u);
      }
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int d = 2 * (lane + 64 * c), dc = d < dim ? d : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int pos = min(max(p0 + i, t.lo), t.hi - 1);
          load2<DT>(p.a.v, (t.row + pos) * p.a.ldv + head0 + dc, x[c * 4 + i / 4][i % 4], x[c * 4 + i / 4][4 + i % 4]);
        }
      }
      // every row that was loaded is one of the call's, so none needs a mask for
      // the maximum: the nearest row only repeats
#pragma unroll
      for (int c = 0; c < 4 * NC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = qm::max_u32(top, __float_as_uint(x[c][e]) & 0x7fffffffu);
      if (p0 >= t.hi || p0 + 16 <= t.lo) top = 0;  // no new position among these 16
    }
  }
  float amax = qm::wave_max_nonneg(__uint_as_float(top));
  float* const scale_at = t.live ? (t.value ? p.c.v_scale : p.c.k_scale) + t.tile : nullptr;
  const float s0 = t.live && t.lo > 0 ? *scale_at : 0.0f;
  if (P > 16) {
    if (lane == 0) tops[wave] = __float_as_uint(amax);
    __syncthreads();
    const int waves = P >> 4, w0 = wave - t.sub;
    uint32_t m = 0;
    for (int w = 0; w < waves; ++w) m = qm::max_u32(m, tops[w0 + w]);
    amax = __uint_as_float(m);
  }
  if (!t.live) return;

  float s, r;
  if constexpr (FP8)
    qm::row_scale_fp8(amax, 0.0f, s, r);
  else
    qm::row_scale(amax, s, r);
  if (__float_as_uint(amax) >= 0x7f800000u) s = amax;  // infinite or NaN, kept
  bool moves = false;
  if (t.lo > 0 && !(s0 <= s)) {  // the earlier tokens' scale is larger, or one of the two is NaN
    s = s != s ? s : s0;
    r = 1.0f / s;
  } else if (t.lo > 0 && s0 != s) {
    moves = true;
  }
  const bool finite = __float_as_uint(s) < 0x7f800000u;
  if (t.lo > 0 && !finite) moves = true;  // codes become 0
  if (t.sub == 0 && lane == 0) *scale_at = s;

  if (!t.value) {
    uint8_t* const tile = p.c.k + t.tile * P * dim;
    uint2 old[NU];
    if (moves) {
#pragma unroll
      for (int i = 0; i < NU; ++i)
        old[i] = *reinterpret_cast<const uint2*>(tile + static_cast<int64_t>(p0) * dim + min(lane + 64 * i, 2 * dim - 1) * 8);
    }
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = lane + 64 * i, rr = (u * p.magic) >> 16, pos = p0 + rr;
      if (u >= 2 * dim || pos >= t.hi || (pos < t.lo && !moves)) continue;
      uint2 w = make_uint2(0, 0);
      if (finite) {
        if (pos >= t.lo) {
          w.x = kv::codes4_of<FP8>(reinterpret_cast<const float(&)[4]>(x[i][0]), s, r);
          w.y = kv::codes4_of<FP8>(reinterpret_cast<const float(&)[4]>(x[i][4]), s, r);
        } else {
          w.x = moved4<FP8>(old[i].x, s0, s, r);
          w.y = moved4<FP8>(old[i].y, s0, s, r);
        }
      }
      *reinterpret_cast<uint2*>(tile + static_cast<int64_t>(p0) * dim + u * 8) = w;
    }
  } else {
    if (p0 >= t.hi || (p0 + 16 <= t.lo && !moves)) return;  // nothing of these 16 positions changes
    uint8_t* const tile = p.c.v + t.tile * P * dim + p0;
    // byte masks of the 16 positions: new ones, earlier ones
    const int nlo = min(max(t.lo - p0, 0), 16), nhi = min(max(t.hi - p0, 0), 16);
    const bool whole = nlo == 0 && nhi == 16;
    uint4 old[NC][2];
    if (!whole) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int d = 2 * (lane + 64 * c);
          old[c][h] = *reinterpret_cast<const uint4*>(tile + static_cast<int64_t>((d < dim ? d : 0) + h) * P);
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = 2 * (lane + 64 * c);
      if (d >= dim) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = finite ? kv::codes4_of<FP8>(reinterpret_cast<const float(&)[4]>(x[c * 4 + i][4 * h]), s, r) : 0u;
        if (!whole) {
          const uint32_t was[4] = {old[c][h].x, old[c][h].y, old[c][h].z, old[c][h].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // bytes of the word's earlier positions, and of those up to the new end
            const int f = min(max(nlo - 4 * i, 0), 4), g = min(max(nhi - 4 * i, 0), 4);
            const uint32_t below = f >= 4 ? 0xffffffffu : (1u << (8 * f)) - 1u;
            const uint32_t upto = g >= 4 ? 0xffffffffu : (1u << (8 * g)) - 1u;
            uint32_t held = was[i];
            if (moves) held = ((finite ? moved4<FP8>(held, s0, s, r) : 0u) & below) | (held & ~below);
            w[i] = (w[i] & upto & ~below) | (held & (below | ~upto));
          }
        }
        *reinterpret_cast<uint4*>(tile + static_cast<int64_t>(d + h) * P) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// Stores of the rows read back: nontemporal, since what reads them next is far
// behind (100003 positions of 8 heads: 129 us with ordinary stores, 119 so).
template <int N, int ALIGN>
__device__ __forceinline__ void store_words(char* p, const uint32_t (&w)[N]) {
  typedef uint32_t words_t __attribute__((ext_vector_type(N), aligned(ALIGN)));
  words_t v;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = w[i];
  __builtin_nontemporal_store(v, reinterpret_cast<words_t*>(p));
}

template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t i, const float (&f)[8]) {
  using E = Elem<DT>;
  char* p = static_cast<char*>(base) + i * E::kBytes;
  if constexpr (DT == QK_F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w[4] = {__float_as_uint(f[4 * h]), __float_as_uint(f[4 * h + 1]), __float_as_uint(f[4 * h + 2]),
                             __float_as_uint(f[4 * h + 3])};
      store_words<4, 4>(p + 16 * h, w);
    }
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = qm::pack2_narrow<DT>(f[2 * e], f[2 * e + 1]);
    store_words<4, 2>(p, w);
  }
}

template <int DT, bool FP8, int DP>
__global__ __launch_bounds__(512) void kv_read_kernel(Params p) {
  constexpr int NU = DP / 32;
  constexpr int NC = DP > 128 ? 2 : 1;
  const int lane = threadIdx.x & 63;
  const Task t = find_task(p);
  if (!t.live) return;
  const int dim = p.c.dim, P = p.c.block;
  const int p0 = t.sub * 16;
  const int64_t head0 = static_cast<int64_t>(t.head) * dim;
  if (!t.value) {
    const float s = p.c.k_scale[t.tile];
    const uint8_t* const tile = p.c.k + t.tile * P * dim + static_cast<int64_t>(p0) * dim;
    uint2 codes[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i)
      codes[i] = *reinterpret_cast<const uint2*>(tile + min(lane + 64 * i, 2 * dim - 1) * 8);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = lane + 64 * i, r = (u * p.magic) >> 16, pos = p0 + r;
      if (u >= 2 * dim || pos < t.lo || pos >= t.hi) continue;
      const uint2 w = codes[i];
      float f[8];
      kv::codes4_to_float<FP8>(w.x, reinterpret_cast<float(&)[4]>(f[0]));
      kv::codes4_to_float<FP8>(w.y, reinterpret_cast<float(&)[4]>(f[4]));
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= s;
      store8<DT>(p.a.k, (t.row + pos) * p.a.ldk + head0 + (u - r * (dim / 8)) * 8, f);
    }
  } else {
    const float s = p.c.v_scale[t.tile];
    const uint8_t* const tile = p.c.v + t.tile * P * dim + p0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = 2 * (lane + 64 * c);
      if (d >= dim) continue;
      const uint4 a4 = *reinterpret_cast<const uint4*>(tile + static_cast<int64_t>(d) * P);
      const uint4 b4 = *reinterpret_cast<const uint4*>(tile + static_cast<int64_t>(d + 1) * P);
      const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float fa[4], fb[4];
        kv::codes4_to_float<FP8>(a[i], fa);
        kv::codes4_to_float<FP8>(b[i], fb);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int pos = p0 + 4 * i + e;
          if (pos < t.lo || pos >= t.hi) continue;
          char* const to = static_cast<char*>(p.a.v) +
                           ((t.row + pos) * p.a.ldv + head0 + d) * static_cast<int64_t>(Elem<DT>::kBytes);
          if constexpr (DT == QK_F32)
            store_words<2, 4>(to, {__float_as_uint(fa[e] * s), __float_as_uint(fb[e] * s)});
          else
            store_words<1, 2>(to, {qm::pack2_narrow<DT>(fa[e] * s, fb[e] * s)});
        }
      }
    }
  }
}

template <bool WRITE, int DT, bool FP8, int DP>
hipError_t go(const Params& p, hipStream_t stream) {
  const int waves = p.c.block == 128 ? 8 : 4;
  const int64_t tasks = p.items * p.c.heads * 2;
  const int64_t groups = (tasks * (p.c.block / 16) + waves - 1) / waves;
  if (!grid_fits(groups, 64 * waves)) return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(groups)), block(64 * waves);
  if constexpr (WRITE)
    return launch(kv_write_kernel<DT, FP8, DP>, grid, block, 0, stream, p);
  else
    return launch(kv_read_kernel<DT, FP8, DP>, grid, block, 0, stream, p);
}

template <bool WRITE, int DT, bool FP8>
hipError_t by_dim(const Params& p, hipStream_t stream) {
  if (p.c.dim <= 64) return go<WRITE, DT, FP8, 64>(p, stream);
  if (p.c.dim <= 128) return go<WRITE, DT, FP8, 128>(p, stream);
  return go<WRITE, DT, FP8, 256>(p, stream);
}

template <bool WRITE>
hipError_t by_type(const KvCacheView& c, const KvRowsArgs& a, hipStream_t stream) {
  const int n = c.dim / 8;
  const Params p{c, a, kv::item_base(a.tokens, 1, c.block, 2, a.seqs), (65536 + n - 1) / n};
  switch (a.dtype) {
    case QK_F32: return c.fp8 ? by_dim<WRITE, QK_F32, true>(p, stream) : by_dim<WRITE, QK_F32, false>(p, stream);
    case QK_BF16: return c.fp8 ? by_dim<WRITE, QK_BF16, true>(p, stream) : by_dim<WRITE, QK_BF16, false>(p, stream);
    default: return c.fp8 ? by_dim<WRITE, QK_F16, true>(p, stream) : by_dim<WRITE, QK_F16, false>(p, stream);
  }
}

}  // namespace

hipError_t launch_kv_cache_write(const KvCacheView& c, const KvRowsArgs& a, hipStream_t stream) {
  return by_type<true>(c, a, stream);
}

hipError_t launch_kv_cache_read(const KvCacheView& c, const KvRowsArgs& a, hipStream_t stream) {
  return by_type<false>(c, a, stream);
}

}  // namespace qk
