// Attention over the paged 8-bit cache for gfx950: softmax(scale q k^T) v with
// a causal mask (the sequence's rows are its last positions), an optional
// sliding window, and grouped heads.
//
// The (row, head) pairs of a sequence that share a kv head are the columns of
// a tile.  Scores are formed transposed, S^T = K Q^T: a lane then holds the
// scores of one column, so the running maximum, the sum and the rescaling of
// the output are plain lane arithmetic, and the probabilities are already
// where the second product, O^T = V^T P^T, wants them.  Its reduction index
// is a position, and the order of positions is free as long as P and V agree:
// the rows of K are taken in such an order that the scores a lane holds are
// those of 16 consecutive positions, which is how V lies in the cache.
//
// Arithmetic.  Codes are exact in binary16 (INT8 and e4m3 alike), so both
// products run on the binary16 matrix cores with binary32 sums.  bf16 queries
// are multiplied by a power of two per column that brings their largest
// element to [2^14, 2^15): exact down to 2^-29 of it, and below that the error
// is 2^-39 of it.  The block's scales never touch the codes: K's multiplies
// the scores, and V's goes into the exponent, p = 2^(s + log2 v_scale - m + 14)
// with m the running maximum of s + log2 v_scale, so that every p is at most
// 2^14 and normal in binary16 down to 2^-28 of the largest.  The sum l adds
// p / v_scale in binary32 from the unrounded p.  Rounding p to 11 bits is the
// only rounding below binary32 before the output's.
#include <algorithm>

#include "kv_common.h"

namespace qk {
namespace {

using kv::half8_t;
using kv::Raw16;

typedef float float4_t __attribute__((ext_vector_type(4)));

constexpr int kCols = 16;       // columns of a tile
constexpr int kGroup = 64;      // positions a wave takes at a time
constexpr int kWaves = 4;
constexpr float kNone = -3.0e38f;  // a maximum over nothing
constexpr float kLift = 14.0f;

struct Params {
  KvCacheView c;
  KvAttentionArgs a;
  int group;      // heads per kv head
  int chunk;      // positions per workgroup
  int splits;     // chunks of the longest range
  int cols;       // columns that the workspace holds per tile
  float scale2;   // scale * log2(e)
  float* part_o;  // [item][kv head][split][cols][dim]
  float* part_ml; // [item][kv head][split][cols][2]
};

// A tile's columns and the positions they see.
struct Tile {
  bool live;
  int seq, rows, len;   // the sequence, its rows, its positions
  int64_t row0;         // its first row
  int col0, ncols;      // the tile's columns of the sequence's rows * group
  int lo, hi;           // positions that some column sees: [lo, hi)
  int splits;
};

__device__ __forceinline__ Tile find_tile(const Params& p, int64_t item) {
  Tile t{};
  int tile;
  if (p.a.cu) {
    t.seq = kv::find_sequence(item, p.a.cu, p.a.seqs, p.group, kCols, 1);
    if (t.seq < 0) return t;
    const int first = p.a.cu[t.seq];
    t.rows = p.a.cu[t.seq + 1] - first;
    if (first < 0 || t.rows <= 0 || t.rows > p.a.tokens - first) return t;
    t.row0 = first;
    tile = static_cast<int>(item - kv::item_base(first, p.group, kCols, 1, t.seq));
  } else {
    const int tiles = (p.group + kCols - 1) / kCols;
    t.seq = static_cast<int>(item / tiles);
    t.rows = 1;
    t.row0 = t.seq;
    tile = static_cast<int>(item - static_cast<int64_t>(t.seq) * tiles);
  }
  const int64_t all = static_cast<int64_t>(t.rows) * p.group;
  t.col0 = tile * kCols;
  if (t.col0 >= all) return t;
  t.ncols = static_cast<int>(min(all - t.col0, static_cast<int64_t>(kCols)));
  t.len = min(max(p.a.lens[t.seq], 0), p.a.max_kv);  // max_kv is at most what the table covers
  const int first_pos = t.len - t.rows + t.col0 / p.group;
  const int last_pos = t.len - t.rows + (t.col0 + t.ncols - 1) / p.group;
  t.hi = min(last_pos + 1, t.len);
  t.lo = p.a.window > 0 ? max(first_pos - p.a.window + 1, 0) : 0;
  t.splits = t.hi > t.lo ? (t.hi - (t.lo & ~(kGroup - 1)) + p.chunk - 1) / p.chunk : 0;
  t.live = true;
  return t;
}

// A workgroup's place in the flat grid: `inner` fastest, then kv heads, then
// items.
struct Place {
  int inner, head;
  int64_t item;
};
__device__ __forceinline__ Place place_of(const Params& p, int inner) {
  const unsigned b = blockIdx.x, r = b / static_cast<unsigned>(inner);
  const unsigned item = r / static_cast<unsigned>(p.c.heads);
  return Place{static_cast<int>(b - r * inner), static_cast<int>(r - item * p.c.heads), item};
}

// Max and sum over the four lanes that hold one column (lane ^ 16, ^ 32).
__device__ __forceinline__ float column_max(float v) {
  uint32_t b = __float_as_uint(v);
  const auto r16 = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  v = __builtin_fmaxf(__uint_as_float(r16[0]), __uint_as_float(r16[1]));
  b = __float_as_uint(v);
  const auto r32 = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __builtin_fmaxf(__uint_as_float(r32[0]), __uint_as_float(r32[1]));
}
__device__ __forceinline__ float column_sum(float v) {
  uint32_t b = __float_as_uint(v);
  const auto r16 = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  v = __uint_as_float(r16[0]) + __uint_as_float(r16[1]);
  b = __float_as_uint(v);
  const auto r32 = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float(r32[0]) + __uint_as_float(r32[1]);
}

template <int DT>
__device__ __forceinline__ uint16_t narrow(float v) {
  if constexpr (DT == QK_BF16)
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

// The column's query as the second operand of K Q^T, and the power of two
// that undoes its scaling.  Lane (g, n) holds, for step 2 c + u, elements
// 64 c + 16 g + 8 u + j: the order in which 16-byte loads bring K.
template <int DT, int DP>
__device__ __forceinline__ float load_query(const void* q, int64_t at, int dim, bool valid,
                                            half8_t (&f)[DP / 32]) {
  const int g = (threadIdx.x & 63) >> 4;
  uint32_t raw[DP / 32][4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < DP / 32; ++i) {
    const int d = 64 * (i >> 1) + 16 * g + 8 * (i & 1);
    Raw16<2> w{{0, 0, 0, 0}};
    if (valid && d < dim) w = *reinterpret_cast<const Raw16<2>*>(static_cast<const char*>(q) + (at + d) * 2);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      raw[i][e] = w.w[e];
      top = qm::max_u32(top, qm::max_u32(w.w[e] & 0x7fffu, (w.w[e] >> 16) & 0x7fffu));
    }
  }
  if constexpr (DT == QK_F16) {
#pragma unroll
    for (int i = 0; i < DP / 32; ++i)
      f[i] = __builtin_bit_cast(half8_t, make_uint4(raw[i][0], raw[i][1], raw[i][2], raw[i][3]));
    return 1.0f;
  } else {
    const float amax = column_max(__uint_as_float(top << 16));
    const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;  // NaN and infinity stay what they are
#pragma unroll
    for (int i = 0; i < DP / 32; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        f[i][2 * w] = static_cast<_Float16>(__builtin_amdgcn_ldexpf(qm::bf16_lo(raw[i][w]), 14 - e));
        f[i][2 * w + 1] = static_cast<_Float16>(__builtin_amdgcn_ldexpf(qm::bf16_hi(raw[i][w]), 14 - e));
      }
    return __builtin_amdgcn_ldexpf(1.0f, e - 14);
  }
}

// One workgroup: one tile of up to 16 columns, one kv head, one chunk of
// positions.  Its four waves take groups of 64 positions in turn, each with a
// maximum, a sum and an output of its own, and join them through LDS at the
// end; nothing is shared before, so no wave waits for another.  A wave keeps a
// group's K and V (16 KB at dim 128) on its way from memory while it works on
// the group before.
template <int DT, bool FP8, int DP>
__global__ __launch_bounds__(64 * kWaves) void kv_attention_cols_kernel(Params p) {
  constexpr int KC = DP / 64;  // 16-byte pieces of a K row per lane
  constexpr int VC = DP / 16;  // 16-row pieces of V
  __shared__ float lds_o[kWaves][kCols][DP + 4];
  __shared__ float lds_m[kWaves][kCols], lds_l[kWaves][kCols];

  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place at = place_of(p, p.splits);
  const int split = at.inner, head = at.head;
  const int64_t item = at.item;
  const Tile t = find_tile(p, item);
  if (!t.live) return;
  const int dim = p.c.dim, P = p.c.block, group = p.group;
  const int begin0 = t.lo & ~(kGroup - 1);
  const int begin = begin0 + split * p.chunk, end = min(begin + p.chunk, t.hi);
  if (split > 0 && begin >= t.hi) return;  // split 0 stays, to write the rows that see nothing

  // this lane's column
  const int col = t.col0 + n;
  const bool valid = n < t.ncols;
  const int row = valid ? col / group : 0;
  const int64_t qrow = t.row0 + row;
  const int qhead = head * group + (valid ? col - row * group : 0);
  const int pos = t.len - t.rows + row;
  const int see_lo = p.a.window > 0 ? max(pos - p.a.window + 1, 0) : 0;
  const int see_hi = valid ? min(pos + 1, t.len) : 0;

  half8_t qf[DP / 32];
  const float unscale = load_query<DT, DP>(p.a.q, qrow * p.a.ldq + static_cast<int64_t>(qhead) * dim, dim, valid, qf);
  const float c_col = unscale * p.scale2;

  float4_t o[VC];
#pragma unroll
  for (int i = 0; i < VC; ++i) o[i] = float4_t{0, 0, 0, 0};
  float m = kNone, l = 0.0f;

  const int64_t head_bytes = static_cast<int64_t>(P) * dim;
  const int* const table = p.c.table + t.seq * p.c.ldt;
  // The block that holds 16 positions from `at` on, held to the range of
  // positions that are seen; entries outside the cache read block 0 and give
  // NaN scales.
  auto piece = [&](int at) { return min(max(at, t.lo & ~15), (t.hi - 1) & ~15); };

  for (int t0 = begin + wave * kGroup; t0 < end; t0 += kWaves * kGroup) {
    // K: lane's row r = n of tile i is position t0 + 16 (r / 4) + 4 i + r % 4
    const int kp = piece(t0 + 16 * (n >> 2)), vp = piece(t0 + 16 * g);
    int kb = table[kp / P], vb = table[vp / P];
    const bool bad = static_cast<unsigned>(vb) >= static_cast<unsigned>(p.c.blocks);
    kb = static_cast<unsigned>(kb) < static_cast<unsigned>(p.c.blocks) ? kb : 0;
    vb = bad ? 0 : vb;
    const int64_t kt = static_cast<int64_t>(kb) * p.c.heads + head, vt = static_cast<int64_t>(vb) * p.c.heads + head;
    const uint8_t* const krow = p.c.k + kt * head_bytes + static_cast<int64_t>((kp & (P - 1)) + (n & 3)) * dim + 16 * g;
    const uint8_t* const vrow = p.c.v + vt * head_bytes + static_cast<int64_t>(n) * P + (vp & (P - 1));
    uint4 kr[4][KC], vr[VC];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        kr[i][c] = make_uint4(0, 0, 0, 0);
        if (64 * c + 16 * g < dim) kr[i][c] = *reinterpret_cast<const uint4*>(krow + 4 * i * dim + 64 * c);
      }
#pragma unroll
    for (int i = 0; i < VC; ++i) {
      vr[i] = make_uint4(0, 0, 0, 0);
      if (16 * i < dim) vr[i] = *reinterpret_cast<const uint4*>(vrow + static_cast<int64_t>(16 * i) * P);
    }
    float ks = p.c.k_scale[vt], vs = p.c.v_scale[vt];
    if (bad) ks = vs = __builtin_nanf("");

    float4_t s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = float4_t{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        s[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv::codes8_to_half<FP8>(kr[i][c].x, kr[i][c].y), qf[2 * c], s[i], 0, 0, 0);
        s[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv::codes8_to_half<FP8>(kr[i][c].z, kr[i][c].w), qf[2 * c + 1], s[i], 0, 0, 0);
      }
    }
    const float c = c_col * ks, lvs = __builtin_amdgcn_logf(vs);
    float top = kNone;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int spot = t0 + 16 * g + 4 * i + e;
        const float y = __builtin_fmaf(s[i][e], c, lvs);
        s[i][e] = spot >= see_lo && spot < see_hi ? y : -__builtin_inff();
        top = __builtin_fmaxf(top, s[i][e]);
      }
    const float m_new = __builtin_fmaxf(m, column_max(top));
    const float shrink = __builtin_amdgcn_exp2f(m - m_new);
    m = m_new;
    float sum = 0.0f;
    half8_t pf[2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float pr = __builtin_amdgcn_exp2f(s[i][e] - m + kLift);
        sum += pr;
        pf[i >> 1][4 * (i & 1) + e] = static_cast<_Float16>(pr);
      }
    // a lane that sees none of these positions must not meet their scale
    l = l * shrink + (sum != 0.0f ? sum / vs : 0.0f);
    if (FP8) {  // positions past the end may hold any bytes, NaN codes among them
      const int have = min(t.len - vp, 16);
      if (have < 16) {
        uint32_t mask[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int b = min(max(have - 4 * w, 0), 4);
          mask[w] = b >= 4 ? 0xffffffffu : (1u << (8 * b)) - 1u;
        }
#pragma unroll
        for (int i = 0; i < VC; ++i) {
          vr[i].x &= mask[0];
          vr[i].y &= mask[1];
          vr[i].z &= mask[2];
          vr[i].w &= mask[3];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < VC; ++i) {
      o[i] *= shrink;
      o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv::codes8_to_half<FP8>(vr[i].x, vr[i].y), pf[0], o[i], 0, 0, 0);
      o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv::codes8_to_half<FP8>(vr[i].z, vr[i].w), pf[1], o[i], 0, 0, 0);
    }
  }

  // join the four waves
  l = column_sum(l);
  if (g == 0) {
    lds_m[wave][n] = m;
    lds_l[wave][n] = l;
  }
#pragma unroll
  for (int i = 0; i < VC; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) lds_o[wave][n][16 * i + 4 * g + e] = o[i][e];
  __syncthreads();

  const int64_t slot = ((item * p.c.heads + head) * p.splits + split) * p.cols;
  for (int k = wave; k < t.ncols; k += kWaves) {
    float mm = lds_m[0][k], ll = 0.0f, f[kWaves];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mm = __builtin_fmaxf(mm, lds_m[w][k]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      f[w] = __builtin_amdgcn_exp2f(lds_m[w][k] - mm);
      ll = __builtin_fmaf(lds_l[w][k], f[w], ll);
    }
    const int kc = t.col0 + k, kr = kc / group, kh = head * group + kc - kr * group;
    const int64_t out_at = (t.row0 + kr) * p.a.heads + kh;
    const bool last = t.splits <= 1;
    const float inv = ll != 0.0f ? 1.0f / ll : 0.0f;
    for (int d = lane; d < dim; d += 64) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v = __builtin_fmaf(lds_o[w][k][d], f[w], v);
      if (last)
        static_cast<uint16_t*>(p.a.out)[out_at * dim + d] = narrow<DT>(v * inv);
      else
        p.part_o[(slot + k) * dim + d] = v;
    }
    if (lane == 0) {
      if (!last) {
        p.part_ml[(slot + k) * 2] = mm;
        p.part_ml[(slot + k) * 2 + 1] = ll;
      } else if (p.a.lse) {
        p.a.lse[out_at] = ll != 0.0f ? (mm - kLift + __builtin_amdgcn_logf(ll)) * 0.6931471805599453f : -__builtin_inff();
      }
    }
  }
}

// Joins the chunks of a tile: one wave per column.
template <int DT, int DP>
__global__ __launch_bounds__(64) void kv_attention_join_kernel(Params p) {
  const Place at = place_of(p, p.cols);
  const int k = at.inner, head = at.head;
  const int64_t item = at.item;
  const Tile t = find_tile(p, item);
  if (!t.live || t.splits <= 1 || k >= t.ncols) return;
  const int lane = threadIdx.x, dim = p.c.dim;
  const int64_t slot = (item * p.c.heads + head) * p.splits;
  const int splits = min(t.splits, p.splits);
  float m = kNone;
  for (int s = lane; s < splits; s += 64) m = __builtin_fmaxf(m, p.part_ml[((slot + s) * p.cols + k) * 2]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = __builtin_fmaxf(m, __shfl_xor(m, o));
  float l = 0.0f, v[DP / 64];
#pragma unroll
  for (int i = 0; i < DP / 64; ++i) v[i] = 0.0f;
  for (int s = 0; s < splits; ++s) {
    const int64_t part = (slot + s) * p.cols + k;
    const float f = __builtin_amdgcn_exp2f(p.part_ml[part * 2] - m);
    l = __builtin_fmaf(p.part_ml[part * 2 + 1], f, l);
#pragma unroll
    for (int i = 0; i < DP / 64; ++i)
      if (lane + 64 * i < dim) v[i] = __builtin_fmaf(p.part_o[part * dim + lane + 64 * i], f, v[i]);
  }
  const int kc = t.col0 + k, kr = kc / p.group, kh = head * p.group + kc - kr * p.group;
  const int64_t out_at = (t.row0 + kr) * p.a.heads + kh;
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int i = 0; i < DP / 64; ++i)
    if (lane + 64 * i < dim) static_cast<uint16_t*>(p.a.out)[out_at * dim + lane + 64 * i] = narrow<DT>(v[i] * inv);
  if (lane == 0 && p.a.lse)
    p.a.lse[out_at] = l != 0.0f ? (m - kLift + __builtin_amdgcn_logf(l)) * 0.6931471805599453f : -__builtin_inff();
}

// How a call is cut: tiles, chunks of positions, workspace.
struct Plan {
  int64_t items;
  int chunk, splits, cols;
  size_t bytes;
};

Plan plan_of(int seqs, int tokens, int heads, int kv_heads, int dim, bool ragged, int max_kv, int window) {
  Plan pl{};
  const int group = heads / kv_heads;
  pl.items = ragged ? kv::item_base(tokens, group, kCols, 1, seqs)
                    : static_cast<int64_t>(seqs) * ((group + kCols - 1) / kCols);
  // positions that one tile can see, from a multiple of 64 on
  int64_t range = max_kv;
  if (window > 0) range = std::min<int64_t>(range, static_cast<int64_t>(window) + kCols);
  range += kGroup;
  const int64_t tiles = std::max<int64_t>(1, pl.items * kv_heads);
  // about 1024 workgroups (four per CU), chunks of 256 positions at least
  int64_t chunk = (range * tiles + 1023) / 1024;
  chunk = std::max<int64_t>(256, (chunk + 255) / 256 * 256);
  chunk = std::min<int64_t>(chunk, (range + 255) / 256 * 256);
  pl.chunk = static_cast<int>(std::min<int64_t>(chunk, 1 << 30));
  pl.splits = static_cast<int>((range + pl.chunk - 1) / pl.chunk);
  pl.cols = ragged ? kCols : std::min(group, kCols);
  if (pl.splits > 1)
    pl.bytes = static_cast<size_t>(pl.items) * kv_heads * pl.splits * pl.cols * (dim + 2) * sizeof(float);
  return pl;
}

template <int DT, bool FP8, int DP>
hipError_t go(const Params& p, int64_t items, hipStream_t stream) {
  const int64_t tiles = items * p.c.heads;
  if (tiles * std::max(p.splits, p.cols) > 0x7fffffff) return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(tiles * p.splits));
  hipError_t e = launch(kv_attention_cols_kernel<DT, FP8, DP>, grid, dim3(64 * kWaves), 0, stream, p);
  if (e != hipSuccess || p.splits <= 1) return e;
  return launch(kv_attention_join_kernel<DT, DP>, dim3(static_cast<unsigned>(tiles * p.cols)), dim3(64), 0, stream, p);
}

template <int DT, bool FP8>
hipError_t by_dim(const Params& p, int64_t items, hipStream_t stream) {
  if (p.c.dim <= 64) return go<DT, FP8, 64>(p, items, stream);
  if (p.c.dim <= 128) return go<DT, FP8, 128>(p, items, stream);
  return go<DT, FP8, 256>(p, items, stream);
}

}  // namespace

size_t kv_attention_workspace_bytes(int seqs, int tokens, int heads, int kv_heads, int dim, int max_kv,
                                    int window) {
  // enough for either form of the call
  return std::max(plan_of(seqs, tokens, heads, kv_heads, dim, true, max_kv, window).bytes,
                  plan_of(seqs, tokens, heads, kv_heads, dim, false, max_kv, window).bytes);
}

hipError_t launch_kv_attention(const KvCacheView& c, const KvAttentionArgs& a, hipStream_t stream) {
  const Plan pl = plan_of(a.seqs, a.tokens, a.heads, c.heads, c.dim, a.cu != nullptr, a.max_kv, a.window);
  Params p{c, a, a.heads / c.heads, pl.chunk, pl.splits, pl.cols, a.scale * 1.4426950408889634f, nullptr, nullptr};
  p.part_o = static_cast<float*>(a.workspace);
  p.part_ml = p.part_o + static_cast<size_t>(pl.items) * c.heads * pl.splits * pl.cols * c.dim;
  if (a.dtype == QK_BF16)
    return c.fp8 ? by_dim<QK_BF16, true>(p, pl.items, stream) : by_dim<QK_BF16, false>(p, pl.items, stream);
  return c.fp8 ? by_dim<QK_F16, true>(p, pl.items, stream) : by_dim<QK_F16, false>(p, pl.items, stream);
}

}  // namespace qk
