// Attention over the paged 8-bit cache for gfx950: softmax(scale q k^T) v with
// a causal mask (the sequence's rows are its last positions), an optional
// sliding window, and grouped heads.
//
// The (row, head) pairs of a sequence that share a kv head are the columns of
// a tile: 16 in kv_attention_cols_kernel (sequences with up to 64 columns:
// single tokens; bound by the cache's bytes), 128 in kv_attention_tile_kernel
// (prompts; bound by the matrix cores and the exponentials).  Scores are formed
// transposed, S^T = K Q^T: a lane then holds the scores of one column, so the
// running maximum, the sum and the rescaling of the output are plain lane
// arithmetic, and the probabilities are already where the second product,
// O^T = V^T P^T, wants them.  Its reduction index
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
// with m at most 1.9 below the running maximum of s + log2 v_scale, so that
// every p is below 2^15.9 and normal in binary16 down to 2^-28 of the largest.
// The sum l adds p / v_scale in binary32 from the unrounded p.  Rounding p to
// 11 bits is the only rounding below binary32 before the output's.
//
// Scales may be any finite numbers.  Where K's is negative, or V's is outside
// [2^-64, 2^126] (a fresh cache's is 0), the scores are multiplied out before
// their maximum is taken, the exponent takes V's magnitude raised to 2^-64, and
// the power of two (or sign, or 0) that is left multiplies p, rounded, or the
// codes in binary16: exact but for binary16's smallest numbers, which costs
// values below 2^-64 an absolute error of 2^-88 at most.  The sum l keeps binary32's precision as
// long as the V scales that a row sees, so raised, lie within 2^92 of each other.
#include <algorithm>
#include <cmath>

#include "kv_common.h"

namespace qk {
namespace {

using kv::half8_t;
using kv::Raw16;

typedef float float4_t __attribute__((ext_vector_type(4)));
typedef float float16_t __attribute__((ext_vector_type(16)));

constexpr int kCols = 16;        // columns of a tile of kv_attention_cols_kernel
constexpr int kSmall = 64;       // columns of a sequence that it takes (in tiles of 16)
constexpr int kTileCols = 128;   // columns of a tile of kv_attention_tile_kernel
constexpr int kGroup = 64;       // positions taken at a time
constexpr int kWaves = 4;
constexpr float kNone = -3.0e38f;  // a maximum over nothing
constexpr float kLift = 14.0f;
constexpr float kSlack = 1.9f;     // 2^(kLift + kSlack) < 65504
constexpr float kLeastScale = 5.421010862427522e-20f;  // 2^-64: V scales from here ...
constexpr float kMostScale = 8.507059173023462e37f;    // ... to 2^126 go into the exponent as they are
constexpr int kJoinHere = 16;      // most chunks that a tile's last workgroup joins
constexpr int kCounters = 16384;   // arrival counters at the front of the workspace
// Partial results of single tokens are held to this: chunks of thousands of
// tiles over long ranges would take gigabytes, and that many tiles fill the
// chip without them.
constexpr int64_t kMostPartials = 1 << 30;

struct Params {
  KvCacheView c;
  KvAttentionArgs a;
  int block_shift;  // log2 of the cache's block
  int group;        // heads per kv head
  int tiles;        // cols kernel: tiles per sequence
  unsigned items;
  int small;        // tile kernel: columns of a sequence that the other kernel takes (kSmall or 0)
  int chunk;        // positions per workgroup
  int splits;       // chunks of the longest range
  int cols;         // columns that the workspace holds per tile
  float scale2;     // |scale| * log2(e)
  uint32_t flip;    // sign bits that turn q where the scale is negative
  bool join_later;  // cols kernel: the chunks are joined by a launch of their own
  unsigned* arrived;  // [item][kv head], zero between calls (cols kernel)
  float* part_o;      // [item][kv head][split][cols][dim]
  float* part_ml;     // [item][kv head][split][cols][2]
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

// The first position that a row at `pos` sees (a row before position 0 none,
// whatever this says; held to 0 first, for windows close to 2^31).
__device__ __forceinline__ int first_seen(const Params& p, int pos) {
  return p.a.window > 0 ? max(max(pos, 0) - p.a.window + 1, 0) : 0;
}

// Columns col0 .. col0 + size of the sequence whose rows are already in t.
__device__ __forceinline__ void set_range(const Params& p, Tile& t, int64_t col0, int size, int len) {
  const int64_t all = static_cast<int64_t>(t.rows) * p.group;
  if (col0 >= all) return;
  t.col0 = static_cast<int>(col0);
  t.ncols = static_cast<int>(min(all - col0, static_cast<int64_t>(size)));
  t.len = min(max(len, 0), p.a.max_kv);  // max_kv is at most what the table covers
  const int first_pos = t.len - t.rows + t.col0 / p.group;
  const int last_pos = t.len - t.rows + (t.col0 + t.ncols - 1) / p.group;
  t.hi = min(last_pos + 1, t.len);
  t.lo = first_seen(p, first_pos);
  t.splits = t.hi > t.lo ? (t.hi - (t.lo & ~(kGroup - 1)) + p.chunk - 1) / p.chunk : 0;
  t.live = true;
}

// Tiles of 16 columns: item = sequence * tiles + tile; longer sequences are
// the other kernel's.  Partial results have room for the columns that max_q
// rows have; rows beyond it, of which only the device knows, stay out of them.
__device__ __forceinline__ Tile find_cols(const Params& p, unsigned item) {
  Tile t{};
  t.seq = static_cast<int>(item / static_cast<unsigned>(p.tiles));
  t.rows = 1;
  t.row0 = t.seq;
  if (p.a.cu) {
    const int first = p.a.cu[t.seq];
    t.rows = p.a.cu[t.seq + 1] - first;
    t.row0 = first;
    if (first < 0 || t.rows <= 0 || t.rows > p.a.tokens - first) return t;
    if (static_cast<int64_t>(t.rows) * p.group > kSmall) return t;
  }
  set_range(p, t, static_cast<int64_t>(item - static_cast<unsigned>(t.seq) * p.tiles) * kCols,
            p.splits > 1 ? p.cols : kCols, p.a.lens[t.seq]);
  return t;
}

// Tiles of 128 columns, laid over the ragged rows: sequence b, from `row` on,
// owns items tile_base(row, b) .. tile_base(next row, b + 1).  n rows of it have
// n * group columns and need ceil(n * group / 128) of them: the first term gives
// floor(n * group / 128), the second, where sequences of up to `small` columns are
// the other kernel's, at least one more to every longer sequence and at most
// one for every small + 1 columns of the call, however many sequences there are.
// A call's columns fit in 31 bits, which the host checks with Int = int64_t; the
// device counts in 32 bits, where an offset outside the call may give any base:
// it is the sequence's alone, and such a sequence is dropped.
template <typename Int>
__host__ __device__ __forceinline__ int64_t tile_base(Int row, int group, int small, Int b) {
  const Int cols = row * static_cast<Int>(group), many = cols / (kSmall + 1);
  return static_cast<int64_t>(cols / kTileCols + (small && many < b ? many : b));
}
__device__ __forceinline__ int64_t tile_base_of(const Params& p, int row, int b) {
  return tile_base<uint32_t>(row, p.group, p.small, b);
}

__device__ __forceinline__ Tile find_tile(const Params& p, int64_t item) {
  Tile t{};
  const kv::Owner o = kv::find_sequence(item, p.a.cu, p.a.lens, p.a.seqs, [&](int row, int seq) {
    return tile_base_of(p, row, seq);
  });
  t.seq = o.seq;
  t.rows = o.next - o.first;
  t.row0 = o.first;
  if (o.seq < 0 || o.first < 0 || t.rows <= 0 || t.rows > p.a.tokens - o.first) return t;
  if (static_cast<int64_t>(t.rows) * p.group <= p.small) return t;
  set_range(p, t, (item - tile_base_of(p, o.first, o.seq)) * kTileCols, kTileCols, o.value);
  return t;
}

// A workgroup's place in the flat grid: `inner` fastest, then kv heads, then
// items.
struct Place {
  int inner, head;
  unsigned item;
};
__device__ __forceinline__ Place place_of(const Params& p, unsigned b, int inner) {
  const unsigned r = b / static_cast<unsigned>(inner);
  const unsigned item = r / static_cast<unsigned>(p.c.heads);
  return Place{static_cast<int>(b - r * inner), static_cast<int>(r - item * p.c.heads), item};
}

// Max and sum over the lanes that hold one column: lane ^ 32, and lane ^ 16
// where a column has four lanes.
template <bool FOUR>
__device__ __forceinline__ float column_max(float v) {
  if constexpr (FOUR) {
    const uint32_t b = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    v = __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  const uint32_t b = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <bool FOUR>
__device__ __forceinline__ float column_sum(float v) {
  if constexpr (FOUR) {
    const uint32_t b = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  const uint32_t b = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A column's place among the query rows, and the positions it sees.
struct Column {
  bool valid;
  int64_t out_row;  // row * heads + head, of out and lse
  int64_t q_at;     // element offset of its query
  int see_lo, see_hi;
};
__device__ __forceinline__ Column column_of(const Params& p, const Tile& t, int head, int k) {
  Column c;
  c.valid = k < t.ncols;
  const int col = t.col0 + (c.valid ? k : 0), row = col / p.group;
  const int h = head * p.group + col - row * p.group;
  c.out_row = (t.row0 + row) * p.a.heads + h;
  c.q_at = (t.row0 + row) * p.a.ldq + static_cast<int64_t>(h) * p.c.dim;
  const int pos = t.len - t.rows + row;
  c.see_lo = first_seen(p, pos);
  c.see_hi = c.valid ? min(pos + 1, t.len) : 0;
  return c;
}

// The column's query as the second operand of K Q^T, and the power of two
// that undoes its scaling.  at(i) is the element that the lane's i-th piece
// of 8 begins with.
template <int DT, int N, bool FOUR, typename At>
__device__ __forceinline__ float load_query(const Params& p, const Column& c, At at, half8_t (&f)[N]) {
  uint32_t raw[N][4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int d = at(i);
    Raw16<2> w{{0, 0, 0, 0}};
    if (c.valid && d < p.c.dim)
      w = *reinterpret_cast<const Raw16<2>*>(static_cast<const char*>(p.a.q) + (c.q_at + d) * 2);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      raw[i][e] = w.w[e] ^ p.flip;
      top = qm::max_u32(top, qm::max_u32(w.w[e] & 0x7fffu, (w.w[e] >> 16) & 0x7fffu));
    }
  }
  if constexpr (DT == QK_F16) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      f[i] = __builtin_bit_cast(half8_t, make_uint4(raw[i][0], raw[i][1], raw[i][2], raw[i][3]));
    return 1.0f;
  } else {
    const float amax = column_max<FOUR>(__uint_as_float(top << 16));
    const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;  // NaN and infinity stay what they are
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        f[i][2 * w] = static_cast<_Float16>(__builtin_amdgcn_ldexpf(qm::bf16_lo(raw[i][w]), 14 - e));
        f[i][2 * w + 1] = static_cast<_Float16>(__builtin_amdgcn_ldexpf(qm::bf16_hi(raw[i][w]), 14 - e));
      }
    return __builtin_amdgcn_ldexpf(1.0f, e - 14);
  }
}

// A wave-uniform element of an array that the kernel does not write, through
// the scalar cache: it has a counter of its own, so that waiting for a block
// number does not mean waiting for the keys and values asked for before it.
__device__ __forceinline__ int scalar_load(const int* p, int i) {
  typedef const __attribute__((address_space(4))) int* constant_t;
  return reinterpret_cast<constant_t>(reinterpret_cast<uintptr_t>(p))[__builtin_amdgcn_readfirstlane(i)];
}

// Bytes of a 16-position piece of V past `have` positions as zeros: what lies
// past a sequence's end may be any bytes, NaN codes among them, and a zero
// probability would not silence those.
__device__ __forceinline__ void keep_first(uint4& w, int have) {
  uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = min(max(have - 4 * i, 0), 4);
    v[i] &= b >= 4 ? 0xffffffffu : (1u << (8 * b)) - 1u;
  }
  w = make_uint4(v[0], v[1], v[2], v[3]);
}

// Partial results travel between workgroups of one launch, which may run on
// dies with L2 caches of their own: device-scope accesses, which go past the
// L2.  With those no cache has to be written back or invalidated; a store is
// done once the wave's vmcnt says so.
__device__ __forceinline__ void put2(float* at, float a, float b) {
  const uint64_t v = static_cast<uint64_t>(__float_as_uint(b)) << 32 | __float_as_uint(a);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(at), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 get2(const float* at) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(at), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32)));
}

// m and log2 l may be large and of opposite signs (small V scales): l's exponent
// is added to m first, as exactly as the two allow.
__device__ __forceinline__ float lse_of(float m, float l) {
  if (l == 0.0f) return -__builtin_inff();
  const float whole = m - kLift + static_cast<float>(__builtin_amdgcn_frexp_expf(l));
  return (whole + __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(l))) * 0.6931471805599453f;
}

// Whether a block's scales need nothing of what split_scale does.
__device__ __forceinline__ bool plain_scales(float ks, float vs) {
  return ks >= 0.0f && vs >= kLeastScale && vs <= kMostScale;
}

// Any scale of V as held * rest: of `held`, positive and 2^-64 or more, the
// exponent takes the logarithm and the sum the reciprocal (formed in two steps,
// being subnormal beyond 2^126); `rest`, a power of two, its negative or 0, is
// left to multiply p or the codes.  Infinity and NaN stay in `held`.
struct SplitScale {
  float log2, inv, rest;
};
__device__ __forceinline__ SplitScale split_scale(float vs) {
  const float mag = __builtin_fabsf(vs);
  const bool low = mag < kLeastScale;
  const int up = low ? -63 - __builtin_amdgcn_frexp_expf(mag) : 0;
  const float held = vs == 0.0f ? kLeastScale : __builtin_amdgcn_ldexpf(mag, up);
  return SplitScale{__builtin_amdgcn_logf(held), __builtin_amdgcn_rcpf(held * 0.0625f) * 0.0625f,
                    vs == 0.0f ? 0.0f : __builtin_copysignf(__builtin_amdgcn_ldexpf(1.0f, -up), vs)};
}

// What a column's sums are multiplied by: 0 for a column that sees nothing, that
// is, whose row stands before position 0; where the scores of one that does
// are all -infinity, l and the sums are 0 and the products NaN.
__device__ __forceinline__ float inverse_of(float l, bool sees) { return sees ? 1.0f / l : 0.0f; }

// One step of the running softmax over a lane's scores of one column: N
// pieces of E raw scores s, whose exponents are y = s c + b with c >= 0 and
// b = log2 v_scale per piece.  Leaves p = 2^(y - m + 14) in s.  m is raised to
// the maximum only where that exceeds it by more than kSlack, so that most
// steps find nothing to rescale; rescale(f) is called, for whole waves, where
// what was summed before shrinks by f.  The maximum is taken of the raw scores
// and the product with c merged into the exponent: one fused multiply-add,
// one max, one exponential and one addition per score.
template <int N, int E, bool FOUR, typename Rescale>
__device__ __forceinline__ void softmax_step(float (&s)[N][E], const float (&c)[N], const float (&b)[N],
                                             const float (&inv_vs)[N], float& m, float& l, Rescale rescale) {
  float top = kNone;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = s[i][0];
#pragma unroll
    for (int e = 1; e < E; ++e) t = __builtin_fmaxf(t, s[i][e]);
    top = __builtin_fmaxf(top, __builtin_fmaf(t, c[i], b[i]));
  }
  top = column_max<FOUR>(top);
  const bool grow = top > m + kSlack;
  if (__any(grow)) {
    const float m_new = grow ? top : m, shrink = __builtin_amdgcn_exp2f(m - m_new);
    m = m_new;
    l *= shrink;
    rescale(shrink);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float off = b[i] - (m - kLift);
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      s[i][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][e], c[i], off));
      sum += s[i][e];
    }
    l = __builtin_fmaf(sum, inv_vs[i], l);
  }
}

// Joins a tile's chunks in order, by the workgroup that arrived last: threads
// over (column, pair of elements).
template <int DT>
__device__ __forceinline__ void join_chunks(const Params& p, const Tile& t, int head, int64_t slot) {
  constexpr int kAhead = 8;  // chunks whose loads are in flight together
  const int pairs = p.c.dim >> 1;
  const int splits = t.splits;
  for (int i = threadIdx.x; i < t.ncols * pairs; i += 64 * kWaves) {
    const int k = i / pairs, d = 2 * (i - k * pairs);
    float m = kNone, l = 0.0f, a = 0.0f, b = 0.0f;
    for (int s0 = 0; s0 < splits; s0 += kAhead) {
      float2 ml[kAhead], o[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t at = slot + static_cast<int64_t>(min(s0 + j, splits - 1)) * p.cols + k;
        ml[j] = get2(p.part_ml + at * 2);
        o[j] = get2(p.part_o + at * p.c.dim + d);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (s0 + j >= splits) break;
        const float m_new = __builtin_fmaxf(m, ml[j].x);
        const float f0 = __builtin_amdgcn_exp2f(m - m_new), f1 = __builtin_amdgcn_exp2f(ml[j].x - m_new);
        m = m_new;
        l = __builtin_fmaf(l, f0, ml[j].y * f1);
        a = __builtin_fmaf(a, f0, o[j].x * f1);
        b = __builtin_fmaf(b, f0, o[j].y * f1);
      }
    }
    const Column col = column_of(p, t, head, k);
    const int64_t out_row = col.out_row;
    const float inv = inverse_of(l, col.see_hi > 0);
    *reinterpret_cast<kv::Raw4<2>*>(static_cast<char*>(p.a.out) + (out_row * p.c.dim + d) * 2) =
        kv::Raw4<2>{qm::pack2_narrow<DT>(a * inv, b * inv)};
    if (d == 0 && p.a.lse) p.a.lse[out_row] = lse_of(m, l);
  }
}

// The bodies share their kernel's dynamic LDS; this many binary16.  (Named in
// the body that uses it: through a pointer from elsewhere the compiler kept
// fewer reads in flight, and a prompt of 1000 rows took 1.08 times as long.)
template <int DP>
constexpr int kLdsHalves = 4 * kGroup * DP;

// One workgroup: one tile of up to 16 columns, one kv head, one chunk of
// positions.  Its four waves take groups of 64 positions in turn, each with a
// maximum, a sum and an output of its own, and join them through LDS at the
// end; nothing is shared before, so no wave waits for another.  The workgroup
// that arrives last at a tile joins its chunks.
//
// 32 heads on 8, dim 128: 64 sequences of 1 to 8192 positions, INT8, 126 us
// (5.0 TB/s; a plain copy reaches 4.9 and a read-only stream 6.1); two
// sequences of about 115000, 64 heads, FP8, 88 us (5.4 TB/s); one of 771
// positions 7 us: the launch, and a chain of table entry, keys, products and
// join.
template <int DT, bool FP8, int DP>
__device__ __forceinline__ void cols_body(const Params& p, unsigned block) {
  // the waves' outputs, [wave][column][element], elements exchanged in fours by
  // the column's number so that columns fall on different banks
  extern __shared__ __align__(16) _Float16 lds_all[];
  float* const lds_o = reinterpret_cast<float*>(lds_all);
  __shared__ struct {
    float m[kWaves][kCols], l[kWaves][kCols];
    unsigned last;
  } lds;
  constexpr int KC = DP / 64;  // 16-byte pieces of a K row per lane
  constexpr int VC = DP / 16;  // 16-row pieces of V

  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place at = place_of(p, block, p.splits);
  // Workgroups go round the eight dies in turn, and early chunks have work in
  // every sequence, late ones in few: the chunks are turned by the tile's
  // number so that no die gets the same one of each (64 requests of up to 8192
  // positions in four chunks: 153 us without, 128 with).
  const int head = at.head, split = static_cast<int>((at.inner + at.item + head) % static_cast<unsigned>(p.splits));
  const Tile t = find_cols(p, at.item);
  if (!t.live) return;
  const int dim = p.c.dim, P = p.c.block;
  const int begin = (t.lo & ~(kGroup - 1)) + split * p.chunk, end = min(begin + p.chunk, t.hi);
  if (split > 0 && begin >= t.hi) return;  // split 0 stays, to write the rows that see nothing

  const Column col = column_of(p, t, head, n);
  half8_t qf[DP / 32];
  // lane (g, n) holds, for step 2 c + u, elements 64 c + 16 g + 8 u + j: the
  // order in which 16-byte loads bring K
  const float unscale = load_query<DT, DP / 32, true>(
      p, col, [&](int i) { return 64 * (i >> 1) + 16 * g + 8 * (i & 1); }, qf);
  const float c_col = unscale * p.scale2;

  float4_t o[VC];
#pragma unroll
  for (int i = 0; i < VC; ++i) o[i] = float4_t{0, 0, 0, 0};
  float m = kNone, l = 0.0f;

  const int64_t head_bytes = static_cast<int64_t>(P) * dim;
  const int* const table = p.c.table + t.seq * p.c.ldt;
  // Table entries are read at any position that the table has, whether seen or
  // not, so that they need not wait for the lengths; a block number outside
  // the cache reads block 0.  Where such a position is seen its scales are
  // NaN; elsewhere scores are masked, and bytes of V that may be NaN codes
  // become zeros.
  auto entry = [&](int pos) { return scalar_load(table, min(pos >> p.block_shift, p.c.width - 1)); };
  auto in_pool = [&](int b) { return static_cast<unsigned>(b) < static_cast<unsigned>(p.c.blocks); };

  // Up to dim 128 the next group's K and V are asked for before this one is
  // worked on; beyond, the registers hold one of each, and the next K is asked
  // for when the scores are done, the next V at the end.
  constexpr int kSets = DP > 128 ? 1 : 2;
  uint4 kr[kSets][4][KC], vr[kSets][VC];
  float ks[kSets], vs[kSets];
  // The blocks of the next group's four pieces of 16 positions.
  int nb0 = 0, nb1 = 0, nb2 = 0, nb3 = 0;
  auto next_blocks = [&](int t0) {
    nb0 = entry(t0);
    nb1 = entry(t0 + 16);
    nb2 = entry(t0 + 32);
    nb3 = entry(t0 + 48);
  };
  auto pick = [&](int j) {
    const int lo = j & 1 ? nb1 : nb0, hi = j & 1 ? nb3 : nb2;
    return j & 2 ? hi : lo;
  };
  auto tile_of = [&](int b) { return static_cast<int64_t>(in_pool(b) ? b : 0) * p.c.heads + head; };
  // Elements past dim come from the front of the row: K's meet zeros of the
  // query there, V's rows past dim are not stored.
  int kpart[KC];
#pragma unroll
  for (int c = 0; c < KC; ++c) kpart[c] = 64 * c + 16 * g < dim ? 64 * c + 16 * g : 0;
  // K: the lane's row n of tile i is position t0 + 16 (n / 4) + 4 i + n % 4
  auto load_k = [&](int t0, auto half) {
    constexpr int S = decltype(half)::value % kSets;
    const uint8_t* const row =
        p.c.k + tile_of(pick(n >> 2)) * head_bytes + (((t0 + 16 * (n >> 2)) & (P - 1)) + (n & 3)) * dim;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < KC; ++c) kr[S][i][c] = *reinterpret_cast<const uint4*>(row + 4 * i * dim + kpart[c]);
  };
  auto load_scales = [&](auto half) {
    constexpr int S = decltype(half)::value % kSets;
    const int b = pick(g);
    ks[S] = p.c.k_scale[tile_of(b)];
    vs[S] = p.c.v_scale[tile_of(b)];
    if (!in_pool(b)) ks[S] = vs[S] = __builtin_nanf("");
  };
  auto load_v = [&](int t0, auto half) {
    constexpr int S = decltype(half)::value % kSets;
    const uint8_t* const row = p.c.v + tile_of(pick(g)) * head_bytes + n * P + ((t0 + 16 * g) & (P - 1));
#pragma unroll
    for (int i = 0; i < VC; ++i) vr[S][i] = *reinterpret_cast<const uint4*>(row + (16 * i < dim ? 16 * i : 0) * P);
  };

  constexpr int kStep = kWaves * kGroup;
  // the group at t0, whose K and V are in registers or on their way; `more`:
  // ask for the next group's
  auto group = [&](int t0, auto half, auto more) {
    constexpr int S = decltype(half)::value % kSets;
    constexpr std::integral_constant<int, 1 - decltype(half)::value> other{};
    if (kSets == 2 && more) {
      load_scales(other);
      load_k(t0 + kStep, other);
      load_v(t0 + kStep, other);
      next_blocks(t0 + 2 * kStep);
    }
    float4_t acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i] = float4_t{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv::codes8_to_half<FP8>(kr[S][i][c].x, kr[S][i][c].y), qf[2 * c], acc[i], 0, 0, 0);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv::codes8_to_half<FP8>(kr[S][i][c].z, kr[S][i][c].w), qf[2 * c + 1], acc[i], 0, 0, 0);
      }
    }
    if (kSets == 1 && more) load_k(t0 + kStep, other);
    float s[1][16];
#pragma unroll
    for (int i = 0; i < 16; ++i) s[0][i] = acc[i >> 2][i & 3];
    float c[1] = {c_col * ks[S]}, bias[1] = {__builtin_amdgcn_logf(vs[S])}, inv_vs[1] = {__builtin_amdgcn_rcpf(vs[S])};
    const bool odd = __any(!plain_scales(ks[S], vs[S]));
    if (t0 < t.lo || t0 + kGroup > t.len - t.rows || p.a.window > 0 || odd) {  // some column may not see all 64
      const int at = t0 + 16 * g;
      if (odd) [[unlikely]] {
        const SplitScale v = split_scale(vs[S]);
        bias[0] = v.log2;
        inv_vs[0] = v.inv;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool seen = at + i >= col.see_lo && at + i < col.see_hi;
        s[0][i] = seen ? __builtin_fmaf(s[0][i], c[0], bias[0]) : -__builtin_inff();
      }
      c[0] = 1.0f;
      bias[0] = 0.0f;
      // a lane that sees none of these positions must not meet their scale
      if (at + 16 <= col.see_lo || at >= col.see_hi) inv_vs[0] = 0.0f;
    }
    softmax_step<1, 16, true>(s, c, bias, inv_vs, m, l, [&](float shrink) {
#pragma unroll
      for (int i = 0; i < VC; ++i) o[i] *= shrink;
    });
    half8_t pf[2];
#pragma unroll
    for (int i = 0; i < 16; ++i) pf[i >> 3][i & 7] = static_cast<_Float16>(s[0][i]);
    // after the rounding, where half as many registers are live (before it: 8
    // spilled for FP8 at dim 128, and short FP8 calls took 1.04 times as long)
    if (__any(!(vs[S] >= kLeastScale))) [[unlikely]] {
      const float rest = split_scale(vs[S]).rest;
#pragma unroll
      for (int i = 0; i < 16; ++i) pf[i >> 3][i & 7] = static_cast<_Float16>(static_cast<float>(pf[i >> 3][i & 7]) * rest);
    }
    if (FP8 && (t0 + kGroup > t.len || t0 < t.lo)) {
      const int have = t0 + 16 * g + 16 > t.lo ? t.len - (t0 + 16 * g) : 0;
#pragma unroll
      for (int i = 0; i < VC; ++i) keep_first(vr[S][i], have);
    }
#pragma unroll
    for (int i = 0; i < VC; ++i) {
      o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv::codes8_to_half<FP8>(vr[S][i].x, vr[S][i].y), pf[0], o[i], 0, 0, 0);
      o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv::codes8_to_half<FP8>(vr[S][i].z, vr[S][i].w), pf[1], o[i], 0, 0, 0);
    }
    if (kSets == 1 && more) {
      load_scales(other);
      load_v(t0 + kStep, other);
      next_blocks(t0 + 2 * kStep);
    }
  };
  constexpr std::integral_constant<int, 0> even{};
  constexpr std::integral_constant<int, 1> odd{};
  int t0 = begin + wave * kGroup;
  if (t0 < end) {
    next_blocks(t0);
    load_scales(even);
    load_k(t0, even);
    load_v(t0, even);
    next_blocks(t0 + kStep);
    if constexpr (kSets == 1) {
      for (; t0 < end; t0 += kStep) group(t0, even, t0 + kStep < end);
    } else {
      for (; t0 + 2 * kStep < end; t0 += 2 * kStep) {
        group(t0, even, std::true_type{});
        group(t0 + kStep, odd, std::true_type{});
      }
      if (t0 + kStep < end) {
        group(t0, even, std::true_type{});
        group(t0 + kStep, odd, std::false_type{});
      } else {
        group(t0, even, std::false_type{});
      }
    }
  }

  // join the four waves
  l = column_sum<true>(l);
  if (g == 0) {
    lds.m[wave][n] = m;
    lds.l[wave][n] = l;
  }
#pragma unroll
  for (int i = 0; i < VC; ++i)
    *reinterpret_cast<float4_t*>(lds_o + (wave * kCols + n) * DP + ((16 * i + 4 * g) ^ (4 * n))) = o[i];
  __syncthreads();

  const unsigned tile_id = at.item * static_cast<unsigned>(p.c.heads) + head;
  const int64_t slot = static_cast<int64_t>(tile_id) * p.splits * p.cols;
  const bool whole = t.splits <= 1;
  const int pairs = dim >> 1;
  for (int i = threadIdx.x; i < t.ncols * pairs; i += 64 * kWaves) {
    const int k = i / pairs, d = 2 * (i - k * pairs);
    float mm = lds.m[0][k], ll = 0.0f, a = 0.0f, b = 0.0f;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mm = __builtin_fmaxf(mm, lds.m[w][k]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(lds.m[w][k] - mm);
      ll = __builtin_fmaf(lds.l[w][k], f, ll);
      const float2 v = *reinterpret_cast<const float2*>(lds_o + (w * kCols + k) * DP + (d ^ (4 * k)));
      a = __builtin_fmaf(v.x, f, a);
      b = __builtin_fmaf(v.y, f, b);
    }
    if (whole) {
      const Column c = column_of(p, t, head, k);
      const int64_t out_row = c.out_row;
      const float inv = inverse_of(ll, c.see_hi > 0);
      *reinterpret_cast<kv::Raw4<2>*>(static_cast<char*>(p.a.out) + (out_row * dim + d) * 2) =
          kv::Raw4<2>{qm::pack2_narrow<DT>(a * inv, b * inv)};
      if (d == 0 && p.a.lse) p.a.lse[out_row] = lse_of(mm, ll);
    } else {
      const int64_t part = slot + static_cast<int64_t>(split) * p.cols + k;
      put2(p.part_o + part * dim + d, a, b);
      if (d == 0) put2(p.part_ml + part * 2, mm, ll);
    }
  }
  if (whole || p.join_later) return;

  // every wave's stores are done before the workgroup counts as arrived
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned before = __hip_atomic_fetch_add(p.arrived + tile_id, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const bool last = before + 1 == static_cast<unsigned>(t.splits);
    if (last) __hip_atomic_store(p.arrived + tile_id, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    lds.last = last;
  }
  __syncthreads();
  if (lds.last) join_chunks<DT>(p, t, head, slot);
}

// One workgroup: one tile of 128 columns, one kv head, one chunk of positions
// in steps of 64.  The four waves share K and V of a step through LDS, as
// binary16 (each code is converted once per workgroup), and have 32 columns
// each.  LDS is doubled: while a step is worked on, the next one's bytes are
// written converted to the other half, and those of the one after it come
// from memory into registers; one barrier per step.  Rows of K lie in the order
// in which the first product's result registers want them, 16-byte pieces of a
// row are exchanged by its number so that consecutive rows fall on different
// banks: 16 rows where a row of K has 16 pieces or more (eight only: 176 us for
// 173 in the case below).
//
// 4096 rows of 32 heads on 8, dim 128, causal: 170-178 us, 770 to 810 TFLOP/s (a
// plain binary16 matrix product of 8192^3 reaches 1280 here), when some 200 calls
// have run before; the first after a pause take 190 to 205.  A wave's step is 1024
// cycles of matrix instructions and some 300 vector instructions (64 codes
// converted, 32 exponentials), of which the two waves of a SIMD overlap a part.
// Measured beside it: 64 columns per wave, which halves the reads of LDS but
// leaves one wave per SIMD, 319 us; the next step's conversion within the
// first product 471 (registers spill); conversion before the products 175;
// a raised wave priority during the products 176; rescaling at every new
// maximum 176.
template <int DT, bool FP8, int DP>
__device__ __forceinline__ void tile_body(const Params& p, unsigned block) {
  extern __shared__ __align__(16) _Float16 lds_all[];
  _Float16(*const lds_k)[kGroup * DP] = reinterpret_cast<_Float16(*)[kGroup * DP]>(lds_all);
  _Float16(*const lds_v)[kGroup * DP] = lds_k + 2;
  __shared__ __align__(16) float lds_s[2][3][4];  // of each 16 positions: k scale, log2 v scale, 1 / v scale
  constexpr int KP = DP / 8;       // 16-byte pieces of a K row (8 binary16)
  constexpr int NC = DP / 64;      // 16-byte loads per thread, of K and of V
  constexpr int ND = DP / 32;      // 32-row pieces of V
  constexpr int RB = DP / 16;      // 16-byte pieces of a row of codes

  auto key_k = [](int row) { return KP >= 16 ? row & 15 : (row >> 1) & 7; };
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  Place at = place_of(p, block, p.splits);
  at.item = p.items - 1 - at.item;  // later rows see more: the longest work first
  const int split = at.inner, head = at.head;
  const Tile t = find_tile(p, at.item);
  if (!t.live) return;
  const int dim = p.c.dim, P = p.c.block;
  const int begin = (t.lo & ~(kGroup - 1)) + split * p.chunk, end = min(begin + p.chunk, t.hi);
  if (split > 0 && begin >= t.hi) return;

  const Column col = column_of(p, t, head, wave * 32 + n);
  half8_t qf[DP / 16];
  const float unscale = load_query<DT, DP / 16, false>(p, col, [&](int i) { return 16 * i + 8 * h; }, qf);
  const float c_col = unscale * p.scale2;
  // positions that all of this wave's columns see, and that any of them sees
  const int w0 = wave * 32, w1 = min(wave * 32 + 31, t.ncols - 1);
  const bool any = w0 < t.ncols;
  const int pos0 = t.len - t.rows + (t.col0 + w0) / p.group, pos1 = t.len - t.rows + (t.col0 + max(w1, 0)) / p.group;
  const int all_hi = min(pos0 + 1, t.len), any_hi = any ? min(pos1 + 1, t.len) : 0;
  const int all_lo = first_seen(p, pos1), any_lo = first_seen(p, pos0);

  float16_t o[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
  float m = kNone, l = 0.0f;

  const int64_t head_bytes = static_cast<int64_t>(P) * dim;
  const int* const table = p.c.table + t.seq * p.c.ldt;
  auto entry = [&](int pos) { return scalar_load(table, min(pos >> p.block_shift, p.c.width - 1)); };  // as above
  auto in_pool = [&](int b) { return static_cast<unsigned>(b) < static_cast<unsigned>(p.c.blocks); };

  // What this thread brings of a step.  K: piece kd of rows krow(i); V: 16
  // positions of rows lane + 64 i.  Either way a wave brings the same 16
  // positions, so one block number and one tile's address, both scalar, serve it.
  // Elements past dim come from the front of the row and rows past dim from
  // the last: they meet zeros of the query, or are not stored.
  const int kd = tid % RB, kcol = 16 * kd < dim ? 16 * kd : 0;
  auto krow = [&](int i) { return 16 * wave + lane / RB + i * (64 / RB); };
  // Up to dim 128 two steps are on their way, so that a load has a whole step
  // to arrive; beyond, the registers hold one.
  constexpr int kSets = DP > 128 ? 1 : 2;
  uint4 kr[kSets][NC], vr[kSets][NC];
  float sk[kSets], sv[kSets];
  int next_block = 0;  // of this wave's 16 positions of the step to load
  auto load_block = [&](int t0) { next_block = entry(t0 + 16 * wave); };
  auto load_step = [&](int t0, auto half) {
    const int S = half % kSets;
    const bool ok = in_pool(next_block);
    const int64_t tile = static_cast<int64_t>(ok ? next_block : 0) * p.c.heads + head;
    const int pos = (t0 + 16 * wave) & (P - 1);
    const uint8_t* const from_k = p.c.k + tile * head_bytes + pos * dim;
    const uint8_t* const from_v = p.c.v + tile * head_bytes + pos;
#pragma unroll
    for (int i = 0; i < NC; ++i)
      kr[S][i] = *reinterpret_cast<const uint4*>(from_k + static_cast<unsigned>((krow(i) & 15) * dim + kcol));
#pragma unroll
    for (int i = 0; i < NC; ++i)
      vr[S][i] = *reinterpret_cast<const uint4*>(from_v + static_cast<unsigned>(min(lane + 64 * i, dim - 1) * P));
    sk[S] = p.c.k_scale[tile];
    sv[S] = p.c.v_scale[tile];
    if (!ok) sk[S] = sv[S] = __builtin_nanf("");
  };
  // the step at t0 into half H of LDS
  auto put_step = [&](int t0, auto half) {
    const int H = half, S = H % kSets;
    half8_t* const kl = reinterpret_cast<half8_t*>(lds_k[H]);
    half8_t* const vl = reinterpret_cast<half8_t*>(lds_v[H]);
    if (FP8 && (t0 + kGroup > t.len || t0 < t.lo)) {
      const int have = t0 + 16 * wave + 16 > t.lo ? t.len - (t0 + 16 * wave) : 0;
#pragma unroll
      for (int i = 0; i < NC; ++i) keep_first(vr[S][i], have);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      // position 32 a + 16 b + 8 c + 4 d + e lies in row 32 a + 16 b + 8 d + 4 c + e
      const int r = krow(i), row = (r & ~12) | ((r & 8) >> 1) | ((r & 4) << 1);
      const int key = key_k(row);
      kl[row * KP + ((2 * kd) ^ key)] = kv::codes8_to_half<FP8>(kr[S][i].x, kr[S][i].y);
      kl[row * KP + ((2 * kd + 1) ^ key)] = kv::codes8_to_half<FP8>(kr[S][i].z, kr[S][i].w);
      const int d = lane + 64 * i;
      vl[d * 8 + ((2 * wave) ^ (d & 7))] = kv::codes8_to_half<FP8>(vr[S][i].x, vr[S][i].y);
      vl[d * 8 + ((2 * wave + 1) ^ (d & 7))] = kv::codes8_to_half<FP8>(vr[S][i].z, vr[S][i].w);
    }
    if (lane == 0) {
      lds_s[H][0][wave] = sk[S];
      lds_s[H][1][wave] = __builtin_amdgcn_logf(sv[S]);
      lds_s[H][2][wave] = __builtin_amdgcn_rcpf(sv[S]);
    }
    if (__any(!plain_scales(sk[S], sv[S]))) [[unlikely]] {  // the wave's 16 positions have one block's scales
      const SplitScale v = split_scale(sv[S]);
      const _Float16 turn = sk[S] < 0.0f ? -1.0f : 1.0f;
#pragma unroll 1
      for (int i = 0; i < 2 * NC; ++i) {
        const int r = krow(i >> 1), row = (r & ~12) | ((r & 8) >> 1) | ((r & 4) << 1), d = lane + 64 * (i >> 1);
        kl[row * KP + ((2 * kd + (i & 1)) ^ key_k(row))] *= turn;
        half8_t& w = vl[d * 8 + ((2 * wave + (i & 1)) ^ (d & 7))];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = static_cast<_Float16>(static_cast<float>(w[e]) * v.rest);
      }
      if (lane == 0) {
        lds_s[H][0][wave] = __builtin_fabsf(sk[S]);
        lds_s[H][1][wave] = v.log2;
        lds_s[H][2][wave] = v.inv;
      }
    }
  };
  // the step at t0, in half H of LDS
  auto work = [&](int t0, auto half) {
    const int H = half;
    if (t0 >= any_hi || t0 + kGroup <= any_lo) return;
    const half8_t* const kl = reinterpret_cast<const half8_t*>(lds_k[H]);
    const half8_t* const vl = reinterpret_cast<const half8_t*>(lds_v[H]);
    float16_t acc[2];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[a][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) {
        acc[a] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kl[(32 * a + n) * KP + ((2 * i + h) ^ key_k(n))], qf[i], acc[a], 0, 0, 0);
      }
    }
    // register 8 b + e of acc[a] is position 32 a + 16 b + 8 h + e
    float s[4][8], c[4], bias[4], inv_vs[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      c[b] = c_col * lds_s[H][0][b];
      bias[b] = lds_s[H][1][b];
      inv_vs[b] = lds_s[H][2][b];
#pragma unroll
      for (int e = 0; e < 8; ++e) s[b][e] = acc[b >> 1][8 * (b & 1) + e];
    }
    if (t0 + kGroup > all_hi || t0 < all_lo) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int first = t0 + 16 * b;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int spot = first + 8 * h + e;
          s[b][e] = spot >= col.see_lo && spot < col.see_hi ? __builtin_fmaf(s[b][e], c[b], bias[b]) : -__builtin_inff();
        }
        c[b] = 1.0f;
        bias[b] = 0.0f;
        // a column that sees none of these positions must not meet their scale
        if (first + 16 <= col.see_lo || first >= col.see_hi) inv_vs[b] = 0.0f;
      }
    }
    softmax_step<4, 8, false>(s, c, bias, inv_vs, m, l, [&](float shrink) {
#pragma unroll
      for (int i = 0; i < ND; ++i) o[i] *= shrink;
    });
    half8_t pf[4];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int e = 0; e < 8; ++e) pf[b][e] = static_cast<_Float16>(s[b][e]);
#pragma unroll
    for (int i = 0; i < ND; ++i) {
#pragma unroll
      for (int s4 = 0; s4 < 4; ++s4)
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vl[(32 * i + n) * 8 + ((2 * s4 + h) ^ (n & 7))], pf[s4], o[i], 0, 0, 0);
    }
  };
  // One step: ask for a later one, work on this one, write the next.
  auto step = [&](int t0, auto half, auto other) {
    if (t0 + kSets * kGroup < end) {
      load_step(t0 + kSets * kGroup, half);  // with one set there is no other
      load_block(t0 + (kSets + 1) * kGroup);
    }
    work(t0, half);
    if (t0 + kGroup < end) put_step(t0 + kGroup, other);
    __syncthreads();
  };

  using Even = std::integral_constant<int, 0>;
  using Odd = std::integral_constant<int, 1>;
  if (begin < end) {
    load_block(begin);
    load_step(begin, Even{});
    load_block(begin + kGroup);
    if (kSets > 1 && begin + kGroup < end) {
      load_step(begin + kGroup, Odd{});
      load_block(begin + 2 * kGroup);
    }
    put_step(begin, Even{});
  }
  __syncthreads();
  if constexpr (kSets == 1) {
    for (int t0 = begin, half = 0; t0 < end; t0 += kGroup, half ^= 1) step(t0, half, half ^ 1);
  } else {
    for (int t0 = begin; t0 < end; t0 += 2 * kGroup) {
      step(t0, Even{}, Odd{});
      if (t0 + kGroup < end) step(t0 + kGroup, Odd{}, Even{});
    }
  }

  if (!col.valid) return;
  l = column_sum<false>(l);
  // register 4 q + e of o[i] is element 32 i + 8 q + 4 h + e
  if (t.splits <= 1) {
    float inv = l != 0.0f ? 1.0f / l : 0.0f;
    // (with col kept for this, calls of few steps took 1.03 to 1.06 times as long)
    if (__any(l == 0.0f)) [[unlikely]] inv = inverse_of(l, column_of(p, t, head, wave * 32 + n).see_hi > 0);
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int d = 32 * i + 8 * q + 4 * h;
        if (d < dim)
          *reinterpret_cast<kv::Raw8<2>*>(static_cast<char*>(p.a.out) + (col.out_row * dim + d) * 2) =
              kv::Raw8<2>{{qm::pack2_narrow<DT>(o[i][4 * q] * inv, o[i][4 * q + 1] * inv),
                           qm::pack2_narrow<DT>(o[i][4 * q + 2] * inv, o[i][4 * q + 3] * inv)}};
      }
    if (h == 0 && p.a.lse) p.a.lse[col.out_row] = lse_of(m, l);
    return;
  }
  const int64_t part = ((static_cast<int64_t>(at.item) * p.c.heads + head) * p.splits + split) * p.cols + wave * 32 + n;
#pragma unroll
  for (int i = 0; i < ND; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int d = 32 * i + 8 * q + 4 * h;
      if (d < dim)
        *reinterpret_cast<float4_t*>(p.part_o + part * dim + d) =
            float4_t{o[i][4 * q], o[i][4 * q + 1], o[i][4 * q + 2], o[i][4 * q + 3]};
    }
  if (h == 0) *reinterpret_cast<float2*>(p.part_ml + part * 2) = make_float2(m, l);
}

template <int DT, bool FP8, int DP>
__global__ __launch_bounds__(64 * kWaves, DP > 128 ? 1 : 2) void kv_attention_cols_kernel(Params p) {
  cols_body<DT, FP8, DP>(p, blockIdx.x);
}
template <int DT, bool FP8, int DP>
__global__ __launch_bounds__(64 * kWaves, DP > 128 ? 1 : 2) void kv_attention_tile_kernel(Params p) {
  tile_body<DT, FP8, DP>(p, blockIdx.x);
}
// A call of both kinds of sequences in one launch, so that the two run side by
// side: the first `tiles` workgroups (the longer ones) are tiles of 128
// columns.  (16 requests of up to 4100 positions, one of them 509 rows, window
// 1024: 37 us one after the other, 26 together.)
template <int DT, bool FP8, int DP>
__global__ __launch_bounds__(64 * kWaves, DP > 128 ? 1 : 2) void kv_attention_both_kernel(Params pt, Params pc,
                                                                                         unsigned tiles) {
  if (blockIdx.x < tiles)
    tile_body<DT, FP8, DP>(pt, blockIdx.x);
  else
    cols_body<DT, FP8, DP>(pc, blockIdx.x - tiles);
}

// Sums chunks first .. last of one column into (m, l, v): the whole wave, four
// elements per lane.
__device__ __forceinline__ void sum_chunks(const Params& p, int64_t slot, int first, int last, float& m, float& l,
                                           float4_t& v) {
  const int lane = threadIdx.x & 63, dim = p.c.dim;
  m = kNone;
  l = 0.0f;
  v = float4_t{0, 0, 0, 0};
  constexpr int kAhead = 8;  // chunks whose loads are in flight together
  for (int s0 = first; s0 < last; s0 += kAhead) {
    float2 ml[kAhead];
    float4_t o[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t part = slot + static_cast<int64_t>(min(s0 + j, last - 1)) * p.cols;
      ml[j] = *reinterpret_cast<const float2*>(p.part_ml + part * 2);
      o[j] = float4_t{0, 0, 0, 0};
      if (4 * lane < dim) o[j] = *reinterpret_cast<const float4_t*>(p.part_o + part * dim + 4 * lane);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (s0 + j >= last) break;
      const float m_new = __builtin_fmaxf(m, ml[j].x);
      const float f0 = __builtin_amdgcn_exp2f(m - m_new), f1 = __builtin_amdgcn_exp2f(ml[j].x - m_new);
      m = m_new;
      l = __builtin_fmaf(l, f0, ml[j].y * f1);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(v[e], f0, o[j][e] * f1);
    }
  }
}

template <int DT>
__device__ __forceinline__ void store_row(const Params& p, int64_t out_row, bool sees, float m, float l,
                                          const float4_t& v) {
  const int lane = threadIdx.x & 63;
  const float inv = inverse_of(l, sees);
  if (4 * lane < p.c.dim)
    *reinterpret_cast<kv::Raw8<2>*>(static_cast<char*>(p.a.out) + (out_row * p.c.dim + 4 * lane) * 2) =
        kv::Raw8<2>{{qm::pack2_narrow<DT>(v[0] * inv, v[1] * inv), qm::pack2_narrow<DT>(v[2] * inv, v[3] * inv)}};
  if (lane == 0 && p.a.lse) p.a.lse[out_row] = lse_of(m, l);
}

// Joins chunks in a launch of its own.  Many chunks of few columns: one
// workgroup per column, its waves a quarter of the chunks each.
template <int DT>
__global__ __launch_bounds__(64 * kWaves) void kv_attention_join_cols_kernel(Params p) {
  __shared__ float lds_o[kWaves][256];
  __shared__ float lds_m[kWaves], lds_l[kWaves];
  const Place at = place_of(p, blockIdx.x, p.cols);
  const Tile t = find_cols(p, at.item);
  if (!t.live || t.splits <= 1 || at.inner >= t.ncols) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t slot = (static_cast<int64_t>(at.item) * p.c.heads + at.head) * p.splits * p.cols + at.inner;
  const int each = (t.splits + kWaves - 1) / kWaves, first = wave * each;
  float m, l;
  float4_t v;
  sum_chunks(p, slot, first, min(first + each, t.splits), m, l, v);
  if (lane == 0) {
    lds_m[wave] = m;
    lds_l[wave] = l;
  }
  *reinterpret_cast<float4_t*>(&lds_o[wave][4 * lane]) = v;
  __syncthreads();
  if (wave != 0) return;
  for (int w = 1; w < kWaves; ++w) m = __builtin_fmaxf(m, lds_m[w]);
  l = 0.0f;
  v = float4_t{0, 0, 0, 0};
  for (int w = 0; w < kWaves; ++w) {
    const float f = __builtin_amdgcn_exp2f(lds_m[w] - m);
    l = __builtin_fmaf(lds_l[w], f, l);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(lds_o[w][4 * lane + e], f, v[e]);
  }
  const Column col = column_of(p, t, at.head, at.inner);
  store_row<DT>(p, col.out_row, col.see_hi > 0, m, l, v);
}

// Few chunks of many columns: one (row, head) pair per wave, over the rows as
// they lie, so that no workgroup is without rows.
template <int DT>
__global__ __launch_bounds__(64 * kWaves) void kv_attention_join_tile_kernel(Params p) {
  const unsigned wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), heads = p.a.heads;
  const unsigned pair = blockIdx.x * kWaves + wave, row_of = pair / heads;  // fewer than 2^31 pairs
  if (row_of >= static_cast<unsigned>(p.a.tokens)) return;
  const int row = static_cast<int>(row_of), h = static_cast<int>(pair - row_of * heads);
  const kv::Owner o = kv::find_sequence(row, p.a.cu, p.a.lens, p.a.seqs, [](int first, int) { return first; });
  Tile t{};
  t.seq = o.seq;
  t.row0 = o.first;
  t.rows = o.next - o.first;
  if (o.seq < 0 || o.first < 0 || row >= o.next || t.rows > p.a.tokens - o.first) return;
  if (static_cast<int64_t>(t.rows) * p.group <= p.small) return;
  const int head = h / p.group;
  const int64_t col = static_cast<int64_t>(row - o.first) * p.group + h - head * p.group;
  const int k = static_cast<int>(col % kTileCols);
  set_range(p, t, col - k, kTileCols, o.value);
  if (t.splits <= 1) return;
  const int64_t item = tile_base_of(p, o.first, o.seq) + col / kTileCols;
  float m, l;
  float4_t v;
  sum_chunks(p, (item * p.c.heads + head) * p.splits * p.cols + k, 0, t.splits, m, l, v);
  store_row<DT>(p, pair, row - o.first >= t.rows - t.len, m, l, v);
}

// How a call is cut: which kernels run, their tiles and chunks of positions.
struct Cut {
  int64_t items;  // 0: the kernel is not needed
  int tiles, chunk, splits, cols;
  size_t bytes;   // of partial results
};

// The positions that one tile can see, from a multiple of 64 on.
int64_t range_of(int max_kv, int window, int rows) {
  int64_t range = max_kv;
  if (window > 0) range = std::min<int64_t>(range, static_cast<int64_t>(window) + rows);
  return (range + 2 * kGroup - 1) / kGroup * kGroup;
}

Cut cut_of(int64_t items, int tiles, int kv_heads, int dim, int cols, int64_t range, int64_t chunk) {
  Cut c{items, tiles, 0, 0, cols, 0};
  const int64_t all = items * kv_heads;
  if (chunk > range || all > kCounters) chunk = range;
  c.chunk = static_cast<int>(chunk);  // at most 2^30, the range of kKvMostPositions
  c.splits = static_cast<int>((range + c.chunk - 1) / c.chunk);
  if (c.splits > 1) c.bytes = static_cast<size_t>(all) * c.splits * cols * (dim + 2) * sizeof(float);
  return c;
}

// Tiles of 16 columns, for sequences of at most kSmall columns.  One workgroup
// per CU keeps HBM busy, and every further chunk costs a start (about 3.5 us)
// and its part of the join, so tiles are cut until there are 256 workgroups;
// where there are that many tiles, only so that ragged lengths even out.
// Measured (dim 128, us in 1 / 2 / 4 / 8 / 16 / 32 / 64 chunks): 16 tiles of
// 121344 positions 652 / 336 / 178 / 105 / 89 / 91 / 96; 8 of 32768 172 / 92 /
// 51 / 31 / 22 / 20 / 22; 128 of 7936 54 / 41 / 44 / 45 / 49; 512 of up to 8192
// 131 / 139 / 128 / 128; 512 of 4096 94 / 102 / 109 / 113.
Cut cut_cols(int seqs, int group, int kv_heads, int dim, bool ragged, int max_q, int max_kv, int window) {
  const int64_t most = ragged ? std::min<int64_t>(static_cast<int64_t>(max_q) * group, kSmall) : group;
  // wide groups, and a call of one long sequence, are the other kernel's alone
  if (ragged && (group > kSmall || (seqs == 1 && max_q * static_cast<int64_t>(group) > kSmall))) return Cut{};
  const int tiles = static_cast<int>((most + kCols - 1) / kCols);
  const int64_t items = static_cast<int64_t>(seqs) * tiles;
  // beside long sequences the others are mostly single tokens
  const bool mixed = ragged && static_cast<int64_t>(max_q) * group > kSmall;
  const int64_t live = (mixed ? static_cast<int64_t>(seqs) * ((group + kCols - 1) / kCols) : items) * kv_heads;
  const int64_t range = range_of(max_kv, window, kCols);
  int64_t chunks = 1;
  if (range > 640 && live < 256) chunks = 256 / live;
  if (range > 6144 && live >= 256) chunks = (range + 2047) / 2048;
  const int64_t cols = std::min<int64_t>(most, kCols), each = items * kv_heads * cols * (dim + 2) * 4;
  chunks = std::min(chunks, std::max<int64_t>(kMostPartials / each, 1));
  constexpr int64_t kStep = kWaves * kGroup;
  const int64_t chunk = ((range + chunks - 1) / chunks + kStep - 1) / kStep * kStep;
  return cut_of(items, tiles, kv_heads, dim, static_cast<int>(cols), range, chunk);
}

// Tiles of 128 columns, for the others: chunks, of 512 positions or more, only
// where there are too few tiles for the CUs (two workgroups fit on one, one
// beyond dim 128) and the range is long.  Measured (us unsplit / split): 500
// rows of 600 positions 24 / 35, 700 of 1400 47 / 30, 300 of 4000 123 / 38, 512
// of 8192 220 / 112.
// A handful of rows (fewer columns than one tile) get short chunks, since the
// bound on the range is mostly what the table covers and they are over before
// it: 30 rows of 32 heads on 8 with a table of 131072, counted as a whole tile /
// a half / a quarter: over 4000 positions 65 / 42 / 32 us, over 20000 69 / 57 /
// 46, over all of them 106 / 126 / 135.
//
// Of the items, which all have room for partial results, few can be without
// columns, so that the workspace stays below some 300 MB.
Cut cut_tile(int seqs, int tokens, int group, int kv_heads, int dim, bool ragged, int max_q, int max_kv, int window,
             int small) {
  if (!ragged || static_cast<int64_t>(max_q) * group <= kSmall) return Cut{};
  const int64_t items = tile_base<int64_t>(tokens, group, small, seqs);
  const int64_t full = static_cast<int64_t>(tokens) * group / kTileCols;
  // in half tiles; a call without a full one counts as a quarter of one
  const int64_t live = full ? 2 * (full + std::min<int64_t>(seqs, full) / 2) * kv_heads : (kv_heads + 1) / 2;
  const int64_t range = range_of(max_kv, window, kTileCols), wanted = dim > 128 ? 512 : 1024;
  int64_t chunk = range;
  if (live < 384 && range > 1024) chunk = ((range * live + wanted - 1) / wanted + 255) / 256 * 256;
  return cut_of(items, 1, kv_heads, dim, kTileCols, range, std::max<int64_t>(chunk, 512));
}

struct Cuts {
  Cut cols, tile;
};
Cuts cuts_of(int seqs, int tokens, int heads, int kv_heads, int dim, bool ragged, int max_q, int max_kv, int window) {
  const int group = heads / kv_heads;
  const Cut c = cut_cols(seqs, group, kv_heads, dim, ragged, max_q, max_kv, window);
  return Cuts{c, cut_tile(seqs, tokens, group, kv_heads, dim, ragged, max_q, max_kv, window, c.items ? kSmall : 0)};
}

template <int DT, bool FP8, int DP>
hipError_t go(const Params& base, const Cut& cc, const Cut& ct, hipStream_t stream) {
  Params pc = base, pt = base;
  pc.tiles = cc.tiles;
  pc.chunk = cc.chunk;
  pc.splits = cc.splits;
  pc.cols = cc.cols;
  pc.join_later = cc.splits > kJoinHere;
  const int64_t all_c = cc.items * base.c.heads, all_t = ct.items * base.c.heads;
  pc.part_ml = pc.part_o + all_c * cc.splits * cc.cols * base.c.dim;
  pt.chunk = ct.chunk;
  pt.splits = ct.splits;
  pt.cols = ct.cols;
  pt.items = static_cast<unsigned>(ct.items);
  pt.small = cc.items ? kSmall : 0;
  pt.part_o = reinterpret_cast<float*>(reinterpret_cast<char*>(base.part_o) + (cc.bytes + 255) / 256 * 256);
  pt.part_ml = pt.part_o + all_t * ct.splits * ct.cols * base.c.dim;
  const unsigned blocks_c = static_cast<unsigned>(all_c * cc.splits), blocks_t = static_cast<unsigned>(all_t * ct.splits);
  const dim3 block(64 * kWaves);
  constexpr size_t lds_c = kWaves * kCols * DP * sizeof(float), lds_t = kLdsHalves<DP> * sizeof(_Float16);
  static_assert(lds_c <= lds_t, "the larger serves both");
  hipError_t e = hipSuccess;
  if (cc.items && ct.items)
    e = launch(kv_attention_both_kernel<DT, FP8, DP>, dim3(blocks_t + blocks_c), block, lds_t, stream, pt, pc,
               blocks_t);
  else if (cc.items)
    e = launch(kv_attention_cols_kernel<DT, FP8, DP>, dim3(blocks_c), block, lds_c, stream, pc);
  else if (ct.items)
    e = launch(kv_attention_tile_kernel<DT, FP8, DP>, dim3(blocks_t), block, lds_t, stream, pt);
  if (e == hipSuccess && cc.items && pc.join_later)
    e = launch(kv_attention_join_cols_kernel<DT>, dim3(static_cast<unsigned>(all_c * cc.cols)), block, 0, stream, pc);
  if (e == hipSuccess && ct.items && ct.splits > 1) {
    const int64_t pairs = static_cast<int64_t>(base.a.tokens) * base.a.heads;
    e = launch(kv_attention_join_tile_kernel<DT>, dim3(static_cast<unsigned>((pairs + kWaves - 1) / kWaves)), block, 0, stream, pt);
  }
  return e;
}

template <int DT, bool FP8>
hipError_t by_dim(const Params& p, const Cut& cc, const Cut& ct, hipStream_t stream) {
  if (p.c.dim <= 64) return go<DT, FP8, 64>(p, cc, ct, stream);
  if (p.c.dim <= 128) return go<DT, FP8, 128>(p, cc, ct, stream);
  return go<DT, FP8, 256>(p, cc, ct, stream);
}

size_t bytes_of(const Cut& cc, const Cut& ct) {
  if (cc.bytes == 0 && ct.bytes == 0) return 0;
  return kCounters * sizeof(unsigned) + (cc.bytes + 255) / 256 * 256 + ct.bytes;
}

}  // namespace

size_t kv_attention_workspace_bytes(int seqs, int tokens, int heads, int kv_heads, int dim, bool ragged, int max_q,
                                    int max_kv, int window) {
  const Cuts c = cuts_of(seqs, tokens, heads, kv_heads, dim, ragged, max_q, max_kv, window);
  return bytes_of(c.cols, c.tile);
}

hipError_t launch_kv_attention(const KvCacheView& c, const KvAttentionArgs& a, hipStream_t stream) {
  const auto [cc, ct] = cuts_of(a.seqs, a.tokens, a.heads, c.heads, c.dim, a.cu != nullptr, a.max_q, a.max_kv, a.window);
  if (!grid_fits((cc.items * cc.splits + ct.items * ct.splits) * c.heads, 64 * kWaves) ||
      static_cast<int64_t>(a.tokens) * a.heads > 0x7fffffff)
    return hipErrorInvalidConfiguration;  // the joins' grids are smaller: they are for few tiles
  Params p{};
  p.c = c;
  p.a = a;
  while (1 << p.block_shift < c.block) ++p.block_shift;
  p.group = a.heads / c.heads;
  p.scale2 = std::fabs(a.scale) * 1.4426950408889634f;
  p.flip = a.scale < 0.0f ? 0x80008000u : 0u;
  p.arrived = static_cast<unsigned*>(a.workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kCounters * sizeof(unsigned));
  if (a.dtype == QK_BF16) return c.fp8 ? by_dim<QK_BF16, true>(p, cc, ct, stream) : by_dim<QK_BF16, false>(p, cc, ct, stream);
  return c.fp8 ? by_dim<QK_F16, true>(p, cc, ct, stream) : by_dim<QK_F16, false>(p, cc, ct, stream);
}

}  // namespace qk
