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

typedef int v4i __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v8i operand(const v4i& w) { return v8i{w[0], w[1], w[2], w[3], 0, 0, 0, 0}; }

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
    const v4i w = *reinterpret_cast<const v4i*>(b + 16 * here);
    const uint32_t ws = in ? sb[here] : kOne;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      v4i x = *reinterpret_cast<const v4i*>(a[f] + 16 * here);
      if (!in) x = v4i{0, 0, 0, 0};
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

// ---- many rows: tiles in LDS ----

__device__ const uint4 kZeros = {0, 0, 0, 0};  // what a block past k is read from

// lds_dma16 by all lanes (who = ~0) or none (0; a load by none counts as one that
// has arrived).  Every lane is active before and after it.  A branch around the
// load instead would let the compiler move the products of a whole loop behind
// it, and their operands into scratch memory.
__device__ __forceinline__ void lds_dma16_by(uint32_t who, const void* sbase, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_mov_b32 exec_lo, %3\n\ts_mov_b32 exec_hi, %3\n\tglobal_load_lds_dwordx4 %0, %1\n\ts_mov_b64 exec, -1"
               :
               : "v"(voff), "s"(sbase), "s"(lds_base), "s"(who)
               : "memory", "m0");
}
__device__ __forceinline__ void lds_dma16_by(uint32_t who, const void* from, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b32 exec_lo, %2\n\ts_mov_b32 exec_hi, %2\n\tglobal_load_lds_dwordx4 %0, off\n\ts_mov_b64 exec, -1"
               :
               : "v"(from), "s"(lds_base), "s"(who)
               : "memory", "m0");
}

// A workgroup has BM x BN outputs, a wave WTM x WTN of them, in steps of 64 k with
// v_mfma_scale_f32_32x32x64_f8f6f4.  Slices of 128 k (64 bytes of a row, four
// blocks) go from memory to LDS in a ring of four stages, three ahead of the one
// that is multiplied; the scales of four slices (16 bytes of a row) in one of two
// buffers.  Half h of a wave takes blocks 2 h and 2 h + 1 of a slice in its two
// steps, for both operands, so that one 16-bit read brings the scales of both
// steps, and the instruction picks the byte: no vector instruction is left
// between the products.
template <int DT, int BM, int BN, int WTM, int WTN, bool KTAIL>
struct Mx4Tile {
  static constexpr int kStages = 4;
  static constexpr int kWavesN = BN / WTN;
  static constexpr int kWaves = (BM / WTM) * kWavesN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRow = 64;                 // bytes of a row in a slice
  static constexpr int kStageA = BM * kRow, kStageB = BN * kRow;
  static constexpr int kScales = kStages * (kStageA + kStageB);  // two buffers of them follow the ring
  static constexpr int kScaleBuf = (BM + BN) * 16;
  static constexpr int kSmem = kScales + 2 * kScaleBuf;
  static constexpr int kOps = (BM + BN) / 16 / kWaves;  // 1 KiB transfers of a slice per wave
  static constexpr int FM = WTM / 32, FN = WTN / 32;
  static constexpr int kElem = DT == QK_F32 ? 4 : 2;
  static_assert(kOps * kWaves * 16 == BM + BN && BM % 16 == 0, "whole transfers");
  static_assert((BM + BN) / 64 <= kWaves, "one transfer of scales per wave");
  static_assert(kSmem <= 163840 && kWaves * 16384 <= kSmem, "LDS; 16 KiB of it per wave for the results");
  static_assert(3 * kStageA + 2048 * (FM - 1) < 65536 && 3 * kStageB + 2048 * (FN - 1) < 65536, "immediate offsets");

  typedef float v16f __attribute__((ext_vector_type(16)));
  typedef __attribute__((address_space(3))) const v4i* lds_v4i;
  typedef __attribute__((address_space(3))) const uint16_t* lds_u16;

  // 16-byte chunks of a row are exchanged by its number: 16 consecutive rows then
  // have a chunk in 16 different places of 256 bytes
  __device__ static int row_offset(int row, int chunk) { return row * kRow + ((chunk ^ ((row >> 2) & 3)) << 4); }

  __device__ static __forceinline__ void run(const Mx4GemmArgs& g, int tm, int tn) {
    __shared__ __attribute__((aligned(1024))) char smem[kSmem];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = tm * BM, n0 = tn * BN;
    const int row_bytes = g.k / 2, blocks = g.k / 32;
    const int KT = (blocks + 3) / 4;
    const uint32_t lds0 = lds_addr(smem);

    // ---- transfers ----
    // part p of a slice: 16 rows (A's, then B's); lane l brings a chunk of row l / 4
    const uint8_t* const base_a = g.a + static_cast<int64_t>(m0) * row_bytes;
    const uint8_t* const base_b = g.b + static_cast<int64_t>(n0) * row_bytes;
    uint32_t voff[kOps];
    const int part0 = wave * kOps;
    auto chunk_of = [&](int row) { return (lane & 3) ^ ((row >> 2) & 3); };
#pragma unroll
    for (int q = 0; q < kOps; ++q) {
      const bool is_a = (part0 + q) * 16 < BM;
      const int row = (part0 + q) * 16 - (is_a ? 0 : BM) + (lane >> 2);
      const int from = is_a ? min(m0 + row, g.m - 1) - m0 : min(n0 + row, g.n - 1) - n0;
      voff[q] = static_cast<uint32_t>(from) * static_cast<uint32_t>(row_bytes) + 16 * chunk_of(row);
    }
    // slice s, if there is one
    auto issue = [&](int s, int q) {
      const bool is_a = (part0 + q) * 16 < BM;
      const uint32_t who = __builtin_amdgcn_readfirstlane(s < KT ? ~0u : 0u);
      const uint32_t to = __builtin_amdgcn_readfirstlane(
          lds0 + (is_a ? (s & 3) * kStageA : kStages * kStageA + (s & 3) * kStageB - BM * kRow) + (part0 + q) * 1024);
      const uint8_t* const from = (is_a ? base_a : base_b) + static_cast<int64_t>(s) * kRow;
      if constexpr (KTAIL) {  // blocks past k: A's are zeros, B's any
        const int row = (part0 + q) * 16 - (is_a ? 0 : BM) + (lane >> 2);
        const int past = 4 * s + chunk_of(row) - (blocks - 1);
        const uint8_t* const src = from + voff[q];
        const uint8_t* const other = is_a ? reinterpret_cast<const uint8_t*>(&kZeros) : src - 16 * past;
        lds_dma16_by(who, past > 0 ? other : src, to);
      } else {
        lds_dma16_by(who, from, voff[q], to);
      }
    };
    // scales of slices 4 group .. 4 group + 3, 64 rows per wave; a wave beyond the
    // rows brings some a second time
    const int piece = wave % ((BM + BN) / 64);
    const uint8_t* scale_from;
    {
      const int row = piece * 64 + lane;
      scale_from = piece * 64 < BM ? g.scale_a + min(m0 + row, g.m - 1) * g.ldsa
                                   : g.scale_b + min(n0 + row - BM, g.n - 1) * g.ldsb;
    }
    auto issue_scales = [&](int group) {
      lds_dma16_by(__builtin_amdgcn_readfirstlane(4 * group < KT ? ~0u : 0u), scale_from + 16 * group,
                   __builtin_amdgcn_readfirstlane(lds0 + kScales + (group & 1) * kScaleBuf + piece * 1024));
    };

    // ---- fragments ----
    const int wm = wave / kWavesN, wn = wave % kWavesN;
    const int i32 = lane & 31, h = lane >> 5;
    auto opaque = [](uint32_t x) {
      asm("" : "+v"(x));
      return x;
    };
    uint32_t a_base[2], b_base[2];  // [step]
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      a_base[s] = opaque(lds0 + row_offset(wm * WTM + i32, 2 * h + s));
      b_base[s] = opaque(lds0 + kStages * kStageA + row_offset(wn * WTN + i32, 2 * h + s));
    }
    const uint32_t sa_base = opaque(lds0 + kScales + (wm * WTM + i32) * 16 + 2 * h);
    const uint32_t sb_base = opaque(lds0 + kScales + (BM + wn * WTN + i32) * 16 + 2 * h);
    auto read_a = [&](int S, int i, int s) { return *reinterpret_cast<lds_v4i>(a_base[s] + S * kStageA + 2048 * i); };
    auto read_b = [&](int S, int j, int s) { return *reinterpret_cast<lds_v4i>(b_base[s] + S * kStageB + 2048 * j); };
    // S8: the slice's number modulo 8
    auto read_sa = [&](int S8, int i) -> int {
      return *reinterpret_cast<lds_u16>(sa_base + (S8 >> 2) * kScaleBuf + (S8 & 3) * 4 + 512 * i);
    };
    auto read_sb = [&](int S8, int j) -> int {
      return *reinterpret_cast<lds_u16>(sb_base + (S8 >> 2) * kScaleBuf + (S8 & 3) * 4 + 512 * j);
    };
    // the scales of blocks past k become 1: whatever lies there may be NaN
    int keep = 0xffff, fill = 0;
    if (KTAIL) {
      const int valid = blocks - 4 * (KT - 1);
      if (2 * h >= valid) keep &= 0xff00, fill |= kOne;
      if (2 * h + 1 >= valid) keep &= 0x00ff, fill |= kOne << 8;
    }

    v16f acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    v4i fa[2][FM], fb[2][FN];
    int sa[FM], sb[FN], na[FM], nb[FN];
    auto settle = [&](int kt) {  // the scales just read are slice kt's
      if constexpr (KTAIL) {
        const int k = kt == KT - 1 ? keep : 0xffff, f = kt == KT - 1 ? fill : 0;
#pragma unroll
        for (int i = 0; i < FM; ++i) sa[i] = (sa[i] & k) | f;
#pragma unroll
        for (int j = 0; j < FN; ++j) sb[j] = (sb[j] & k) | f;
      }
    };

    if (KT > 0) {
      issue_scales(0);
#pragma unroll
      for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int q = 0; q < kOps; ++q) issue(s, q);
      wait_vmcnt<2 * kOps>();
      __syncthreads();
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[0][j] = read_b(0, j, 0), sb[j] = read_sb(0, j);
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[0][i] = read_a(0, i, 0), sa[i] = read_sa(0, i);
      settle(0);
    }
    auto barrier = [] {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    auto pin = [] { __builtin_amdgcn_sched_barrier(0); };
    // Slice kt, S8 its number modulo 8.  While step 0 is multiplied step 1's
    // fragments are read; then slice kt + 1 has landed, and slice kt - 1's stage is
    // free, for every wave; while step 1 is multiplied the next slice's step 0
    // is read and slice kt + 3 asked for.
    auto slice = [&](int S8, int kt) __attribute__((always_inline)) {
      const int S = S8 & 3, N8 = (S8 + 1) & 7;
#pragma unroll
      for (int n = 0; n < FM * FN; ++n) {
        const int i = n / FN, j = n % FN;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fb[0][j]), operand(fa[0][i]), acc[i][j], kFp4,
                                                                   kFp4, 0, sb[j], 0, sa[i]);
        pin();
        if (n < FN) fb[1][n] = read_b(S, n, 1);
        if (n < FM) fa[1][n] = read_a(S, n, 1);
        pin();
      }
      wait_vmcnt<kOps>();  // what may still be under way is slice kt + 2
      barrier();
#pragma unroll
      for (int n = 0; n < FM * FN; ++n) {
        const int i = n / FN, j = n % FN;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fb[1][j]), operand(fa[1][i]), acc[i][j], kFp4,
                                                                   kFp4, 1, sb[j], 1, sa[i]);
        pin();
        // after the last slice these come from a stage that is there and are not used
        if (n < FN) fb[0][n] = read_b(N8 & 3, n, 0), nb[n] = read_sb(N8, n);
        if (n < FM) fa[0][n] = read_a(N8 & 3, n, 0), na[n] = read_sa(N8, n);
        if (n == 0 && (S8 & 3) == 1) issue_scales((kt + 3) >> 2);
        if (n < kOps) issue(kt + 3, n);
        pin();
      }
      static_assert(FM * FN >= kOps && FM * FN >= FM && FM * FN >= FN, "a place for every read and transfer");
#pragma unroll
      for (int i = 0; i < FM; ++i) sa[i] = na[i];
#pragma unroll
      for (int j = 0; j < FN; ++j) sb[j] = nb[j];
      settle(kt + 1);
    };
    int kt = 0;
    for (; kt + 8 <= KT; kt += 8) {
      slice(0, kt);
      slice(1, kt + 1);
      slice(2, kt + 2);
      slice(3, kt + 3);
      slice(4, kt + 4);
      slice(5, kt + 5);
      slice(6, kt + 6);
      slice(7, kt + 7);
    }
    if (kt < KT) slice(0, kt);
    if (kt + 1 < KT) slice(1, kt + 1);
    if (kt + 2 < KT) slice(2, kt + 2);
    if (kt + 3 < KT) slice(3, kt + 3);
    if (kt + 4 < KT) slice(4, kt + 4);
    if (kt + 5 < KT) slice(5, kt + 5);
    if (kt + 6 < KT) slice(6, kt + 6);

    // ---- results ----
    // register 4 q + e of a fragment is row (of out) i32, column 8 q + 4 h + e.  A wave
    // puts rows of WTN results into its 16 KiB of LDS, as many at a time as fit,
    // and stores them 16 bytes per lane.
    __syncthreads();
    constexpr int kRowOut = WTN * kElem;                   // bytes
    constexpr int kChunks = kRowOut / 16;
    constexpr int kFrags = 16384 / (32 * kRowOut) < FM ? 16384 / (32 * kRowOut) : FM;  // fragments of rows at a time
    char* const stage = smem + wave * 16384;
    auto place = [](int row, int chunk) { return row * kRowOut + ((chunk ^ (row & (kChunks - 1))) << 4); };
#pragma unroll
    for (int i0 = 0; i0 < FM; i0 += kFrags) {
      if (i0 > 0) __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int ii = 0; ii < kFrags; ++ii)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[i0 + ii][j][4 * q + e] * g.output_scale;
            const int row = ii * 32 + i32, col = j * 32 + 8 * q + 4 * h;
            if constexpr (DT == QK_F32)
              *reinterpret_cast<float4*>(stage + place(row, col / 4)) = make_float4(v[0], v[1], v[2], v[3]);
            else
              *reinterpret_cast<uint2*>(stage + place(row, col / 8) + (col & 4) * 2) =
                  make_uint2(qm::pack2_narrow<DT>(v[0], v[1]), qm::pack2_narrow<DT>(v[2], v[3]));
          }
      __builtin_amdgcn_wave_barrier();
      constexpr int kRowsAt = 64 / kChunks;  // rows that the wave's lanes take together
      const int chunk = lane % kChunks, col = n0 + wn * WTN + chunk * (16 / kElem);
#pragma unroll 4
      for (int r = lane / kChunks; r < kFrags * 32; r += kRowsAt) {
        typedef unsigned v4u __attribute__((ext_vector_type(4)));
        const v4u w = *reinterpret_cast<const v4u*>(stage + place(r, chunk));
        const int row = m0 + wm * WTM + i0 * 32 + r;
        if (row >= g.m || col >= g.n) continue;
        char* const to = static_cast<char*>(g.out) + (static_cast<int64_t>(row) * g.n + col) * kElem;
        if (col + 16 / kElem <= g.n && reinterpret_cast<uintptr_t>(to) % 16 == 0) {
          __builtin_nontemporal_store(w, reinterpret_cast<v4u*>(to));
        } else {
#pragma unroll
          for (int e = 0; e < 16 / kElem; ++e) {
            if (col + e >= g.n) continue;
            if constexpr (DT == QK_F32)
              reinterpret_cast<uint32_t*>(to)[e] = w[e];
            else
              reinterpret_cast<uint16_t*>(to)[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
          }
        }
      }
    }
  }
};

template <typename Tile>
__global__ __launch_bounds__(Tile::kThreads, 2) void mx4_gemm_tile_kernel(Mx4GemmArgs g, int tiles_m, int tiles_n) {
  int tm, tn;
  tile::tile_coords(tiles_m, tiles_n, tm, tn);
  Tile::run(g, tm, tn);
}

template <int DT, int BM, int BN, int WTM, int WTN>
hipError_t tiles(const Mx4GemmArgs& g, hipStream_t stream) {
  using Whole = Mx4Tile<DT, BM, BN, WTM, WTN, false>;
  using Tail = Mx4Tile<DT, BM, BN, WTM, WTN, true>;
  const int tm = (g.m + BM - 1) / BM, tn = (g.n + BN - 1) / BN;
  const dim3 grid(static_cast<unsigned>(tm) * static_cast<unsigned>(tn)), block(Whole::kThreads);
  if (!grid_fits(static_cast<int64_t>(tm) * tn, Whole::kThreads)) return hipErrorInvalidConfiguration;
  if (g.k % 128) return launch(mx4_gemm_tile_kernel<Tail>, grid, block, 0, stream, g, tm, tn);
  return launch(mx4_gemm_tile_kernel<Whole>, grid, block, 0, stream, g, tm, tn);
}

template <int DT>
hipError_t by_size(const Mx4GemmArgs& g, hipStream_t stream) {
  if (g.m <= 16) return rows<DT, 1, 4>(g, stream);
  if (g.m <= 64) return rows<DT, 4, 4>(g, stream);
  const int64_t large = static_cast<int64_t>((g.m + 255) / 256) * ((g.n + 255) / 256);
  if (large >= 256) return tiles<DT, 256, 256, 128, 64>(g, stream);
  return tiles<DT, 128, 128, 64, 64>(g, stream);
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
