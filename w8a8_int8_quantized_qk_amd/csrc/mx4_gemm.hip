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
#include "mx4.h"
#include "mx4_rule.h"

namespace qk {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;       // the instruction's number of the element type

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

// ---- few rows ----

// Bound by the weight's bytes.  A workgroup has 16 R columns (rows of the weight)
// and 16 F rows of A; its W waves take stretches of S slices of 128 k in turn, and
// their sums meet in LDS in the order of the waves.  A wave brings its own operands
// through LDS of its own, 64 S bytes of a row at a time: loaded straight into the
// registers that the instruction wants (16 bytes of 16 rows from neighbouring lanes)
// they came at a quarter of the rate.  Nothing is shared until the end, so no wave
// waits for another, and several workgroups of a CU keep the weight coming.
// 1 x 14336 x 4096 (m, n, k) 6.9 us (4.5 TB/s, the launch included; loaded straight 10.6), 24 rows 8.0.
template <int DT, int F, int R, int W, int S>
__global__ __launch_bounds__(64 * W) void mx4_gemm_rows_kernel(Mx4GemmArgs g, unsigned tiles_n) {
  constexpr int kRow = 64 * S, kChunks = 4 * S;  // bytes, and 16-byte chunks, of a row in a stretch
  constexpr int kTile = 16 * kRow;               // 16 rows
  constexpr int kOps = kTile / 1024;
  constexpr int kRowsAt = 64 / kChunks;          // rows of one transfer
  constexpr int kWave = (F + R) * kTile;
  static_assert(W * kWave <= 81920 && F * R * 1024 <= kWave, "LDS: two workgroups or more on a CU; the sums");
  __shared__ __attribute__((aligned(1024))) char smem[W * kWave];
  typedef __attribute__((address_space(3))) const v4i* lds_v4i;
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned tile_m = blockIdx.x / tiles_n;
  const int n0 = (blockIdx.x - tile_m * tiles_n) * 16 * R, m0 = tile_m * 16 * F;
  const int blocks = g.k / 32, stretches = (blocks + kChunks - 1) / kChunks;
  const int64_t row_bytes = g.k / 2;
  const uint32_t own = lds_addr(smem) + wave * kWave;
  const uint8_t *sb[R], *sa[F];
#pragma unroll
  for (int i = 0; i < R; ++i) sb[i] = g.scale_b + min(n0 + 16 * i + r, g.n - 1) * g.ldsb;
#pragma unroll
  for (int f = 0; f < F; ++f) sa[f] = g.scale_a + min(m0 + 16 * f + r, g.m - 1) * g.ldsa;
  v4f acc[F][R];
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int i = 0; i < R; ++i) acc[f][i] = v4f{0, 0, 0, 0};
  // Chunks of a row are exchanged by its number, so that a chunk of 16 rows lies in 16
  // different places of 256 bytes (8 where a row has 8 chunks).
  auto key = [](int row) { return kChunks == 16 ? row & 15 : (row >> 1) & 7; };
  for (int t = wave; t < stretches; t += W) {
    // Blocks past k are read from the row's last one, and their scales become
    // 2^-127 in both operands: products of codes are then 2^-247 at most, nothing in
    // binary32.
    auto bring = [&](const uint8_t* base, int row0, int rows, uint32_t to) {
#pragma unroll
      for (int q = 0; q < kOps; ++q) {
        const int row = q * kRowsAt + lane / kChunks;
        const int chunk = min(t * kChunks + ((lane % kChunks) ^ key(row)), blocks - 1);
        lds_dma16(base + min(row0 + row, rows - 1) * row_bytes + 16 * chunk, to + 1024 * q);
      }
    };
#pragma unroll
    for (int i = 0; i < R; ++i) bring(g.b, n0 + 16 * i, g.n, own + i * kTile);
#pragma unroll
    for (int f = 0; f < F; ++f) bring(g.a, m0 + 16 * f, g.m, own + (R + f) * kTile);
    uint32_t ws[R][S], xs[F][S];
    auto scales = [&](const uint8_t* from, uint32_t (&v)[S]) {
#pragma unroll
      for (int s = 0; s < S; ++s) v[s] = reinterpret_cast<const uint32_t*>(from)[t * S + s];
    };
#pragma unroll
    for (int i = 0; i < R; ++i) scales(sb[i], ws[i]);
#pragma unroll
    for (int f = 0; f < F; ++f) scales(sa[f], xs[f]);
    wait_vmcnt<0>();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const bool past = t * kChunks + 4 * s + c >= blocks;
      auto at = [&](int tile) { return *reinterpret_cast<lds_v4i>(own + tile * kTile + r * kRow + (((4 * s + c) ^ key(r)) << 4)); };
      auto scale = [&](uint32_t w) { return static_cast<int>(past ? 0u : w >> (8 * c)); };
      v4i w[R];
#pragma unroll
      for (int i = 0; i < R; ++i) w[i] = at(i);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const v4i x = at(R + f);
#pragma unroll
        for (int i = 0; i < R; ++i)
          acc[f][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w[i]), operand(x), acc[f][i], kFp4, kFp4, 0,
                                                                      scale(ws[i][s]), 0, scale(xs[f][s]));
      }
    }
    // the next stretch's transfers come over what has been read
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
  }
  v4f* const sums = reinterpret_cast<v4f*>(smem + wave * kWave);
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int i = 0; i < R; ++i) sums[(f * R + i) * 64 + lane] = acc[f][i];
  __syncthreads();
  for (int x = wave; x < F * R; x += W) {
    auto of = [&](int w) { return reinterpret_cast<const v4f*>(smem + w * kWave)[x * 64 + lane]; };
    v4f v = of(0);
#pragma unroll
    for (int w = 1; w < W; ++w) v += of(w);
    const int row = m0 + 16 * (x / R) + r, col = n0 + 16 * (x % R) + 4 * c;
    if (row >= g.m) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < g.n) put<DT>(g.out, static_cast<int64_t>(row) * g.n + col + e, v[e] * g.output_scale);
  }
}

template <int DT, int F, int R, int W, int S>
hipError_t rows(const Mx4GemmArgs& g, hipStream_t stream) {
  const int64_t gn = (g.n + 16 * R - 1) / (16 * R), groups = gn * ((g.m + 16 * F - 1) / (16 * F));
  if (!grid_fits(groups, 64 * W)) return hipErrorInvalidConfiguration;
  return launch(mx4_gemm_rows_kernel<DT, F, R, W, S>, dim3(static_cast<unsigned>(groups)), dim3(64 * W), 0, stream, g,
                static_cast<unsigned>(gn));
}

// The same for up to 16 rows that are not quantised yet: one launch for a whole
// linear layer.  A lane's operand is one block of one row, so it quantises its 32 values
// by itself, into the registers and the scale byte that the instruction wants.  The
// values come through LDS too, 128 B k at a time (512 bytes of a row), and every
// workgroup quantises them again.  Stretches, waves and the order of the sums are those of
// mx4_gemm_rows_kernel, and so are the results.
template <int DT, int XT, int R, int W>
__global__ __launch_bounds__(64 * W) void mx4_linear_rows_kernel(Mx4GemmArgs g, const char* x, int64_t ldx) {
  constexpr int XB = qm::Elem<XT>::kBytes;
  constexpr int B = 4 / XB;                      // slices at a time
  constexpr int kRowX = 128 * B * XB, kChunksX = kRowX / 16;  // of a row of values
  constexpr int kRowW = 64 * B, kChunksW = 4 * B;
  constexpr int kTileX = 16 * kRowX, kTileW = 16 * kRowW;
  constexpr int kWave = kTileX + R * kTileW;
  static_assert(W * kWave <= 81920 && R * 1024 <= kWave, "LDS: two workgroups or more on a CU; the sums");
  __shared__ __attribute__((aligned(1024))) char smem[W * kWave];
  typedef __attribute__((address_space(3))) const v4i* lds_v4i;
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16 * R;
  const int blocks = g.k / 32, pieces = (blocks + kChunksW - 1) / kChunksW;
  const int64_t row_bytes = g.k / 2;
  const uint32_t own = lds_addr(smem) + wave * kWave;
  const uint8_t* sb[R];
#pragma unroll
  for (int i = 0; i < R; ++i) sb[i] = g.scale_b + min(n0 + 16 * i + r, g.n - 1) * g.ldsb;
  v4f acc[R];
#pragma unroll
  for (int i = 0; i < R; ++i) acc[i] = v4f{0, 0, 0, 0};
  // Chunks of a row are exchanged by its number, as in the other kernel; a row of the
  // weight has 64 or 128 bytes here, one of the values 512.
  auto key_w = [](int row) { return kChunksW == 8 ? row & 7 : (row >> 1) & 3; };
  auto key_x = [](int row) { return row >> 2 | (row & 3) << 2; };
  // piece p: B slices; a wave's stretches of four slices are those of the other kernel
  for (int p = wave * (4 / B); p < pieces; p = p % (4 / B) == 4 / B - 1 ? p + 1 + (W - 1) * (4 / B) : p + 1) {
#pragma unroll
    for (int q = 0; q < kTileX / 1024; ++q) {
      const int row = q * (64 / kChunksX) + lane / kChunksX;
      if (q * (64 / kChunksX) >= g.m) break;  // rows that are not there: any values, in columns of their own
      const int chunk = min(p * kChunksX + ((lane % kChunksX) ^ key_x(row)), blocks * 2 * XB - 1);
      lds_dma16(x + min(row, g.m - 1) * ldx * XB + 16 * static_cast<int64_t>(chunk), own + 1024 * q);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int q = 0; q < kTileW / 1024; ++q) {
        const int row = q * (64 / kChunksW) + lane / kChunksW;
        const int chunk = min(p * kChunksW + ((lane % kChunksW) ^ key_w(row)), blocks - 1);
        lds_dma16(g.b + min(n0 + 16 * i + row, g.n - 1) * row_bytes + 16 * chunk, own + kTileX + i * kTileW + 1024 * q);
      }
    uint32_t ws[R][B];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int s = 0; s < B; ++s) ws[i][s] = reinterpret_cast<const uint32_t*>(sb[i])[p * B + s];
    wait_vmcnt<0>();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int s = 0; s < B; ++s) {
      const bool past = (p * B + s) * 4 + c >= blocks;
      float v[32];
#pragma unroll
      for (int j = 0; j < 2 * XB; ++j) {
        const v4i u = *reinterpret_cast<lds_v4i>(own + r * kRowX + ((((4 * s + c) * 2 * XB + j) ^ key_x(r)) << 4));
        qm::Elem<XT>::unpack(make_uint4(u[0], u[1], u[2], u[3]), v + j * qm::Elem<XT>::kPerUnit);
      }
      const mx4::Block b = mx4::quantised(v);
      const v4i a = {static_cast<int>(b.codes[0]), static_cast<int>(b.codes[1]), static_cast<int>(b.codes[2]), static_cast<int>(b.codes[3])};
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const v4i w = *reinterpret_cast<lds_v4i>(own + kTileX + i * kTileW + r * kRowW + (((4 * s + c) ^ key_w(r)) << 4));
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(a), acc[i], kFp4, kFp4, 0,
                                                                 static_cast<int>(past ? 0u : ws[i][s] >> (8 * c)), 0,
                                                                 static_cast<int>(past ? 0u : b.scale));
      }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the next piece comes over what has been read
    asm volatile("" ::: "memory");
  }
  v4f* const sums = reinterpret_cast<v4f*>(smem + wave * kWave);
#pragma unroll
  for (int i = 0; i < R; ++i) sums[i * 64 + lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < R; i += W) {
    auto of = [&](int w) { return reinterpret_cast<const v4f*>(smem + w * kWave)[i * 64 + lane]; };
    v4f v = of(0);
#pragma unroll
    for (int w = 1; w < W; ++w) v += of(w);
    const int col = n0 + 16 * i + 4 * c;
    if (r >= g.m) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < g.n) put<DT>(g.out, static_cast<int64_t>(r) * g.n + col + e, v[e] * g.output_scale);
  }
}

template <int DT, int XT>
hipError_t linear_rows(const Mx4GemmArgs& g, const void* x, int64_t ldx, hipStream_t stream) {
  const char* const from = static_cast<const char*>(x);
  auto grid = [&](int cols) { return dim3(static_cast<unsigned>((g.n + cols - 1) / cols)); };
  if (g.n >= kMx4Cols64) return launch(mx4_linear_rows_kernel<DT, XT, 4, 4>, grid(64), dim3(256), 0, stream, g, from, ldx);
  if (g.n >= kMx4Cols32) return launch(mx4_linear_rows_kernel<DT, XT, 2, 4>, grid(32), dim3(256), 0, stream, g, from, ldx);
  return launch(mx4_linear_rows_kernel<DT, XT, 1, 8>, grid(16), dim3(512), 0, stream, g, from, ldx);
}

template <int DT>
hipError_t linear_by_type(const Mx4GemmArgs& g, const void* x, int64_t ldx, int x_dtype, hipStream_t stream) {
  switch (x_dtype) {
    case QK_F32: return linear_rows<DT, QK_F32>(g, x, ldx, stream);
    case QK_BF16: return linear_rows<DT, QK_BF16>(g, x, ldx, stream);
    default: return linear_rows<DT, QK_F16>(g, x, ldx, stream);
  }
}

// ---- many rows: tiles in LDS ----

// lds_dma16_split by all lanes where i < n (both uniform), else by none, which
// counts as a load that has arrived.  Every lane is active before and after it.  A
// branch around the load instead would let the compiler move the products of a
// whole loop behind it, and their operands into scratch memory.
__device__ __forceinline__ void lds_dma16_below(int i, int n, const void* sbase, uint32_t voff, uint32_t lds_base) {
  asm volatile(
      "s_mov_b32 m0, %2\n\ts_cmp_lt_i32 %3, %4\n\ts_cselect_b64 exec, -1, 0\n\tglobal_load_lds_dwordx4 %0, %1\n\t"
      "s_mov_b64 exec, -1"
      :
      : "v"(voff), "s"(sbase), "s"(lds_base), "s"(i), "s"(n)
      : "memory", "m0", "scc");
}

// A pointer that all lanes hold alike, in scalar registers.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(hi) << 32 | lo);
}

// A workgroup has BM x BN outputs, a wave WTM x WTN of them, with
// v_mfma_scale_f32_16x16x128_f8f6f4 (measured alone, on random codes: 7.3
// PFLOP/s, where 32x32x64 reaches 6.7; with all codes 0 both reach 9.5: the
// power that the operands take holds the clock down).
//
// Slices of 128 k (64 bytes of a row, four blocks) go from memory to LDS in pairs,
// so that a transfer touches 8 whole lines of 128 bytes and not 16 halves (8192 x 28672 x
// 8192: 837 us for 898; 2048 x 4096 x 14336: 60.5 for 69), into a ring of as many pairs
// as LDS holds: two, or in 128 x 128 tiles four (512 x 4096 x 14336: 32.5 us; 35.9 with two
// such workgroups on a CU and slices one by one, 39.7 with two of two pairs each).  A part of
// the ring is free as soon as every wave has read its fragments, and is then asked for the
// next pair.
//
// Figures: 8192 x 28672 x 8192 840 to 865 us (4.4 to 4.6 PFLOP/s; the products alone, from
// LDS that nothing is brought to, 718; the stores, while which nothing is multiplied, 84
// of both), 4096 x 4096 x 14336 97 to 101, 2048 x 4096 x 4096 21.7 to 23.1 (of which stores
// 4), 512 x 4096 x 4096 13.2.  Columns that are no multiple of 16 bytes of results are
// stored one by one and through the caches: 2048 x 4097 x 4096 42, 8192 x 28671 x 8192 1120.
// With 16-bit results 16 bytes of the arguments lie in scratch memory per lane, written
// ahead of the loop and read behind it.
//
// A lane's quarter of a wave is its block of a slice, and the byte of its scale
// register that the instruction picks is the slice: the scales of four slices, 16
// bytes of a row, have to be transposed as a 4 x 4 matrix of bytes for that.
// Each thread does so for one row, 16 slices at a time, in place in LDS; a
// fragment's scales are then one 32-bit read in four slices, and no vector
// instruction stands between the products.  (64 bytes of a row are asked for at
// a time because a transfer costs by the lines that it touches: with 16 bytes
// of 64 rows in each, the scales cost a tenth of the kernel.)
template <int DT, int BM, int BN, int WTM, int WTN, bool KTAIL>
struct Mx4Tile {
  static constexpr int kWavesN = BN / WTN;
  static constexpr int kWaves = (BM / WTM) * kWavesN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRing = BM * BN > 128 * 128 ? 2 : 4;  // pairs of slices
  static constexpr int kRow = 128;                           // bytes of a row in a pair
  static constexpr int kStageA = BM * kRow, kStageB = BN * kRow;
  static constexpr int kScales = kRing * (kStageA + kStageB);  // rows of 64 bytes of scales follow the ring
  static constexpr int kUsed = kScales + kWaves * 64 * 64;
  // All of a CU's LDS, or half of it: workgroups of anything between were
  // started one after the other, some 50 ns apart (2048 x 4096 x 4096 on 256 tiles,
  // with 136 KiB each: 34.6 us; with 160: 23.8).
  static constexpr int kSmem = 163840;
  static constexpr int kRowsAt = 1024 / kRow;             // rows of a transfer
  static constexpr int kOps = (BM + BN) / kRowsAt / kWaves;  // transfers of a pair per wave
  static constexpr int kPieces = (BM + BN) / 64;
  static constexpr int FM = WTM / 16, FN = WTN / 16;
  static constexpr int kElem = DT == QK_F32 ? 4 : 2;
  static_assert(kOps * kWaves * kRowsAt == BM + BN && BM % 64 == 0 && BN % 64 == 0, "whole transfers");
  static_assert(kPieces <= kWaves, "a thread for every row of scales");
  static_assert(kUsed <= kSmem && kWaves * 16384 <= kSmem, "LDS; 16 KiB of it per wave for the results");
  static_assert((kRing - 1) * kStageA + 16 * kRow * (FM - 1) < 65536 && (kRing - 1) * kStageB + 16 * kRow * (FN - 1) < 65536, "immediate offsets");
  static_assert((FM == 8 || FM == 4) && FN == 4 && kOps <= 8, "the orders below");

  typedef __attribute__((address_space(3))) const v4i* lds_v4i;
  typedef __attribute__((address_space(3))) v4i* lds_v4i_out;
  typedef __attribute__((address_space(3))) const int* lds_int;

  // 16-byte chunks of a row are exchanged by its number.  The 64 lanes' reads of a
  // fragment (chunk c of rows 0 .. 15, c = 0 .. 3) go in sets of 16 that take half of their rows
  // from one chunk and half from the next; those fall on 16 different places of 256 bytes
  // with this key and not with, say, row / 4 of 64-byte rows, which took twice as long.
  __device__ static int key(int row) { return row & 7; }
  __device__ static int row_offset(int row, int chunk) { return row * kRow + ((chunk ^ key(row)) << 4); }
  __device__ static int scale_offset(int row, int chunk) { return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4); }

  __device__ static __forceinline__ void run(const Mx4GemmArgs& g, int tm, int tn) {
    __shared__ __attribute__((aligned(1024))) char smem[kSmem];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = tm * BM, n0 = tn * BN;
    const int row_bytes = g.k / 2, blocks = g.k / 32;
    const int KT = (blocks + 3) / 4;
    const uint32_t lds0 = lds_addr(smem);

    // What is needed in few slices is formed where it is used, from a value that the
    // compiler does not know there: kept over the loop it would cost the registers that
    // the fragments need.
    auto here = [](int x) {
      asm volatile("" : "+v"(x));
      return x;
    };

    // ---- transfers ----
    // part p of a pair: 8 rows (A's, then B's); the lanes bring their chunks
    const uint8_t* const base_a = uniform(g.a + static_cast<int64_t>(m0) * row_bytes);
    const uint8_t* const base_b = uniform(g.b + static_cast<int64_t>(n0) * row_bytes);
    uint32_t voff[kOps];
    const int part0 = wave * kOps;
    const int row_at = lane / 8, chunk = lane % 8 ^ key(row_at);  // as row_offset has it
#pragma unroll
    for (int q = 0; q < kOps; ++q) {
      const bool is_a = (part0 + q) * kRowsAt < BM;
      const int row = (part0 + q) * kRowsAt - (is_a ? 0 : BM) + row_at;
      const int from = is_a ? min(m0 + row, g.m - 1) - m0 : min(n0 + row, g.n - 1) - n0;
      voff[q] = static_cast<uint32_t>(from) * static_cast<uint32_t>(row_bytes) + (KTAIL ? 0 : 16 * chunk);
    }
    // slices s and s + 1 (s even), if there is s; blocks past k are read from the row's last
    auto issue = [&](int s, int q) {
      const bool is_a = (part0 + q) * kRowsAt < BM;
      const int at = s / 2 & (kRing - 1);
      const uint32_t to =
          lds0 + (is_a ? at * kStageA : kRing * kStageA + at * kStageB - BM * kRow) + (part0 + q) * 1024;
      const uint8_t* const from = is_a ? base_a : base_b;
      if constexpr (KTAIL)
        lds_dma16_below(s, KT, from, voff[q] + 16 * min(4 * s + here(chunk), blocks - 1), to);
      else
        lds_dma16_below(s, KT, from + static_cast<int64_t>(s) * 64, voff[q], to);
    };
    // Scales of 16 slices: 64 bytes (chunks of four slices' 16) of each of this
    // wave's 64 rows, laid out and exchanged as a slice's.  Chunks past the row's
    // last are read from that.  A wave past the rows has room of its own, and brings
    // nothing.
    const bool scales_a = wave * 64 < BM;
    const uint8_t* const base_s = uniform(scales_a ? g.scale_a + m0 * g.ldsa : g.scale_b + n0 * g.ldsb);
    const uint32_t lds_s = static_cast<uint32_t>(scales_a ? g.ldsa : g.ldsb);
    const int rows_s = (scales_a ? g.m - m0 : g.n - n0) - 1, row_s = wave * 64 - (scales_a ? 0 : BM);
    const int last_chunk = (KT - 1) >> 2;
    const uint32_t wave_scales = lds0 + kScales + wave * 64 * 64;
    auto issue_scales = [&](int batch, int q) {
      const int l = here(lane), c = (l & 3) ^ ((l >> 3) & 3);
      const uint32_t row = static_cast<uint32_t>(min(row_s + q * 16 + (l >> 2), rows_s));
      lds_dma16_below(wave < kPieces ? 16 * batch : KT, KT, base_s, row * lds_s + 16 * min(4 * batch + c, last_chunk),
                   wave_scales + q * 1024);
    };
    auto own_scales = [&](int x) { return wave_scales + here(lane) * 64 + 16 * x; };  // of this thread's row
    auto raw_scales = [&](int x) { return *reinterpret_cast<lds_v4i>(own_scales(x)); };
    auto put_scales = [&](int batch, int x, v4i w) {
      // Those of blocks past k, where anything may lie, become 2^-127 in both
      // operands: products of codes are then 2^-247 at most, nothing in binary32.
      if constexpr (KTAIL) {
        const int left = blocks - 16 * (4 * batch + (x ^ ((here(lane) >> 1) & 3)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int have = left - 4 * i;
          const uint32_t keep = have >= 4 ? ~0u : have <= 0 ? 0u : (1u << (8 * have)) - 1u;
          w[i] = static_cast<int>(static_cast<uint32_t>(w[i]) & keep);
        }
      }
      uint32_t t[4];
      tile::transpose4x4(w[0], w[1], w[2], w[3], t[0], t[1], t[2], t[3]);
      *reinterpret_cast<lds_v4i_out>(own_scales(x)) =
          v4i{static_cast<int>(t[0]), static_cast<int>(t[1]), static_cast<int>(t[2]), static_cast<int>(t[3])};
    };

    // ---- fragments ----
    const int wm = wave / kWavesN, wn = wave % kWavesN;
    const int i16 = lane & 15, c4 = lane >> 4;
    auto opaque = [](uint32_t x) {
      asm("" : "+v"(x));
      return x;
    };
    const uint32_t a_base = opaque(lds0 + row_offset(wm * WTM + i16, c4));
    const uint32_t b_base = opaque(lds0 + kRing * kStageA + row_offset(wn * WTN + i16, c4));
    const uint32_t sa_base = opaque(lds0 + kScales + scale_offset(wm * WTM + i16, 0) + 4 * c4);
    const uint32_t sb_base = opaque(lds0 + kScales + scale_offset(BM + wn * WTN + i16, 0) + 4 * c4);
    // of slice S of the ring's
    auto read_a = [&](int S, int i) { return *reinterpret_cast<lds_v4i>((a_base ^ (S % 2) << 6) + S / 2 * kStageA + 16 * kRow * i); };
    auto read_b = [&](int S, int j) { return *reinterpret_cast<lds_v4i>((b_base ^ (S % 2) << 6) + S / 2 * kStageB + 16 * kRow * j); };
    v4f acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = v4f{0, 0, 0, 0};
    v4i fa[FM], fb[FN];
    int sa[FM], sb[FN];  // of four slices
    int ta[FM], tb[FN];  // small tiles: of the next four
    auto scale_a = [&](int chunk, int i) { return *reinterpret_cast<lds_int>((sa_base ^ (chunk << 4)) + 1024 * i); };
    auto scale_b = [&](int chunk, int j) { return *reinterpret_cast<lds_int>((sb_base ^ (chunk << 4)) + 1024 * j); };
    auto barrier = [] {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    auto pin = [] { __builtin_amdgcn_sched_barrier(0); };

    if (KT > 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q) issue_scales(0, q);
#pragma unroll
      for (int s = 0; s < 2 * kRing; s += 2)
#pragma unroll
        for (int q = 0; q < kOps; ++q) issue(s, q);
      wait_vmcnt<(kRing - 1) * kOps>();
#pragma unroll
      for (int x = 0; x < 4; ++x) put_scales(0, x, raw_scales(x));
      __syncthreads();
#pragma unroll
      for (int j = 0; j < FN; ++j) sb[j] = scale_b(0, j), fb[j] = read_b(0, j);
#pragma unroll
      for (int i = 0; i < FM; ++i) sa[i] = scale_a(0, i), fa[i] = read_a(0, i);
    }

    // Slice kt, X its number modulo 16 (a constant wherever it is used).  At the
    // barrier in an odd slice the next pair has landed, for every wave, and every wave
    // has read the last of this one, whose part of the ring is then asked for the next
    // pair but kRing - 1.  The last scales of a batch are read in slice 11 or, half of them
    // where FM is 8, in slice 12 ahead of its barrier, so the next batch may come over it
    // from that barrier on; in slice 14 it is there, each thread transposes what its own
    // wave brought, and it is read behind slice 15's barrier.
    // (Loads arrive in order: the waits count those that may still be under way, in
    // slice 13 the scales among them.)
    auto meet = [&](int X) {
      if (X % 2 == 0 && X != 12) return;
      if (X == 13) wait_vmcnt<(kRing - 2) * kOps + 4>();
      else if (X != 12) wait_vmcnt<(kRing - 2) * kOps>();
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
      barrier();
    };
    auto slice = [&](int X, int kt) __attribute__((always_inline)) {
      const int S = X & (2 * kRing - 1), SN = (X + 1) & (2 * kRing - 1);
      const int next = (kt >> 4) + 1;  // the next batch of scales
      auto mfma = [&](int i, int j) {
        // the byte's number is part of the instruction
        if ((X & 3) == 0) acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(fb[j]), operand(fa[i]), acc[i][j], kFp4, kFp4, 0, sb[j], 0, sa[i]);
        if ((X & 3) == 1) acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(fb[j]), operand(fa[i]), acc[i][j], kFp4, kFp4, 1, sb[j], 1, sa[i]);
        if ((X & 3) == 2) acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(fb[j]), operand(fa[i]), acc[i][j], kFp4, kFp4, 2, sb[j], 2, sa[i]);
        if ((X & 3) == 3) acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(fb[j]), operand(fa[i]), acc[i][j], kFp4, kFp4, 3, sb[j], 3, sa[i]);
        pin();
      };
      auto dma = [&](int q) {
        if (X == 12) issue_scales(next, q);
        pin();
      };
      auto data = [&](int q) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (X % 2 == 1 && 2 * q + j < kOps) issue(kt + 2 * kRing - 1, 2 * q + j);
        pin();
      };
      v4i raw[2];
      auto scales = [&](int part) {  // work on scales between the last products: 12 parts
        const int chunk = ((X + 1) >> 2) & 3;
        if ((X & 3) == 3 && FM == 8) {  // the first half's; the others are still in use
          if (part >= 6 && part < 10) sa[part - 6] = scale_a(chunk, part - 6);
          if (part >= 10) sb[part - 10] = scale_b(chunk, part - 10);
        }
        if ((X & 3) == 3 && FM == 4) {
          if (part < FN) tb[part] = scale_b(chunk, part);
          else if (part < FN + FM) ta[part - FN] = scale_a(chunk, part - FN);
        }
        if (X == 14 && part == 0) {
          wait_vmcnt<kOps>();
          asm volatile("" ::: "memory");
        }
        if (X == 14 && (part == 0 || part == 1 || part == 6 || part == 7)) raw[part & 1] = raw_scales(part < 6 ? part : part - 4);
        if (X == 14 && (part == 4 || part == 5 || part == 10 || part == 11))
          put_scales(next, part < 6 ? part - 4 : part - 8, raw[part & 1]);
        pin();
      };
      if constexpr (FM == 8) {
        // Each fragment is read several products before its first use, and the
        // slice's last well before the barrier.  In hand: A 0 .. 3, B 0 .. 1.
        mfma(0, 0);
        fa[4] = read_a(S, 4);
        fa[5] = read_a(S, 5);
        mfma(0, 1);
        fa[6] = read_a(S, 6);
        fa[7] = read_a(S, 7);
        mfma(1, 0);
        fb[2] = read_b(S, 2);
        fb[3] = read_b(S, 3);
        mfma(1, 1);
        if ((X & 3) == 0) {
#pragma unroll
          for (int x = 0; x < 4; ++x) sa[4 + x] = scale_a(X >> 2, 4 + x);
          sb[2] = scale_b(X >> 2, 2);
          sb[3] = scale_b(X >> 2, 3);
          pin();
        }
        mfma(2, 0);
        mfma(2, 1);
        mfma(3, 0);
        mfma(3, 1);
        meet(X);
        if (X == 12) {
#pragma unroll
          for (int q = 0; q < 4; ++q) dma(q);
        }
        // after the last slice these come from a stage that is there and are not used
        v4i na[4], nb[2];
        mfma(4, 0);
        scales(0);
        mfma(5, 0);
        data(0);
        mfma(6, 0);
        scales(1);
        mfma(7, 0);
        nb[0] = read_b(SN, 0);
        mfma(4, 1);
        scales(2);
        mfma(5, 1);
        data(1);
        mfma(6, 1);
        scales(3);
        mfma(7, 1);
        nb[1] = read_b(SN, 1);
        mfma(0, 2);
        scales(4);
        mfma(0, 3);
        na[0] = read_a(SN, 0);
        mfma(1, 2);
        data(2);
        mfma(1, 3);
        na[1] = read_a(SN, 1);
        mfma(2, 2);
        scales(5);
        mfma(2, 3);
        na[2] = read_a(SN, 2);
        mfma(3, 2);
        data(3);
        mfma(3, 3);
        na[3] = read_a(SN, 3);
        mfma(4, 2);
        scales(6);
        mfma(4, 3);
        scales(7);
        mfma(5, 2);
        scales(8);
        mfma(5, 3);
        scales(9);
        mfma(6, 2);
        scales(10);
        mfma(6, 3);
        scales(11);
        mfma(7, 2);
        mfma(7, 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) fa[i] = na[i];
        fb[0] = nb[0];
        fb[1] = nb[1];
      } else {
        // Small sets of fragments are held twice: after the barrier the next slice's
        // are read while this one's, read before it, are multiplied.
        meet(X);
        if (X == 12) {
#pragma unroll
          for (int q = 0; q < 4; ++q) dma(q);
        }
        v4i na[FM], nb[FN];
#pragma unroll
        for (int x = 0; x < FM * FN; ++x) {
          mfma(x / FN, x % FN);
          if (x < FN) nb[x] = read_b(SN, x);
          else if (x < FN + FM) na[x - FN] = read_a(SN, x - FN);
          if (x % 2 == 1 && x / 2 < 4) data(x / 2);
          scales(x < 12 ? x : 99);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[i] = na[i];
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[j] = nb[j];
        if ((X & 3) == 3) {
#pragma unroll
          for (int i = 0; i < FM; ++i) sa[i] = ta[i];
#pragma unroll
          for (int j = 0; j < FN; ++j) sb[j] = tb[j];
        }
      }
    };
    int kt = 0;
    for (; kt + 16 <= KT; kt += 16) {
      slice(0, kt + 0);
      slice(1, kt + 1);
      slice(2, kt + 2);
      slice(3, kt + 3);
      slice(4, kt + 4);
      slice(5, kt + 5);
      slice(6, kt + 6);
      slice(7, kt + 7);
      slice(8, kt + 8);
      slice(9, kt + 9);
      slice(10, kt + 10);
      slice(11, kt + 11);
      slice(12, kt + 12);
      slice(13, kt + 13);
      slice(14, kt + 14);
      slice(15, kt + 15);
    }
    if (kt + 0 < KT) slice(0, kt + 0);
    if (kt + 1 < KT) slice(1, kt + 1);
    if (kt + 2 < KT) slice(2, kt + 2);
    if (kt + 3 < KT) slice(3, kt + 3);
    if (kt + 4 < KT) slice(4, kt + 4);
    if (kt + 5 < KT) slice(5, kt + 5);
    if (kt + 6 < KT) slice(6, kt + 6);
    if (kt + 7 < KT) slice(7, kt + 7);
    if (kt + 8 < KT) slice(8, kt + 8);
    if (kt + 9 < KT) slice(9, kt + 9);
    if (kt + 10 < KT) slice(10, kt + 10);
    if (kt + 11 < KT) slice(11, kt + 11);
    if (kt + 12 < KT) slice(12, kt + 12);
    if (kt + 13 < KT) slice(13, kt + 13);
    if (kt + 14 < KT) slice(14, kt + 14);

    // ---- results ----
    // register e of a fragment is row (of out) i16, column 4 c4 + e.  A wave puts
    // rows of WTN results into its 16 KiB of LDS, as many at a time as fit, and
    // stores them 16 bytes per lane.
    __syncthreads();
    constexpr int kRowOut = WTN * kElem;                   // bytes
    constexpr int kChunks = kRowOut / 16;
    constexpr int kFrags = 16384 / (16 * kRowOut) < FM ? 16384 / (16 * kRowOut) : FM;  // fragments of rows at a time
    char* const stage = smem + wave * 16384;
    auto place = [](int row, int chunk) { return row * kRowOut + ((chunk ^ (row & (kChunks - 1))) << 4); };
#pragma unroll
    for (int i0 = 0; i0 < FM; i0 += kFrags) {
      if (i0 > 0) __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int ii = 0; ii < kFrags; ++ii)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const v4f v = acc[i0 + ii][j] * g.output_scale;
          const int row = ii * 16 + i16, col = j * 16 + 4 * c4;
          if constexpr (DT == QK_F32)
            *reinterpret_cast<v4f*>(stage + place(row, col / 4)) = v;
          else
            *reinterpret_cast<uint2*>(stage + place(row, col / 8) + (col & 4) * 2) =
                make_uint2(qm::pack2_narrow<DT>(v[0], v[1]), qm::pack2_narrow<DT>(v[2], v[3]));
        }
      __builtin_amdgcn_wave_barrier();
      constexpr int kRowsAt = 64 / kChunks;  // rows that the wave's lanes take together
      const int chunk = lane % kChunks, col = n0 + wn * WTN + chunk * (16 / kElem);
#pragma unroll 4
      for (int r = lane / kChunks; r < kFrags * 16; r += kRowsAt) {
        typedef unsigned v4u __attribute__((ext_vector_type(4)));
        const v4u w = *reinterpret_cast<const v4u*>(stage + place(r, chunk));
        const int row = m0 + wm * WTM + i0 * 16 + r;
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
  if (g.k % 256) return launch(mx4_gemm_tile_kernel<Tail>, grid, block, 0, stream, g, tm, tn);
  return launch(mx4_gemm_tile_kernel<Whole>, grid, block, 0, stream, g, tm, tn);
}

template <int DT>
hipError_t by_size(const Mx4GemmArgs& g, hipStream_t stream) {
  switch (mx4_kernel_of(g.m, g.n, g.k)) {
    case Mx4Kernel::kRows16x64: return rows<DT, 1, 4, 4, 4>(g, stream);
    case Mx4Kernel::kRows16x32: return rows<DT, 1, 2, 4, 4>(g, stream);
    case Mx4Kernel::kRows16x16: return rows<DT, 1, 1, 8, 4>(g, stream);
    case Mx4Kernel::kRows32x32: return rows<DT, 2, 2, 2, 4>(g, stream);
    case Mx4Kernel::kRows32x16: return rows<DT, 2, 1, 4, 4>(g, stream);
    case Mx4Kernel::kManyRows32: return rows<DT, 2, 2, 4, 4>(g, stream);
    case Mx4Kernel::kManyRows64: return rows<DT, 4, 4, 4, 2>(g, stream);
    case Mx4Kernel::kTile128: return tiles<DT, 128, 128, 64, 64>(g, stream);
    case Mx4Kernel::kTile128x256: return tiles<DT, 128, 256, 64, 64>(g, stream);
    default: return tiles<DT, 256, 256, 128, 64>(g, stream);
  }
}

}  // namespace

hipError_t launch_gemm_mx4(const Mx4GemmArgs& g, hipStream_t stream) {
  switch (g.out_dtype) {
    case QK_F32: return by_size<QK_F32>(g, stream);
    case QK_BF16: return by_size<QK_BF16>(g, stream);
    default: return by_size<QK_F16>(g, stream);
  }
}

hipError_t launch_linear_mx4_rows(const Mx4GemmArgs& g, const void* x, int64_t ldx, int x_dtype, hipStream_t stream) {
  switch (g.out_dtype) {
    case QK_F32: return linear_by_type<QK_F32>(g, x, ldx, x_dtype, stream);
    case QK_BF16: return linear_by_type<QK_BF16>(g, x, ldx, x_dtype, stream);
    default: return linear_by_type<QK_F16>(g, x, ldx, x_dtype, stream);
  }
}

}  // namespace qk
