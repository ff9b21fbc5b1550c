// The choices of the 4-bit product and layer: host code without any other part of the
// library, so that the binding, which allocates codes and scales only for the calls that
// need them, and tests have the same.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace qk {

// Whether x [m][k], its rows row_bytes apart, is quantised within its product with a
// weight of n rows, in one launch: where the weight is small.  One launch / two, from
// a graph, and called one by one (where a second launch costs the host 3 us): 1 x
// 4096 x 4096 4.7 / 4.7 and 4.7 / 7.9 us; 16 x 4096 x 4096 5.8 / 5.4 and 5.7 / 7.8;
// 1 x 14336 x 4096 10.0 / 9.0 and 9.7 / 8.7; 16 x 4096 x 14336 13.5 / 9.3 and 13.2 / 9.1:
// quantising again in every workgroup grows with n k.
inline bool mx4_linear_at_once(int64_t m, int64_t n, int64_t k, const void* x, int64_t row_bytes) {
  return m <= 16 && k > 0 && n * k <= int64_t{1} << 24 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
         (m <= 1 || row_bytes % 16 == 0);
}

// The product's kernels: workgroups of few rows (rows x columns), the same for many
// rows, and tiles in LDS.
enum class Mx4Kernel {
  kRows16x64, kRows16x32, kRows16x16, kRows32x32, kRows32x16,
  kManyRows32, kManyRows64,                // 32 x 32 and 64 x 64
  kTile128, kTile128x256, kTile256,        // 128 x 128, 128 x 256 and 256 x 256
};

// Columns from which a workgroup of few rows has 64, or 32, of them: 400 workgroups.
constexpr int kMx4Cols64 = 64 * 400, kMx4Cols32 = 32 * 400;

// How many tiles one of 256 CUs takes one after the other, in times of a tile on a full
// chip: the last ones, on a part of the CUs, take less, down to `least` (clock and
// memory are theirs).
inline double mx4_rounds(double tiles, double least) {
  const double full = std::ceil(tiles / 256) - 1, part = tiles / 256 - full;
  return full + least + (1 - least) * part * part * part;
}

// Up to 32 rows: as many columns to a workgroup as leave enough of them (28672,
// 14336 and 4096 columns in 64 / 32 / 16: one row of 4096 k 7.9 / 6.9 / 7.4 us with
// 14336, 16 rows of 8192 k 28.6 / 29.8 / 30.2 with 28672, of 4096 k 5.9 / 4.6 / 3.8
// with 4096; 24 rows of 4096 k 8.0 in 32 by two waves, 9.0 by four, 9.7 in 16 with 14336;
// 32 rows of 8192 k 34.2 / 35.2 / 39.5 with 28672; 24 of 4096 k 5.8 / 5.2 / 4.7 with 4096).
//
// Beyond, the least estimated time, in us: a workgroup's time grows with k, a CU takes
// one after the other.  The tiles' numbers are fitted to 48 to 6000 rows of 1024 to 14336
// columns and k, which they meet within 3% at the mean; the kernel taken there is the
// fastest one or within 4% of it but for 96 to 1500 rows of k 1024 or few tiles, where
// workgroups of few rows take up to 1.17 of it.  Measured, of rows in 64 x 64 / tiles of
// 128 x 128 / 128 x 256 / 256 x 256: 256 x 4096 x 14336 22.5 / 32 / 54 / -; 512 x 4096 x
// 14336 39.6 / 32.3 / 53.9 / -; 1024 x 4096 x 4096 - / 13.8 / 19.5 / 28; 2048 x 4096 x 4096
// - / 26.2 / 21.6 / 27.3; 2048 x 4096 x 14336 - / 74.1 / 61.3 / 74.8; 3000 x 4096 x 4096
// - / 38.8 / 39.0 / 29.2; 4096 x 6144 x 14336 - / 221 / 185 / 170.  (Without the part of a
// last round that is saved, 128 x 128 was taken for the other two where a CU has three of
// its tiles for one or two of theirs: up to 1.35 of their time.)
inline Mx4Kernel mx4_kernel_of(int m, int n, int k) {
  if (m <= 16) return n >= kMx4Cols64 ? Mx4Kernel::kRows16x64 : n >= kMx4Cols32 ? Mx4Kernel::kRows16x32 : Mx4Kernel::kRows16x16;
  if (m <= 32) return n >= kMx4Cols32 ? Mx4Kernel::kRows32x32 : Mx4Kernel::kRows32x16;
  auto count = [&](int bm, int bn) { return static_cast<double>((m + bm - 1) / bm) * ((n + bn - 1) / bn); };
  const double slices = (k + 127) / 128;
  const double rows32 = 3.0 + 0.075 * slices * std::max(count(32, 32) / 256, 1.0);
  const double rows64 = 3.5 + 0.24 * slices * std::max(count(64, 64) / 256, 1.0);
  const double tile1 = 2.3 + (3.4 + 0.285 * slices) * mx4_rounds(count(128, 128), 0.86);
  const double tile2 = 1.5 + (4.2 + 0.51 * slices) * mx4_rounds(count(128, 256), 0.86);
  const double tile4 = 1.5 + (7.0 + 0.81 * slices) * mx4_rounds(count(256, 256), 0.75);
  const double best = std::min({rows32, rows64, tile1, tile2, tile4});
  if (best == tile4) return Mx4Kernel::kTile256;
  if (best == tile2) return Mx4Kernel::kTile128x256;
  if (best == tile1) return Mx4Kernel::kTile128;
  return best == rows64 ? Mx4Kernel::kManyRows64 : Mx4Kernel::kManyRows32;
}

}  // namespace qk
