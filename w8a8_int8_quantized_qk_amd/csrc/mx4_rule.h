// The choice of the 4-bit layer, for the library and for the binding, which
// allocates codes and scales only for the calls that need them.
#pragma once

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

}  // namespace qk
