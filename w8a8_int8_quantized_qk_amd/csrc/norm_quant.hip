// Root-mean-square norm with the residual's addition and an 8-bit output with
// per-token scales, one launch, for gfx950.
//
// Per row of k elements (all binary32 unless stated):
//   r      = x + residual                  (or x when there is no residual)
//   inv    = RN32(1 / sqrt(sum r^2 / k + eps))   (the sum, the mean, the root
//            and the division in binary64, rounded once)
//   y      = (r * inv) * w
//   scale  = max(max |y|, 1e-12) / qmax    qmax 127 (INT8) or 448 (FP8 e4m3fn)
//   code   = rint(y / scale)  or  e4m3fn(y / scale)   (exact quotient)
//   residual_out = r rounded to the type of x.
// The norm works on the unrounded r; only what is stored is rounded.
//
// Why binary64 for one sum: every other step is one IEEE operation, so codes
// and scales are reproducible bit for bit as long as inv is; a binary32 sum of
// squares would change its last bits with the order of addition.  It costs a
// conversion and a fused multiply-add per element, below the memory time.
//
// A row whose sum of squares or whose max |y| is not finite (an infinity or a
// NaN among x, residual or w) gets that maximum's non-finite scale and codes
// 0, so whatever the codes are multiplied into is NaN and not silently wrong.
//
// What bounds it: HBM, 2 reads and 1 write of the row's type plus the codes
// (7 bytes per bf16 element).  A row's values stay in registers between the
// two reductions, so x and the residual are read once.  bf16 with a residual:
// 8192 rows of 8192 in 72 us (6.5 TB/s), 2048 of 4096 in 11 us (5.3 TB/s); 8
// rows of 4096 in 6 us, which is the launch and one row's chain of a load and
// two reductions.
#include <algorithm>

#include "quant_math.h"

namespace qk {
namespace {

using qm::Elem;

constexpr int kBlock = 256;
constexpr int kMaxUnits = 8;  // units of P elements held per thread

// Calls that read more than this pass the caches by.  What they read was
// written too long ago to be in the 256 MB last-level cache, and filling that
// cache costs.  Rows of 8192 bf16 elements with a residual, through the
// caches / past them: 2048 rows (67 MB read) 19.3 / 23.5 us, 4096 (134 MB)
// 40.1 / 40.5, 6144 (201 MB) 56.7 / 56.5, 8192 80.9 / 73.4, 16384 159 / 140.
// The stored sum goes past them at every size: the next to read it is a whole
// layer half away (512 rows 8.4 -> 7.6 us, 6144 rows 63.9 -> 56.7).
constexpr double kReadOnceBytes = 160e6;

// 16 bytes at any alignment the element type allows (rows of odd widths)
template <int ALIGN>
struct __attribute__((packed, aligned(ALIGN))) Raw16 {
  uint32_t w[4];
};
template <int ALIGN>
struct __attribute__((packed, aligned(ALIGN))) Raw8 {
  uint32_t w[2];
};
struct __attribute__((packed, aligned(1))) Raw4 {
  uint32_t w;
};

template <int DT>
__device__ __forceinline__ void load_full(const void* row, int u, float (&v)[Elem<DT>::kPerUnit]) {
  using E = Elem<DT>;
  const auto raw = *reinterpret_cast<const Raw16<E::kBytes>*>(static_cast<const char*>(row) +
                                                              static_cast<size_t>(u) * 16);
  E::unpack(make_uint4(raw.w[0], raw.w[1], raw.w[2], raw.w[3]), v);
}

// The P values of unit u of a row of k elements; those past the row's end are 0.
template <int DT>
__device__ __forceinline__ void load_values(const void* row, int k, int u,
                                            float (&v)[Elem<DT>::kPerUnit]) {
  constexpr int P = Elem<DT>::kPerUnit;
  if ((u + 1) * P <= k) {
    load_full<DT>(row, u, v);
  } else {
#pragma unroll
    for (int e = 0; e < P; ++e) v[e] = u * P + e < k ? Elem<DT>::load(row, u * P + e) : 0.0f;
  }
}

// The same for the weight, which is of the row's type or binary32.
template <int DT>
__device__ __forceinline__ void load_weight(const void* w, bool w_f32, int k, int u,
                                            float (&v)[Elem<DT>::kPerUnit]) {
  constexpr int P = Elem<DT>::kPerUnit;
  if (DT == QK_F32 || !w_f32) {
    load_values<DT>(w, k, u, v);
  } else {
    float a[4];
#pragma unroll
    for (int h = 0; h < P / 4; ++h) {
      load_values<QK_F32>(w, k, u * (P / 4) + h, a);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[h * 4 + e] = a[e];
    }
  }
}

template <int DT>
__device__ __forceinline__ uint32_t narrow_bits(float v) {
  if constexpr (DT == QK_F32) return __float_as_uint(v);
  if constexpr (DT == QK_BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  return __builtin_bit_cast(uint16_t, static_cast<_Float16>(qm::rounded_f32(v)));
}

template <int DT>
__device__ __forceinline__ void store_values(void* row, int k, int u,
                                             const float (&v)[Elem<DT>::kPerUnit]) {
  using E = Elem<DT>;
  constexpr int P = E::kPerUnit;
  if ((u + 1) * P <= k) {
    Raw16<E::kBytes> raw;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == QK_F32)
        raw.w[i] = narrow_bits<DT>(v[i]);
      else
        raw.w[i] = qm::pack2_narrow<DT>(v[2 * i], v[2 * i + 1]);
    }
    *reinterpret_cast<Raw16<E::kBytes>*>(static_cast<char*>(row) + static_cast<size_t>(u) * 16) = raw;
  } else {
    for (int e = 0; u * P + e < k; ++e) {
      if constexpr (DT == QK_F32)
        static_cast<uint32_t*>(row)[u * P + e] = narrow_bits<DT>(v[e]);
      else
        static_cast<uint16_t*>(row)[u * P + e] = static_cast<uint16_t>(narrow_bits<DT>(v[e]));
    }
  }
}

// Four codes of values in units of the scale, packed little-endian.
template <bool FP8>
__device__ __forceinline__ uint32_t codes4(const float* y, float s, float r) {
  if constexpr (FP8) {
    return qm::pack4_fp8(qm::fp8_ratio_own(y[0], s, r), qm::fp8_ratio_own(y[1], s, r),
                         qm::fp8_ratio_own(y[2], s, r), qm::fp8_ratio_own(y[3], s, r));
  } else {
    return qm::pack4_low_bytes(qm::code_word_dynamic(y[0], s, r), qm::code_word_dynamic(y[1], s, r),
                               qm::code_word_dynamic(y[2], s, r), qm::code_word_dynamic(y[3], s, r));
  }
}

template <int DT, bool FP8>
__device__ __forceinline__ void store_row_codes(uint8_t* qrow, int k, int u, bool finite,
                                                const float (&y)[Elem<DT>::kPerUnit], float s, float r) {
  constexpr int P = Elem<DT>::kPerUnit;
  uint32_t w[P / 4];
#pragma unroll
  for (int i = 0; i < P / 4; ++i) w[i] = finite ? codes4<FP8>(y + 4 * i, s, r) : 0u;
  if ((u + 1) * P <= k) {
    if constexpr (P == 8)
      *reinterpret_cast<Raw8<1>*>(qrow + static_cast<size_t>(u) * P) = Raw8<1>{{w[0], w[1]}};
    else
      *reinterpret_cast<Raw4*>(qrow + static_cast<size_t>(u) * P) = Raw4{w[0]};
  } else {
    for (int e = 0; u * P + e < k; ++e)
      qrow[u * P + e] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
  }
}

struct NormParams {
  int k;
  const void* x;
  int64_t ldx;  // row strides in elements
  const void* residual;
  int64_t ldr;
  const void* weight;
  int w_f32;
  double eps;
  void* r_out;
  int64_t ldo;
  uint8_t* q;
  float* scale;
  int once;  // x and residual are read past the caches
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Sum over the row's threads: one wave, or four through LDS.
template <int THREADS>
__device__ __forceinline__ double row_sum(double v) {
  v = wave_sum(v);
  if constexpr (THREADS > 64) {
    __shared__ double part[THREADS / 64];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) v += part[w];
  }
  return v;
}
// Max of |y| as bit patterns: NaN orders above infinity, so it is kept.
template <int THREADS>
__device__ __forceinline__ float row_max_abs(float v) {
  if constexpr (THREADS > 64)
    return qm::block_max<THREADS>(v);
  else
    return qm::wave_max_nonneg(v);
}

__device__ __forceinline__ float max_abs_bits(float top, float y) {
  return __uint_as_float(qm::max_u32(__float_as_uint(top), __float_as_uint(y) & 0x7fffffffu));
}

__device__ __forceinline__ float inverse_rms(double sum, int k, double eps) {
  return static_cast<float>(1.0 / sqrt(sum / static_cast<double>(k) + eps));
}

// scale and r = RN(1 / scale) of a row; whether its codes are formed.
template <bool FP8>
__device__ __forceinline__ bool row_scale_of(float top, float& s, float& r) {
  const bool finite = __float_as_uint(top) < 0x7f800000u;
  if constexpr (FP8)
    qm::row_scale_fp8(top, 0.0f, s, r);
  else
    qm::row_scale(top, s, r);
  if (!finite) s = top;
  return finite;
}

// 16 bytes of a row from element `at` on, as they are, and as values.
template <int DT>
__device__ __forceinline__ void raw_load(Raw16<Elem<DT>::kBytes>& r, const void* row, int at) {
  r = *reinterpret_cast<const Raw16<Elem<DT>::kBytes>*>(static_cast<const char*>(row) +
                                                        static_cast<size_t>(at) * Elem<DT>::kBytes);
}
// The same past the caches, and the store past them.
typedef uint32_t words4 __attribute__((ext_vector_type(4)));
typedef words4 words4_16bit __attribute__((aligned(2)));
typedef words4 words4_32bit __attribute__((aligned(4)));
template <int DT>
__device__ __forceinline__ void raw_load_once(Raw16<Elem<DT>::kBytes>& r, const void* row, int at) {
  const char* from = static_cast<const char*>(row) + static_cast<size_t>(at) * Elem<DT>::kBytes;
  words4 w;
  if constexpr (DT == QK_F32)
    w = __builtin_nontemporal_load(reinterpret_cast<const words4_32bit*>(from));
  else
    w = __builtin_nontemporal_load(reinterpret_cast<const words4_16bit*>(from));
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] = w[i];
}
template <int DT>
__device__ __forceinline__ void raw_store_once(void* to, const Raw16<Elem<DT>::kBytes>& r) {
  const words4 w = {r.w[0], r.w[1], r.w[2], r.w[3]};
  if constexpr (DT == QK_F32)
    __builtin_nontemporal_store(w, static_cast<words4_32bit*>(to));
  else
    __builtin_nontemporal_store(w, static_cast<words4_16bit*>(to));
}
template <int DT>
__device__ __forceinline__ void raw_values(const Raw16<Elem<DT>::kBytes>& r, float* v) {
  Elem<DT>::unpack(make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]), v);
}

// A row in registers: THREADS threads (one wave, four rows per workgroup; or
// one workgroup) with UPT units each; k is at least one unit.  Every load is
// unconditional and asked for before the first is used: a thread without a
// unit loads the row's last elements, and a row's last, partial unit is moved
// back to end with the row, so it computes the elements before it a second
// time, with the same results; only the sum leaves them out.  W32: a binary32
// weight beside a 16-bit row.
template <int DT, bool RES, bool FP8, int UPT, int THREADS, bool W32>
__global__ __launch_bounds__(kBlock) void norm_rows(NormParams p, int m) {
  using E = Elem<DT>;
  constexpr int P = E::kPerUnit;
  constexpr int WT = W32 ? QK_F32 : DT, WN = P / Elem<WT>::kPerUnit;
  const int t = THREADS == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t row = THREADS == 64 ? static_cast<int64_t>(blockIdx.x) * (kBlock / 64) + (threadIdx.x >> 6)
                                    : blockIdx.x;
  if (row >= m) return;  // whole waves leave, and only in the variant without barriers
  const int k = p.k, units = (k + P - 1) / P;
  const char* xrow = static_cast<const char*>(p.x) + row * p.ldx * E::kBytes;
  const char* rrow = RES ? static_cast<const char*>(p.residual) + row * p.ldr * E::kBytes : nullptr;

  Raw16<E::kBytes> xr[UPT], rr[UPT];
  Raw16<Elem<WT>::kBytes> wr[UPT][WN];
  int at[UPT];
#pragma unroll
  for (int j = 0; j < UPT; ++j) at[j] = min((t + j * THREADS) * P, k - P);
  if (p.once) {
#pragma unroll
    for (int j = 0; j < UPT; ++j) {
      raw_load_once<DT>(xr[j], xrow, at[j]);
      if constexpr (RES) raw_load_once<DT>(rr[j], rrow, at[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < UPT; ++j) {
      raw_load<DT>(xr[j], xrow, at[j]);
      if constexpr (RES) raw_load<DT>(rr[j], rrow, at[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < UPT; ++j)
#pragma unroll
    for (int h = 0; h < WN; ++h) raw_load<WT>(wr[j][h], p.weight, at[j] + h * (P / WN));

  float v[UPT][P];
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < UPT; ++j) {
    raw_values<DT>(xr[j], v[j]);
    if constexpr (RES) {
      float a[P];
      raw_values<DT>(rr[j], a);
#pragma unroll
      for (int e = 0; e < P; ++e) v[j][e] += a[e];
    }
    const int first = (t + j * THREADS) * P;  // the unit's own elements begin here
    if (first + P <= k) {
#pragma unroll
      for (int e = 0; e < P; ++e) sum = __builtin_fma(static_cast<double>(v[j][e]), static_cast<double>(v[j][e]), sum);
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const double d = at[j] + e >= first ? static_cast<double>(v[j][e]) : 0.0;
        sum = __builtin_fma(d, d, sum);
      }
    }
  }
  const float inv = inverse_rms(row_sum<THREADS>(sum), k, p.eps);

  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < UPT; ++j) {
    if constexpr (RES) {
      if (t + j * THREADS < units) {
        Raw16<E::kBytes> o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (DT == QK_F32)
            o.w[i] = __float_as_uint(v[j][i]);
          else
            o.w[i] = qm::pack2_narrow<DT>(v[j][2 * i], v[j][2 * i + 1]);
        }
        raw_store_once<DT>(static_cast<char*>(p.r_out) + (row * p.ldo + at[j]) * E::kBytes, o);
      }
    }
    float w[P];
#pragma unroll
    for (int h = 0; h < WN; ++h) raw_values<WT>(wr[j][h], w + h * (P / WN));
#pragma unroll
    for (int e = 0; e < P; ++e) {
      v[j][e] = v[j][e] * inv * w[e];
      top = max_abs_bits(top, v[j][e]);
    }
  }
  top = row_max_abs<THREADS>(top);
  float s, r;
  const bool finite = row_scale_of<FP8>(top, s, r);
  if (t == 0) p.scale[row] = s;
#pragma unroll
  for (int j = 0; j < UPT; ++j) {
    if (t + j * THREADS >= units) continue;
    uint32_t c[P / 4];
#pragma unroll
    for (int i = 0; i < P / 4; ++i) c[i] = finite ? codes4<FP8>(v[j] + 4 * i, s, r) : 0u;
    uint8_t* const q = p.q + row * static_cast<int64_t>(k) + at[j];
    if constexpr (P == 8)
      *reinterpret_cast<Raw8<1>*>(q) = Raw8<1>{{c[0], c[1]}};
    else
      *reinterpret_cast<Raw4*>(q) = Raw4{c[0]};
  }
}

// Rows longer than the registers hold, or shorter than a unit: three passes.  The
// residual's sum is stored in the last one, by the thread that read it in
// every pass, so it may replace the residual or x in place.
template <int DT, bool RES, bool FP8>
__global__ __launch_bounds__(kBlock) void norm_rows_long(NormParams p) {
  using E = Elem<DT>;
  constexpr int P = E::kPerUnit;
  const int64_t row = blockIdx.x;
  const int k = p.k, units = (k + P - 1) / P;
  const char* xrow = static_cast<const char*>(p.x) + row * p.ldx * E::kBytes;
  const char* rrow = RES ? static_cast<const char*>(p.residual) + row * p.ldr * E::kBytes : nullptr;
  auto values = [&](int u, float(&v)[P]) {
    load_values<DT>(xrow, k, u, v);
    if constexpr (RES) {
      float a[P];
      load_values<DT>(rrow, k, u, a);
#pragma unroll
      for (int e = 0; e < P; ++e) v[e] += a[e];
    }
  };
  double sum = 0.0;
  for (int u = threadIdx.x; u < units; u += kBlock) {
    float v[P];
    values(u, v);
#pragma unroll
    for (int e = 0; e < P; ++e) sum = __builtin_fma(static_cast<double>(v[e]), static_cast<double>(v[e]), sum);
  }
  const float inv = inverse_rms(row_sum<kBlock>(sum), k, p.eps);
  float top = 0.0f;
  for (int u = threadIdx.x; u < units; u += kBlock) {
    float v[P], w[P];
    values(u, v);
    load_weight<DT>(p.weight, p.w_f32, k, u, w);
#pragma unroll
    for (int e = 0; e < P; ++e)
      if (u * P + e < k) top = max_abs_bits(top, v[e] * inv * w[e]);
  }
  top = row_max_abs<kBlock>(top);
  float s, r;
  const bool finite = row_scale_of<FP8>(top, s, r);
  if (threadIdx.x == 0) p.scale[row] = s;
  for (int u = threadIdx.x; u < units; u += kBlock) {
    float v[P], w[P];
    values(u, v);
    if constexpr (RES) store_values<DT>(static_cast<char*>(p.r_out) + row * p.ldo * E::kBytes, k, u, v);
    load_weight<DT>(p.weight, p.w_f32, k, u, w);
#pragma unroll
    for (int e = 0; e < P; ++e) v[e] = v[e] * inv * w[e];
    store_row_codes<DT, FP8>(p.q + row * static_cast<int64_t>(k), k, u, finite, v, s, r);
  }
}

template <int DT, bool RES, bool FP8, bool W32>
hipError_t dispatch(int m, const NormParams& p, hipStream_t stream) {
  constexpr int P = Elem<DT>::kPerUnit;
  const int units = p.k / P + (p.k % P != 0);
  const dim3 block(kBlock), rows(static_cast<unsigned>(m)), quads((static_cast<unsigned>(m) + 3) / 4);
  if (p.k < P || units > kBlock * kMaxUnits)
    return launch(norm_rows_long<DT, RES, FP8>, rows, block, 0, stream, p);
  if (units <= 64) return launch(norm_rows<DT, RES, FP8, 1, 64, W32>, quads, block, 0, stream, p, m);
  if (units <= 128) return launch(norm_rows<DT, RES, FP8, 2, 64, W32>, quads, block, 0, stream, p, m);
  if (units <= kBlock) return launch(norm_rows<DT, RES, FP8, 1, kBlock, W32>, rows, block, 0, stream, p, m);
  if (units <= kBlock * 2) return launch(norm_rows<DT, RES, FP8, 2, kBlock, W32>, rows, block, 0, stream, p, m);
  if (units <= kBlock * 4) return launch(norm_rows<DT, RES, FP8, 4, kBlock, W32>, rows, block, 0, stream, p, m);
  return launch(norm_rows<DT, RES, FP8, kMaxUnits, kBlock, W32>, rows, block, 0, stream, p, m);
}

template <int DT, bool RES, bool FP8>
hipError_t dispatch_weight(int m, const NormParams& p, hipStream_t stream) {
  if constexpr (DT != QK_F32)
    if (p.w_f32) return dispatch<DT, RES, FP8, true>(m, p, stream);
  return dispatch<DT, RES, FP8, false>(m, p, stream);
}

template <int DT>
hipError_t dispatch_dtype(const RmsNormQuantArgs& a, hipStream_t stream) {
  const double read = static_cast<double>(a.m) * a.k * Elem<DT>::kBytes * (a.residual ? 2 : 1);
  const NormParams p{a.k,     a.x,      a.ldx, a.residual, a.ldr,   a.weight,            a.weight_f32,
                     a.eps,   a.r_out,  a.ldo, a.q,        a.scale, read > kReadOnceBytes};
  if (a.residual)
    return a.fp8 ? dispatch_weight<DT, true, true>(a.m, p, stream) : dispatch_weight<DT, true, false>(a.m, p, stream);
  return a.fp8 ? dispatch_weight<DT, false, true>(a.m, p, stream) : dispatch_weight<DT, false, false>(a.m, p, stream);
}

}  // namespace

// More rows than a grid of one workgroup each may have go in several launches.
hipError_t launch_rms_norm_quant(const RmsNormQuantArgs& a, hipStream_t stream) {
  constexpr int kRows = 1 << 23;
  static_assert(kRows <= 0xffffffffll / kBlock, "a launch's work items fit in 32 bits");
  const int64_t bytes = a.dtype == QK_F32 ? 4 : 2;
  for (int64_t row = 0; row < a.m; row += kRows) {
    RmsNormQuantArgs s = a;
    s.m = static_cast<int>(std::min<int64_t>(a.m - row, kRows));
    s.x = static_cast<const char*>(a.x) + row * a.ldx * bytes;
    if (a.residual) {
      s.residual = static_cast<const char*>(a.residual) + row * a.ldr * bytes;
      s.r_out = static_cast<char*>(a.r_out) + row * a.ldo * bytes;
    }
    s.q = a.q + row * a.k;
    s.scale = a.scale + row;
    const hipError_t e = a.dtype == QK_F32    ? dispatch_dtype<QK_F32>(s, stream)
                         : a.dtype == QK_BF16 ? dispatch_dtype<QK_BF16>(s, stream)
                                              : dispatch_dtype<QK_F16>(s, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qk
