// C ABI of libqk: argument validation, kernel choice by shape, launches on the
// caller's stream.  Declarations and the contract of each call are in qk.h.
#include <cstdint>
#include <mutex>

#include "mx4_rule.h"
#include "qk_internal.h"

#define QK_STR2(x) #x
#define QK_STR(x) QK_STR2(x)

namespace qk {
namespace {

// 16 bytes per lane, grid-stride; the last (bytes % 16) bytes one per thread
// of the first workgroup.
__global__ __launch_bounds__(256) void zero_fill_kernel(uint4* __restrict__ p, size_t n16,
                                                        unsigned char* __restrict__ tail,
                                                        unsigned ntail) {
  const size_t stride = static_cast<size_t>(gridDim.x) * 256;
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < n16; i += stride)
    p[i] = make_uint4(0, 0, 0, 0);
  if (blockIdx.x == 0 && threadIdx.x < ntail) tail[threadIdx.x] = 0;
}

}  // namespace

hipError_t launch_zero_fill(void* p, size_t bytes, hipStream_t stream) {
  if (bytes == 0) return hipSuccess;
  const size_t n16 = bytes / 16;
  const unsigned ntail = static_cast<unsigned>(bytes % 16);
  const size_t want = (n16 + 255) / 256;
  const unsigned blocks = static_cast<unsigned>(want == 0 ? 1 : (want < 4096 ? want : 4096));
  return launch(zero_fill_kernel, dim3(blocks), dim3(256), 0, stream, static_cast<uint4*>(p), n16,
                static_cast<unsigned char*>(p) + n16 * 16, ntail);
}

}  // namespace qk

namespace {

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool known_input_dtype(int dt) { return dt == QK_F32 || dt == QK_BF16 || dt == QK_F16; }

int status_of(hipError_t e) { return e == hipSuccess ? QK_OK : static_cast<int>(e); }

bool workspace_ok(const void* ws, size_t bytes, int n) {
  return ws && aligned(ws, 256) && bytes >= qk::gemv_workspace_bytes(n);
}

int check_rows(int m, int k, const void* src, const void* q, const void* scale, int dtype) {
  if (m < 0 || k < 0) return QK_ERR_INVALID_VALUE;
  if (!known_input_dtype(dtype)) return QK_ERR_INVALID_VALUE;
  if (m > 0 && (!scale || (k > 0 && (!src || !q)))) return QK_ERR_INVALID_VALUE;
  return QK_OK;
}

int gemm_common(int m, int n, int k, const int8_t* a, const int8_t* b, int32_t* c,
                const float* scale_a, const float* scale_b, float output_scale, void* out,
                int out_dtype, int b_layout, void* workspace, size_t workspace_bytes, int kernel,
                hipStream_t stream) {
  if (m < 0 || n < 0 || k < 0 || k > QK_MAX_K) return QK_ERR_INVALID_VALUE;
  if (b_layout != QK_B_KN && b_layout != QK_B_NK) return QK_ERR_INVALID_VALUE;
  if (kernel != QK_KERNEL_AUTO && kernel != QK_KERNEL_MFMA && kernel != QK_KERNEL_GEMV)
    return QK_ERR_INVALID_VALUE;
  if (k % 16 != 0) return QK_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return QK_OK;  // empty tensors may have NULL data pointers
  if (!c && !out) return QK_ERR_INVALID_VALUE;
  if (out && out_dtype != QK_F32 && out_dtype != QK_BF16) return QK_ERR_INVALID_VALUE;
  if (k > 0 && (!a || !b)) return QK_ERR_INVALID_VALUE;
  if (out && (!scale_a || !scale_b)) return QK_ERR_INVALID_VALUE;
  if (!aligned(a, 16) || !aligned(b, 16)) return QK_ERR_UNSUPPORTED;
  if (c && !aligned(c, 4)) return QK_ERR_UNSUPPORTED;
  if (out && !aligned(out, out_dtype == QK_BF16 ? 2 : 4)) return QK_ERR_UNSUPPORTED;

  bool gemv;
  if (kernel == QK_KERNEL_GEMV) {
    if (m > qk::kGemvMaxM || b_layout != QK_B_KN) return QK_ERR_UNSUPPORTED;
    gemv = true;
  } else if (kernel == QK_KERNEL_MFMA) {
    gemv = false;
  } else {
    gemv = m <= qk::kGemvMaxRows && b_layout == QK_B_KN;
  }
  if (gemv) {
    if (!workspace_ok(workspace, workspace_bytes, n)) return QK_ERR_WORKSPACE;
    qk::GemvArgs g{m, n, k, a, -1, b, c, scale_a, scale_b, output_scale, out, out_dtype, nullptr,
                   nullptr, workspace};
    return status_of(qk::launch_gemv(g, stream));
  }
  if (!qk::gemm_mfma_supported(m, n, k)) return QK_ERR_UNSUPPORTED;
  // the workspace, when given, lets an output with few tiles split k
  const bool ws = workspace && aligned(workspace, 256);
  qk::GemmArgs g{m, n, k, a, b, c, scale_a, scale_b, output_scale, out, out_dtype, b_layout,
                 ws ? workspace : nullptr, ws ? workspace_bytes : 0};
  return status_of(qk::launch_gemm_mfma(g, stream));
}

// Host checks of the whole-layer call (both entry points).  On QK_OK, *noop
// tells that there is nothing to do (m or n is 0) and *fused which path runs:
// the single decode launch or quantization + tiled GEMM.
int linear_check(int m, int n, int k, const void* x, int x_dtype, const int8_t* b,
                 const float* scale_b, const void* out, int out_dtype, int b_layout,
                 const int8_t* q_out, const float* scale_out, const int32_t* c_out, int kernel,
                 bool* fused, bool* noop) {
  if (m < 0 || n < 0 || k < 0 || k > QK_MAX_K) return QK_ERR_INVALID_VALUE;
  if (!known_input_dtype(x_dtype)) return QK_ERR_INVALID_VALUE;
  if (b_layout != QK_B_KN && b_layout != QK_B_NK) return QK_ERR_INVALID_VALUE;
  if (kernel != QK_KERNEL_AUTO && kernel != QK_KERNEL_MFMA && kernel != QK_KERNEL_GEMV)
    return QK_ERR_INVALID_VALUE;
  if (out && out_dtype != QK_F32 && out_dtype != QK_BF16) return QK_ERR_INVALID_VALUE;
  if (k % 16 != 0) return QK_ERR_UNSUPPORTED;
  *noop = m == 0 || n == 0;
  if (*noop) return QK_OK;
  if (!out && !c_out) return QK_ERR_INVALID_VALUE;
  if ((out && !scale_b) || (k > 0 && (!x || !b))) return QK_ERR_INVALID_VALUE;
  if (!aligned(b, 16) || !aligned(x, x_dtype == QK_F32 ? 4 : 2)) return QK_ERR_UNSUPPORTED;
  if (out && !aligned(out, out_dtype == QK_BF16 ? 2 : 4)) return QK_ERR_UNSUPPORTED;
  if (c_out && !aligned(c_out, 4)) return QK_ERR_UNSUPPORTED;
  if (q_out && !aligned(q_out, 16)) return QK_ERR_UNSUPPORTED;
  if (scale_out && !aligned(scale_out, 4)) return QK_ERR_UNSUPPORTED;

  if (kernel == QK_KERNEL_GEMV) {
    if (m > qk::kGemvMaxM || b_layout != QK_B_KN) return QK_ERR_UNSUPPORTED;
    *fused = true;
  } else if (kernel == QK_KERNEL_MFMA) {
    *fused = false;
  } else {
    *fused = m <= qk::kGemvMaxRows && b_layout == QK_B_KN;
  }
  if (*fused && !aligned(x, 16)) {
    if (kernel == QK_KERNEL_GEMV) return QK_ERR_UNSUPPORTED;
    *fused = false;  // the fused launch reads x with 128-bit loads
  }
  if (!*fused) {
    // two launches: the codes and scales go through q_out / scale_out
    if (!q_out || !scale_out) return QK_ERR_INVALID_VALUE;
    if (!qk::gemm_mfma_supported(m, n, k)) return QK_ERR_UNSUPPORTED;
  }
  return QK_OK;
}

// Enqueues a checked whole-layer call; the workspace (valid and large enough
// for the decode launch when `fused`) lets the tiled GEMM split k when its
// partial sums fit.
int linear_launch(int m, int n, int k, const void* x, int x_dtype, const int8_t* b,
                  const float* scale_b, float output_scale, void* out, int out_dtype,
                  int b_layout, int8_t* q_out, float* scale_out, int32_t* c_out, bool fused,
                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (fused) {
    qk::GemvArgs g{m, n, k, x, x_dtype, b, c_out, nullptr, scale_b, output_scale, out,
                   out_dtype, q_out, scale_out, workspace};
    return status_of(qk::launch_gemv(g, stream));
  }
  hipError_t e = qk::launch_quant_rows(m, k, x, x_dtype, q_out, scale_out, stream);
  if (e != hipSuccess) return status_of(e);
  const bool ws = workspace && aligned(workspace, 256);
  qk::GemmArgs g{m, n, k, q_out, b, c_out, scale_out, scale_b, output_scale, out, out_dtype,
                 b_layout, ws ? workspace : nullptr, ws ? workspace_bytes : 0};
  return status_of(qk::launch_gemm_mfma(g, stream));
}

// ---- static scratch of qk_linear_w8a8_noalloc ----
// The memory the no-allocation entry point uses in place of a caller's
// workspace: a file-scope device array, one copy per GPU, held until the
// process ends.  Its name is a host-side stand-in in host code, so the device
// address is looked up once per device (hipGetSymbolAddress, with that device
// current) and only that address is ever passed to kernels.  The first call
// on a device, and the first call after a failed launch, clear it on the
// caller's stream before using it (a kernel, so that a captured call stays
// valid); every successful call leaves it all zeros again.
constexpr size_t kScratchBytes = QK_SCRATCH_BYTES;
static __device__ __align__(256) unsigned char scratch[kScratchBytes];

constexpr int kMaxDevices = 64;
struct ScratchSlot {
  void* ptr = nullptr;    // device address of `scratch` on this device
  bool needs_clear = true;
};
std::mutex g_scratch_mutex;
ScratchSlot g_scratch[kMaxDevices];

hipError_t scratch_for_call(hipStream_t stream, int* dev, void** ptr) {
  hipError_t e = hipGetDevice(dev);
  if (e != hipSuccess) return e;
  if (*dev < 0 || *dev >= kMaxDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mutex);
  ScratchSlot& slot = g_scratch[*dev];
  if (!slot.ptr) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return e;
    slot.ptr = p;
  }
  if (slot.needs_clear) {
    e = qk::launch_zero_fill(slot.ptr, kScratchBytes, stream);
    if (e != hipSuccess) return e;
    slot.needs_clear = false;
  }
  *ptr = slot.ptr;
  return hipSuccess;
}

void scratch_mark_dirty(int dev) {
  std::lock_guard<std::mutex> lock(g_scratch_mutex);
  g_scratch[dev].needs_clear = true;
}

}  // namespace

extern "C" {

int qk_abi_version(void) { return QK_ABI_VERSION; }

const char* qk_status_string(int status) {
  switch (status) {
    case QK_OK: return "QK_OK: success";
    case QK_ERR_INVALID_VALUE:
      return "QK_ERR_INVALID_VALUE: negative size, NULL pointer, or unknown dtype/layout/kernel";
    case QK_ERR_UNSUPPORTED:
      return "QK_ERR_UNSUPPORTED: k not a multiple of 16, misaligned pointer, or kernel/shape "
             "combination not provided";
    case QK_ERR_WORKSPACE:
      return "QK_ERR_WORKSPACE: workspace missing, misaligned, or smaller than "
             "qk_gemm_workspace_size()";
    case QK_ERR_SCRATCH_LIMIT:
      return "QK_ERR_SCRATCH_LIMIT: the call needs more than the QK_SCRATCH_BYTES of static "
             "scratch that qk_linear_w8a8_noalloc uses (the decode launch needs 64 bytes per "
             "output column)";
    default: return hipGetErrorString(static_cast<hipError_t>(status));
  }
}

const char* qk_build_info(void) {
  return "libqk ABI " QK_STR(QK_ABI_VERSION) "; code objects: gfx950; HIP " QK_STR(
      HIP_VERSION_MAJOR) "." QK_STR(HIP_VERSION_MINOR) "." QK_STR(HIP_VERSION_PATCH) "; built " __DATE__
                                                                                       " " __TIME__;
}

int qk_quant_per_token(int m, int k, const void* x, int x_dtype, int8_t* q, float* scale,
                       hipStream_t stream) {
  const int rc = check_rows(m, k, x, q, scale, x_dtype);
  if (rc != QK_OK || m == 0) return rc;
  return status_of(qk::launch_quant_rows(m, k, x, x_dtype, q, scale, stream));
}

int qk_silu_mul_quant_per_token(int m, int d, const void* h, int h_dtype, int8_t* q,
                                float* scale, hipStream_t stream) {
  const int rc = check_rows(m, d, h, q, scale, h_dtype);
  if (rc != QK_OK || m == 0) return rc;
  if (static_cast<long long>(d) * 2 > 0x7fffffffLL) return QK_ERR_UNSUPPORTED;
  return status_of(qk::launch_silu_quant_rows(m, d, h, h_dtype, q, scale, stream));
}

int qk_silu_mul(int m, int d, const void* h, int h_dtype, float* out, hipStream_t stream) {
  if (m < 0 || d < 0 || !known_input_dtype(h_dtype)) return QK_ERR_INVALID_VALUE;
  if (m == 0 || d == 0) return QK_OK;  // empty tensors may have NULL data pointers
  if (!h || !out) return QK_ERR_INVALID_VALUE;
  if (static_cast<long long>(d) * 2 > 0x7fffffffLL) return QK_ERR_UNSUPPORTED;
  return status_of(qk::launch_silu_mul(m, d, h, h_dtype, out, stream));
}

size_t qk_gemm_workspace_size(int m, int n, int k) {
  if (m <= 0 || n <= 0 || k < 0) return 0;
  // the decode kernel's words (m <= 16), and the tiled kernel's split-K
  // partial sums when the output has few tiles (the plan is the same for
  // either weight layout)
  const size_t gemv = m <= qk::kGemvMaxM ? qk::gemv_workspace_bytes(n) : 0;
  const size_t split = qk::splitk_plan(m, n, k, QK_B_KN).bytes;
  return gemv > split ? gemv : split;
}

int qk_workspace_init(void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (workspace_bytes == 0) return QK_OK;
  if (!workspace) return QK_ERR_INVALID_VALUE;
  if (!aligned(workspace, 256)) return QK_ERR_WORKSPACE;
  return status_of(qk::launch_zero_fill(workspace, workspace_bytes, stream));
}

int qk_gemm_i8_scaled(int m, int n, int k, const int8_t* a, const int8_t* b, int32_t* c,
                      const float* scale_a, const float* scale_b, float output_scale, void* out,
                      int out_dtype, int b_layout, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
  return gemm_common(m, n, k, a, b, c, scale_a, scale_b, output_scale, out, out_dtype, b_layout,
                     workspace, workspace_bytes, QK_KERNEL_AUTO, stream);
}

int qk_gemm_i8_scaled_ex(int m, int n, int k, const int8_t* a, const int8_t* b, int32_t* c,
                         const float* scale_a, const float* scale_b, float output_scale,
                         void* out, int out_dtype, int b_layout, void* workspace,
                         size_t workspace_bytes, int kernel, hipStream_t stream) {
  return gemm_common(m, n, k, a, b, c, scale_a, scale_b, output_scale, out, out_dtype, b_layout,
                     workspace, workspace_bytes, kernel, stream);
}

int qk_linear_w8a8(int m, int n, int k, const void* x, int x_dtype, const int8_t* b,
                   const float* scale_b, float output_scale, void* out, int out_dtype,
                   int b_layout, int8_t* q_out, float* scale_out, int32_t* c_out,
                   void* workspace, size_t workspace_bytes, int kernel, hipStream_t stream) {
  bool fused = false, noop = false;
  const int rc = linear_check(m, n, k, x, x_dtype, b, scale_b, out, out_dtype, b_layout, q_out,
                              scale_out, c_out, kernel, &fused, &noop);
  if (rc != QK_OK || noop) return rc;
  if (fused && !workspace_ok(workspace, workspace_bytes, n)) return QK_ERR_WORKSPACE;
  return linear_launch(m, n, k, x, x_dtype, b, scale_b, output_scale, out, out_dtype, b_layout,
                       q_out, scale_out, c_out, fused, workspace, workspace_bytes, stream);
}

int qk_linear_w8a8_noalloc(int m, int n, int k, const void* x, int x_dtype, const int8_t* b,
                           const float* scale_b, float output_scale, void* out, int out_dtype,
                           int b_layout, int8_t* q_out, float* scale_out, int32_t* c_out,
                           int kernel, hipStream_t stream) {
  bool fused = false, noop = false;
  const int rc = linear_check(m, n, k, x, x_dtype, b, scale_b, out, out_dtype, b_layout, q_out,
                              scale_out, c_out, kernel, &fused, &noop);
  if (rc != QK_OK || noop) return rc;
  // the decode launch needs its words; the tiled GEMM splits k only when its
  // partial sums fit, and otherwise runs unsplit
  if (fused && qk::gemv_workspace_bytes(n) > kScratchBytes) return QK_ERR_SCRATCH_LIMIT;
  int dev = 0;
  void* ptr = nullptr;
  hipError_t e = scratch_for_call(stream, &dev, &ptr);
  if (e != hipSuccess) return status_of(e);
  const int st = linear_launch(m, n, k, x, x_dtype, b, scale_b, output_scale, out, out_dtype,
                               b_layout, q_out, scale_out, c_out, fused, ptr, kScratchBytes, stream);
  if (st != QK_OK) scratch_mark_dirty(dev);  // a launch failed after others may have run
  return st;
}

int qk_quant_per_token_fp8(int m, int k, const void* x, int x_dtype, float scale_ub, uint8_t* q,
                           float* scale, hipStream_t stream) {
  const int rc = check_rows(m, k, x, q, scale, x_dtype);
  if (rc != QK_OK) return rc;
  if (scale_ub != scale_ub) return QK_ERR_INVALID_VALUE;  // NaN bound
  if (m == 0) return QK_OK;
  return status_of(qk::launch_quant_rows_fp8(m, k, x, x_dtype, q, scale, scale_ub, stream));
}

int qk_silu_mul_quant_per_token_fp8(int m, int d, const void* h, int h_dtype, float scale_ub,
                                    uint8_t* q, float* scale, hipStream_t stream) {
  const int rc = check_rows(m, d, h, q, scale, h_dtype);
  if (rc != QK_OK) return rc;
  if (scale_ub != scale_ub) return QK_ERR_INVALID_VALUE;
  if (m == 0) return QK_OK;
  if (static_cast<long long>(d) * 2 > 0x7fffffffLL) return QK_ERR_UNSUPPORTED;
  return status_of(qk::launch_silu_quant_rows_fp8(m, d, h, h_dtype, q, scale, scale_ub, stream));
}

int qk_gemm_fp8_scaled(int m, int n, int k, const uint8_t* a, const uint8_t* b, float* c,
                       const float* scale_a, const float* scale_b, float output_scale, void* out,
                       int out_dtype, int b_layout, hipStream_t stream) {
  if (m < 0 || n < 0 || k < 0 || k > QK_MAX_K) return QK_ERR_INVALID_VALUE;
  if (b_layout != QK_B_KN && b_layout != QK_B_NK) return QK_ERR_INVALID_VALUE;
  if (k % 16 != 0) return QK_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return QK_OK;
  if (!c && !out) return QK_ERR_INVALID_VALUE;
  if (out && out_dtype != QK_F32 && out_dtype != QK_BF16) return QK_ERR_INVALID_VALUE;
  if (k > 0 && (!a || !b)) return QK_ERR_INVALID_VALUE;
  if (out && (!scale_a || !scale_b)) return QK_ERR_INVALID_VALUE;
  if (!aligned(a, 16) || !aligned(b, 16)) return QK_ERR_UNSUPPORTED;
  if (c && !aligned(c, 4)) return QK_ERR_UNSUPPORTED;
  if (out && !aligned(out, out_dtype == QK_BF16 ? 2 : 4)) return QK_ERR_UNSUPPORTED;
  if (!qk::gemm_mfma_supported(m, n, k)) return QK_ERR_UNSUPPORTED;
  qk::SliceGemmArgs g{m, n, k, reinterpret_cast<const int8_t*>(a), reinterpret_cast<const int8_t*>(b),
                      c, scale_a, scale_b, output_scale, out, out_dtype, b_layout};
  return status_of(qk::launch_gemm_fp8(g, stream));
}

int qk_linear_fp8(int m, int n, int k, const void* x, int x_dtype, float scale_ub,
                  const uint8_t* b, const float* scale_b, float output_scale, void* out,
                  int out_dtype, int b_layout, uint8_t* q_out, float* scale_out,
                  hipStream_t stream) {
  if (m < 0 || n < 0 || k < 0 || k > QK_MAX_K) return QK_ERR_INVALID_VALUE;
  if (!known_input_dtype(x_dtype)) return QK_ERR_INVALID_VALUE;
  if (b_layout != QK_B_KN && b_layout != QK_B_NK) return QK_ERR_INVALID_VALUE;
  if (out_dtype != QK_F32 && out_dtype != QK_BF16) return QK_ERR_INVALID_VALUE;
  if (scale_ub != scale_ub) return QK_ERR_INVALID_VALUE;
  if (k % 16 != 0) return QK_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return QK_OK;
  if (!out || !scale_b || !q_out || !scale_out || (k > 0 && (!x || !b)))
    return QK_ERR_INVALID_VALUE;
  if (!aligned(b, 16) || !aligned(q_out, 16) || !aligned(scale_out, 4)) return QK_ERR_UNSUPPORTED;
  if (!aligned(x, x_dtype == QK_F32 ? 4 : 2)) return QK_ERR_UNSUPPORTED;
  if (!aligned(out, out_dtype == QK_BF16 ? 2 : 4)) return QK_ERR_UNSUPPORTED;
  if (!qk::gemm_mfma_supported(m, n, k)) return QK_ERR_UNSUPPORTED;
  hipError_t e = qk::launch_quant_rows_fp8(m, k, x, x_dtype, q_out, scale_out, scale_ub, stream);
  if (e != hipSuccess) return status_of(e);
  qk::SliceGemmArgs g{m, n, k, reinterpret_cast<const int8_t*>(q_out),
                      reinterpret_cast<const int8_t*>(b), nullptr, scale_out, scale_b, output_scale,
                      out, out_dtype, b_layout};
  return status_of(qk::launch_gemm_fp8(g, stream));
}

int qk_gemm_i8_grouped(int m, int n, int k, int group, const int8_t* a, const int8_t* b, float* c,
                       const float* scale_a, const float* scale_b, float output_scale, void* out,
                       int out_dtype, int b_layout, hipStream_t stream) {
  if (m < 0 || n < 0 || k < 0 || k > QK_MAX_K) return QK_ERR_INVALID_VALUE;
  if (b_layout != QK_B_KN && b_layout != QK_B_NK) return QK_ERR_INVALID_VALUE;
  if (group != 64 && group != 128) return QK_ERR_UNSUPPORTED;
  if (k % group != 0) return QK_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return QK_OK;
  if (!c && !out) return QK_ERR_INVALID_VALUE;
  if (out && out_dtype != QK_F32 && out_dtype != QK_BF16) return QK_ERR_INVALID_VALUE;
  if (k > 0 && (!a || !b || !scale_b)) return QK_ERR_INVALID_VALUE;
  if (out && !scale_a) return QK_ERR_INVALID_VALUE;
  if (!aligned(a, 16) || !aligned(b, 16) || (scale_b && !aligned(scale_b, 4)))
    return QK_ERR_UNSUPPORTED;
  if (c && !aligned(c, 4)) return QK_ERR_UNSUPPORTED;
  if (out && !aligned(out, out_dtype == QK_BF16 ? 2 : 4)) return QK_ERR_UNSUPPORTED;
  if (!qk::gemm_mfma_supported(m, n, k)) return QK_ERR_UNSUPPORTED;
  qk::SliceGemmArgs g{m, n, k, a, b, c, scale_a, scale_b, output_scale, out, out_dtype, b_layout};
  return status_of(qk::launch_gemm_i8_grouped(g, group, stream));
}

int qk_moe_gemm_i8_scaled(int experts, int m, int n, int k, const int* expert_offsets,
                          const int8_t* a, const int8_t* b, int32_t* c, const float* scale_a,
                          const float* scale_b, float output_scale, void* out, int out_dtype,
                          int b_layout, hipStream_t stream) {
  if (experts < 1 || experts > qk::moe_max_experts()) return QK_ERR_INVALID_VALUE;
  if (m < 0 || n < 0 || k < 0 || k > QK_MAX_K) return QK_ERR_INVALID_VALUE;
  if (b_layout != QK_B_KN && b_layout != QK_B_NK) return QK_ERR_INVALID_VALUE;
  if (k % 16 != 0) return QK_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return QK_OK;
  if (!expert_offsets || (!c && !out)) return QK_ERR_INVALID_VALUE;
  if (out && out_dtype != QK_F32 && out_dtype != QK_BF16) return QK_ERR_INVALID_VALUE;
  if (k > 0 && (!a || !b)) return QK_ERR_INVALID_VALUE;
  if (out && (!scale_a || !scale_b)) return QK_ERR_INVALID_VALUE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(expert_offsets, 4)) return QK_ERR_UNSUPPORTED;
  if (c && !aligned(c, 4)) return QK_ERR_UNSUPPORTED;
  if (out && !aligned(out, out_dtype == QK_BF16 ? 2 : 4)) return QK_ERR_UNSUPPORTED;
  if (!qk::gemm_mfma_supported(m, n, k)) return QK_ERR_UNSUPPORTED;
  // k % 16 == 0 keeps every expert's weight (k n bytes apart) and every row
  // group's codes 16-byte aligned
  qk::GemmArgs g{m, n, k, a, b, c, scale_a, scale_b, output_scale, out, out_dtype, b_layout,
                 nullptr, 0};
  return status_of(qk::launch_gemm_moe(g, expert_offsets, experts, stream));
}

static int quant_static_common(int m, int k, const void* x, int x_dtype, const float* scale,
                               void* q, bool silu, bool fp8, hipStream_t stream) {
  const int rc = check_rows(m, k, x, q, scale, x_dtype);
  if (rc != QK_OK || m == 0 || k == 0) return rc;
  if (silu && static_cast<long long>(k) * 2 > 0x7fffffffLL) return QK_ERR_UNSUPPORTED;
  return status_of(qk::launch_quant_static(m, k, x, x_dtype, silu, fp8, scale,
                                           static_cast<int8_t*>(q), stream));
}

int qk_quant_static(int m, int k, const void* x, int x_dtype, const float* scale, int8_t* q,
                    hipStream_t stream) {
  return quant_static_common(m, k, x, x_dtype, scale, q, false, false, stream);
}

int qk_silu_mul_quant_static(int m, int d, const void* h, int h_dtype, const float* scale,
                             int8_t* q, hipStream_t stream) {
  return quant_static_common(m, d, h, h_dtype, scale, q, true, false, stream);
}

int qk_quant_static_fp8(int m, int k, const void* x, int x_dtype, const float* scale, uint8_t* q,
                        hipStream_t stream) {
  return quant_static_common(m, k, x, x_dtype, scale, q, false, true, stream);
}

int qk_silu_mul_quant_static_fp8(int m, int d, const void* h, int h_dtype, const float* scale,
                                 uint8_t* q, hipStream_t stream) {
  return quant_static_common(m, d, h, h_dtype, scale, q, true, true, stream);
}

int qk_quant_per_token_asym(int m, int k, const void* x, int x_dtype, int8_t* q, float* scale,
                            int32_t* zero_point, hipStream_t stream) {
  const int rc = check_rows(m, k, x, q, scale, x_dtype);
  if (rc != QK_OK) return rc;
  if (m > 0 && !zero_point) return QK_ERR_INVALID_VALUE;
  if (m == 0) return QK_OK;
  return status_of(qk::launch_quant_rows_asym(m, k, x, x_dtype, q, scale, zero_point, stream));
}

int qk_weight_colsum(int k, int n, const int8_t* b, int b_layout, int32_t* wsum, hipStream_t stream) {
  if (k < 0 || n < 0 || k > QK_MAX_K) return QK_ERR_INVALID_VALUE;
  if (b_layout != QK_B_KN && b_layout != QK_B_NK) return QK_ERR_INVALID_VALUE;
  if (n == 0) return QK_OK;
  if (!wsum || (k > 0 && !b)) return QK_ERR_INVALID_VALUE;
  return status_of(qk::launch_weight_colsum(k, n, b, b_layout, wsum, stream));
}

int qk_gemm_i8_asym(int m, int n, int k, const int8_t* a, const int32_t* zero_point,
                    const int8_t* b, const int32_t* wsum, int32_t* c, const float* scale_a,
                    const float* scale_b, float output_scale, void* out, int out_dtype,
                    int b_layout, hipStream_t stream) {
  if (m < 0 || n < 0 || k < 0 || k > QK_MAX_K_ASYM) return QK_ERR_INVALID_VALUE;
  if (b_layout != QK_B_KN && b_layout != QK_B_NK) return QK_ERR_INVALID_VALUE;
  if (k % 16 != 0) return QK_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return QK_OK;
  if (!c && !out) return QK_ERR_INVALID_VALUE;
  if (!zero_point || !wsum) return QK_ERR_INVALID_VALUE;
  if (out && out_dtype != QK_F32 && out_dtype != QK_BF16) return QK_ERR_INVALID_VALUE;
  if (k > 0 && (!a || !b)) return QK_ERR_INVALID_VALUE;
  if (out && (!scale_a || !scale_b)) return QK_ERR_INVALID_VALUE;
  if (!aligned(a, 16) || !aligned(b, 16)) return QK_ERR_UNSUPPORTED;
  if (c && !aligned(c, 4)) return QK_ERR_UNSUPPORTED;
  if (out && !aligned(out, out_dtype == QK_BF16 ? 2 : 4)) return QK_ERR_UNSUPPORTED;
  if (!qk::gemm_mfma_supported(m, n, k)) return QK_ERR_UNSUPPORTED;
  qk::GemmArgs g{m, n, k, a, b, c, scale_a, scale_b, output_scale, out, out_dtype, b_layout,
                 nullptr, 0};
  return status_of(qk::launch_gemm_asym(g, zero_point, wsum, stream));
}

// Whether some row of `in` (m rows of `row_in` bytes, ld_in bytes apart) overlaps
// a row of `out` (of `row_out` bytes), other than, with `own`, the same row in place.
static bool rows_overlap(const void* in, int64_t ld_in, int64_t row_in, const void* out, int64_t ld_out,
                         int64_t row_out, int64_t m, bool own) {
  const int64_t a = reinterpret_cast<intptr_t>(in), b = reinterpret_cast<intptr_t>(out);
  if (row_in == 0 || row_out == 0 || a + (m - 1) * ld_in + row_in <= b || b + (m - 1) * ld_out + row_out <= a)
    return false;
  if (m == 1) return !own || a != b;
  // row i of `in` overlaps row j of `out` where j lies past its start less
  // row_out and before its end; rows of either do not overlap each other, so with
  // ld_out >= row_out there are few such j
  const int64_t last = ld_in == ld_out ? 1 : m;  // with one stride the distance depends on j - i alone
  for (int64_t i = 0; i < last; ++i) {
    const int64_t from = a + i * ld_in;
    const int64_t near = (from - b) / ld_out - (from < b);
    for (int64_t j = near; j <= near + 1 || b + j * ld_out < from + row_in; ++j) {
      const bool there = ld_in == ld_out ? j > -m && j < m : j >= 0 && j < m;
      const int64_t off = from - (b + j * ld_out);
      if (there && off < row_out && off > -row_in && !(own && off == 0 && i == j)) return true;
    }
  }
  return false;
}
static bool rows_clash(const void* in, int64_t ld_in, const void* out, int64_t ld_out, int64_t m, int64_t row) {
  return rows_overlap(in, ld_in, row, out, ld_out, row, m, true);
}

int qk_rms_norm_quant(int m, int k, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                      const void* weight, int dtype, int weight_dtype, double eps, int code,
                      void* residual_out, int64_t ldo, void* q, float* scale, hipStream_t stream) {
  if (m < 0 || k < 0 || !known_input_dtype(dtype)) return QK_ERR_INVALID_VALUE;
  if (weight_dtype != dtype && weight_dtype != QK_F32) return QK_ERR_INVALID_VALUE;
  if (code != QK_CODE_I8 && code != QK_CODE_FP8) return QK_ERR_INVALID_VALUE;
  if (!(eps >= 0.0)) return QK_ERR_INVALID_VALUE;
  if (m == 0) return QK_OK;
  if (!scale || (k > 0 && (!x || !weight || !q || (residual && !residual_out)))) return QK_ERR_INVALID_VALUE;
  if (ldx < k || (residual && (ldr < k || ldo < k))) return QK_ERR_INVALID_VALUE;
  if (k > 1 << 30) return QK_ERR_UNSUPPORTED;
  const uintptr_t e = dtype == QK_F32 ? 4 : 2;
  if (!aligned(x, e) || !aligned(weight, weight_dtype == QK_F32 ? 4 : 2) || !aligned(scale, 4))
    return QK_ERR_UNSUPPORTED;
  if (residual && (!aligned(residual, e) || !aligned(residual_out, e))) return QK_ERR_UNSUPPORTED;
  const int64_t b = static_cast<int64_t>(e);
  if (residual && (rows_clash(x, ldx * b, residual_out, ldo * b, m, k * b) ||
                   rows_clash(residual, ldr * b, residual_out, ldo * b, m, k * b)))
    return QK_ERR_INVALID_VALUE;
  const qk::RmsNormQuantArgs a{m,        k,          x,        ldx, residual,
                               ldr,      weight,     dtype,    weight_dtype == QK_F32,
                               eps,      residual_out, ldo,    code == QK_CODE_FP8,
                               static_cast<uint8_t*>(q), scale};
  return status_of(qk::launch_rms_norm_quant(a, stream));
}

// Checks of the cache and its tables, the same for every call on it.
static int kv_check(int seqs, int tokens, int kv_heads, int dim, const void* k_cache, const void* v_cache,
                    const float* k_scale, const float* v_scale, int blocks, int block, int code,
                    const int* table, int64_t ldt, int width, const int* lens) {
  if (seqs < 0 || tokens < 0 || kv_heads < 1 || blocks < 0 || width < 0) return QK_ERR_INVALID_VALUE;
  if (dim < 16 || dim > 256 || dim % 16 != 0) return QK_ERR_INVALID_VALUE;
  if (block != 16 && block != 32 && block != 64 && block != 128) return QK_ERR_INVALID_VALUE;
  if (code != QK_CODE_I8 && code != QK_CODE_FP8) return QK_ERR_INVALID_VALUE;
  if (seqs == 0 || tokens == 0) return QK_OK;
  if (ldt < width || !lens || (width > 0 && !table)) return QK_ERR_INVALID_VALUE;
  if (blocks == 0 || !k_cache || !v_cache || !k_scale || !v_scale) return QK_ERR_INVALID_VALUE;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
      !aligned(table, 4) || !aligned(lens, 4))
    return QK_ERR_UNSUPPORTED;
  return QK_OK;
}

static qk::KvCacheView kv_view(int kv_heads, int dim, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, int blocks, int block, int code,
                               const int* table, int64_t ldt, int width) {
  return qk::KvCacheView{blocks,
                         kv_heads,
                         block,
                         dim,
                         code == QK_CODE_FP8,
                         static_cast<uint8_t*>(const_cast<void*>(k_cache)),
                         static_cast<uint8_t*>(const_cast<void*>(v_cache)),
                         const_cast<float*>(k_scale),
                         const_cast<float*>(v_scale),
                         table,
                         ldt,
                         width};
}

// A grid beyond what a launch takes is an argument error here.
static int status_of_cut(hipError_t e) {
  return e == hipErrorInvalidConfiguration ? QK_ERR_UNSUPPORTED : status_of(e);
}

static int kv_rows(bool write, int seqs, int tokens, int kv_heads, int dim, void* k, int64_t ldk, void* v,
                   int64_t ldv, int dtype, const void* k_cache, const void* v_cache, const float* k_scale,
                   const float* v_scale, int blocks, int block, int code, const int* table, int64_t ldt,
                   int width, const int* start, const int* cu, hipStream_t stream) {
  if (!known_input_dtype(dtype)) return QK_ERR_INVALID_VALUE;
  const int rc = kv_check(seqs, tokens, kv_heads, dim, k_cache, v_cache, k_scale, v_scale, blocks, block, code,
                          table, ldt, width, start);
  if (rc != QK_OK || seqs == 0 || tokens == 0) return rc;
  const int64_t row = static_cast<int64_t>(kv_heads) * dim;
  if (!k || !v || !cu || ldk < row || ldv < row) return QK_ERR_INVALID_VALUE;
  const uintptr_t e = dtype == QK_F32 ? 4 : 2;
  if (!aligned(k, e) || !aligned(v, e) || !aligned(cu, 4)) return QK_ERR_UNSUPPORTED;
  const qk::KvCacheView c = kv_view(kv_heads, dim, k_cache, v_cache, k_scale, v_scale, blocks, block, code, table,
                                    ldt, width);
  const qk::KvRowsArgs a{seqs, tokens, dtype, start, cu, k, ldk, v, ldv};
  return status_of_cut(write ? qk::launch_kv_cache_write(c, a, stream) : qk::launch_kv_cache_read(c, a, stream));
}

int qk_kv_cache_write(int seqs, int tokens, int kv_heads, int dim, const void* k, int64_t ldk,
                      const void* v, int64_t ldv, int dtype, void* k_cache, void* v_cache,
                      float* k_scale, float* v_scale, int blocks, int block, int code,
                      const int* table, int64_t ldt, int width, const int* start, const int* cu,
                      hipStream_t stream) {
  return kv_rows(true, seqs, tokens, kv_heads, dim, const_cast<void*>(k), ldk, const_cast<void*>(v), ldv, dtype,
                 k_cache, v_cache, k_scale, v_scale, blocks, block, code, table, ldt, width, start, cu, stream);
}

int qk_kv_cache_read(int seqs, int tokens, int kv_heads, int dim, void* k, int64_t ldk, void* v,
                     int64_t ldv, int dtype, const void* k_cache, const void* v_cache,
                     const float* k_scale, const float* v_scale, int blocks, int block, int code,
                     const int* table, int64_t ldt, int width, const int* start, const int* cu,
                     hipStream_t stream) {
  return kv_rows(false, seqs, tokens, kv_heads, dim, k, ldk, v, ldv, dtype, k_cache, v_cache, k_scale, v_scale,
                 blocks, block, code, table, ldt, width, start, cu, stream);
}

size_t qk_kv_attention_sinks_workspace_size(int seqs, int tokens, int heads, int kv_heads, int dim, int ragged,
                                            int max_q, int max_kv, int window, int sinks) {
  if (seqs <= 0 || tokens <= 0 || kv_heads < 1 || heads < kv_heads || heads % kv_heads != 0 || dim < 16 ||
      dim > 256 || max_q < 1 || max_kv < 0 || max_kv > qk::kKvMostPositions || window < 0 || sinks < 0)
    return 0;
  return qk::kv_attention_workspace_bytes(seqs, tokens, heads, kv_heads, dim, ragged != 0, max_q, max_kv, window,
                                          sinks);
}

size_t qk_kv_attention_workspace_size(int seqs, int tokens, int heads, int kv_heads, int dim, int ragged,
                                      int max_q, int max_kv, int window) {
  return qk_kv_attention_sinks_workspace_size(seqs, tokens, heads, kv_heads, dim, ragged, max_q, max_kv, window, 0);
}

int qk_kv_attention_sinks(int seqs, int tokens, int heads, int kv_heads, int dim, const void* q,
                          int64_t ldq, int dtype, const void* k_cache, const void* v_cache,
                          const float* k_scale, const float* v_scale, int blocks, int block, int code,
                          const int* table, int64_t ldt, int width, const int* lens, const int* cu,
                          int max_q, int max_kv, float scale, int window, int sinks, void* out,
                          float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (dtype != QK_BF16 && dtype != QK_F16) return QK_ERR_INVALID_VALUE;
  if (kv_heads < 1 || heads < 1 || heads % kv_heads != 0) return QK_ERR_INVALID_VALUE;
  if (max_q < 1 || max_kv < 0 || window < 0 || sinks < 0 || !(scale - scale == 0.0f)) return QK_ERR_INVALID_VALUE;
  const int rc = kv_check(seqs, tokens, kv_heads, dim, k_cache, v_cache, k_scale, v_scale, blocks, block, code,
                          table, ldt, width, lens);
  if (rc != QK_OK || seqs == 0 || tokens == 0) return rc;
  if (!q || !out || ldq < static_cast<int64_t>(heads) * dim || (!cu && tokens != seqs))
    return QK_ERR_INVALID_VALUE;
  if (!aligned(q, 2) || !aligned(out, 2) || !aligned(lse, 4) || !aligned(cu, 4)) return QK_ERR_UNSUPPORTED;
  const int64_t reach = static_cast<int64_t>(width) * block;
  if (reach < max_kv) max_kv = static_cast<int>(reach);
  if (max_kv > qk::kKvMostPositions) return QK_ERR_UNSUPPORTED;
  const size_t need =
      qk::kv_attention_workspace_bytes(seqs, tokens, heads, kv_heads, dim, cu != nullptr, max_q, max_kv, window, sinks);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return QK_ERR_WORKSPACE;
  const qk::KvCacheView c = kv_view(kv_heads, dim, k_cache, v_cache, k_scale, v_scale, blocks, block, code, table,
                                    ldt, width);
  const qk::KvAttentionArgs a{seqs, tokens, heads, dtype, q, ldq, lens, cu, max_q, max_kv, scale, window, sinks, out, lse,
                              workspace, workspace_bytes};
  return status_of_cut(qk::launch_kv_attention(c, a, stream));
}

int qk_kv_attention(int seqs, int tokens, int heads, int kv_heads, int dim, const void* q,
                    int64_t ldq, int dtype, const void* k_cache, const void* v_cache,
                    const float* k_scale, const float* v_scale, int blocks, int block, int code,
                    const int* table, int64_t ldt, int width, const int* lens, const int* cu,
                    int max_q, int max_kv, float scale, int window, void* out, float* lse,
                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return qk_kv_attention_sinks(seqs, tokens, heads, kv_heads, dim, q, ldq, dtype, k_cache, v_cache, k_scale, v_scale,
                               blocks, block, code, table, ldt, width, lens, cu, max_q, max_kv, scale, window, 0, out,
                               lse, workspace, workspace_bytes, stream);
}

// ---- microscaled 4-bit rows ----

constexpr int64_t kMx4Most = int64_t{1} << 35;  // values of one call, eight to a work item

// Checks of one operand's codes and scales.
static int mx4_operand(int64_t rows, int k, const uint8_t* q, const uint8_t* scale, int64_t lds) {
  if (rows == 0 || k == 0) return QK_OK;
  if (!q || !scale || lds < k / 32) return QK_ERR_INVALID_VALUE;
  if (lds % 16 != 0 || !aligned(q, 16) || !aligned(scale, 16)) return QK_ERR_UNSUPPORTED;
  return QK_OK;
}

static int mx4_rows(bool back, bool silu, int m, int k, void* x, int64_t ldx, int dtype, uint8_t* q, uint8_t* scale,
                    int64_t lds, hipStream_t stream) {
  if (m < 0 || k < 0 || !known_input_dtype(dtype)) return QK_ERR_INVALID_VALUE;
  if (k % 32 != 0) return QK_ERR_UNSUPPORTED;
  if (m == 0 || k == 0) return QK_OK;
  if (!x || ldx < (silu ? 2 : 1) * static_cast<int64_t>(k)) return QK_ERR_INVALID_VALUE;
  const int rc = mx4_operand(m, k, q, scale, lds);
  if (rc != QK_OK) return rc;
  if (!aligned(x, dtype == QK_F32 ? 4 : 2) || static_cast<int64_t>(m) * k >= kMx4Most) return QK_ERR_UNSUPPORTED;
  return status_of_cut(qk::launch_mx4_rows(qk::Mx4RowsArgs{m, k, x, ldx, dtype, silu, q, scale, lds}, back, stream));
}

int qk_quant_mx4(int m, int k, const void* x, int64_t ldx, int x_dtype, uint8_t* q, uint8_t* scale, int64_t lds,
                 hipStream_t stream) {
  return mx4_rows(false, false, m, k, const_cast<void*>(x), ldx, x_dtype, q, scale, lds, stream);
}

int qk_silu_mul_quant_mx4(int m, int d, const void* h, int64_t ldh, int h_dtype, uint8_t* q, uint8_t* scale,
                          int64_t lds, hipStream_t stream) {
  return mx4_rows(false, true, m, d, const_cast<void*>(h), ldh, h_dtype, q, scale, lds, stream);
}

int qk_dequant_mx4(int m, int k, const uint8_t* q, const uint8_t* scale, int64_t lds, void* x, int64_t ldx,
                   int x_dtype, hipStream_t stream) {
  return mx4_rows(true, false, m, k, x, ldx, x_dtype, const_cast<uint8_t*>(q), const_cast<uint8_t*>(scale), lds,
                  stream);
}

// The product's kernels reach 256 rows from a base with 32-bit offsets.
constexpr int kMx4MostRows = 1 << 24, kMx4MostK = 1 << 24;
constexpr int64_t kMx4MostStride = 1 << 23;
static bool mx4_fits(int m, int n, int k, int64_t ldsa, int64_t ldsb) {
  return m <= kMx4MostRows && n <= kMx4MostRows && k <= kMx4MostK && ldsa <= kMx4MostStride && ldsb <= kMx4MostStride;
}

int qk_gemm_mx4_scaled(int m, int n, int k, const uint8_t* a, const uint8_t* scale_a, int64_t ldsa, const uint8_t* b,
                       const uint8_t* scale_b, int64_t ldsb, float output_scale, void* out, int out_dtype,
                       hipStream_t stream) {
  if (m < 0 || n < 0 || k < 0 || !known_input_dtype(out_dtype)) return QK_ERR_INVALID_VALUE;
  if (k % 32 != 0) return QK_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return QK_OK;
  if (!out) return QK_ERR_INVALID_VALUE;
  int rc = mx4_operand(m, k, a, scale_a, ldsa);
  if (rc == QK_OK) rc = mx4_operand(n, k, b, scale_b, ldsb);
  if (rc != QK_OK) return rc;
  if (!aligned(out, out_dtype == QK_F32 ? 4 : 2) || !mx4_fits(m, n, k, ldsa, ldsb)) return QK_ERR_UNSUPPORTED;
  const qk::Mx4GemmArgs g{m, n, k, a, scale_a, ldsa, b, scale_b, ldsb, output_scale, out, out_dtype};
  return status_of_cut(qk::launch_gemm_mx4(g, stream));
}

int qk_linear_mx4(int m, int n, int k, const void* x, int64_t ldx, int x_dtype, const uint8_t* b,
                  const uint8_t* scale_b, int64_t ldsb, float output_scale, void* out, int out_dtype, uint8_t* q_out,
                  uint8_t* scale_out, int64_t lds_out, hipStream_t stream) {
  // everything is checked before anything is enqueued
  if (m < 0 || n < 0 || k < 0 || !known_input_dtype(x_dtype) || !known_input_dtype(out_dtype))
    return QK_ERR_INVALID_VALUE;
  if (k % 32 != 0) return QK_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return QK_OK;
  if (!out || (k > 0 && (!x || ldx < k))) return QK_ERR_INVALID_VALUE;
  const int rc = mx4_operand(n, k, b, scale_b, ldsb);
  if (rc != QK_OK) return rc;
  if (!aligned(x, x_dtype == QK_F32 ? 4 : 2) || !aligned(out, out_dtype == QK_F32 ? 4 : 2) ||
      !mx4_fits(m, n, k, 0, ldsb))
    return QK_ERR_UNSUPPORTED;
  const qk::Mx4GemmArgs g{m, n, k, q_out, scale_out, lds_out, b, scale_b, ldsb, output_scale, out, out_dtype};
  if (qk::mx4_linear_at_once(m, n, k, x, ldx * (x_dtype == QK_F32 ? 4 : 2)))
    return status_of_cut(qk::launch_linear_mx4_rows(g, x, ldx, x_dtype, stream));
  if (lds_out > kMx4MostStride) return QK_ERR_UNSUPPORTED;
  const int quantised = qk_quant_mx4(m, k, x, ldx, x_dtype, q_out, scale_out, lds_out, stream);
  if (quantised != QK_OK) return quantised;
  return qk_gemm_mx4_scaled(m, n, k, q_out, scale_out, lds_out, b, scale_b, ldsb, output_scale, out, out_dtype,
                            stream);
}

// ---- norm and rotation of queries and keys ----

int qk_norm_rope(int seqs, int tokens, int heads, int kv_heads, int dim, const void* q, int64_t ldq, const void* k,
                 int64_t ldk, const void* q_weight, const void* k_weight, int dtype, int weight_dtype, float eps,
                 const double* freqs, int rotary, int interleaved, const int* start, const int* cu, void* q_out,
                 int64_t ldqo, void* k_out, int64_t ldko, hipStream_t stream) {
  if (seqs < 0 || tokens < 0 || heads < 0 || kv_heads < 0 || !known_input_dtype(dtype)) return QK_ERR_INVALID_VALUE;
  if (weight_dtype != dtype && weight_dtype != QK_F32) return QK_ERR_INVALID_VALUE;
  if (dim < 16 || dim > 256 || dim % 16 != 0 || rotary < 0 || rotary > dim || rotary % 2 != 0)
    return QK_ERR_INVALID_VALUE;
  if (!(eps >= 0.0f)) return QK_ERR_INVALID_VALUE;
  if (seqs == 0 || tokens == 0 || heads + static_cast<int64_t>(kv_heads) == 0) return QK_OK;
  if (!start || (rotary > 0 && !freqs) || (!cu && tokens != seqs)) return QK_ERR_INVALID_VALUE;
  const uintptr_t e = dtype == QK_F32 ? 4 : 2, we = weight_dtype == QK_F32 ? 4 : 2;
  const int64_t b = static_cast<int64_t>(e);
  struct Side {
    int heads;
    const void* x;
    int64_t ldx;
    const void* weight;
    void* out;
    int64_t ldo;
  } sides[] = {{heads, q, ldq, q_weight, q_out, ldqo}, {kv_heads, k, ldk, k_weight, k_out, ldko}};
  for (const Side& s : sides) {
    const int64_t row = static_cast<int64_t>(s.heads) * dim;
    if (row == 0) continue;
    if (!s.x || !s.out || s.ldx < row || s.ldo < row) return QK_ERR_INVALID_VALUE;
    if (!aligned(s.x, e) || !aligned(s.out, e) || !aligned(s.weight, we)) return QK_ERR_UNSUPPORTED;
  }
  if (!aligned(start, 4) || !aligned(cu, 4) || !aligned(freqs, 8)) return QK_ERR_UNSUPPORTED;
  if (static_cast<int64_t>((heads > kv_heads ? heads : kv_heads)) * dim > 1 << 24) return QK_ERR_UNSUPPORTED;
  for (const Side& out : sides)
    for (const Side& in : sides) {
      const int64_t wo = static_cast<int64_t>(out.heads) * dim * b, wi = static_cast<int64_t>(in.heads) * dim * b;
      if (wo == 0 || wi == 0) continue;
      // each output against each input, and against the other output
      const bool own = &out == &in;
      if (rows_overlap(in.x, in.ldx * b, wi, out.out, out.ldo * b, wo, tokens, own)) return QK_ERR_INVALID_VALUE;
      if (!own && rows_overlap(in.out, in.ldo * b, wi, out.out, out.ldo * b, wo, tokens, false))
        return QK_ERR_INVALID_VALUE;
    }
  const qk::NormRopeArgs a{seqs, tokens, heads, kv_heads, dim, rotary, q, ldq, k, ldk, q_weight, k_weight, dtype,
                           weight_dtype == QK_F32, eps, freqs, interleaved != 0, start, cu, q_out, ldqo, k_out, ldko};
  return status_of_cut(qk::launch_norm_rope(a, stream));
}

}  // extern "C"
