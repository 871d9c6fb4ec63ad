// C-ABI entry points of the operators around the fused expert FFN: grouped
// matmul, block-scaled FP8 matmul with its quantisers, layer norm.  Argument
// checks only; every check comes before anything is enqueued.
#include <cmath>

#include "internal.h"
#include "matmul_util.cuh"

using namespace moe;

namespace {

bool ok16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ws(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }
int as_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
long long up(long long a, long long b) { return (a + b - 1) / b; }

// Widths up to this: kernels round them up to whole tiles in 31 bits.
constexpr int kMaxWidth = INT32_MAX - 65536;

// Sizes and groups of a matmul.  offsets == NULL: one group of all rows.
int check_matmul(int64_t rows, const int32_t* offsets, int experts, int n, int k) {
  if (rows < 0 || experts <= 0 || n <= 0 || k <= 0) return MOE_ERR_ARG;
  if (offsets == nullptr ? experts != 1 : !ok16(offsets)) return MOE_ERR_ARG;
  if (experts > kMatmulMaxGroups || rows > kMaxWidth || n > kMaxWidth || k > kMaxWidth)
    return MOE_ERR_UNSUPPORTED;
  // output tiles (at least 64 x 64) are numbered in 31 bits, and so are 128-wide blocks
  const long long wide = up(n > k ? n : k, 64);
  if ((rows / 64 + experts) * wide > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (up(n, 64) * up(k, 64) > INT32_MAX / experts) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_grouped(int64_t rows, const int32_t* offsets, int experts, int n, int k, int dtype,
                  const void* ws) {
  const int rc = check_matmul(rows, offsets, experts, n, k);
  if (rc != MOE_OK) return rc;
  if (!ok_ws(ws)) return MOE_ERR_ARG;
  if (dtype != MOE_DTYPE_FP32 && dtype != MOE_DTYPE_BF16) return MOE_ERR_UNSUPPORTED;
  if (dtype == MOE_DTYPE_BF16 && (n % 8 != 0 || k % 8 != 0)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int grouped(int mode, const void* a, int64_t rows, const int32_t* offsets, int experts,
            const void* w, int n, int k, int dtype, void* out, void* ws, void* stream) {
  const int rc = check_grouped(rows, offsets, experts, n, k, dtype, ws);
  if (rc != MOE_OK) return rc;
  if (!ok16(w)) return MOE_ERR_ARG;
  if (rows == 0) return MOE_OK;
  if (!ok16(a) || !ok16(out)) return MOE_ERR_ARG;
  if (dtype == MOE_DTYPE_BF16)
    return launch_grouped_matmul_bf16(mode, a, (int)rows, offsets, experts, w, n, k, out, ws,
                                      as_stream(stream));
  return launch_grouped_matmul_fp32(mode, static_cast<const float*>(a),
                                    static_cast<const float*>(w), (int)rows, offsets, experts, n,
                                    k, static_cast<float*>(out), ws, as_stream(stream));
}

int fp8(int dx, const void* a_codes, int a_format, const float* a_scales, int64_t scale_ld,
        int64_t rows, const int32_t* offsets, int experts, const void* w_codes,
        const float* w_scales, int n, int k, void* out, void* ws, void* stream) {
  const int rc = check_matmul(rows, offsets, experts, n, k);
  if (rc != MOE_OK) return rc;
  if (!ok_ws(ws) || !ok16(w_codes) || !ok16(w_scales)) return MOE_ERR_ARG;
  if (a_format != MOE_FP8_E4M3 && a_format != MOE_FP8_E5M2) return MOE_ERR_UNSUPPORTED;
  if (k % 16 != 0 || (dx && n % 16 != 0)) return MOE_ERR_UNSUPPORTED;
  if (scale_ld < rows) return MOE_ERR_ARG;
  if (rows == 0) return MOE_OK;
  if (!ok16(a_codes) || !ok16(a_scales) || !ok16(out)) return MOE_ERR_ARG;
  return launch_matmul_fp8(dx, a_format == MOE_FP8_E5M2, a_codes, a_scales, scale_ld, (int)rows,
                           offsets, experts, w_codes, w_scales, n, k, out, ws, as_stream(stream));
}

int check_norm(int64_t rows, int d, int dtype) {
  if (rows < 0 || d <= 0) return MOE_ERR_ARG;
  if (dtype != MOE_DTYPE_FP32 && dtype != MOE_DTYPE_BF16) return MOE_ERR_UNSUPPORTED;
  if (d > layer_norm_max_d() || rows > kMaxWidth) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_matmul_workspace_size(void) { return 256; }

int moe_grouped_matmul(const void* x, int64_t rows, const int32_t* offsets, int experts,
                       const void* w, int n, int k, int dtype, void* y, void* ws, void* stream) {
  return grouped(0, x, rows, offsets, experts, w, n, k, dtype, y, ws, stream);
}

int moe_grouped_matmul_dx(const void* dy, int64_t rows, const int32_t* offsets, int experts,
                          const void* w, int n, int k, int dtype, void* dx, void* ws,
                          void* stream) {
  return grouped(1, dy, rows, offsets, experts, w, n, k, dtype, dx, ws, stream);
}

int moe_grouped_matmul_dw(const void* dy, const void* x, int64_t rows, const int32_t* offsets,
                          int experts, int n, int k, int dtype, void* dw, void* ws,
                          void* stream) {
  const int rc = check_grouped(rows, offsets, experts, n, k, dtype, ws);
  if (rc != MOE_OK) return rc;
  if (!ok16(dw)) return MOE_ERR_ARG;
  const size_t bytes = (size_t)experts * n * k * dtype_bytes(dtype);
  if (rows == 0)
    return as_status(note_cuda(cudaMemsetAsync(dw, 0, bytes, as_stream(stream)),
                               "grouped matmul weight gradient: clear"));
  if (!ok16(dy) || !ok16(x)) return MOE_ERR_ARG;
  if (dtype == MOE_DTYPE_BF16)
    return launch_grouped_matmul_dw_bf16(dy, x, (int)rows, offsets, experts, n, k, dw, ws,
                                         as_stream(stream));
  return launch_grouped_matmul_fp32(2, static_cast<const float*>(dy), static_cast<const float*>(x),
                                    (int)rows, offsets, experts, n, k, static_cast<float*>(dw), ws,
                                    as_stream(stream));
}

int moe_quantize_rows_fp8(const void* x, int64_t rows, int cols, int format, uint8_t* codes,
                          float* scales, int64_t scale_ld, void* stream) {
  if (rows < 0 || cols <= 0 || scale_ld < rows) return MOE_ERR_ARG;
  if (format != MOE_FP8_E4M3 && format != MOE_FP8_E5M2) return MOE_ERR_UNSUPPORTED;
  if (cols % 16 != 0 || cols > kMaxWidth) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!ok16(x) || !ok16(codes) || !ok16(scales)) return MOE_ERR_ARG;
  return as_status(launch_quantize_rows_fp8(x, rows, cols, format == MOE_FP8_E5M2, codes, scales,
                                            scale_ld, as_stream(stream)));
}

int moe_quantize_blocks_fp8(const void* w, int experts, int n, int k, uint8_t* codes,
                            float* scales, void* stream) {
  if (experts <= 0 || n <= 0 || k <= 0) return MOE_ERR_ARG;
  if (n > kMaxWidth || k > kMaxWidth) return MOE_ERR_UNSUPPORTED;
  if (k % 16 != 0 || up(n, 128) * up(k, 128) > INT32_MAX / experts) return MOE_ERR_UNSUPPORTED;
  if (!ok16(w) || !ok16(codes) || !ok16(scales)) return MOE_ERR_ARG;
  return as_status(launch_quantize_blocks_fp8(w, experts, n, k, codes, scales, as_stream(stream)));
}

int moe_matmul_fp8(const void* x_codes, int x_format, const float* x_scales, int64_t scale_ld,
                   int64_t rows, const int32_t* offsets, int experts, const void* w_codes,
                   const float* w_scales, int n, int k, void* y, void* ws, void* stream) {
  return fp8(0, x_codes, x_format, x_scales, scale_ld, rows, offsets, experts, w_codes, w_scales,
             n, k, y, ws, stream);
}

int moe_matmul_fp8_dx(const void* dy_codes, int dy_format, const float* dy_scales,
                      int64_t scale_ld, int64_t rows, const int32_t* offsets, int experts,
                      const void* w_codes, const float* w_scales, int n, int k, void* dx, void* ws,
                      void* stream) {
  return fp8(1, dy_codes, dy_format, dy_scales, scale_ld, rows, offsets, experts, w_codes,
             w_scales, n, k, dx, ws, stream);
}

size_t moe_layer_norm_workspace_size(int64_t rows, int d) {
  if (check_norm(rows, d, MOE_DTYPE_FP32) != MOE_OK) return 0;
  return (layer_norm_ws_bytes((int)rows, d) + 255) & ~size_t(255);
}

int moe_layer_norm(const void* x, const float* weight, const float* bias, float eps, int64_t rows,
                   int d, int dtype, void* y, float* mean, float* rstd, void* stream) {
  const int rc = check_norm(rows, d, dtype);
  if (rc != MOE_OK) return rc;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return MOE_ERR_ARG;
  if (!ok16(weight) || (bias != nullptr && !ok16(bias))) return MOE_ERR_ARG;
  if (rows == 0) return MOE_OK;
  if (!ok16(x) || !ok16(y) || !ok16(mean) || !ok16(rstd)) return MOE_ERR_ARG;
  return as_status(launch_layer_norm(dtype, x, weight, bias, eps, (int)rows, d, y, mean, rstd,
                                     as_stream(stream)));
}

int moe_layer_norm_backward(const void* dy, const void* x, const float* weight, const float* mean,
                            const float* rstd, int64_t rows, int d, int dtype, void* dx,
                            float* dweight, float* dbias, void* ws, void* stream) {
  const int rc = check_norm(rows, d, dtype);
  if (rc != MOE_OK) return rc;
  if (!ok16(weight) || !ok16(dweight) || (dbias != nullptr && !ok16(dbias))) return MOE_ERR_ARG;
  if (rows == 0) {
    cudaError_t e = cudaMemsetAsync(dweight, 0, (size_t)d * 4, as_stream(stream));
    if (e == cudaSuccess && dbias != nullptr)
      e = cudaMemsetAsync(dbias, 0, (size_t)d * 4, as_stream(stream));
    return as_status(note_cuda(e, "layer norm backward: clear"));
  }
  if (!ok16(dy) || !ok16(x) || !ok16(mean) || !ok16(rstd) || !ok16(dx) || !ok_ws(ws))
    return MOE_ERR_ARG;
  return as_status(launch_layer_norm_backward(dtype, dy, x, weight, mean, rstd, (int)rows, d, dx,
                                              dweight, dbias, ws, as_stream(stream)));
}

}  // extern "C"
