// C ABI of libmxfp4: argument validation on the host, then one kernel
// launch on the caller's stream. The contract of every entry point (layouts,
// ownership, errors) is stated in include/mxfp4.h.
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/mxfp4.h"
#include "launch.cuh"

namespace {

bool aligned16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// The optional status word (NULL passes).
bool aligned4(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

// rows, cols > 0, each at most MXFP4_MAX_DIM, product below 2^46.
bool dims_ok(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return false;
  if (rows > MXFP4_MAX_DIM || cols > MXFP4_MAX_DIM) return false;
  return rows <= (int64_t(1) << 46) / cols;
}

bool dtype_ok(int dt) { return dt == MXFP4_F32 || dt == MXFP4_BF16; }
bool axis_ok(int a) { return a == MXFP4_ROWS || a == MXFP4_COLS; }
bool rounding_ok(int r) { return r == MXFP4_RNE || r == MXFP4_SR; }

mxfp4_status from_cuda(cudaError_t e) {
  return e == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA;
}

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

namespace {

mxfp4_status quantize_with_rule(const void* x, int dtype, int64_t rows,
                                int64_t cols, int axis, int rounding,
                                uint64_t seed, uint8_t* codes,
                                uint8_t* scales, void* stream, bool oas) {
  if (!dtype_ok(dtype) || !axis_ok(axis) || !rounding_ok(rounding))
    return MXFP4_ERR_ENUM;
  if (!x || !codes || !scales) return MXFP4_ERR_NULL;
  if (!dims_ok(rows, cols)) return MXFP4_ERR_SHAPE;
  if ((axis == MXFP4_ROWS ? cols : rows) % 32 != 0) return MXFP4_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(codes)) return MXFP4_ERR_ALIGN;
  const bool bf16 = dtype == MXFP4_BF16, sr = rounding == MXFP4_SR;
  if (axis == MXFP4_ROWS)
    return from_cuda(mxfp4::launch_quant_rows(x, bf16, rows, cols, sr, seed,
                                              codes, scales, as_stream(stream),
                                              oas));
  return from_cuda(mxfp4::launch_quant_cols(x, bf16, rows, cols, sr, seed,
                                            codes, scales, as_stream(stream),
                                            oas));
}

}  // namespace

mxfp4_status mxfp4_quantize(const void* x, int dtype, int64_t rows,
                            int64_t cols, int axis, int rounding,
                            uint64_t seed, uint8_t* codes, uint8_t* scales,
                            void* stream) {
  return quantize_with_rule(x, dtype, rows, cols, axis, rounding, seed, codes,
                            scales, stream, false);
}

mxfp4_status mxfp4_quantize_oas(const void* x, int dtype, int64_t rows,
                                int64_t cols, int axis, int rounding,
                                uint64_t seed, uint8_t* codes, uint8_t* scales,
                                void* stream) {
  return quantize_with_rule(x, dtype, rows, cols, axis, rounding, seed, codes,
                            scales, stream, true);
}

mxfp4_status mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales,
                              int64_t rows, int64_t cols, int axis, void* y,
                              int out_dtype, void* stream) {
  if (!dtype_ok(out_dtype) || !axis_ok(axis)) return MXFP4_ERR_ENUM;
  if (!codes || !scales || !y) return MXFP4_ERR_NULL;
  if (!dims_ok(rows, cols)) return MXFP4_ERR_SHAPE;
  if ((axis == MXFP4_ROWS ? cols : rows) % 32 != 0) return MXFP4_ERR_SHAPE;
  if (!aligned16(codes) || !aligned16(y)) return MXFP4_ERR_ALIGN;
  return from_cuda(mxfp4::launch_dequant(codes, scales, rows * cols / 32, y,
                                         out_dtype == MXFP4_BF16,
                                         as_stream(stream)));
}

static mxfp4_status double_quantize_with_rule(const void* x, int dtype, int64_t rows,
                                              int64_t cols, uint64_t seed,
                                              uint8_t* row_codes, uint8_t* row_scales,
                                              uint8_t* col_codes, uint8_t* col_scales,
                                              void* stream, bool oas) {
  if (!dtype_ok(dtype)) return MXFP4_ERR_ENUM;
  if (!x || !row_codes || !row_scales || !col_codes || !col_scales)
    return MXFP4_ERR_NULL;
  if (!dims_ok(rows, cols) || rows % 32 || cols % 32) return MXFP4_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(row_codes) || !aligned16(col_codes))
    return MXFP4_ERR_ALIGN;
  return from_cuda(mxfp4::launch_double_quant(
      x, dtype == MXFP4_BF16, rows, cols, seed, row_codes, row_scales,
      col_codes, col_scales, as_stream(stream), oas));
}

mxfp4_status mxfp4_double_quantize(const void* x, int dtype, int64_t rows,
                                   int64_t cols, uint64_t seed,
                                   uint8_t* row_codes, uint8_t* row_scales,
                                   uint8_t* col_codes, uint8_t* col_scales,
                                   void* stream) {
  return double_quantize_with_rule(x, dtype, rows, cols, seed, row_codes, row_scales,
                                   col_codes, col_scales, stream, false);
}

mxfp4_status mxfp4_double_quantize_oas(const void* x, int dtype, int64_t rows,
                                       int64_t cols, uint64_t seed,
                                       uint8_t* row_codes, uint8_t* row_scales,
                                       uint8_t* col_codes, uint8_t* col_scales,
                                       void* stream) {
  return double_quantize_with_rule(x, dtype, rows, cols, seed, row_codes, row_scales,
                                   col_codes, col_scales, stream, true);
}

static mxfp4_status rht_quantize_with_rule(const void* x, int dtype, int64_t rows,
                                           int64_t cols, uint64_t sign_seed,
                                           int rounding, uint64_t sr_seed,
                                           uint8_t* codes, uint8_t* scales,
                                           float* rotated, int* status, void* stream,
                                           bool oas) {
  if (!dtype_ok(dtype) || !rounding_ok(rounding)) return MXFP4_ERR_ENUM;
  if (!x || !codes || !scales) return MXFP4_ERR_NULL;
  if (!dims_ok(rows, cols) || cols % 32) return MXFP4_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(codes) || (rotated && !aligned16(rotated)) ||
      !aligned4(status))
    return MXFP4_ERR_ALIGN;
  return from_cuda(mxfp4::launch_rht_quant(
      x, dtype == MXFP4_BF16, rows, cols, sign_seed, rounding == MXFP4_SR,
      sr_seed, codes, scales, rotated, status, as_stream(stream), oas));
}

mxfp4_status mxfp4_rht_quantize(const void* x, int dtype, int64_t rows,
                                int64_t cols, uint64_t sign_seed,
                                int rounding, uint64_t sr_seed,
                                uint8_t* codes, uint8_t* scales,
                                float* rotated, int* status, void* stream) {
  return rht_quantize_with_rule(x, dtype, rows, cols, sign_seed, rounding, sr_seed, codes,
                                scales, rotated, status, stream, false);
}

mxfp4_status mxfp4_rht_quantize_oas(const void* x, int dtype, int64_t rows,
                                    int64_t cols, uint64_t sign_seed,
                                    int rounding, uint64_t sr_seed,
                                    uint8_t* codes, uint8_t* scales,
                                    float* rotated, int* status, void* stream) {
  return rht_quantize_with_rule(x, dtype, rows, cols, sign_seed, rounding, sr_seed, codes,
                                scales, rotated, status, stream, true);
}

mxfp4_status mxfp4_osc_step(float* w, float* w_snap, float* d_w, float* d_q,
                            int64_t rows, int64_t cols, int window_end,
                            float threshold, unsigned long long* n_flagged,
                            void* stream) {
  if (!w || !w_snap || !d_w || !d_q) return MXFP4_ERR_NULL;
  if (!dims_ok(rows, cols) || cols % 32) return MXFP4_ERR_SHAPE;
  if (!aligned16(w) || !aligned16(w_snap) || !aligned16(d_w) ||
      !aligned16(d_q))
    return MXFP4_ERR_ALIGN;
  return from_cuda(mxfp4::launch_osc_step(w, w_snap, d_w, d_q, rows, cols,
                                          window_end != 0, threshold,
                                          n_flagged, as_stream(stream)));
}

mxfp4_status mxfp4_qramp_step(float* w, const float* delta, float* w_snap,
                              float* d_w, float* d_q, float* acc, uint8_t* flag,
                              int64_t rows, int64_t cols, int64_t iter,
                              int64_t track_iters, float k1, int64_t k2,
                              unsigned long long* n_flagged, void* stream) {
  if (!w || !delta || !w_snap || !d_w || !d_q || !acc || !flag) return MXFP4_ERR_NULL;
  if (!dims_ok(rows, cols) || cols % 32) return MXFP4_ERR_SHAPE;
  if (iter < 0 || track_iters < 0 || k2 < 1) return MXFP4_ERR_SHAPE;
  if (!aligned16(w) || !aligned16(delta) || !aligned16(w_snap) || !aligned16(d_w) ||
      !aligned16(d_q) || !aligned16(acc) || !aligned16(flag))
    return MXFP4_ERR_ALIGN;
  return from_cuda(mxfp4::launch_qramp_step(w, delta, w_snap, d_w, d_q, acc, flag, rows,
                                            cols, iter, track_iters, k1, k2, n_flagged,
                                            as_stream(stream)));
}

mxfp4_status mxfp4_osc_synthetic_update(float* w, int64_t rows, int64_t cols,
                                        uint64_t seed, uint32_t step,
                                        float rel_step, void* stream) {
  if (!w) return MXFP4_ERR_NULL;
  if (!dims_ok(rows, cols)) return MXFP4_ERR_SHAPE;
  if (!aligned16(w)) return MXFP4_ERR_ALIGN;
  return from_cuda(mxfp4::launch_osc_update(w, rows * cols, seed, step,
                                            rel_step, as_stream(stream)));
}

mxfp4_status mxfp4_qema_quantize(const float* w, float* w_ema, int64_t rows,
                                 int64_t cols, float beta, uint8_t* codes,
                                 uint8_t* scales, void* stream) {
  if (!w || !w_ema || !codes || !scales) return MXFP4_ERR_NULL;
  if (!dims_ok(rows, cols) || cols % 32) return MXFP4_ERR_SHAPE;
  if (!aligned16(w) || !aligned16(w_ema) || !aligned16(codes))
    return MXFP4_ERR_ALIGN;
  return from_cuda(mxfp4::launch_qema_quant(w, w_ema, rows, cols, beta,
                                            codes, scales, as_stream(stream)));
}

mxfp4_status mxfp4_scales_to_blocked(const uint8_t* scales, int64_t rows,
                                     int64_t groups, uint8_t* blocked,
                                     void* stream) {
  if (!scales || !blocked) return MXFP4_ERR_NULL;
  if (!dims_ok(rows, groups)) return MXFP4_ERR_SHAPE;
  if (!aligned16(blocked)) return MXFP4_ERR_ALIGN;
  return from_cuda(mxfp4::launch_scales_blocked(scales, rows, groups, blocked,
                                                as_stream(stream)));
}

mxfp4_status mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales,
                        const uint8_t* b_codes, const uint8_t* b_scales,
                        int64_t m, int64_t n, int64_t k, float* c,
                        int* status, void* stream) {
  if (!a_codes || !a_scales || !b_codes || !b_scales || !c)
    return MXFP4_ERR_NULL;
  if (!dims_ok(m, k) || !dims_ok(n, k) || !dims_ok(m, n) || k % 32)
    return MXFP4_ERR_SHAPE;
  if ((m + 127) / 128 > 65535) return MXFP4_ERR_SHAPE;  // grid y
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(b_codes) ||
      !aligned16(b_scales) || !aligned16(c) || !aligned4(status))
    return MXFP4_ERR_ALIGN;
  return from_cuda(mxfp4::launch_gemm_mxf4(a_codes, a_scales, b_codes,
                                           b_scales, m, n, k, c, status,
                                           as_stream(stream)));
}

mxfp4_status mxfp4_gemm_quantize_a(const void* x, int64_t m, int64_t n, int64_t k,
                                   int rounding, uint64_t seed, const uint8_t* b_codes,
                                   const uint8_t* b_scales, float* c, uint8_t* a_codes,
                                   uint8_t* a_scales, int* status, void* stream) {
  if (!rounding_ok(rounding)) return MXFP4_ERR_ENUM;
  if (!x || !b_codes || !b_scales || !c || (a_codes == nullptr) != (a_scales == nullptr))
    return MXFP4_ERR_NULL;
  if (!dims_ok(m, k) || !dims_ok(n, k) || !dims_ok(m, n) || k % 256)
    return MXFP4_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(b_codes) || !aligned16(b_scales) || !aligned16(c) ||
      !aligned16(a_codes) || !aligned4(status))
    return MXFP4_ERR_ALIGN;
  return from_cuda(mxfp4::launch_gemm_qa(x, m, n, k, rounding == MXFP4_SR, seed, b_codes,
                                         b_scales, c, a_codes, a_scales, status,
                                         as_stream(stream)));
}

namespace {

// An element-aligned pointer (NULL passes).
bool aligned_to(const void* p, uintptr_t size) {
  return (reinterpret_cast<uintptr_t>(p) & (size - 1)) == 0;
}

bool eps_ok(float eps) { return eps >= 0.0f && eps <= 3.4e38f; }

// ld >= cols, and the strided rows stay within the size limit.
bool stride_ok(int64_t rows, int64_t cols, int64_t ld) {
  return ld >= cols && ld <= (int64_t(1) << 46) / rows;
}

mxfp4_status layernorm_args(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                            const float* weight, const float* bias, float eps, const void* y,
                            const float* mean, const float* rstd) {
  if (!dtype_ok(dtype)) return MXFP4_ERR_ENUM;
  if (!dims_ok(rows, cols) || !stride_ok(rows, cols, ldx)) return MXFP4_ERR_SHAPE;
  if (!eps_ok(eps)) return MXFP4_ERR_VALUE;
  const uintptr_t size = dtype == MXFP4_BF16 ? 2 : 4;
  if (!aligned_to(x, size) || !aligned_to(y, size) || !aligned_to(weight, 4) ||
      !aligned_to(bias, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return MXFP4_ERR_ALIGN;
  return MXFP4_OK;
}

}  // namespace

namespace {
bool gemv_dims_ok(int64_t m, int64_t n, int64_t k) {
  return dims_ok(m, k) && dims_ok(n, k) && dims_ok(m, n) && k % 32 == 0 &&
         m <= (int64_t(1) << 19) && k <= (int64_t(1) << 30);  // grids, 32-bit k counts
}
}  // namespace

int64_t mxfp4_gemv_workspace(int64_t m, int64_t n, int64_t k) {
  return gemv_dims_ok(m, n, k) ? mxfp4::gemv_workspace(m, n, k) : -1;
}

mxfp4_status mxfp4_gemv(const void* x, int64_t m, int64_t n, int64_t k, int64_t ldx,
                        const uint8_t* b_codes, const uint8_t* b_scales, void* y, int y_dtype,
                        void* workspace, int64_t workspace_bytes, int* status, void* stream) {
  if (!dtype_ok(y_dtype)) return MXFP4_ERR_ENUM;
  if (!x || !b_codes || !b_scales || !y) return MXFP4_ERR_NULL;
  if (!gemv_dims_ok(m, n, k) || !stride_ok(m, k, ldx) || ldx % 8) return MXFP4_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(b_codes) || !aligned16(b_scales) || !aligned16(y) ||
      !aligned16(workspace) || !aligned4(status))
    return MXFP4_ERR_ALIGN;
  const int64_t need = mxfp4::gemv_workspace(m, n, k);
  if (need > 0 && workspace == nullptr) return MXFP4_ERR_NULL;
  if (workspace_bytes < need) return MXFP4_ERR_WORKSPACE;
  return from_cuda(mxfp4::launch_gemv(x, m, n, k, ldx, b_codes, b_scales, y,
                                      y_dtype == MXFP4_BF16, workspace, status,
                                      as_stream(stream)));
}

int64_t mxfp4_newton_schulz_workspace(int64_t rows, int64_t cols) {
  if (!dims_ok(rows, cols) || rows > MXFP4_NS_MAX_DIM || cols > MXFP4_NS_MAX_DIM) return -1;
  return mxfp4::newton_schulz_workspace(rows, cols);
}

mxfp4_status mxfp4_newton_schulz(const void* g, int dtype, int64_t rows, int64_t cols, int steps,
                                 float a, float b, float c, float eps, float scale, void* out,
                                 int out_dtype, void* workspace, int64_t workspace_bytes,
                                 int* status, void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype)) return MXFP4_ERR_ENUM;
  if (!g || !out || !workspace) return MXFP4_ERR_NULL;
  const int64_t need = mxfp4_newton_schulz_workspace(rows, cols);
  if (need < 0) return MXFP4_ERR_SHAPE;
  const float lim = 1e4f;
  if (steps < 1 || steps > 1000 || !eps_ok(eps) || !(a >= -lim && a <= lim) ||
      !(b >= -lim && b <= lim) || !(c >= -lim && c <= lim) ||
      !(scale >= -3.4e38f && scale <= 3.4e38f))
    return MXFP4_ERR_VALUE;
  if (!aligned16(g) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || !aligned4(status))
    return MXFP4_ERR_ALIGN;
  if (workspace_bytes < need) return MXFP4_ERR_WORKSPACE;
  return from_cuda(mxfp4::launch_newton_schulz(g, dtype == MXFP4_BF16, rows, cols, steps, a, b,
                                               c, eps, scale, out, out_dtype == MXFP4_BF16,
                                               workspace, status, as_stream(stream)));
}

mxfp4_status mxfp4_layernorm(const void* x, int dtype, int64_t rows, int64_t cols,
                             int64_t ldx, const float* weight, const float* bias, float eps,
                             void* y, float* mean, float* rstd, void* stream) {
  if (!x || !y) return MXFP4_ERR_NULL;
  const mxfp4_status st =
      layernorm_args(x, dtype, rows, cols, ldx, weight, bias, eps, y, mean, rstd);
  if (st != MXFP4_OK) return st;
  return from_cuda(mxfp4::launch_layernorm(x, dtype == MXFP4_BF16, rows, cols, ldx, weight,
                                           bias, eps, y, mean, rstd, nullptr, nullptr,
                                           as_stream(stream)));
}

mxfp4_status mxfp4_layernorm_quantize(const void* x, int dtype, int64_t rows, int64_t cols,
                                      int64_t ldx, const float* weight, const float* bias,
                                      float eps, void* y, float* mean, float* rstd,
                                      uint8_t* codes, uint8_t* scales, void* stream) {
  if (!x || !codes || !scales) return MXFP4_ERR_NULL;
  const mxfp4_status st =
      layernorm_args(x, dtype, rows, cols, ldx, weight, bias, eps, y, mean, rstd);
  if (st != MXFP4_OK) return st;
  if (cols % 32) return MXFP4_ERR_SHAPE;
  if (!aligned16(codes)) return MXFP4_ERR_ALIGN;
  return from_cuda(mxfp4::launch_layernorm(x, dtype == MXFP4_BF16, rows, cols, ldx, weight,
                                           bias, eps, y, mean, rstd, codes, scales,
                                           as_stream(stream)));
}

int64_t mxfp4_layernorm_backward_workspace(int64_t rows, int64_t cols) {
  if (!dims_ok(rows, cols)) return -1;
  return mxfp4::layernorm_backward_partials(rows) * 2 * cols * int64_t(sizeof(float));
}

mxfp4_status mxfp4_layernorm_backward(const void* dy, const void* x, int dtype, int64_t rows,
                                      int64_t cols, int64_t lddy, int64_t ldx,
                                      const float* weight, const float* mean, const float* rstd,
                                      void* dx, float* dw, float* db, void* workspace,
                                      int64_t workspace_bytes, void* stream) {
  if (!dy || !x || !mean || !rstd || !dx || (dw == nullptr) != (db == nullptr) ||
      (dw != nullptr && workspace == nullptr))
    return MXFP4_ERR_NULL;
  const mxfp4_status st =
      layernorm_args(x, dtype, rows, cols, ldx, weight, nullptr, 0.0f, dx, mean, rstd);
  if (st != MXFP4_OK) return st;
  if (!stride_ok(rows, cols, lddy)) return MXFP4_ERR_SHAPE;
  if (!aligned_to(dy, dtype == MXFP4_BF16 ? 2 : 4) || !aligned_to(dw, 4) ||
      !aligned_to(db, 4) || !aligned16(workspace))
    return MXFP4_ERR_ALIGN;
  if (dw != nullptr && workspace_bytes < mxfp4_layernorm_backward_workspace(rows, cols))
    return MXFP4_ERR_WORKSPACE;
  return from_cuda(mxfp4::launch_layernorm_backward(
      dy, x, dtype == MXFP4_BF16, rows, cols, lddy, ldx, weight, mean, rstd, dx, dw, db,
      static_cast<float*>(workspace), as_stream(stream)));
}

const char* mxfp4_status_string(int status) {
  switch (status) {
    case MXFP4_OK: return "ok";
    case MXFP4_ERR_NULL: return "a required pointer is NULL";
    case MXFP4_ERR_SHAPE:
      return "bad shape: rows/cols must be positive, within the size limit, "
             "and the group axis a multiple of 32 (of 256 for the fused GEMM)";
    case MXFP4_ERR_ALIGN:
      return "a tensor pointer is not 16-byte aligned (a status word: 4-byte)";
    case MXFP4_ERR_ENUM: return "dtype, axis or rounding out of range";
    case MXFP4_ERR_CUDA: return "CUDA launch failed";
    case MXFP4_ERR_VALUE: return "a numeric argument is outside its stated range";
    case MXFP4_ERR_WORKSPACE: return "the workspace is too small";
    default: return "unknown status";
  }
}

}  // extern "C"
