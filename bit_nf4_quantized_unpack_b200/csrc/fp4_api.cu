// fp4_api.cu -- the extern "C" entry points of the microscaled 4-bit operators: host-side
// validation (nothing is launched when an argument is rejected) and dispatch.
#include "internal.h"

namespace qlora {
namespace {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 256;  // tile coordinates are 32-bit
// A CTA pair multiplies 256 columns in about 0.4 us, and no role of a kernel may wait for
// another one longer than the 2 s after which waits give up: 2^28 columns take 0.4 s.
constexpr int64_t kMaxCols = int64_t{1} << 28;
constexpr int64_t kMaxValues = int64_t{1} << 40;        // grid dimensions of the codec kernels
constexpr int64_t kMaxWeightRows = int64_t{65535} * 32;  // the weight kernel's grid
constexpr size_t kWeightWorkspace = kFp4MaxTops * sizeof(uint32_t);

bool known_format(int32_t f) { return f == QLORA_FP4_MX || f == QLORA_FP4_NV; }
bool known_dtype(qlora_dtype d) { return d == QLORA_F32 || d == QLORA_BF16; }

qlora_status check_shape(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > kMaxRows || cols < 32 || cols > kMaxCols || cols % 32 != 0)
    return QLORA_ERR_SHAPE;
  if (rows > kMaxValues / cols) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

qlora_status check_matrix(const qlora_fp4_matrix& q) {
  if (!known_format(q.format)) return QLORA_ERR_INVALID_ARG;
  qlora_status s = check_shape(q.rows, q.cols);
  if (s != QLORA_OK) return s;
  if (q.rows == 0) return QLORA_OK;
  if (!q.codes || !q.scales) return QLORA_ERR_INVALID_ARG;
  if (q.gscale && q.gscale_rows != 1 && q.gscale_rows != q.rows) return QLORA_ERR_SHAPE;
  if (!is_aligned16(q.codes) || !is_aligned16(q.scales) || (q.gscale && !is_aligned16(q.gscale)))
    return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

// Whether `an` bytes at a and `bn` bytes at b share memory.
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

bool finite_scale(float s) { return s == s && s <= 3.0e38f && s >= -3.0e38f; }

// The checks both directions of the linear layer share; w is the weight in either form.
qlora_status check_fp4_linear(int64_t M, const qlora_fp4_matrix& w, int r, float scale) {
  qlora_status q = check_matrix(w);
  if (q != QLORA_OK) return q;
  if (w.rows < 32 || w.rows % 32 != 0) return QLORA_ERR_SHAPE;
  if (w.gscale && w.gscale_rows != 1) return QLORA_ERR_SHAPE;
  if (r < 8 || r > 64 || r % 8 != 0 || !finite_scale(scale)) return QLORA_ERR_INVALID_ARG;
  q = check_shape(M, w.cols);
  return q != QLORA_OK ? q : check_shape(M, w.rows);
}

bool linear_sizes(int64_t M, int64_t n, int64_t k, int r, int32_t format) {
  return known_format(format) && n >= 32 && n % 32 == 0 && r >= 8 && r <= 64 && r % 8 == 0 &&
         check_shape(M, k) == QLORA_OK && check_shape(M, n) == QLORA_OK;
}

}  // namespace
}  // namespace qlora

using namespace qlora;

extern "C" {

size_t qlora_fp4_scales_bytes(int64_t rows, int64_t cols, int32_t format) {
  if (!known_format(format) || check_shape(rows, cols) != QLORA_OK) return 0;
  return fp4_scales_bytes(rows, cols, format);
}

qlora_status qlora_fp4_quantize(const void* X, qlora_dtype x_dtype, int64_t rows, int64_t cols,
                                int32_t format, uint8_t* codes, uint8_t* scales, float* gscale,
                                void* stream) {
  if (!known_format(format) || !known_dtype(x_dtype)) return QLORA_ERR_INVALID_ARG;
  qlora_status q = check_shape(rows, cols);
  if (q != QLORA_OK) return q;
  if (rows == 0) return QLORA_OK;
  const bool nv = format == QLORA_FP4_NV;
  if (!X || !codes || !scales || (nv && !gscale)) return QLORA_ERR_INVALID_ARG;
  if (!is_aligned16(X) || !is_aligned16(codes) || !is_aligned16(scales) ||
      (nv && !is_aligned16(gscale)))
    return QLORA_ERR_ALIGN;
  q = check_device();
  if (q != QLORA_OK) return q;
  return cuda_status(launch_fp4_quantize(X, x_dtype == QLORA_BF16, rows, cols, format,
                                         Fp4Out{codes, scales, gscale},
                                         static_cast<cudaStream_t>(stream)));
}

size_t qlora_fp4_quantize_weight_workspace_size(void) { return kWeightWorkspace; }

qlora_status qlora_fp4_quantize_weight(const void* W, qlora_dtype w_dtype, int64_t n_out,
                                       int64_t k_in, int32_t format, uint8_t* codes,
                                       uint8_t* scales, float* gscale, uint8_t* t_codes,
                                       uint8_t* t_scales, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  if (!known_format(format) || !known_dtype(w_dtype)) return QLORA_ERR_INVALID_ARG;
  qlora_status q = check_shape(n_out, k_in);
  if (q != QLORA_OK) return q;
  if (n_out < 32 || n_out % 32 != 0 || n_out > kMaxWeightRows) return QLORA_ERR_SHAPE;
  const bool nv = format == QLORA_FP4_NV;
  if (!W || !codes || !scales || (nv && !gscale) || !t_codes != !t_scales)
    return QLORA_ERR_INVALID_ARG;
  if (!is_aligned16(W) || !is_aligned16(codes) || !is_aligned16(scales) ||
      (nv && !is_aligned16(gscale)) || (t_codes && !is_aligned16(t_codes)) ||
      (t_scales && !is_aligned16(t_scales)))
    return QLORA_ERR_ALIGN;
  if (!workspace || workspace_bytes < kWeightWorkspace) return QLORA_ERR_WORKSPACE;
  if (!is_aligned16(workspace)) return QLORA_ERR_ALIGN;
  q = check_device();
  if (q != QLORA_OK) return q;
  return cuda_status(launch_fp4_quantize_weight(
      W, w_dtype == QLORA_BF16, n_out, k_in, format, Fp4Out{codes, scales, gscale},
      Fp4Out{t_codes, t_scales, nullptr}, workspace, static_cast<cudaStream_t>(stream)));
}

qlora_status qlora_fp4_dequant(qlora_fp4_matrix m, qlora_dtype out_dtype, void* out,
                               void* stream) {
  if (!known_dtype(out_dtype)) return QLORA_ERR_INVALID_ARG;
  qlora_status q = check_matrix(m);
  if (q != QLORA_OK) return q;
  if (m.rows == 0) return QLORA_OK;
  if (!out) return QLORA_ERR_INVALID_ARG;
  if (!is_aligned16(out)) return QLORA_ERR_ALIGN;
  q = check_device();
  if (q != QLORA_OK) return q;
  return cuda_status(launch_fp4_dequant(m, out_dtype == QLORA_BF16, out,
                                        static_cast<cudaStream_t>(stream)));
}

qlora_status qlora_fp4_matmul(qlora_fp4_matrix a, qlora_fp4_matrix b, qlora_dtype out_dtype,
                              void* out, void* stream) {
  if (!known_dtype(out_dtype)) return QLORA_ERR_INVALID_ARG;
  qlora_status q = check_matrix(a);
  if (q == QLORA_OK) q = check_matrix(b);
  if (q != QLORA_OK) return q;
  if (a.format != b.format) return QLORA_ERR_INVALID_ARG;
  if (a.cols != b.cols || b.rows < 8 || b.rows % 8 != 0) return QLORA_ERR_SHAPE;
  if (a.rows == 0) return QLORA_OK;
  if (!out) return QLORA_ERR_INVALID_ARG;
  if (!is_aligned16(out)) return QLORA_ERR_ALIGN;
  q = check_device();
  if (q != QLORA_OK) return q;
  return fp4_product(a, b, nullptr, out, out_dtype == QLORA_F32, false,
                     static_cast<cudaStream_t>(stream));
}

size_t qlora_fp4_linear_fwd_workspace_size(int64_t M, int64_t n_out, int64_t k_in, int r,
                                           int32_t format) {
  if (!linear_sizes(M, n_out, k_in, r, format)) return 0;
  return fp4_fwd_workspace(LinearShape{M, n_out, k_in, r, 1.f}, format);
}

qlora_status qlora_fp4_linear_fwd(const uint16_t* X, int64_t M, qlora_fp4_matrix w,
                                  const uint16_t* A, const uint16_t* B, int r, float scale,
                                  uint16_t* Y, float* T_save, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  qlora_status q = check_fp4_linear(M, w, r, scale);
  if (q != QLORA_OK) return q;
  if (M == 0) return QLORA_OK;  // empty batch: nothing to compute (X, Y may be NULL)
  if (!X || !A || !B || !Y) return QLORA_ERR_INVALID_ARG;
  if (!is_aligned16(X) || !is_aligned16(A) || !is_aligned16(B) || !is_aligned16(Y) ||
      (T_save && !is_aligned16(T_save)))
    return QLORA_ERR_ALIGN;
  const LinearShape s{M, w.rows, w.cols, r, scale};
  if (!workspace || workspace_bytes < fp4_fwd_workspace(s, w.format)) return QLORA_ERR_WORKSPACE;
  if (!is_aligned16(workspace)) return QLORA_ERR_ALIGN;
  q = check_device();
  if (q != QLORA_OK) return q;
  return fp4_forward(X, w, A, B, s, Y, T_save, workspace, static_cast<cudaStream_t>(stream));
}

size_t qlora_fp4_linear_bwd_workspace_size(int64_t M, int64_t n_out, int64_t k_in, int r,
                                           int32_t format) {
  if (!linear_sizes(M, n_out, k_in, r, format)) return 0;
  return fp4_bwd_workspace(LinearShape{M, n_out, k_in, r, 1.f}, format);
}

qlora_status qlora_fp4_linear_bwd(const uint16_t* dY, const uint16_t* X, const float* T_saved,
                                  int64_t M, qlora_fp4_matrix wt, const uint16_t* A,
                                  const uint16_t* B, int r, float scale, uint16_t* dX, float* dA,
                                  float* dB, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  qlora_status q = check_fp4_linear(M, wt, r, scale);
  if (q != QLORA_OK) return q;
  if (!dA || !dB) return QLORA_ERR_INVALID_ARG;
  if (!is_aligned16(dA) || !is_aligned16(dB)) return QLORA_ERR_ALIGN;
  const LinearShape s{M, wt.cols, wt.rows, r, scale};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (M == 0) {  // empty batch: the gradients of A and B are zero
    q = check_device();
    if (q != QLORA_OK) return q;
    cudaError_t e = cudaMemsetAsync(dA, 0, static_cast<size_t>(s.K) * r * 4, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(dB, 0, static_cast<size_t>(s.N) * r * 4, st);
    return cuda_status(e);
  }
  if (!dY || !X || !A || !B) return QLORA_ERR_INVALID_ARG;
  if (!is_aligned16(dY) || !is_aligned16(X) || !is_aligned16(A) || !is_aligned16(B) ||
      (dX && !is_aligned16(dX)) || (T_saved && !is_aligned16(T_saved)))
    return QLORA_ERR_ALIGN;
  if (!workspace || workspace_bytes < fp4_bwd_workspace(s, wt.format)) return QLORA_ERR_WORKSPACE;
  if (!is_aligned16(workspace)) return QLORA_ERR_ALIGN;
  // dA and dB read X and dY beside or behind the product that writes dX
  const size_t x_bytes = static_cast<size_t>(M) * s.K * 2, y_bytes = static_cast<size_t>(M) * s.N * 2;
  if (dX && (overlap(dX, x_bytes, X, x_bytes) || overlap(dX, x_bytes, dY, y_bytes)))
    return QLORA_ERR_INVALID_ARG;
  q = check_device();
  if (q != QLORA_OK) return q;
  return fp4_backward(dY, X, T_saved, wt, A, B, s, dX, dA, dB, workspace, st);
}

}  // extern "C"
