// layer_checks.hpp -- argument checks of the operators around the FP4 product
// (host only).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4.h"

namespace fp4chk {

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline bool dtype_ok(int t) { return t == FP4_DTYPE_F32 || t == FP4_DTYPE_BF16; }
inline bool act_ok(int a) { return a >= FP4_ACT_NONE && a <= FP4_ACT_SILU; }

// Rows and columns each index a launch dimension or a lane's 32-bit column (its byte
// offset too); offsets into a matrix are 64-bit. 2^25 columns are more than any
// product has: its operands' codes stay below 2^31 bytes and its K is at least 128.
inline bool dims_ok(int64_t rows, int64_t cols) {
  return rows >= 1 && cols >= 1 && rows <= INT32_MAX && cols <= (int64_t(1) << 25);
}

// A rows x cols matrix of dt (valid) with leading dimension ld.
inline fp4_status check_mat(const void* p, int dt, int64_t rows, int64_t cols, int64_t ld) {
  if (!dims_ok(rows, cols) || ld < cols || ld > INT64_MAX / 8 / rows) return FP4_ERR_SHAPE;
  return aligned(p, dt == FP4_DTYPE_F32 ? 4 : 2) ? FP4_OK : FP4_ERR_ALIGN;
}
inline fp4_status check_opt(const void* p, int dt, int64_t rows, int64_t cols, int64_t ld) {
  return p ? check_mat(p, dt, rows, cols, ld) : FP4_OK;
}

// An output over an input has its rows where the input's are: others would be
// written before they are read.
inline fp4_status check_over(const void* out, int64_t ld_out, const void* in, int64_t ld_in, int64_t rows) {
  return out && out == in && ld_out != ld_in && rows > 1 ? FP4_ERR_UNSUPPORTED : FP4_OK;
}

inline fp4_status check_mx8(const fp4_mx8* q, int64_t rows, int64_t cols) {
  if (!q->codes || !q->scales) return FP4_ERR_NULL;
  if (!dims_ok(rows, cols) || q->rows != rows || q->cols != cols) return FP4_ERR_SHAPE;
  const int64_t blocks = (cols + 31) / 32;
  if (q->ld < blocks * 32 || q->ld % 32 != 0 || q->lds < blocks) return FP4_ERR_SHAPE;
  if (q->ld > INT64_MAX / 8 / rows || q->lds > INT64_MAX / 8 / rows) return FP4_ERR_SHAPE;
  return aligned(q->codes, 16) ? FP4_OK : FP4_ERR_ALIGN;
}

inline fp4_status launched() { return hipGetLastError() == hipSuccess ? FP4_OK : FP4_ERR_HIP; }

}  // namespace fp4chk
