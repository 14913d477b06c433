// epilogue.hpp -- the FP4 product's epilogue: z = alpha sum + bias, act(z) +
// residual, the 8-bit form of z. Shared by the tiled kernels (gemm_core.hpp with
// EPI) and the few-row kernel (gemm_rows.hip).
#pragma once
#include "fp4.h"
#include "fp4_internal.hpp"
#include "row_device.hpp"

namespace {

struct EpiArgs {
  void* c;           // the output; the residual may be the same buffer
  const void* bias;  // null or N values
  const char* res;   // null or M x N
  int64_t ld_res;
  fp4row::Mx8Out z8;
  int act;
  bool bias_bf16, res_bf16;
};
template <bool EPI>
struct EpiOf {};
template <>
struct EpiOf<true> : EpiArgs {};

inline EpiOf<true> epi_args(const fp4_epilogue& f, void* c) {
  EpiOf<true> e;
  e.c = c;
  e.bias = f.bias;
  e.res = static_cast<const char*>(f.residual);
  e.ld_res = f.ld_residual;
  e.z8 = f.z8 ? fp4row::Mx8Out{f.z8->codes, f.z8->scales, f.z8->ld, f.z8->lds}
              : fp4row::Mx8Out{nullptr, nullptr, 0, 0};
  e.act = f.act;
  e.bias_bf16 = f.bias_t == FP4_DTYPE_BF16;
  e.res_bf16 = f.residual_t == FP4_DTYPE_BF16;
  return e;
}

// Eight columns of one output row: z (alpha times the accumulators, plus bias),
// its 8-bit form, the activation, the residual, the store. The lanes of a quad
// hold 32 consecutive columns from a multiple of 32 on and call it together
// (needed with z8 only). Columns past N and rows past M stand as zeros and are not
// stored.
__device__ __forceinline__ void epi_row8(const EpiArgs& e, float z[8], const float bias[8], const float res[8],
                                         float alpha, uint32_t row, uint32_t col, uint32_t M, uint32_t N, bool obf,
                                         int64_t ldc) {
  const uint32_t n = row < M ? N : 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = col + i < N ? __builtin_fmaf(z[i], alpha, bias[i]) : 0.0f;
  if (e.z8.codes) {
    uint32_t m;
    fp4row::mx8_store(e.z8, row, col, n, z, m);
  }
  fp4row::act8(e.act, z);
  if (e.res) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += res[i];
  }
  if (col < n) {
    if (obf) fp4row::store_chunk<true>(static_cast<char*>(e.c) + (int64_t)row * ldc * 2, col, n, z);
    else fp4row::store_chunk<false>(static_cast<char*>(e.c) + (int64_t)row * ldc * 4, col, n, z);
  }
}

// The same where every column and row of the caller's tile is inside the output: a
// lane's addresses, moved on from row to row (a 64-bit product for each took a
// fifth of the epilogue's instructions). Stores are marked as not to be kept, as
// fp4_gemm's are.
template <bool OBF>
struct EpiWhole {
  char* c;
  uint8_t *codes, *scales;
  int64_t dc, dcodes, dscales;  // bytes from one of the lane's rows to the next
  bool first;                   // the lane holds the first columns of a block

  __device__ __forceinline__ EpiWhole(const EpiArgs& e, uint32_t row, uint32_t col, uint32_t step, int64_t ldc) {
    constexpr int ES = OBF ? 2 : 4;
    c = static_cast<char*>(e.c) + ((int64_t)row * ldc + col) * ES;
    dc = (int64_t)step * ldc * ES;
    codes = e.z8.codes + (int64_t)row * e.z8.ld + col;
    dcodes = (int64_t)step * e.z8.ld;
    scales = e.z8.scales + (int64_t)row * e.z8.lds + col / 32;
    dscales = (int64_t)step * e.z8.lds;
    first = col % 32 == 0;
  }
  __device__ __forceinline__ void row8(const EpiArgs& e, float z[8], const float bias[8], const float res[8],
                                       float alpha) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __builtin_fmaf(z[i], alpha, bias[i]);
    if (e.z8.codes) {
      const uint32_t byte = fp4row::mx8_byte(fp4row::quad_max(fp4row::number_max8_bits(z)));
      const uint2 w = fp4row::mx8_pack8(z, fp4row::mx8_factor(byte));
      __builtin_nontemporal_store((fp4row::v2u){w.x, w.y}, reinterpret_cast<fp4row::v2u*>(codes));
      if (first) *scales = (uint8_t)byte;
      codes += dcodes;
      scales += dscales;
    }
    fp4row::act8(e.act, z);
    if (e.res) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] += res[i];
    }
    fp4row::store8_any<OBF, OBF>(c, z);
    c += dc;
  }
};

// The residual of the same columns as it lies in memory (bf16: in w[0]). EDGE: some
// of the columns or the row may lie outside the output; zeros there.
template <bool EDGE>
__device__ __forceinline__ void epi_residual8(const EpiArgs& e, uint32_t row, uint32_t col, uint32_t M, uint32_t N,
                                              fp4dev::v4u (&w)[2]) {
  const char* const p = e.res + (int64_t)row * e.ld_res * (e.res_bf16 ? 2 : 4);
  const uint32_t n = row < M ? N : 0;
  if (e.res_bf16) {
    const fp4row::Raw8<true> r = EDGE ? fp4row::raw_chunk<true>(p, col, n) : fp4row::raw8_any<true>(p + (int64_t)col * 2);
    w[0] = r.w[0];
  } else {
    const fp4row::Raw8<false> r = EDGE ? fp4row::raw_chunk<false>(p, col, n) : fp4row::raw8_any<false>(p + (int64_t)col * 4);
    w[0] = r.w[0];
    w[1] = r.w[1];
  }
}
// The same as values; zeros without a residual.
__device__ __forceinline__ void epi_residual8(const EpiArgs& e, uint32_t row, uint32_t col, uint32_t M, uint32_t N,
                                              float res[8]) {
  fp4row::load_chunk_rt(e.res + (int64_t)row * e.ld_res * (e.res_bf16 ? 2 : 4), e.res_bf16, col,
                        e.res && row < M ? N : 0, res);
}

}  // namespace

// Launchers: the tiled product, and the one of few tiles; which one a product takes.
void fp4i_launch_gemm_fused(const GemmArgs& g, const fp4_epilogue& f, hipStream_t s);
void fp4i_launch_gemm_rows(const GemmArgs& g, const fp4_epilogue& f, hipStream_t s);
bool fp4i_gemm_rows_pays(int64_t M, int64_t N, int64_t K, int fmt);
