// act.hip -- the gradient of the product's epilogue: dz = dy act'(z), the
// bias's gradient (the column sums of dz) and max |dz| (NaN left out), in one pass
// that is bound by HBM (2 + 2 + 1 + 1/32 bytes per bf16 value with z in 8 bits).
//
// A workgroup takes a slab of 256 columns over a range of rows: 32 lanes along
// the columns (chunks of 8), 8 along the rows, kUnroll rows of each lane in
// flight. A lane keeps its columns' sums in registers over all its rows; the 8
// row lanes meet in LDS at the end, and the workgroup leaves one partial row of
// sums and one maximum for k_col_reduce. No atomics, so the sums' order, and
// their bits, depend on the shape alone.
#include "layer_internal.hpp"
#include "row_device.hpp"

#include <type_traits>

using namespace fp4row;

namespace {

constexpr int kUnroll = 4;

struct Act {
  const char *dy, *z;
  int64_t ld_dy, ld_z;
  Mx8In z8;
  char* dz;
  int64_t ld_dz;
  float* part;         // [gridDim.y][cols] or null
  uint32_t* max_part;  // [gridDim.y][gridDim.x] or null
  int64_t rows, part_rows;
  uint32_t cols;
};

template <bool BF16, bool Z8>
using RawZ = std::conditional_t<Z8, RawMx8, Raw8<BF16>>;

template <bool BF16, bool Z8, int ACT, bool NT>
__global__ __launch_bounds__(256) void k_act_bwd(Act a) {
  constexpr int ES = BF16 ? 2 : 4;
  __shared__ float sums[8][256];
  __shared__ uint32_t tops[4];
  const int col_lane = threadIdx.x & 31, row_lane = threadIdx.x >> 5;
  const uint32_t c = (blockIdx.x * 32 + col_lane) * 8;
  const int64_t first = a.part_rows * blockIdx.y, last = min(first + a.part_rows, a.rows);
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  uint32_t top = 0;
  for (int64_t r0 = first + row_lane; r0 < last; r0 += 8 * kUnroll) {
    Raw8<BF16> dr[kUnroll];
    RawZ<BF16, Z8> zr[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int64_t r = r0 + 8 * k;
      const uint32_t n = r < last ? a.cols : 0;
      dr[k] = raw_chunk<BF16, NT>(a.dy + r * a.ld_dy * ES, c, n);
      if constexpr (Z8) zr[k] = mx8_raw<NT>(a.z8, r, c, n);
      else zr[k] = raw_chunk<BF16, NT>(a.z + r * a.ld_z * ES, c, n);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int64_t r = r0 + 8 * k;
      float d[8], z[8];
      expand<BF16>(dr[k], d);
      if constexpr (Z8) expand(zr[k], c, a.cols, z);
      else expand<BF16>(zr[k], z);
      act_slope8(ACT, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] *= z[i];
        acc[i] += d[i];
      }
      top = max(top, number_max8_bits(d));
      if (r < last && c < a.cols) store_chunk<BF16, NT>(a.dz + r * a.ld_dz * ES, c, a.cols, d);
      // One row's values at a time in registers (all at once took 140).
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (a.part) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[row_lane][col_lane * 8 + i] = acc[i];
    __syncthreads();
    const uint32_t cc = blockIdx.x * 256 + threadIdx.x;
    if (cc < a.cols) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += sums[i][threadIdx.x];
      a.part[(int64_t)blockIdx.y * a.cols + cc] = s;
    }
  }
  if (a.max_part) {
    top = wave_max(BF16 ? bf16_bits(top) : top);  // of the values as stored
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0)
      a.max_part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  }
}

template <bool BF16, bool Z8, bool NT>
void pick_act(int act, dim3 g, const Act& a, hipStream_t s) {
  if (act == ACT_RELU) hipLaunchKernelGGL((k_act_bwd<BF16, Z8, ACT_RELU, NT>), g, dim3(256), 0, s, a);
  else if (act == ACT_GELU) hipLaunchKernelGGL((k_act_bwd<BF16, Z8, ACT_GELU, NT>), g, dim3(256), 0, s, a);
  else if (act == ACT_SILU) hipLaunchKernelGGL((k_act_bwd<BF16, Z8, ACT_SILU, NT>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_act_bwd<BF16, Z8, ACT_NONE, NT>), g, dim3(256), 0, s, a);
}
template <bool BF16, bool Z8>
void pick_stream(int act, dim3 g, const Act& a, hipStream_t s) {
  if (streaming(a.rows, a.cols, BF16 ? 2 : 4, rows_on_16(a.dz, a.ld_dz, BF16 ? 2 : 4))) pick_act<BF16, Z8, true>(act, g, a, s);
  else pick_act<BF16, Z8, false>(act, g, a, s);
}

}  // namespace

ActPlan fp4i_act_plan(int64_t rows, int64_t cols) {
  ActPlan p;
  p.slabs = (cols + 255) / 256;
  // Whole sets of 8 kUnroll rows to a workgroup, as many as leave about 3072
  // workgroups: enough to even out their ends, few partial rows to add.
  const int64_t sets = (rows + 8 * kUnroll - 1) / (8 * kUnroll), want = 3072 / p.slabs > 0 ? 3072 / p.slabs : 1;
  const int64_t per = (sets + want - 1) / want;
  p.rows = per * 8 * kUnroll;
  p.parts = (sets + per - 1) / per;
  return p;
}

void fp4i_launch_act_bwd(const fp4_act_bwd& n, hipStream_t s) {
  const ActPlan p = fp4i_act_plan(n.rows, n.cols);
  // One workgroup's sums and maximum are the result; a single range of rows
  // gives the sums whole.
  const bool one = p.parts * p.slabs == 1;
  float* const part = static_cast<float*>(n.ws);
  uint32_t* const tops = reinterpret_cast<uint32_t*>(part + p.parts * n.cols);
  Act a;
  a.dy = static_cast<const char*>(n.dy);
  a.z = static_cast<const char*>(n.z);
  a.ld_dy = n.ld_dy;
  a.ld_z = n.ld_z;
  a.z8 = n.z8 ? Mx8In{n.z8->codes, n.z8->scales, n.z8->ld, n.z8->lds} : Mx8In{nullptr, nullptr, 0, 0};
  a.dz = static_cast<char*>(n.dz);
  a.ld_dz = n.ld_dz;
  a.part = !n.dbias ? nullptr : p.parts == 1 ? n.dbias : part;
  a.max_part = !n.amax ? nullptr : one ? reinterpret_cast<uint32_t*>(n.amax) : tops;
  a.rows = n.rows;
  a.cols = (uint32_t)n.cols;
  a.part_rows = p.rows;
  const dim3 g((uint32_t)p.slabs, (uint32_t)p.parts);
  if (n.dtype == FP4_DTYPE_BF16) {
    if (n.z8) pick_stream<true, true>(n.act, g, a, s);
    else pick_stream<true, false>(n.act, g, a, s);
  } else {
    if (n.z8) pick_stream<false, true>(n.act, g, a, s);
    else pick_stream<false, false>(n.act, g, a, s);
  }
  const bool sum = n.dbias && p.parts > 1, top = n.amax && !one;
  if (sum || top)
    fp4i_launch_col_reduce(part, p.parts, n.cols, sum ? n.dbias : nullptr, tops, p.parts * p.slabs,
                           top ? n.amax : nullptr, s);
}
