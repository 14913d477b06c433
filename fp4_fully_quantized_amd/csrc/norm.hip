// norm.hip -- root-mean-square norm with the residual's addition and its
// gradient.
//
//   forward   h = x + residual; rstd = (mean h^2 + eps)^-1/2; y = h rstd gamma
//   backward  xhat = h rstd; m = mean(dy gamma xhat);
//             dx = rstd (dy gamma - xhat m) + dres; dgamma = sum_rows dy xhat
//
// Both read a row once: T lanes hold it whole in registers (NCH chunks of 8
// columns each), so the row's sum, its reduction over the lanes and the outputs
// need no second read; gamma, and the backward pass's dgamma sums, stay in
// registers over all the rows a workgroup takes. They are bound by HBM. Rows
// too long for registers go through k_*_long, which read them twice.
#include "layer_internal.hpp"
#include "row_device.hpp"

#include <type_traits>

using namespace fp4row;

namespace {

__global__ void k_zero_amax(float* p) { *p = 0.0f; }

// A workgroup's first row for this lane; the same for a whole wave, and told so to
// the compiler, which then keeps the rows' addresses in scalar registers.
template <int T>
__device__ __forceinline__ int64_t first_row() {
  constexpr uint32_t PER = T > 256 ? 1 : 256 / T;
  return blockIdx.x * PER + (PER == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / T));
}

// Sum over the T lanes of a row, given to all of them. One row of a workgroup
// of T > 64: a word per wave in LDS, two sets of them in turn, so one barrier
// per row is enough (a set is written again only after the next row's barrier,
// which every wave reaches after it has read it).
template <int T>
__device__ __forceinline__ float row_sum(float v, float (*part)[T / 64 > 0 ? T / 64 : 1], int turn) {
  v = wave_sum(v);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) part[turn][threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v += part[turn][i];
  }
  return v;
}

// Largest m of a workgroup (bits of a magnitude) into *amax: plainly by the
// only workgroup of a launch, else an atomic maximum (order does not matter to
// it) that only a workgroup issues whose maximum exceeds the value it reads.
template <int BLOCK>
__device__ __forceinline__ void amax_out(uint32_t m, float* amax) {
  __shared__ uint32_t part[BLOCK / 64];
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < BLOCK / 64; ++i) m = max(m, part[i]);
    unsigned int* const a = reinterpret_cast<unsigned int*>(amax);
    if (gridDim.x == 1) *a = m;
    else if (m > __atomic_load_n(a, __ATOMIC_RELAXED)) atomicMax(a, m);
  }
}

struct Fwd {
  const char *x, *res;
  int64_t ld_x, ld_res;
  const void* gamma;
  char *h, *y;
  int64_t ld_h, ld_y;
  Mx8Out y8, h8;
  float* rstd;
  float* amax;
  int64_t rows;
  uint32_t cols;
  float inv_cols, eps;
  bool gamma_bf16;
};

// The outputs of one chunk of a row whose h and rstd are known. Returns the
// largest magnitude of y as it is stored, NaN left out; of a bf16 y that before
// the rounding (stored_max).
template <bool BF16, bool NT>
__device__ __forceinline__ uint32_t norm_out(const Fwd& a, int64_t r, uint32_t c, const float h[8], const float g[8],
                                             float rstd) {
  constexpr int ES = BF16 ? 2 : 4;
  uint32_t top = 0, m;
  if (a.h && c < a.cols) store_chunk<BF16, NT>(a.h + r * a.ld_h * ES, c, a.cols, h);
  if (a.h8.codes) mx8_store<NT>(a.h8, r, c, a.cols, h, m);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = h[i] * rstd * g[i];
  if (a.y8.codes) {
    const uint32_t byte = mx8_store<NT>(a.y8, r, c, a.cols, y, m);
    if (a.amax && !a.y && byte != 255) {
      // The block's largest stored value: rounding keeps the order. A block with an
      // infinity stands for NaN, and is left out as one.
      const float one[8] = {__uint_as_float(m), 0, 0, 0, 0, 0, 0, 0};
      float v[8];
      mx8_unpack8(mx8_pack8(one, mx8_factor(byte)), mx8_scale(byte), v);
      top = __float_as_uint(v[0]);
    }
  }
  if (a.y && c < a.cols) {
    store_chunk<BF16, NT>(a.y + r * a.ld_y * ES, c, a.cols, y);
    if (a.amax) top = number_max8_bits(y);
  }
  return top;
}

// The maximum over norm_out's results as the stored values' own.
template <bool BF16>
__device__ __forceinline__ uint32_t stored_max(const Fwd& a, uint32_t top) {
  return BF16 && a.y ? bf16_bits(top) : top;
}

// A lane's part of one row as it lies in memory (zeros from row a.rows on).
template <bool BF16, bool RES, int NCH>
struct FwdRow {
  Raw8<BF16> x[NCH], q[RES ? NCH : 1];
};
template <bool BF16, bool RES, int T, int NCH, bool NT>
__device__ __forceinline__ void load_row(const Fwd& a, int64_t r, int t, FwdRow<BF16, RES, NCH>& v) {
  constexpr int ES = BF16 ? 2 : 4;
  const uint32_t n = r < a.rows ? a.cols : 0;
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    v.x[k] = raw_chunk<BF16, NT>(a.x + r * a.ld_x * ES, (k * T + t) * 8, n);
    if constexpr (RES) v.q[k] = raw_chunk<BF16, NT>(a.res + r * a.ld_res * ES, (k * T + t) * 8, n);
  }
}

// The next row is loaded while the current one is worked on, so that the wait for
// the row's sum does not leave the memory idle. h and y may be x's or the
// residual's buffer: a row is written after it was read, and no other row is.
template <bool BF16, bool RES, int T, int NCH, bool NT>
__global__ __launch_bounds__(T > 256 ? T : 256) void k_norm(Fwd a) {
  constexpr int BLOCK = T > 256 ? T : 256, PER = BLOCK / T;
  __shared__ float part[2][T / 64];
  const int t = PER == 1 ? threadIdx.x : threadIdx.x % T;
  float g[NCH][8];
#pragma unroll
  for (int k = 0; k < NCH; ++k) load_chunk_rt(a.gamma, a.gamma_bf16, (k * T + t) * 8, a.cols, g[k]);
  uint32_t top = 0;
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * PER;
  int64_t r = first_row<T>();
  FwdRow<BF16, RES, NCH> row;
  load_row<BF16, RES, T, NCH, NT>(a, r, t, row);
  for (; r < a.rows; r += step) {
    float h[NCH][8];
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      expand<BF16>(row.x[k], h[k]);
      if constexpr (RES) {
        float q[8];
        expand<BF16>(row.q[k], q);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] += q[i];
      }
    }
    load_row<BF16, RES, T, NCH, NT>(a, r + step, t, row);
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s = __builtin_fmaf(h[k][i], h[k][i], s);
    s = row_sum<T>(s, part, turn);
    turn ^= 1;
    const float rstd = 1.0f / sqrtf(s * a.inv_cols + a.eps);
    if (a.rstd && t == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int k = 0; k < NCH; ++k) top = max(top, norm_out<BF16, NT>(a, r, (k * T + t) * 8, h[k], g[k], rstd));
  }
  if (a.amax) amax_out<BLOCK>(stored_max<BF16>(a, top), a.amax);
}

// Rows of any length: one for the sum, once more for the outputs.
template <bool BF16, bool RES>
__global__ __launch_bounds__(1024) void k_norm_long(Fwd a) {
  constexpr int ES = BF16 ? 2 : 4;
  constexpr int T = 1024;
  __shared__ float part[2][T / 64];
  const uint32_t end = (a.cols + 31) / 32 * 32;  // the four lanes of a block stay together
  uint32_t top = 0;
  int turn = 0;
  auto load = [&](int64_t r, uint32_t c, float h[8]) {
    load_chunk<BF16>(a.x + r * a.ld_x * ES, c, a.cols, h);
    if constexpr (RES) {
      float q[8];
      load_chunk<BF16>(a.res + r * a.ld_res * ES, c, a.cols, q);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] += q[i];
    }
  };
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float s = 0.0f;
    for (uint32_t c = threadIdx.x * 8; c < end; c += T * 8) {
      float h[8];
      load(r, c, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = __builtin_fmaf(h[i], h[i], s);
    }
    s = row_sum<T>(s, part, turn);
    turn ^= 1;
    const float rstd = 1.0f / sqrtf(s * a.inv_cols + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
    for (uint32_t c = threadIdx.x * 8; c < end; c += T * 8) {
      float h[8], g[8];
      load(r, c, h);
      load_chunk_rt(a.gamma, a.gamma_bf16, c, a.cols, g);
      top = max(top, norm_out<BF16, false>(a, r, c, h, g, rstd));
    }
  }
  if (a.amax) amax_out<T>(stored_max<BF16>(a, top), a.amax);
}

struct Bwd {
  const char *dy, *h, *dres;
  int64_t ld_dy, ld_h, ld_dres;
  Mx8In h8;
  const void* gamma;
  const float* rstd;
  char* dx;
  int64_t ld_dx;
  float* part;  // dgamma sums of each workgroup [gridDim.x][cols], or null
  int64_t rows;
  uint32_t cols;
  float inv_cols;
  bool gamma_bf16;
};

template <bool BF16, bool H8>
__device__ __forceinline__ void load_h(const Bwd& a, int64_t r, uint32_t c, float h[8]) {
  if constexpr (H8) mx8_load(a.h8, r, c, a.cols, h);
  else load_chunk<BF16>(a.h + r * a.ld_h * (BF16 ? 2 : 4), c, a.cols, h);
}

// A lane's part of one row as it lies in memory: the next row is loaded while
// the current one is worked on, so that the barrier in the middle of a row does
// not leave the memory idle. Nothing is read from row a.rows on. dx may be dy's or
// dres's buffer: a row is written after it was read, and no other row is.
template <bool BF16, bool H8, int NCH>
struct BwdRow {
  Raw8<BF16> d[NCH], q[NCH];
  std::conditional_t<H8, RawMx8, Raw8<BF16>> h[NCH];
  float rstd;
};
template <bool BF16, bool H8, int T, int NCH, bool NT>
__device__ __forceinline__ void load_row(const Bwd& a, int64_t r, int t, BwdRow<BF16, H8, NCH>& v) {
  constexpr int ES = BF16 ? 2 : 4;
  const uint32_t n = r < a.rows ? a.cols : 0, nq = a.dres ? n : 0;
  v.rstd = n ? a.rstd[r] : 0.0f;
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const uint32_t c = (k * T + t) * 8;
    v.d[k] = raw_chunk<BF16, NT>(a.dy + r * a.ld_dy * ES, c, n);
    if constexpr (H8) v.h[k] = mx8_raw<NT>(a.h8, r, c, n);
    else v.h[k] = raw_chunk<BF16, NT>(a.h + r * a.ld_h * ES, c, n);
    v.q[k] = raw_chunk<BF16, NT>(a.dres + r * a.ld_dres * ES, c, nq);
  }
}

template <bool BF16, bool H8, int T, int NCH, bool NT>
__global__ __launch_bounds__(T > 256 ? T : 256) void k_norm_bwd(Bwd a) {
  constexpr int ES = BF16 ? 2 : 4;
  constexpr int BLOCK = T > 256 ? T : 256, PER = BLOCK / T;
  __shared__ float part[2][T / 64];
  __shared__ float sums[PER > 1 ? PER : 1][PER > 1 ? T * 8 : 1];
  const int t = PER == 1 ? threadIdx.x : threadIdx.x % T;
  // gamma: in registers, or where two chunks of a 1024-lane workgroup leave none for
  // it (128 a lane), in LDS; a lane reads what it wrote.
  constexpr bool GLDS = T * NCH == 2048;
  __shared__ v4f gl[GLDS ? 2 * NCH : 1][GLDS ? T : 1];
  float g[GLDS ? 1 : NCH][8], acc[NCH][8];
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    float (&gk)[8] = g[GLDS ? 0 : k];
    load_chunk_rt(a.gamma, a.gamma_bf16, (k * T + t) * 8, a.cols, gk);
    if constexpr (GLDS) {
      gl[2 * k][t] = (v4f){gk[0], gk[1], gk[2], gk[3]};
      gl[2 * k + 1][t] = (v4f){gk[4], gk[5], gk[6], gk[7]};
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[k][i] = 0.0f;
  }
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * PER;
  int64_t r = first_row<T>();
  BwdRow<BF16, H8, NCH> row;
  load_row<BF16, H8, T, NCH, NT>(a, r, t, row);
  for (; r < a.rows; r += step) {
    float d[NCH][8], x[NCH][8];
    Raw8<BF16> q[NCH];
    const float rstd = row.rstd;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      expand<BF16>(row.d[k], d[k]);
      if constexpr (H8) expand(row.h[k], (k * T + t) * 8, a.cols, x[k]);
      else expand<BF16>(row.h[k], x[k]);
      q[k] = row.q[k];
    }
    load_row<BF16, H8, T, NCH, NT>(a, r + step, t, row);
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float (&gk)[8] = g[GLDS ? 0 : k];
      if constexpr (GLDS) {
        const v4f lo = gl[2 * k][t], hi = gl[2 * k + 1][t];
#pragma unroll
        for (int i = 0; i < 8; ++i) gk[i] = i < 4 ? lo[i] : hi[i - 4];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[k][i] *= rstd;
        acc[k][i] = __builtin_fmaf(d[k][i], x[k][i], acc[k][i]);
        d[k][i] *= gk[i];
        s = __builtin_fmaf(d[k][i], x[k][i], s);
      }
    }
    const float m = row_sum<T>(s, part, turn) * a.inv_cols;
    turn ^= 1;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float w[8];
      expand<BF16>(q[k], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[k][i] = __builtin_fmaf(rstd, __builtin_fmaf(-m, x[k][i], d[k][i]), w[i]);
      if ((k * T + t) * 8 < a.cols) store_chunk<BF16, NT>(a.dx + r * a.ld_dx * ES, (k * T + t) * 8, a.cols, d[k]);
    }
  }
  if (!a.part) return;
  char* out = reinterpret_cast<char*>(a.part + (int64_t)blockIdx.x * a.cols);
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const uint32_t c = (k * T + t) * 8;
    if constexpr (PER > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[threadIdx.x / T][t * 8 + i] = acc[k][i];
      __syncthreads();
#pragma unroll
      for (int p = 0; p < PER; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[k][i] = p ? acc[k][i] + sums[p][t * 8 + i] : sums[p][t * 8 + i];
    }
    if (threadIdx.x < T && c < a.cols) store_chunk<false>(out, c, a.cols, acc[k]);
  }
}

// Rows of any length, read twice; a workgroup's dgamma sums live in its row of
// `part`, each column in the hands of one lane.
template <bool BF16, bool H8>
__global__ __launch_bounds__(1024) void k_norm_bwd_long(Bwd a) {
  constexpr int ES = BF16 ? 2 : 4;
  constexpr int T = 1024;
  __shared__ float part[2][T / 64];
  int turn = 0;
  char* out = reinterpret_cast<char*>(a.part + (int64_t)blockIdx.x * a.cols);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const float rstd = a.rstd[r];
    float s = 0.0f;
    for (uint32_t c = threadIdx.x * 8; c < a.cols; c += T * 8) {
      float d[8], x[8], g[8];
      load_chunk<BF16>(a.dy + r * a.ld_dy * ES, c, a.cols, d);
      load_h<BF16, H8>(a, r, c, x);
      load_chunk_rt(a.gamma, a.gamma_bf16, c, a.cols, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = __builtin_fmaf(d[i] * g[i], x[i] * rstd, s);
    }
    const float m = row_sum<T>(s, part, turn) * a.inv_cols;
    turn ^= 1;
    for (uint32_t c = threadIdx.x * 8; c < a.cols; c += T * 8) {
      float d[8], x[8], g[8], q[8], w[8];
      load_chunk<BF16>(a.dy + r * a.ld_dy * ES, c, a.cols, d);
      load_h<BF16, H8>(a, r, c, x);
      load_chunk_rt(a.gamma, a.gamma_bf16, c, a.cols, g);
      load_chunk<BF16>(a.dres + r * a.ld_dres * ES, c, a.dres ? a.cols : 0, q);
      load_chunk<false>(out, c, a.part && r != blockIdx.x ? a.cols : 0, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] *= rstd;
        w[i] = __builtin_fmaf(d[i], x[i], w[i]);
        d[i] = __builtin_fmaf(rstd, __builtin_fmaf(-m, x[i], d[i] * g[i]), q[i]);
      }
      store_chunk<BF16>(a.dx + r * a.ld_dx * ES, c, a.cols, d);
      if (a.part) store_chunk<false>(out, c, a.cols, w);
    }
  }
}

// Sums of the partial rows. A workgroup takes 64 columns, a wave every 16th
// row; the 16 sums are added in order.
__global__ __launch_bounds__(1024) void k_col_reduce(const float* __restrict__ part, int64_t parts, int64_t cols,
                                                      float* __restrict__ out, const uint32_t* __restrict__ max_part,
                                                      int64_t n_max, float* amax) {
  __shared__ float sums[16][64];
  __shared__ uint32_t tops[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (out) {
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < cols) {
      int64_t p = wave;
      for (; p + 112 < parts; p += 128) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = part[(p + 16 * i) * cols + c];
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[i];
      }
      for (; p < parts; p += 16) s += part[p * cols + c];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < cols) {
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) s += sums[i][lane];
      out[c] = s;
    }
  }
  if (amax && blockIdx.x == 0) {
    uint32_t m = 0;
    for (int64_t i = threadIdx.x; i < n_max; i += 1024) m = max(m, max_part[i]);
    m = wave_max(m);
    if (lane == 0) tops[wave] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < 16; ++i) m = max(m, tops[i]);
      *amax = __uint_as_float(m);
    }
  }
}

// Lanes of a launch at most (1024 workgroups of 256, or as many lanes in larger
// ones): each then works through several rows with the next one on its way. More
// workgroups, to the chip's full occupancy and past it, measured the same or up to
// 10% slower (32768 x 4096 bf16 205 us at 1024, 213 to 225 at 1536 to 2048).
// Whole sets of one to each of the 256 CUs.
constexpr int64_t kLanes = 1024 * 256;
constexpr int64_t most_groups(int block) { return kLanes / block / 256 * 256; }

template <bool BF16, bool RES, int T, int NCH>
void run_fwd(const Fwd& a, hipStream_t s) {
  constexpr int BLOCK = T > 256 ? T : 256, PER = BLOCK / T;
  const int64_t want = (a.rows + PER - 1) / PER, cap = most_groups(BLOCK);
  const uint32_t g = (uint32_t)(want < cap ? want : cap);
  if (a.amax && g > 1) hipLaunchKernelGGL(k_zero_amax, dim3(1), dim3(1), 0, s, a.amax);
  constexpr int ES = BF16 ? 2 : 4;
  if (streaming(a.rows, a.cols, ES, rows_on_16(a.h, a.ld_h, ES) && rows_on_16(a.y, a.ld_y, ES)))
    hipLaunchKernelGGL((k_norm<BF16, RES, T, NCH, true>), dim3(g), dim3(BLOCK), 0, s, a);
  else
    hipLaunchKernelGGL((k_norm<BF16, RES, T, NCH, false>), dim3(g), dim3(BLOCK), 0, s, a);
}

// Lanes and chunks by the row's length. A wave alone needs no barrier; from 1024
// columns on a row is spread over as many lanes as a workgroup has, which leaves
// registers for the row ahead (32768 x 4096 bf16: 512 lanes of one chunk 205 us,
// 256 of two 214; 4000 x 5003 fp32: 1024 of one 72, 512 of two 80). Two chunks are
// better where a bf16 row would leave a single workgroup of 1024 on a CU (4096 x
// 8192: 512 of two 48, 1024 of one 54).
template <bool BF16, bool RES>
void pick_fwd(const Fwd& a, hipStream_t s) {
  if (a.cols <= 512) run_fwd<BF16, RES, 64, 1>(a, s);
  else if (a.cols <= 1024) run_fwd<BF16, RES, 64, 2>(a, s);
  else if (a.cols <= 2048) run_fwd<BF16, RES, 256, 1>(a, s);
  else if (a.cols <= 4096) run_fwd<BF16, RES, 512, 1>(a, s);
  else if (a.cols <= 8192) run_fwd<BF16, RES, BF16 ? 512 : 1024, BF16 ? 2 : 1>(a, s);
  else if (a.cols <= 16384) run_fwd<BF16, RES, 1024, 2>(a, s);
  else {
    const uint32_t g = (uint32_t)(a.rows < 512 ? a.rows : 512);
    if (a.amax && g > 1) hipLaunchKernelGGL(k_zero_amax, dim3(1), dim3(1), 0, s, a.amax);
    hipLaunchKernelGGL((k_norm_long<BF16, RES>), dim3(g), dim3(1024), 0, s, a);
  }
}

// Workgroups of the backward pass, each leaving one partial row: 1024 of 256
// lanes hold the chip's registers, and their partial rows stay a few percent of
// what the pass moves.
struct BwdShape {
  int t, per;
  int64_t grid;
};
// 768 lanes leave a bf16 row registers for two chunks and gamma (8192 x 11008 bf16 129
// us; 1024 lanes, whose 128 registers push gamma into LDS, 148). What does not fit all
// the same goes to scratch memory: fp32 rows 20 B a lane of 768 with h in 8 bits and 68
// with h as a matrix (8192 x 11008 263 us, 4.1 TB/s), 184 and 216 B of 1024 (4096 x
// 16384 343 us, 2.4 TB/s); bf16 rows 36 and 24 B of 1024 (4096 x 16384 from 8 bits 90
// us, 3.8 TB/s).
BwdShape bwd_shape(int64_t rows, int64_t cols) {
  BwdShape b;
  b.t = cols <= 512 ? 64 : cols <= 2048 ? 256 : cols <= 4096 ? 512 : cols > 8192 && cols <= 12288 ? 768 : 1024;
  b.per = b.t < 256 ? 256 / b.t : 1;
  const int64_t want = (rows + b.per - 1) / b.per, cap = most_groups(b.t < 256 ? 256 : b.t);
  b.grid = want < cap ? want : cap;
  return b;
}

template <bool BF16, bool H8, bool NT>
void pick_bwd(const Bwd& a, hipStream_t s) {
  const BwdShape b = bwd_shape(a.rows, a.cols);
  const dim3 g((uint32_t)b.grid);
  if (a.cols <= 512) hipLaunchKernelGGL((k_norm_bwd<BF16, H8, 64, 1, NT>), g, dim3(256), 0, s, a);
  else if (a.cols <= 2048) hipLaunchKernelGGL((k_norm_bwd<BF16, H8, 256, 1, NT>), g, dim3(256), 0, s, a);
  else if (a.cols <= 4096) hipLaunchKernelGGL((k_norm_bwd<BF16, H8, 512, 1, NT>), g, dim3(512), 0, s, a);
  else if (a.cols <= 8192) hipLaunchKernelGGL((k_norm_bwd<BF16, H8, 1024, 1, NT>), g, dim3(1024), 0, s, a);
  else if (a.cols <= 12288) hipLaunchKernelGGL((k_norm_bwd<BF16, H8, 768, 2, NT>), g, dim3(768), 0, s, a);
  else if (a.cols <= 16384) hipLaunchKernelGGL((k_norm_bwd<BF16, H8, 1024, 2, NT>), g, dim3(1024), 0, s, a);
  else hipLaunchKernelGGL((k_norm_bwd_long<BF16, H8>), g, dim3(1024), 0, s, a);
}
template <bool BF16, bool H8>
void pick_bwd(const Bwd& a, hipStream_t s) {
  if (streaming(a.rows, a.cols, BF16 ? 2 : 4, rows_on_16(a.dx, a.ld_dx, BF16 ? 2 : 4))) pick_bwd<BF16, H8, true>(a, s);
  else pick_bwd<BF16, H8, false>(a, s);
}

}  // namespace

void fp4i_launch_rmsnorm(const fp4_rmsnorm_fwd& n, hipStream_t s) {
  Fwd a;
  a.x = static_cast<const char*>(n.x);
  a.res = static_cast<const char*>(n.residual);
  a.ld_x = n.ld_x;
  a.ld_res = n.ld_residual;
  a.gamma = n.gamma;
  a.h = static_cast<char*>(n.h);
  a.y = static_cast<char*>(n.y);
  a.ld_h = n.ld_h;
  a.ld_y = n.ld_y;
  a.y8 = n.y8 ? Mx8Out{n.y8->codes, n.y8->scales, n.y8->ld, n.y8->lds} : Mx8Out{nullptr, nullptr, 0, 0};
  a.h8 = n.h8 ? Mx8Out{n.h8->codes, n.h8->scales, n.h8->ld, n.h8->lds} : Mx8Out{nullptr, nullptr, 0, 0};
  a.rstd = n.rstd;
  a.amax = n.amax;
  a.rows = n.rows;
  a.cols = (uint32_t)n.cols;
  a.inv_cols = 1.0f / (float)n.cols;
  a.eps = n.eps;
  a.gamma_bf16 = n.gamma_t == FP4_DTYPE_BF16;
  if (n.dtype == FP4_DTYPE_BF16) {
    if (n.residual) pick_fwd<true, true>(a, s);
    else pick_fwd<true, false>(a, s);
  } else {
    if (n.residual) pick_fwd<false, true>(a, s);
    else pick_fwd<false, false>(a, s);
  }
}

int64_t fp4i_rmsnorm_bwd_parts(int64_t rows, int64_t cols) { return bwd_shape(rows, cols).grid; }

void fp4i_launch_rmsnorm_bwd(const fp4_rmsnorm_bwd& n, hipStream_t s) {
  const int64_t parts = fp4i_rmsnorm_bwd_parts(n.rows, n.cols);
  Bwd a;
  a.dy = static_cast<const char*>(n.dy);
  a.h = static_cast<const char*>(n.h);
  a.dres = static_cast<const char*>(n.dres);
  a.ld_dy = n.ld_dy;
  a.ld_h = n.ld_h;
  a.ld_dres = n.ld_dres;
  a.h8 = n.h8 ? Mx8In{n.h8->codes, n.h8->scales, n.h8->ld, n.h8->lds} : Mx8In{nullptr, nullptr, 0, 0};
  a.gamma = n.gamma;
  a.rstd = n.rstd;
  a.dx = static_cast<char*>(n.dx);
  a.ld_dx = n.ld_dx;
  a.part = !n.dgamma ? nullptr : parts > 1 ? static_cast<float*>(n.ws) : n.dgamma;
  a.rows = n.rows;
  a.cols = (uint32_t)n.cols;
  a.inv_cols = 1.0f / (float)n.cols;
  a.gamma_bf16 = n.gamma_t == FP4_DTYPE_BF16;
  if (n.dtype == FP4_DTYPE_BF16) {
    if (n.h8) pick_bwd<true, true>(a, s);
    else pick_bwd<true, false>(a, s);
  } else {
    if (n.h8) pick_bwd<false, true>(a, s);
    else pick_bwd<false, false>(a, s);
  }
  if (n.dgamma && parts > 1)
    fp4i_launch_col_reduce(a.part, parts, n.cols, n.dgamma, nullptr, 0, nullptr, s);
}

void fp4i_launch_col_reduce(const float* part, int64_t parts, int64_t cols, float* out, const uint32_t* max_part,
                            int64_t n_max, float* amax, hipStream_t s) {
  const uint32_t g = out ? (uint32_t)((cols + 63) / 64) : 1u;
  hipLaunchKernelGGL(k_col_reduce, dim3(g), dim3(1024), 0, s, part, parts, cols, out, max_part, n_max, amax);
}
