// gemm_rows.hip -- the FP4 product with its epilogue where the tiled kernel has too
// few 256 x 256 tiles for the chip: the tokens of a serving loop against a weight
// matrix, a small batch, a narrow layer.
//
//   z[i][j] = alpha sum_k A[i][k] B[j][k] + bias[j];  C = act(z) + residual
//
// Few rows are bound by reading B once (0.56 or 0.53 bytes a value), so the kernel
// is made to keep loads in flight, not to reuse tiles: a workgroup owns 16 MT rows
// and 16 NT columns of the output, its waves split K between them, and every wave
// loads its operands straight into the registers of the MFMAs (16x16, so one row
// costs no more than 16). The waves' partial sums meet in LDS, are added in wave
// order and go through the epilogue there: one launch, no workspace.
//
// K is cut into steps of 128 values, a wave's steps one after the other. The MFMA
// wants neighbouring lanes to hold different rows; loaded so, every lane's 16 bytes
// are an access of their own, and the 26,000 accesses of a 64 x 64 x 4096 tile took
// most of its 35,000 cycles. So a wave loads four lanes to a row (64 bytes of codes
// in one access; the scales of four steps at once), and turns lanes into rows
// through an LDS area of its own, which needs no barrier: a wave's LDS accesses run
// in order, and the compiler keeps that of a fragment's store and load, whose addresses
// are the same in some lanes (a wave-wide fence between them changed no result and cost
// up to 10%: NVFP4 128 x 11008 x 4096 23.9 -> 26.5 us). NVFP4 is decoded to f16 exactly
// and MXFP4 runs on the scaled FP4 MFMA, as in the tiled kernels.
#include "epilogue.hpp"
#include "fp4_device.hpp"

#include <algorithm>
#include <type_traits>

using namespace fp4dev;

namespace {

constexpr int NV = 0;
constexpr int MX = 1;

// NVFP4: eight values (code word q) of a lane's 32, whose two scales are sd, as an
// f16 operand.
__device__ __forceinline__ v8h decode_nv(const v4u& code, v2h sd, int q) {
  const uint32_t w = code[q];
  const v2h m = q < 2 ? sd.xx : sd.yy;
  const v2h h0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * m;
  const v2h h1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * m;
  const v2h h2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * m;
  const v2h h3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * m;
  return (v8h){h0[0], h0[1], h1[0], h1[1], h2[0], h2[1], h3[0], h3[1]};
}

__device__ __forceinline__ v4f mfma_mx16(const v4u& a, const v4u& b, const v4f& c, uint32_t sa, uint32_t sb) {
  const v8i av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const v8i bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// Most waves of a workgroup: 16 need at most 128 registers a lane, 8 twice that.
constexpr int max_waves(int fragments) { return fragments == 1 ? 16 : 8; }

// LDS of a wave, bytes: a step's codes (16 rows of 64 for each fragment) and four
// steps' scales (NVFP4 8, MXFP4 4 a row and step).
constexpr int codes_lds(int frags) { return frags * 1024; }
constexpr int wave_lds(int frags, int fmt) { return codes_lds(frags) + frags * 16 * 4 * (fmt == NV ? 8 : 4); }

// A bijection on [0, n) that gives each of the 8 XCDs (workgroup b runs on b % 8)
// one range.
__device__ __forceinline__ uint32_t xcd_range(uint32_t b, uint32_t n) {
  const uint32_t x = b % 8, per = n / 8, rem = n % 8;
  return x * per + min(x, rem) + b / 8;
}

template <int FMT, int MT, int NT>
__global__ __launch_bounds__((64 * max_waves(MT * NT))) void k_gemm_rows(const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as,
                                                     const uint8_t* __restrict__ bc, const uint8_t* __restrict__ bs,
                                                     const float* __restrict__ a_ts, const float* __restrict__ b_ts,
                                                     uint32_t M, uint32_t N, uint32_t K, bool obf, int64_t ldc,
                                                     EpiOf<true> epi) {
  extern __shared__ v4f red[];  // [waves][MT * NT][64]; before that the waves' areas
  constexpr int F = MT + NT;    // fragments: A's, then B's
  constexpr uint32_t SB = FMT == NV ? 8 : 4;     // scale bytes of a row and step
  typedef std::conditional_t<FMT == NV, fp4row::v2u, uint32_t> ScaleWord;  // read back as bytes and halves
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, lr = lane & 15;
  // Workgroups go round robin over the 8 XCDs; each XCD takes one range of the
  // columns, all rows of a set of columns in turn, so that B is read from HBM into
  // one L2.
  const uint32_t tile = xcd_range(blockIdx.x, gridDim.x), sets = (M + 16 * MT - 1) / (16 * MT);
  const uint32_t n0 = tile / sets * (16 * NT), m0 = tile % sets * (16 * MT);

  // Loads: lane 4 r + p takes part p of row r of a fragment. Byte offsets (an
  // operand's codes stay below 2^31 bytes); rows past the last read the last, their
  // sums are not used.
  const uint32_t lrow = lane >> 2, part = lane & 3;
  uint32_t coff[F], soff[F];
#pragma unroll
  for (int i = 0; i < F; ++i) {
    const uint32_t row = i < MT ? min(m0 + i * 16 + lrow, M - 1) : min(n0 + (i - MT) * 16 + lrow, N - 1);
    coff[i] = row * (K / 2) + part * 16;
    soff[i] = row * (K / 128 * SB);
  }
  const int steps = (int)(K / 128), first = wave * steps / waves, last = (wave + 1) * steps / waves;

  // The wave's area. A row's four parts are permuted by (row / 4), so that 16 lanes
  // reading one part of 16 rows hit all banks once.
  uint8_t* const area = reinterpret_cast<uint8_t*>(red) + wave * wave_lds(F, FMT);
  uint8_t* const put = area + lrow * 64 + (part ^ (lrow >> 2)) * 16;
  const uint8_t* const get = area + lr * 64 + (g ^ (lr >> 2)) * 16;
  uint8_t* const sput = area + codes_lds(F) + lane * SB;
  const uint8_t* const sget = area + codes_lds(F) + lr * (4 * SB) + g * (SB / 4);

  v4f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = (v4f){0, 0, 0, 0};

  struct Codes {
    v4u v[F];
  };
  auto load_codes = [&](Codes& c, int st) {
#pragma unroll
    for (int i = 0; i < F; ++i)
      c.v[i] = *reinterpret_cast<const v4u*>((i < MT ? ac : bc) + st * 64 + coff[i]);
  };
  ScaleWord scales[F];  // of the four steps from `st` on, part p those of step st + p
  auto load_scales = [&](int st) {
    const uint32_t at = (uint32_t)min(st + (int)part, last - 1) * SB;
#pragma unroll
    for (int i = 0; i < F; ++i) scales[i] = *reinterpret_cast<const ScaleWord*>((i < MT ? as : bs) + at + soff[i]);
  };

  // The next step is on its way while one is multiplied. Two ahead: NVFP4 128 x 4096 x
  // 4096 on 32 x 32 11.9 -> 12.9 us, 64 x 11008 x 4096 on 64 x 32 17.6 -> 20.0; it won
  // (up to 15%) only at thousands of rows, where the tiled kernel runs.
  Codes next;
  load_scales(first);
  load_codes(next, first);
#pragma unroll 1
  for (int st = first; st < last; ++st) {
    const int in4 = (st - first) & 3;
    if (in4 == 0) {
#pragma unroll
      for (int i = 0; i < F; ++i) *reinterpret_cast<ScaleWord*>(sput + i * (64 * SB)) = scales[i];
      load_scales(min(st + 4, last - 1));
    }
#pragma unroll
    for (int i = 0; i < F; ++i) *reinterpret_cast<v4u*>(put + i * 1024) = next.v[i];
    load_codes(next, min(st + 1, last - 1));

    v4u code[F];
    uint32_t sc[F];
#pragma unroll
    for (int i = 0; i < F; ++i) {
      code[i] = *reinterpret_cast<const v4u*>(get + i * 1024);
      const uint8_t* const q = sget + i * (64 * SB) + in4 * SB;
      if constexpr (FMT == NV) sc[i] = *reinterpret_cast<const uint16_t*>(q);
      else sc[i] = *q;
    }
    if constexpr (FMT == MX) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = mfma_mx16(code[MT + n], code[m], acc[m][n], sc[MT + n], sc[m]);
    } else {
      v2h sd[F];
#pragma unroll
      for (int i = 0; i < F; ++i) sd[i] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sc[i], 1.0f, false);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v8h bo[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) bo[n] = decode_nv(code[MT + n], sd[MT + n], q);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const v8h ao = decode_nv(code[m], sd[m], q);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(bo[n], ao, acc[m][n], 0, 0, 0);
        }
      }
    }
  }
  __syncthreads();  // every wave is done with its area

  // The B fragment comes first in the MFMA, so lane l of fragment (m, n) holds
  // row 16 m + l % 16 and columns 16 n + 4 (l / 16) .. + 3.
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) red[(wave * (MT * NT) + m * NT + n) * 64 + lane] = acc[m][n];
  __syncthreads();
  float alpha = 1.0f;
  if constexpr (FMT == NV) alpha = (*a_ts) * (*b_ts);
  constexpr uint32_t CH = 2 * NT;  // chunks of 8 columns
  const uint32_t rows = min(M - m0, (uint32_t)(16 * MT));
  for (uint32_t t = threadIdx.x; t < rows * CH; t += blockDim.x) {
    const uint32_t r = t / CH, row = m0 + r, ch = t % CH, col = n0 + ch * 8;
    const int at = ((r / 16) * NT + ch / 2) * 64 + (ch & 1) * 32 + r % 16;
    float bias[8], res[8];
    fp4row::load_chunk_rt(epi.bias, epi.bias_bf16, col, epi.bias ? N : 0, bias);
    epi_residual8(epi, row, col, M, N, res);
    v4f lo = red[at], hi = red[at + 16];
    for (int w = 1; w < waves; ++w) {
      lo += red[w * (MT * NT * 64) + at];
      hi += red[w * (MT * NT * 64) + at + 16];
    }
    float z[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    epi_row8(epi, z, bias, res, alpha, row, col, M, N, obf, ldc);
  }
}

template <int FMT, int MT, int NT>
void launch(const GemmArgs& g, const EpiOf<true>& e, hipStream_t s) {
  const uint32_t tiles = (uint32_t)((g.N + 16 * NT - 1) / (16 * NT) * ((g.M + 16 * MT - 1) / (16 * MT)));
  const uint32_t steps = (uint32_t)(g.K / 128);
  // Waves: about 16 for each of the 256 CUs in all, as far as K has steps for
  // them.
  uint32_t waves = 1;
  while (waves < (uint32_t)max_waves(MT * NT) && tiles * waves < 4096 && 2 * waves <= steps) waves *= 2;
  const uint32_t lds = waves * (uint32_t)std::max(wave_lds(MT + NT, FMT), MT * NT * 1024);
  hipLaunchKernelGGL((k_gemm_rows<FMT, MT, NT>), dim3(tiles), dim3(64 * waves), lds, s, g.a_codes, g.a_scales,
                     g.b_codes, g.b_scales, g.a_tscale, g.b_tscale, (uint32_t)g.M, (uint32_t)g.N, (uint32_t)g.K,
                     g.bf16out, g.ldc, e);
}

// What a product takes on a shape of this kernel, in us: a start, and for every 256
// workgroups (one to a CU) a part that does not and a part that does grow with K.
// Fitted to a sweep made before every shape loaded one step ahead; the kernel now
// takes 0.63 to 1.5 of these times, and the order between the shapes, which is what
// they are for, mostly stands. Over M = 1 .. 2048 by 4096 x 4096, 11008 x 4096, 4096 x
// 11008, 2560 x 8192, 1000 x 1280, 2048 x 640 and 8192 x 640 (N x K), both formats,
// what is picked is within 10% of the best shape (or the tiled kernel) in 138 of 168
// and 2% slower in the median; the worst are at K = 640 (fp4i_gemm_rows_pays) and
// 1000 x 1280 (2048 rows NVFP4 18.4 us on 64 x 64, 13.2 on 64 x 32). NVFP4 x 4096 x
// 4096 on the shapes in order, replays of a graph over three weight matrices: 64 rows
// 10.4, 9.2, 8.0, 10.2 and 13.8 us; 512 rows 55, 41, 31, 28 and 28.
struct Shape {
  int mt, nt;
  double nv, mx;   // us per 256 workgroups at K = 4096
};
constexpr Shape kShapes[] = {{1, 1, 1.55, 1.05}, {1, 2, 2.4, 1.8}, {2, 2, 4.1, 2.6}, {4, 2, 6.0, 3.8}, {4, 4, 11.2, 6.2}};
constexpr double kStartUs = 5.0;

double shape_us(const Shape& h, int64_t M, int64_t N, int64_t K, bool nv) {
  const double groups = (double)((M + 16 * h.mt - 1) / (16 * h.mt)) * (double)((N + 16 * h.nt - 1) / (16 * h.nt));
  // The two large shapes run one workgroup to a CU: whole rounds.
  double rounds = std::max(1.0, groups / 256);
  if (h.mt == 4) rounds = (double)(int64_t)(rounds + 0.999);
  return kStartUs + rounds * (nv ? h.nv : h.mx) * (0.12 + 0.88 * (double)K / 4096);
}
int best_shape(int64_t M, int64_t N, int64_t K, bool nv, bool wide) {
  int best = wide ? 1 : 0;   // the 8-bit form needs 32 columns in one workgroup
  for (int i = best + 1; i < 5; ++i)
    if (shape_us(kShapes[i], M, N, K, nv) < shape_us(kShapes[best], M, N, K, nv)) best = i;
  return best;
}

template <int FMT>
void pick_shape(const GemmArgs& g, const EpiOf<true>& e, hipStream_t s) {
  switch (best_shape(g.M, g.N, g.K, FMT == NV, e.z8.codes)) {
    case 0: return launch<FMT, 1, 1>(g, e, s);
    case 1: return launch<FMT, 1, 2>(g, e, s);
    case 2: return launch<FMT, 2, 2>(g, e, s);
    case 3: return launch<FMT, 4, 2>(g, e, s);
    default: return launch<FMT, 4, 4>(g, e, s);
  }
}

}  // namespace

// Whether the product takes this kernel: the tiled one's time is that of its K
// tiles (256 values: 4.7 us NVFP4, 1.45 MXFP4, whatever the number of tiles up to
// one to a CU) after a start and an epilogue of 8 and 7 us. NVFP4 x 4096 x 4096 (N x
// K), this kernel against that with the same epilogue, measured as above: 64 rows 8.2
// us and 45, 512 28 and 47, 1024 47 and 75, 1536 67 and 76, 2048 94 and 76; MXFP4 128
// rows 7.6 and 25, 512 19 and 26, 1024 27.7 and 28.8, 1536 40 and 30. Too low for the
// tiled kernel where K is no multiple of 256 (its K tile is then 128): MXFP4 512 x 8192
// x 640 takes 18.4 us there, 9.8 on 64 x 32; 2048 x 2048 x 640 18.2 and 9.9.
bool fp4i_gemm_rows_pays(int64_t M, int64_t N, int64_t K, int fmt) {
  const bool nv = fmt == NV;
  const TilePlan p = fp4i_gemm_tiles(M, N, K);
  const double one = (double)K / 256 * (nv ? 4.7 : 1.45);
  const double tiled = (nv ? 8.0 : 7.0) + (double)((p.whole + 255) / 256) * one + (p.split > 1 ? one / p.split + 5 : 0);
  return shape_us(kShapes[best_shape(M, N, K, nv, false)], M, N, K, nv) < tiled;
}

void fp4i_launch_gemm_rows(const GemmArgs& g, const fp4_epilogue& f, hipStream_t s) {
  const EpiOf<true> e = epi_args(f, g.c);
  if (g.fmt == NV) pick_shape<NV>(g, e, s);
  else pick_shape<MX>(g, e, s);
}
