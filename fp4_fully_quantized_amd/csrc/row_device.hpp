// row_device.hpp -- device helpers of the row-wise kernels (mx8.hip, norm.hip,
// act.hip) and of the product's epilogue: 8-column chunks of a row, the 8-bit
// block format, activations and workgroup reductions.
//
// A row is cut into chunks of 8 columns and a lane holds whole chunks, so four
// neighbouring lanes hold one 32-column block of the 8-bit format and its
// maximum takes two DPP exchanges. Chunks are read and written with 16-byte
// accesses at element alignment: gfx950 does these unaligned in hardware, so
// odd leading dimensions and sub-matrices run on the same code; only the last,
// partial chunk of a row goes element by element.
#pragma once
#include "fp4_device.hpp"

namespace fp4row {

using namespace fp4dev;

typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u_e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned v4u_e4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight elements as they lie in memory. Kernels that load the next row ahead keep
// it in this form: half the registers for bf16.
template <bool BF16>
struct Raw8 {
  v4u w[BF16 ? 1 : 2];
};
struct RawMx8 {
  uint2 w;
  uint32_t byte;
};

template <bool BF16>
__device__ __forceinline__ void expand(const Raw8<BF16>& r, float x[8]) {
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(r.w[0][i]);
      x[2 * i + 1] = bf16_hi(r.w[0][i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r.w[i / 4][i % 4]);
  }
}

// NT: the access is marked as not to be kept in the caches (streaming()).
template <bool NT, class V>
__device__ __forceinline__ v4u load16(const char* p) {
  if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
  else return *reinterpret_cast<const V*>(p);
}
template <bool NT, class V>
__device__ __forceinline__ void store16(char* p, v4u v) {
  if constexpr (NT) __builtin_nontemporal_store((V)v, reinterpret_cast<V*>(p));
  else *reinterpret_cast<V*>(p) = v;
}

template <bool BF16, bool NT = false>
__device__ __forceinline__ Raw8<BF16> raw8_any(const char* p) {
  Raw8<BF16> r;
  if constexpr (BF16) {
    r.w[0] = load16<NT, v4u_e2>(p);
  } else {
    r.w[0] = load16<NT, v4u_e4>(p);
    r.w[1] = load16<NT, v4u_e4>(p + 16);
  }
  return r;
}

// Columns c .. c + 7 of the row at p, zeros from column n on.
template <bool BF16, bool NT = false>
__device__ __forceinline__ Raw8<BF16> raw_chunk(const char* p, uint32_t c, uint32_t n) {
  constexpr int ES = BF16 ? 2 : 4;
  if (c + 8 <= n) return raw8_any<BF16, NT>(p + (uint32_t)(c * ES));
  Raw8<BF16> r;
#pragma unroll
  for (int h = 0; h < (BF16 ? 1 : 2); ++h) r.w[h] = (v4u){0, 0, 0, 0};
  if (c < n) {
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      if (c + i < n) {
        if constexpr (BF16) r.w[0][i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[c + i] << (16 * (i % 2));
        else r.w[i / 4][i % 4] = reinterpret_cast<const uint32_t*>(p)[c + i];
      }
    }
  }
  return r;
}
template <bool BF16, bool NT = false>
__device__ __forceinline__ void load_chunk(const char* p, uint32_t c, uint32_t n, float x[8]) {
  expand<BF16>(raw_chunk<BF16, NT>(p, c, n), x);
}

// As load_chunk, the type known at run time (gamma and bias, read rarely).
__device__ __forceinline__ void load_chunk_rt(const void* p, bool bf16, uint32_t c, uint32_t n, float x[8]) {
  if (bf16) load_chunk<true>(static_cast<const char*>(p), c, n, x);
  else load_chunk<false>(static_cast<const char*>(p), c, n, x);
}

// Two FP32 values to one word of bf16, each rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){a, b}, v2bf));
}

template <bool BF16, bool NT = false>
__device__ __forceinline__ void store8_any(char* d, const float x[8]) {
  if constexpr (BF16) {
    store16<NT, v4u_e2>(d, (v4u){pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])});
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      store16<NT, v4u_e4>(d + 16 * h, (v4u){__float_as_uint(x[4 * h]), __float_as_uint(x[4 * h + 1]),
                                            __float_as_uint(x[4 * h + 2]), __float_as_uint(x[4 * h + 3])});
  }
}

template <bool BF16, bool NT = false>
__device__ __forceinline__ void store_chunk(char* p, uint32_t c, uint32_t n, const float x[8]) {
  constexpr int ES = BF16 ? 2 : 4;
  if (c + 8 <= n) {
    store8_any<BF16, NT>(p + (uint32_t)(c * ES), x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c + i >= n) break;
      if constexpr (BF16) reinterpret_cast<uint16_t*>(p)[c + i] = (uint16_t)pack_bf16(x[i], x[i]);
      else reinterpret_cast<float*>(p)[c + i] = x[i];
    }
  }
}

// max |x| over the values that are no NaN, 0 if none (the maximum of a number and a
// NaN is the number, so it starts from one; the sign is dropped for free, unlike in
// integers). A signalling NaN, which only memory can hold, is made quiet first: the
// instruction would return it. On values that were computed that costs nothing.
__device__ __forceinline__ float number_max8(const float x[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(__builtin_canonicalizef(x[i])));
  return m;
}
// The bits of that maximum: magnitudes of floats order as unsigned integers.
__device__ __forceinline__ uint32_t number_max8_bits(const float x[8]) { return __float_as_uint(number_max8(x)); }
// A maximum of values as bf16 stores them, from that of the values (rounding keeps
// the order).
__device__ __forceinline__ uint32_t bf16_bits(uint32_t m) { return pack_bf16(0.0f, __uint_as_float(m)) & 0xFFFF0000u; }

// ---- 8 bits: E4M3 values, one E8M0 byte per 32 -----------------------------
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));
  return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));
}

// Scale byte of a block whose largest magnitude has the bits m: e + 127 with e
// the smallest exponent for which 448 * 2^e = 1.75 * 2^(e + 8) >= max. With m's
// exponent field F, e + 127 = F - 8, or F - 7 where the mantissa exceeds .75
// (the addition below carries into the field exactly then), 0 at least; 255
// for an infinity.
__device__ __forceinline__ uint32_t mx8_byte(uint32_t m) {
  const int b = (int)((m + 0x1FFFFFu) >> 23) - 8;
  return m >= 0x7F800000u ? 255u : (uint32_t)(b > 0 ? b : 0);
}
// 2^-e (always a normal number: the byte is at most 247), NaN for byte 255.
__device__ __forceinline__ float mx8_factor(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : (254u - byte) << 23);
}
// 2^e (subnormal for byte 0), NaN for byte 255.
__device__ __forceinline__ float mx8_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
}
__device__ __forceinline__ uint2 mx8_pack8(const float x[8], float f) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * f, x[1] * f, lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * f, x[3] * f, lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * f, x[5] * f, hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] * f, x[7] * f, hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}
__device__ __forceinline__ void mx8_unpack8(uint2 w, float s, float x[8]) {
  const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, true);
  const v2f c = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, false), d = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, true);
  x[0] = a[0] * s; x[1] = a[1] * s; x[2] = b[0] * s; x[3] = b[1] * s;
  x[4] = c[0] * s; x[5] = c[1] * s; x[6] = d[0] * s; x[7] = d[1] * s;
}

struct Mx8Out {
  uint8_t* codes;  // null: not wanted
  uint8_t* scales;
  int64_t ld, lds;
};
struct Mx8In {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t ld, lds;
};

// Stores the chunk at column c of row r in 8 bits. The four lanes of a block
// call it together (zeros, or NaN, past the last column); a lane whose block lies
// past the row stores nothing. Returns the scale byte.
template <bool NT = false>
__device__ __forceinline__ uint32_t mx8_store(const Mx8Out& q, int64_t r, uint32_t c, uint32_t n, const float x[8],
                                              uint32_t& block_mag) {
  block_mag = quad_max(number_max8_bits(x));
  const uint32_t byte = mx8_byte(block_mag);
  uint2 w = mx8_pack8(x, mx8_factor(byte));
  if (c + 8 > n) {
    // Codes past the last column are zeros whatever x holds there (a norm's row whose
    // rstd is not finite) and whatever its factor is (byte 255's NaN).
    const uint32_t k = n > c ? n - c : 0;
    w.x &= k >= 4 ? ~0u : (1u << 8 * k) - 1;
    w.y &= k >= 4 ? (1u << 8 * (k - 4)) - 1 : 0u;
  }
  if ((c & ~31u) < n) {
    v2u* const d = reinterpret_cast<v2u*>(q.codes + r * q.ld + c);
    if constexpr (NT) __builtin_nontemporal_store((v2u){w.x, w.y}, d);
    else *d = (v2u){w.x, w.y};
    if ((c & 31) == 0) q.scales[r * q.lds + (c >> 5)] = (uint8_t)byte;
  }
  return byte;
}
template <bool NT = false>
__device__ __forceinline__ RawMx8 mx8_raw(const Mx8In& q, int64_t r, uint32_t c, uint32_t n) {
  RawMx8 v = {make_uint2(0, 0), 0};
  if (c < n) {
    const v2u* const p = reinterpret_cast<const v2u*>(q.codes + r * q.ld + c);
    v2u w;
    if constexpr (NT) w = __builtin_nontemporal_load(p);
    else w = *p;
    v.w = make_uint2(w.x, w.y);
    v.byte = q.scales[r * q.lds + (c >> 5)];
  }
  return v;
}
// Zeros from column n on (what lies there in the codes is the caller's).
__device__ __forceinline__ void expand(const RawMx8& v, uint32_t c, uint32_t n, float x[8]) {
  mx8_unpack8(v.w, mx8_scale(v.byte), x);
  if (c + 8 > n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i >= n) x[i] = 0.0f;
  }
}
template <bool NT = false>
__device__ __forceinline__ void mx8_load(const Mx8In& q, int64_t r, uint32_t c, uint32_t n, float x[8]) {
  expand(mx8_raw<NT>(q, r, c, n), c, n, x);
}

// ---- activations -----------------------------------------------------------
constexpr int ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_SILU = 3;
constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// 1 / (1 + e^-t) is taken with the hardware's base-2 exponential and reciprocal
// (1 ulp each; the argument's rounding adds |t| 2^-24 relative). Far left the
// exponential is infinite and the result 0.
// relu keeps NaN; gelu and silu are z sigmoid(t), with the base-2 exponent's
// factor folded into gelu's constants.
__device__ __forceinline__ void act8(int act, float z[8]) {
  constexpr float kLog2e = 1.4426950408889634f;
  if (act == ACT_RELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = z[i] < 0.0f ? 0.0f : z[i];
  } else if (act == ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = z[i] * __builtin_fmaf(-kGelu2C * kGeluA * kLog2e, z[i] * z[i], -kGelu2C * kLog2e);
      z[i] *= __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u));
    }
  } else if (act == ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z[i] * -kLog2e));
  }
}

// act'(z) = s + z t'(z) s (1 - s) with s = sigmoid(t(z)). From e = e^-|t|: s (1 - s)
// = e / (1 + e)^2 without the difference 1 - s, which would leave few digits
// where s is near 1. z t' is kept finite, so that it drops out where e is 0 (a NaN
// comes through s).
__device__ __forceinline__ float slope(float z, float u, float rate) {
  const float e = __builtin_amdgcn_exp2f(-__builtin_fabsf(u));  // u = -t log2(e)
  const float p = __builtin_amdgcn_rcpf(1.0f + e), q = e * p;
  const float zr = __builtin_amdgcn_fmed3f(z * rate, -1e30f, 1e30f);
  return __builtin_fmaf(zr, q * p, u > 0.0f ? q : p);
}
__device__ __forceinline__ void act_slope8(int act, float z[8]) {
  constexpr float kLog2e = 1.4426950408889634f;
  if (act == ACT_RELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = z[i] > 0.0f ? 1.0f : z[i] == z[i] ? 0.0f : z[i];
  } else if (act == ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float z2 = z[i] * z[i];
      z[i] = slope(z[i], z[i] * __builtin_fmaf(-kGelu2C * kGeluA * kLog2e, z2, -kGelu2C * kLog2e),
                   __builtin_fmaf(3.0f * kGelu2C * kGeluA, z2, kGelu2C));
    }
  } else if (act == ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = slope(z[i], z[i] * -kLog2e, 1.0f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = 1.0f;
  }
}

// Whether a pass over a rows x cols matrix of es-byte values marks its accesses as
// not to be kept (NT). A matrix of more than 160 MiB, read and written, is past what
// the 256 MiB cache before HBM can hold between calls, and keeping parts of it only
// pushes out what others left there: 32768 x 11008 bf16, act backward 384 -> 345 us,
// to 8 bits 266 -> 249; a norm of 32768 x 4096 and the quantization that reads it
// 363 -> 310. A smaller one finds its input there, and leaves its output, when it
// does not (norm of 16384 x 1024 28 us against 32). Rows that do not start on 16
// bytes are written in parts of lines, which then have to meet in the caches (8 bits
// to 16384 x 5003 fp32 129 us marked, 100 not).
inline bool rows_on_16(const void* p, int64_t ld, int es) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0);
}
inline bool streaming(int64_t rows, int64_t cols, int es, bool outputs_on_16) {
  return outputs_on_16 && rows * cols * es >= int64_t(160) << 20;
}

// ---- reductions ------------------------------------------------------------
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  return v;
}

}  // namespace fp4row
