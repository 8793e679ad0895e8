// zn_mx.h -- microscaled numbers: constants and device helpers shared by the
// quantiser, the norm and the product, and their launch interface.
//
// A row of K values is stored as Kp = 32 * ceil(K / 32) codes (the rest zero)
// and one scale byte s per 32 codes: a value is code * 2^(s - 127), s = 255 a
// NaN.  Codes are E4M3 bytes (zn_dtype FP8) or E2M1 nibbles (FP4X2).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zn_common.h"

namespace zn {

constexpr uint32_t kMxBlock = 32;
constexpr uint64_t kMxMaxK = 1ull << 30;       // longest row
constexpr uint64_t kMxMaxRows = 0x7FFFFFFFull;  // most rows

struct MxQuantArgs {
  const uint8_t *x;      // [rows] rows of k elements, x_stride elements apart
  uint64_t rows, k, x_stride;
  uint8_t *codes, *scales;
};
struct MxDequantArgs {
  const uint8_t *codes, *scales;
  uint64_t rows, k;
  uint8_t *out;
  uint64_t out_stride;
};
struct MxNormArgs {
  const uint8_t *x, *res, *w;   // res: NULL for a norm of x itself
  uint8_t *h;                   // the stored sum (NULL without res)
  uint64_t rows, k, x_stride, res_stride, h_stride;
  float eps;
  double over_k;                // 1 / k
  uint8_t *codes, *scales;
};
struct MxMatmulArgs {
  const uint8_t *a, *as, *w, *ws;
  uint64_t m, n, k;              // k whole blocks of 32
  uint8_t *out;
  uint64_t out_stride;           // elements
  uint8_t *scratch;
  uint64_t scratch_bytes;
};

hipError_t launch_mx_quantize(int in_dtype, int fmt, const MxQuantArgs &a, hipStream_t s);
hipError_t launch_mx_dequantize(int fmt, int out_dtype, const MxDequantArgs &a, hipStream_t s);
hipError_t launch_mx_norm(int dtype, int fmt, const MxNormArgs &a, hipStream_t s);
uint64_t mx_matmul_scratch(int a_fmt, int w_fmt, uint64_t m, uint64_t n, uint64_t k);
hipError_t launch_mx_matmul(int a_fmt, int w_fmt, int out_dtype, bool fast, const MxMatmulArgs &a, hipStream_t s);

// ------------------------------------------------------------ device side --

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
// 16 bytes at the alignment of one element: rows of odd lengths take wide
// loads and stores too, which gfx950 does at any address
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4 u32x4_byte __attribute__((aligned(1)));  // scale bytes

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// Two values rounded to nearest even, the first in the low half; a NaN stays a NaN.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t f32_bf16x2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ uint16_t f32_bf16(float f) { return __builtin_bit_cast(uint16_t, __bf16(f)); }

// The larger bits of the lanes of this lane's group of G = 4 lanes (a block of
// 32 values, 8 a lane), by two exchanges inside the quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  v = v > o ? v : o;
  o = uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x4E, 0xF, 0xF, true));           // lanes 2 3 0 1
  return v > o ? v : o;
}

// The scale byte of a block from the bits of its largest magnitude:
// floor(log2) is the exponent field, emax that of the format's largest value
// (E4M3 2^8, E2M1 2^2).  Zero and subnormal maxima give byte 0.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  constexpr int emax = FMT == FP8 ? 8 : 2;
  const int e = int(top >> 23) - emax;
  return top >= 0x7F800000u ? 255u : uint32_t(e < 0 ? 0 : e);
}

// 2^(127 - s), exact: s is at most 252 when the maximum is finite in FP32.
__device__ __forceinline__ float mx_inverse(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// Eight values times inv, rounded to nearest even and saturated: 8 bytes of
// E4M3 or 4 bytes of E2M1 pairs (in the low word).  Without kClamp the values
// are known to be under 464.
template <int FMT, bool kClamp = true>
__device__ __forceinline__ u32x2 mx_codes8(const float (&v)[8], float inv) {
  u32x2 c = {0, 0};
  if constexpr (FMT == FP8) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; i++) q[i] = kClamp ? __builtin_amdgcn_fmed3f(v[i] * inv, -448.0f, 448.0f) : v[i] * inv;
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    c[0] = uint32_t(lo);
    c[1] = uint32_t(hi);
  } else {
    // |v| * inv < 8: the conversion saturates at 6
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * inv, v[1] * inv, 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * inv, v[3] * inv, 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * inv, v[5] * inv, 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * inv, v[7] * inv, 1.0f, 3);
    c[0] = w;
  }
  return c;
}

// 2^(s - 127) as a float: byte 0 is the subnormal 2^-127, 255 a NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255u ? 0x7FC00000u : s << 23);
}

// Division of n < 2^31 by a constant 1 <= d < 2^31: with s = ceil(log2 d) and
// mul = floor(2^(31+s) / d) + 1 (at most 32 bits), n * mul >> (31 + s) is exact:
// mul * d exceeds 2^(31+s) by at most d <= 2^s, so n * (mul * d - 2^(31+s)) < 2^(31+s).
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t v) : d(v) {
    uint32_t s = 0;
    while ((1ull << s) < v) s++;
    shift = 31 + s;
    mul = uint32_t(((1ull << shift) / v) + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return uint32_t((uint64_t(n) * mul) >> shift); }
};

}  // namespace zn
