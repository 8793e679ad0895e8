// zn_mx.hip -- microscaled numbers (E4M3 or E2M1 codes, one E8M0 scale per 32
// values): quantisation, reading back, and the root-mean-square norm whose
// output is quantised in the same pass.
#include "zn_mx.h"

namespace zn {
namespace {

// Eight consecutive elements of a row from k0 on; zeros past k.
template <int DT>
__device__ __forceinline__ void load8(const uint8_t *row, uint32_t k0, uint32_t k, float (&v)[8]) {
  if (k0 + 8 <= k) {
    if constexpr (DT == BF16) {
      const u32x4 w = *reinterpret_cast<const u32x4_any *>(row + 2 * uint64_t(k0));
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4_any *>(row + 4 * uint64_t(k0));
      const f32x4 b = *reinterpret_cast<const f32x4_any *>(row + 4 * uint64_t(k0) + 16);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; i++) {
    v[i] = 0.0f;
    if (k0 + i < k) {
      if constexpr (DT == BF16)
        v[i] = bf16_lo(*reinterpret_cast<const uint16_t *>(row + 2 * uint64_t(k0 + i)));
      else
        v[i] = *reinterpret_cast<const float *>(row + 4 * uint64_t(k0 + i));
    }
  }
}

// Eight consecutive elements of a row, those below k; v is already rounded
// to DT's grid or is rounded here.
template <int DT>
__device__ __forceinline__ void store8(uint8_t *row, uint32_t k0, uint32_t k, const float (&v)[8]) {
  if (k0 + 8 <= k) {
    if constexpr (DT == BF16) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; i++) w[i] = f32_bf16x2(v[2 * i], v[2 * i + 1]);
      *reinterpret_cast<u32x4_any *>(row + 2 * uint64_t(k0)) = w;
    } else {
      f32x4 a, b;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        a[i] = v[i];
        b[i] = v[4 + i];
      }
      *reinterpret_cast<f32x4_any *>(row + 4 * uint64_t(k0)) = a;
      *reinterpret_cast<f32x4_any *>(row + 4 * uint64_t(k0) + 16) = b;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; i++)
    if (k0 + i < k) {
      if constexpr (DT == BF16)
        *reinterpret_cast<uint16_t *>(row + 2 * uint64_t(k0 + i)) = f32_bf16(v[i]);
      else
        *reinterpret_cast<float *>(row + 4 * uint64_t(k0 + i)) = v[i];
    }
}

// Bits of the largest magnitude of eight; a NaN's where there is one.
__device__ __forceinline__ uint32_t top8(const float (&v)[8]) {
  float t = __builtin_fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; i++) t = __builtin_elementwise_maximum(t, __builtin_fabsf(v[i]));
  return __float_as_uint(t) & 0x7FFFFFFFu;
}

// Codes and scale byte of group gi (8 values, a quarter of a block) of a
// tensor whose groups are numbered through all rows.  The four lanes of a
// quad hold one block.
template <int FMT>
__device__ __forceinline__ void put_codes(uint8_t *codes, uint8_t *scales, uint64_t gi, u32x2 c, uint32_t s, bool live) {
  if (!live) return;
  if constexpr (FMT == FP8)
    *reinterpret_cast<u32x2 *>(codes + 8 * gi) = c;
  else
    *reinterpret_cast<uint32_t *>(codes + 4 * gi) = c[0];
  if ((gi & 3) == 0) scales[gi >> 2] = uint8_t(s);
}

// ---------------------------------------------------------------- quantise --
// A lane takes 8 consecutive values (16 bytes of BF16), a quad one block of
// 32; the block's maximum is exchanged inside the quad.  Bound by memory: two
// groups a lane keep enough loads in flight for a copy's rate (28672 x 4096
// BF16 to FP4, 297 MB, 65 us, 4.6 TB/s; one token 1.7 us).
template <int DT, int FMT, int U>
__global__ __launch_bounds__(256) void k_mx_quantize(MxQuantArgs a, FastDiv gpr, uint32_t groups) {
  const uint32_t first = blockIdx.x * (256u * U) + threadIdx.x;
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const uint32_t g = first + 256u * u;
    const uint32_t gc = g < groups ? g : 0;
    const uint32_t row = gpr.div(gc), k0 = (gc - row * gpr.d) * 8;
    load8<DT>(a.x + row * a.x_stride * esize(DT), k0, uint32_t(a.k), v[u]);
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    const uint32_t s = mx_scale_byte<FMT>(quad_max(top8(v[u])));
    // a block with an infinity or a NaN gets codes 0
    const u32x2 c = s == 255u ? u32x2{0, 0} : mx_codes8<FMT>(v[u], mx_inverse(s));
    put_codes<FMT>(a.codes, a.scales, first + 256u * u, c, s, first + 256u * u < groups);
  }
}

// ------------------------------------------------------------------- read --
template <int FMT>
__device__ __forceinline__ void values8(const uint8_t *codes, uint64_t gi, float s, float (&v)[8]) {
  if constexpr (FMT == FP8) {
    const u32x2 c = *reinterpret_cast<const u32x2 *>(codes + 8 * gi);
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const f32x2 p = __builtin_amdgcn_cvt_pk_f32_fp8(int(c[i]), false), q = __builtin_amdgcn_cvt_pk_f32_fp8(int(c[i]), true);
      v[4 * i] = p[0] * s;
      v[4 * i + 1] = p[1] * s;
      v[4 * i + 2] = q[0] * s;
      v[4 * i + 3] = q[1] * s;
    }
  } else {
    const uint32_t c = *reinterpret_cast<const uint32_t *>(codes + 4 * gi);
    const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
#pragma unroll
    for (int i = 0; i < 2; i++) {
      v[i] = p0[i] * s;
      v[2 + i] = p1[i] * s;
      v[4 + i] = p2[i] * s;
      v[6 + i] = p3[i] * s;
    }
  }
}

// Bound by memory: 28672 x 4096 FP4 to BF16, 297 MB, 52 us, 5.7 TB/s (the codes
// partly from the 256 MB cache).
template <int FMT, int DT, int U>
__global__ __launch_bounds__(256) void k_mx_dequantize(MxDequantArgs a, FastDiv gpr, uint32_t groups) {
  const uint32_t first = blockIdx.x * (256u * U) + threadIdx.x;
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const uint32_t g = first + 256u * u;
    const uint32_t gc = g < groups ? g : 0;
    values8<FMT>(a.codes, gc, mx_scale_value(a.scales[gc >> 2]), v[u]);
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    const uint32_t g = first + 256u * u;
    if (g >= groups) return;
    const uint32_t row = gpr.div(g), k0 = (g - row * gpr.d) * 8;
    store8<DT>(a.out + row * a.out_stride * esize(DT), k0, uint32_t(a.k), v[u]);
  }
}

// ------------------------------------------------------------------- norm --
// y = h w / sqrt(mean(h^2) + eps), h = x + res rounded to DT, quantised.
//
// The squares are summed in 64 bits, so no finite row overflows or vanishes,
// and 1 / sqrt is split into a power of two and a 24-bit fraction for the
// same reason: h is scaled by the power exactly before it meets the fraction.
// y then has three FP32 roundings, under 2^-22, and a code or a scale that
// could come out otherwise is computed again in 64 bits: the result is the
// 64-bit formula's, and the second way is taken by one or two groups in 10,000.
// So are blocks that FP32 cannot hold: |y| past 2^128, or h / rms under 2^-126,
// where it has fewer bits, if that can matter.  It cannot where the block's
// maximum is at least kLow = 2^-80 and |w| under kWide = 2^24: codes change at
// multiples of 2^-98 then (2^-10 of a scale of at least 2^-88), and y has
// passed 2^-122 before the weight there.
// One pass over memory with the row in registers: 8192 x 4096 BF16 with the
// addition, 236 MB, 40 us in a row (5.9 TB/s with what the 256 MB cache holds),
// 3.1 us for one row; without the second look it was 38 and 2.8, and 613 x 5003
// FP32 6.6 for 7.5: its registers leave six waves a SIMD where eight would fit.
struct RowScale {
  int e;
  float m;
  double sum;
};
__device__ __forceinline__ RowScale row_scale(double sum, double over_k, float eps) {
  const double a = sum * over_k + double(eps);
  double r = __builtin_amdgcn_rsq(a);
  // one Newton step takes the instruction's 2^-26 to 64-bit rounding
  const double t = __builtin_fma(-a * r, r, 1.0);
  const double n = __builtin_fma(0.5 * r, t, r);
  r = (a > 0 && a < __builtin_inf()) ? n : r;  // 0 gives infinity, infinity gives 0, a NaN stays
  RowScale s;
  // the power is kept apart only where FP32 could not carry it
  const int e = __builtin_amdgcn_frexp_exp(r);
  const bool far = e < -60 || e > 60;
  s.e = far ? e : 0;
  s.m = far ? float(__builtin_amdgcn_frexp_mant(r)) : float(r);
  s.sum = sum;
  return s;
}

// A 64-bit value in FP32, inexact ones to the odd neighbour: a later rounding to
// fewer bits gives what it would have given from 64.
__device__ __forceinline__ float to_odd(double v) {
  float f = float(v);
  const double d = double(f);
  if (d != v) {
    uint32_t b = __float_as_uint(f);
    if (__builtin_fabs(d) > __builtin_fabs(v)) b -= 1;
    f = __uint_as_float(b | 1u);
  }
  return f;
}

// Codes and scale of a group from the formula in 64 bits; all four lanes of a
// quad come here together.
template <int FMT>
__device__ __forceinline__ u32x2 exact8(const MxNormArgs &a, double sum, const float (&h)[8], const float (&w)[8], uint32_t &s) {
  constexpr int emax = FMT == FP8 ? 8 : 2;
  const double q = __builtin_sqrt(sum / double(a.k) + double(a.eps)), over = 1.0 / q;
  double y[8];
  uint32_t top = 0;  // the exponent of the largest
#pragma unroll
  for (int i = 0; i < 8; i++) {
    // h / q by its reciprocal and one correction, which would make -0 a +0
    const double x = double(h[i]), t = x * over;
    y[i] = __builtin_copysign(__builtin_fma(__builtin_fma(-t, q, x), over, t), x) * double(w[i]);
    const uint32_t b = uint32_t(__double_as_longlong(y[i]) >> 52) & 0x7FFu;
    top = top > b ? top : b;
  }
  top = quad_max(top);
  const int e = int(top) - 1023 + 127 - emax;
  s = top == 0x7FFu ? 255u : uint32_t(e < 0 ? 0 : e > 254 ? 254 : e);
  if (s == 255u) return u32x2{0, 0};
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = to_odd(__builtin_amdgcn_ldexp(y[i], 127 - int(s)));
  return mx_codes8<FMT>(v, 1.0f);
}

template <int DT>
__device__ __forceinline__ float rounded(float v) {
  return DT == BF16 ? __uint_as_float(uint32_t(f32_bf16(v)) << 16) : v;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// h of one group: loaded, added, rounded, stored
template <int DT>
__device__ __forceinline__ void take8(const MxNormArgs &a, uint64_t row, uint32_t k0, float (&h)[8]) {
  load8<DT>(a.x + row * a.x_stride * esize(DT), k0, uint32_t(a.k), h);
  if (a.res) {
    float r[8];
    load8<DT>(a.res + row * a.res_stride * esize(DT), k0, uint32_t(a.k), r);
#pragma unroll
    for (int i = 0; i < 8; i++) h[i] = rounded<DT>(h[i] + r[i]);
    store8<DT>(a.h + row * a.h_stride * esize(DT), k0, uint32_t(a.k), h);
  }
}

__device__ __forceinline__ double squares8(const float (&h)[8]) {
  double s = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) s = __builtin_fma(double(h[i]), double(h[i]), s);
  return s;
}

constexpr uint32_t kLow = uint32_t(127 - 80) << 23, kWide = uint32_t(127 + 24) << 23;

// `wide`: one of this lane's weights is kWide or more, an infinity or a NaN.
template <int FMT>
__device__ __forceinline__ void norm8(const MxNormArgs &a, uint64_t gi, const RowScale &r, const float (&h)[8],
                                      const float (&w)[8], bool wide, bool live) {
  float y[8];
  if (r.e) {
#pragma unroll
    for (int i = 0; i < 8; i++) y[i] = __builtin_amdgcn_ldexpf(h[i], r.e) * r.m * w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) y[i] = h[i] * r.m * w[i];
  }
  const uint32_t top = quad_max(top8(y));
  uint32_t s = mx_scale_byte<FMT>(top);
  u32x2 c = {0, 0};
  bool again = true;
  if (s != 255u) {
    const float inv = mx_inverse(s);
    if constexpr (FMT == FP8) {  // saturated before it is scaled, once for both
      const float most = 448.0f * mx_scale_value(s);
#pragma unroll
      for (int i = 0; i < 8; i++) y[i] = __builtin_amdgcn_fmed3f(y[i], -most, most);
    }
    // y and its product with the scale are off by at most 4 x 2^-24
    c = mx_codes8<FMT, false>(y, inv * (1.0f - 5 * 0x1p-24f));
    const u32x2 above = mx_codes8<FMT, false>(y, inv * (1.0f + 6 * 0x1p-24f));
    // in doubt: a maximum within 8 steps of a power of two or too small, a code
    // between two, a wide weight; nothing but zeros only where h has no others
    bool block = ((top + 8) ^ (top - 8)) >> 23 != 0 || top < kLow;
    if (top == 0) block = top8(h) != 0;
    again = quad_max(block || wide || c[0] != above[0] || c[1] != above[1]);
  }
  // a row that holds an infinity or a NaN has only zeros and NaNs, as they are
  if (again && r.sum < __builtin_inf()) c = exact8<FMT>(a, r.sum, h, w, s);
  put_codes<FMT>(a.codes, a.scales, gi, c, s, live);
}

// The sum over a workgroup; `slot` alternates between rows so that one barrier
// a row is enough.
__device__ __forceinline__ double group_sum(double s, double (*part)[16], int slot) {
  s = wave_sum(s);
  if (blockDim.x == 64) return s;
  if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0;
  for (uint32_t i = 0; i < blockDim.x / 64; i++) s += part[slot][i];
  return s;
}

// Rows of at most CH groups of 8 a lane stay in registers; a workgroup has as
// many waves as its row needs.  kFour: rows of one wave, four to a workgroup.
template <int DT, int FMT, int CH, bool kFour>
__global__ __launch_bounds__(kFour ? 256 : 1024, CH == 1 ? 6 : 1) void k_mx_norm(MxNormArgs a, uint32_t gpr) {
  __shared__ double part[2][16];
  const uint32_t t = kFour ? threadIdx.x & 63 : threadIdx.x, team = kFour ? 64 : blockDim.x;
  float w[CH][8];
  bool wide = false;
#pragma unroll
  for (int c = 0; c < CH; c++) {
    load8<DT>(a.w, (c * team + t) * 8, uint32_t(a.k), w[c]);
    wide |= top8(w[c]) >= kWide;
  }
  int slot = 0;
  const uint64_t step = uint64_t(gridDim.x) * (kFour ? 4 : 1);
  for (uint64_t row = uint64_t(blockIdx.x) * (kFour ? 4 : 1) + (kFour ? threadIdx.x >> 6 : 0); row < a.rows; row += step, slot ^= 1) {
    float h[CH][8];
    double s = 0;
#pragma unroll
    for (int c = 0; c < CH; c++) {
      take8<DT>(a, row, (c * team + t) * 8, h[c]);
      s += squares8(h[c]);
    }
    const RowScale r = row_scale(kFour ? wave_sum(s) : group_sum(s, part, slot), a.over_k, a.eps);
#pragma unroll
    for (int c = 0; c < CH; c++) {
      const uint32_t g = c * team + t;
      norm8<FMT>(a, row * gpr + g, r, h[c], w[c], wide, g < gpr);
    }
  }
}

// Longer rows are read twice, the second time as they were stored.
template <int DT, int FMT>
__global__ __launch_bounds__(1024, 8) void k_mx_norm_long(MxNormArgs a, uint32_t gpr) {
  __shared__ double part[2][16];
  int slot = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, slot ^= 1) {
    double s = 0;
    for (uint32_t g = threadIdx.x; g < gpr; g += 1024) {
      float h[8];
      take8<DT>(a, row, g * 8, h);
      s += squares8(h);
    }
    const RowScale r = row_scale(group_sum(s, part, slot), a.over_k, a.eps);
    const uint8_t *src = a.res ? a.h + row * a.h_stride * esize(DT) : a.x + row * a.x_stride * esize(DT);
    // gpr is a multiple of 4: the lanes of a quad stay together
    for (uint32_t g = threadIdx.x; g < gpr; g += 1024) {
      float h[8], w[8];
      load8<DT>(src, g * 8, uint32_t(a.k), h);
      load8<DT>(a.w, g * 8, uint32_t(a.k), w);
      norm8<FMT>(a, row * gpr + g, r, h, w, top8(w) >= kWide, true);
    }
  }
}

// Calls f(first row, rows) for pieces whose groups of 8 stay below 2^31.
template <class F>
hipError_t by_pieces(uint64_t rows, uint32_t gpr, F f) {
  const uint64_t most = 0x7FFF0000u / gpr;
  for (uint64_t r = 0; r < rows; r += most) {
    const hipError_t e = f(r, rows - r < most ? rows - r : most);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int FMT>
hipError_t quantize(const MxQuantArgs &a, hipStream_t s) {
  constexpr int U = 2;
  const uint32_t gpr = uint32_t((a.k + kMxBlock - 1) / kMxBlock * 4);
  return by_pieces(a.rows, gpr, [&](uint64_t r0, uint64_t rows) {
    MxQuantArgs p = a;
    p.x += r0 * a.x_stride * esize(DT);
    p.codes += r0 * gpr * (FMT == FP8 ? 8 : 4);
    p.scales += r0 * (gpr / 4);
    p.rows = rows;
    const uint32_t groups = uint32_t(rows * gpr);
    k_mx_quantize<DT, FMT, U><<<(groups + 256 * U - 1) / (256 * U), 256, 0, s>>>(
        p, FastDiv(gpr), groups);
    return hipGetLastError();
  });
}

template <int FMT, int DT>
hipError_t dequantize(const MxDequantArgs &a, hipStream_t s) {
  constexpr int U = 2;
  const uint32_t gpr = uint32_t((a.k + kMxBlock - 1) / kMxBlock * 4);
  return by_pieces(a.rows, gpr, [&](uint64_t r0, uint64_t rows) {
    MxDequantArgs p = a;
    p.codes += r0 * gpr * (FMT == FP8 ? 8 : 4);
    p.scales += r0 * (gpr / 4);
    p.out += r0 * a.out_stride * esize(DT);
    p.rows = rows;
    const uint32_t groups = uint32_t(rows * gpr);
    k_mx_dequantize<FMT, DT, U><<<(groups + 256 * U - 1) / (256 * U), 256, 0, s>>>(
        p, FastDiv(gpr), groups);
    return hipGetLastError();
  });
}

template <int DT, int FMT>
hipError_t norm(const MxNormArgs &a, hipStream_t s) {
  const uint32_t gpr = uint32_t((a.k + kMxBlock - 1) / kMxBlock * 4);
  const uint32_t grid = uint32_t(a.rows < 4096 ? a.rows : 4096);
  // One group of 8 a lane wherever 1024 lanes are enough: two a lane took, at
  // 8192 x 4096 BF16 with the addition, 4% longer (a single row 25%), and at
  // 4096 x 8192 8%.  Waves as needed and no power of two of them: 613 x 5003 FP32
  // 8% shorter.
  if (gpr <= 64)
    k_mx_norm<DT, FMT, 1, true><<<uint32_t((a.rows + 3) / 4 < 4096 ? (a.rows + 3) / 4 : 4096), 256, 0, s>>>(a, gpr);
  else if (gpr <= 1024)
    k_mx_norm<DT, FMT, 1, false><<<grid, (gpr + 63) / 64 * 64, 0, s>>>(a, gpr);
  else if (gpr <= 2048)
    k_mx_norm<DT, FMT, 2, false><<<grid, (gpr + 127) / 128 * 64, 0, s>>>(a, gpr);
  else
    k_mx_norm_long<DT, FMT><<<grid, 1024, 0, s>>>(a, gpr);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(int in_dtype, int fmt, const MxQuantArgs &a, hipStream_t s) {
  if (in_dtype == BF16) return fmt == FP8 ? quantize<BF16, FP8>(a, s) : quantize<BF16, FP4X2>(a, s);
  return fmt == FP8 ? quantize<FP32, FP8>(a, s) : quantize<FP32, FP4X2>(a, s);
}
hipError_t launch_mx_dequantize(int fmt, int out_dtype, const MxDequantArgs &a, hipStream_t s) {
  if (out_dtype == BF16) return fmt == FP8 ? dequantize<FP8, BF16>(a, s) : dequantize<FP4X2, BF16>(a, s);
  return fmt == FP8 ? dequantize<FP8, FP32>(a, s) : dequantize<FP4X2, FP32>(a, s);
}
hipError_t launch_mx_norm(int dtype, int fmt, const MxNormArgs &a, hipStream_t s) {
  if (dtype == BF16) return fmt == FP8 ? norm<BF16, FP8>(a, s) : norm<BF16, FP4X2>(a, s);
  return fmt == FP8 ? norm<FP32, FP8>(a, s) : norm<FP32, FP4X2>(a, s);
}

}  // namespace zn
