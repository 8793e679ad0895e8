// zn_mxmm.hip -- the product of microscaled activations and weights on the
// scaled matrix instruction of gfx950.
//
//   out[m, n] = sum over blocks b of 2^(sa[m,b] + sw[n,b] - 254) *
//               sum over the block's 32 values of a[m, k] w[n, k],
// summed in FP32 and rounded once to the output's type.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes 128 values (four blocks) of 16 rows
// on each side.  Lane l stands for row l % 16 and lane group g = l / 16; its
// scale byte is that of block g.  Its values are, as measured with one value
// set at a time: E2M1 k = 32 g + 0..31 (16 bytes), E4M3 k = 16 g + 0..15 and
// k = 64 + 16 g + 0..15 (twice 16 bytes).  The weights are the instruction's
// first operand, so a lane ends with 4 consecutive n of one m (row 4 g + i of
// the tile in register i, column l % 16).
#include "zn_mx.h"

namespace zn {
namespace {

template <int F>
__device__ __forceinline__ constexpr int code_bytes() { return F == FP8 ? 32 : 16; }  // of one block
template <int F>
constexpr int kFmtBits = F == FP8 ? 0 : 4;  // the instruction's format field

template <int FW, int FA>
__device__ __forceinline__ f32x4 mfma(i32x8 w, i32x8 a, f32x4 c, uint32_t sw, uint32_t sa) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, kFmtBits<FW>, kFmtBits<FA>, 0, int(sw), 0, int(sa));
}

// A lane's operand for step t from its row in memory; blocks past nb are
// zero codes under scale 1.
template <int F>
__device__ __forceinline__ i32x8 load_codes(const uint8_t *row, uint32_t t, uint32_t g, uint32_t nb) {
  i32x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
  u32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
  if constexpr (F == FP8) {
    const uint8_t *p = row + 128ull * t + 16 * g;
    if (4 * t + g / 2 < nb) lo = *reinterpret_cast<const u32x4 *>(p);
    if (4 * t + 2 + g / 2 < nb) hi = *reinterpret_cast<const u32x4 *>(p + 64);
  } else {
    if (4 * t + g < nb) lo = *reinterpret_cast<const u32x4 *>(row + 64ull * t + 16 * g);
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[i] = int(lo[i]);
    v[4 + i] = int(hi[i]);
  }
  return v;
}
__device__ __forceinline__ uint32_t load_scale(const uint8_t *row, uint32_t t, uint32_t g, uint32_t nb) {
  return 4 * t + g < nb ? row[4 * t + g] : 127u;
}

// Four consecutive n of row m.
template <int OUT>
__device__ __forceinline__ void store4(const MxMatmulArgs &p, uint64_t m, uint64_t n, f32x4 c, bool wide) {
  if (m >= p.m) return;
  uint8_t *row = p.out + m * p.out_stride * esize(OUT);
  if (wide && n + 4 <= p.n) {
    if constexpr (OUT == BF16) {
      const u32x2 v = {f32_bf16(c[0]) | (f32_bf16(c[1]) << 16), f32_bf16(c[2]) | (f32_bf16(c[3]) << 16)};
      *reinterpret_cast<u32x2 *>(row + 2 * n) = v;
    } else {
      *reinterpret_cast<f32x4 *>(row + 4 * n) = c;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (n + i < p.n) {
      if constexpr (OUT == BF16)
        *reinterpret_cast<uint16_t *>(row + 2 * (n + i)) = uint16_t(f32_bf16(c[i]));
      else
        *reinterpret_cast<float *>(row + 4 * (n + i)) = c[i];
    }
}

// Few rows: a workgroup of KS waves makes 16 n by 16 MT m, each wave a piece
// of k straight from memory, joined in LDS in the order of the waves.
template <int FA, int FW, int OUT, int MT, int KS>
__global__ __launch_bounds__(64 * KS) void k_mx_few(MxMatmulArgs p, uint32_t nb, bool wide) {
  __shared__ f32x4 part[KS > 1 ? KS : 1][MT][64];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const uint64_t n0 = uint64_t(blockIdx.x) * 16, m0 = uint64_t(blockIdx.y) * (16 * MT);
  const uint32_t steps = (nb + 3) / 4, per = (steps + KS - 1) / KS;
  const uint32_t t0 = wave * per, t1 = t0 + per < steps ? t0 + per : steps;
  // rows past the end are read as the last row and never stored
  const uint64_t n = n0 + r < p.n ? n0 + r : p.n - 1;
  const uint8_t *w = p.w + n * nb * code_bytes<FW>(), *ws = p.ws + n * nb;
  const uint8_t *a[MT], *as[MT];
#pragma unroll
  for (int i = 0; i < MT; i++) {
    const uint64_t m = m0 + 16 * i + r < p.m ? m0 + 16 * i + r : p.m - 1;
    a[i] = p.a + m * nb * code_bytes<FA>();
    as[i] = p.as + m * nb;
  }
  f32x4 c[MT];
#pragma unroll
  for (int i = 0; i < MT; i++) c[i] = f32x4{0, 0, 0, 0};
  for (uint32_t t = t0; t < t1; t++) {
    const i32x8 x = load_codes<FW>(w, t, g, nb);
    const uint32_t sx = load_scale(ws, t, g, nb);
#pragma unroll
    for (int i = 0; i < MT; i++)
      c[i] = mfma<FW, FA>(x, load_codes<FA>(a[i], t, g, nb), c[i], sx, load_scale(as[i], t, g, nb));
  }
  if constexpr (KS > 1) {
#pragma unroll
    for (int i = 0; i < MT; i++) part[wave][i][lane] = c[i];
    __syncthreads();
  }
  for (int i = wave; i < MT; i += KS) {
    f32x4 s;
    if constexpr (KS > 1) {
      s = part[0][i][lane];
#pragma unroll
      for (int j = 1; j < KS; j++) s += part[j][i][lane];
    } else {
      s = c[i];
    }
    store4<OUT>(p, m0 + 16 * i + r, n0 + 4 * g, s, wide);
  }
}

template <int FA, int FW, int OUT>
hipError_t matmul(const MxMatmulArgs &p, hipStream_t s) {
  const uint32_t nb = uint32_t(p.k / kMxBlock);
  const bool wide = (uintptr_t(p.out) & 15) == 0 && p.out_stride % 4 == 0;
  const uint64_t nt = (p.n + 15) / 16, mt = (p.m + 15) / 16;
  if (mt == 1)
    k_mx_few<FA, FW, OUT, 1, 8><<<dim3(uint32_t(nt), 1), 512, 0, s>>>(p, nb, wide);
  else
    for (uint64_t y = 0; y < (mt + 3) / 4; y += 65535) {
      MxMatmulArgs q = p;
      const uint64_t rows = y * 64;
      q.a += rows * nb * (FA == FP8 ? 32 : 16);
      q.as += rows * nb;
      q.out += rows * p.out_stride * esize(OUT);
      q.m -= rows;
      const uint64_t left = (mt + 3) / 4 - y;
      k_mx_few<FA, FW, OUT, 4, 4><<<dim3(uint32_t(nt), uint32_t(left < 65535 ? left : 65535)), 256, 0, s>>>(q, nb, wide);
    }
  return hipGetLastError();
}

template <int FA, int FW>
hipError_t matmul_out(int out_dtype, const MxMatmulArgs &p, hipStream_t s) {
  return out_dtype == BF16 ? matmul<FA, FW, BF16>(p, s) : matmul<FA, FW, FP32>(p, s);
}

}  // namespace

uint64_t mx_matmul_scratch(int, int, uint64_t, uint64_t, uint64_t) { return 0; }

hipError_t launch_mx_matmul(int a_fmt, int w_fmt, int out_dtype, const MxMatmulArgs &p, hipStream_t s) {
  if (a_fmt == FP8) return w_fmt == FP8 ? matmul_out<FP8, FP8>(out_dtype, p, s) : matmul_out<FP8, FP4X2>(out_dtype, p, s);
  return w_fmt == FP8 ? matmul_out<FP4X2, FP8>(out_dtype, p, s) : matmul_out<FP4X2, FP4X2>(out_dtype, p, s);
}

}  // namespace zn
