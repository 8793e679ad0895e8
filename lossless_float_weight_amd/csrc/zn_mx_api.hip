// zn_mx_api.hip -- the C ABI of the microscaled operators (include/zn.h):
// argument checks and the launch; nothing here allocates or synchronises.
#include <math.h>

#include "../../include/zn.h"
#include "zn_mx.h"

using namespace zn;

namespace {

bool plain(int dt) { return dt == ZN_BF16 || dt == ZN_FP32; }
bool coded(int dt) { return dt == ZN_FP8_E4M3 || dt == ZN_FP4X2_E2M1; }
bool good_rows(uint64_t rows, uint64_t k) { return rows <= kMxMaxRows && k >= 1 && k <= kMxMaxK; }
// a row pitch in elements, whose products with rows stay in 64 bits; that rows do
// not run into each other is asked where they are written
bool good_stride(uint64_t stride) { return stride <= (1ull << 40); }
// elements are read and written whole
bool at(const void *p, int dt) { return p && uintptr_t(p) % (dt == ZN_FP32 ? 4 : 2) == 0; }
bool at16(const void *p) { return p && uintptr_t(p) % 16 == 0; }

zn_status done(hipError_t e) { return e == hipSuccess ? ZN_OK : ZN_ERR_HIP; }

}  // namespace

extern "C" zn_status zn_mx_quantize(zn_dtype dtype, const void *d_x, uint64_t x_stride, uint64_t rows, uint64_t k,
                                    zn_dtype fmt, void *d_codes, void *d_scales, hipStream_t stream) {
  if (!plain(dtype) || !coded(fmt) || !good_rows(rows, k) || !good_stride(x_stride)) return ZN_ERR_ARG;
  if (rows == 0) return ZN_OK;
  if (!at(d_x, dtype) || !at16(d_codes) || !d_scales) return ZN_ERR_ARG;
  MxQuantArgs a;
  a.x = static_cast<const uint8_t *>(d_x);
  a.rows = rows;
  a.k = k;
  a.x_stride = x_stride;
  a.codes = static_cast<uint8_t *>(d_codes);
  a.scales = static_cast<uint8_t *>(d_scales);
  return done(launch_mx_quantize(dtype, fmt, a, stream));
}

extern "C" zn_status zn_mx_dequantize(zn_dtype fmt, const void *d_codes, const void *d_scales, uint64_t rows,
                                      uint64_t k, zn_dtype dtype, void *d_out, uint64_t out_stride,
                                      hipStream_t stream) {
  if (!plain(dtype) || !coded(fmt) || !good_rows(rows, k) || !good_stride(out_stride)) return ZN_ERR_ARG;
  if (rows > 1 && out_stride < k) return ZN_ERR_ARG;
  if (rows == 0) return ZN_OK;
  if (!at(d_out, dtype) || !at16(d_codes) || !d_scales) return ZN_ERR_ARG;
  MxDequantArgs a;
  a.codes = static_cast<const uint8_t *>(d_codes);
  a.scales = static_cast<const uint8_t *>(d_scales);
  a.rows = rows;
  a.k = k;
  a.out = static_cast<uint8_t *>(d_out);
  a.out_stride = out_stride;
  return done(launch_mx_dequantize(fmt, dtype, a, stream));
}

extern "C" zn_status zn_mx_rms_norm(zn_dtype dtype, const void *d_x, uint64_t x_stride, const void *d_residual,
                                    uint64_t residual_stride, const void *d_weight, float eps, uint64_t rows,
                                    uint64_t k, void *d_residual_out, uint64_t residual_out_stride, zn_dtype fmt,
                                    void *d_codes, void *d_scales, hipStream_t stream) {
  if (!plain(dtype) || !coded(fmt) || !good_rows(rows, k) || !good_stride(x_stride)) return ZN_ERR_ARG;
  if (!(eps >= 0.0f) || !isfinite(eps)) return ZN_ERR_ARG;
  if ((d_residual != nullptr) != (d_residual_out != nullptr)) return ZN_ERR_ARG;
  if (d_residual && (!good_stride(residual_stride) || !good_stride(residual_out_stride) ||
                     (rows > 1 && residual_out_stride < k)))
    return ZN_ERR_ARG;
  if (rows == 0) return ZN_OK;
  if (!at(d_x, dtype) || !at(d_weight, dtype) || !at16(d_codes) || !d_scales) return ZN_ERR_ARG;
  if (d_residual && (!at(d_residual, dtype) || !at(d_residual_out, dtype))) return ZN_ERR_ARG;
  MxNormArgs a;
  a.x = static_cast<const uint8_t *>(d_x);
  a.res = static_cast<const uint8_t *>(d_residual);
  a.w = static_cast<const uint8_t *>(d_weight);
  a.h = static_cast<uint8_t *>(d_residual_out);
  a.rows = rows;
  a.k = k;
  a.x_stride = x_stride;
  a.res_stride = residual_stride;
  a.h_stride = residual_out_stride;
  a.eps = eps;
  a.over_k = 1.0 / double(k);
  a.codes = static_cast<uint8_t *>(d_codes);
  a.scales = static_cast<uint8_t *>(d_scales);
  return done(launch_mx_norm(dtype, fmt, a, stream));
}

extern "C" zn_status zn_mx_matmul_scratch_bytes(zn_dtype a_fmt, zn_dtype w_fmt, uint64_t m, uint64_t n, uint64_t k,
                                                uint64_t *bytes) {
  if (!coded(a_fmt) || !coded(w_fmt) || m > kMxMaxRows || n > kMxMaxRows || k < kMxBlock || k > kMxMaxK ||
      k % kMxBlock || !bytes)
    return ZN_ERR_ARG;
  *bytes = m && n ? mx_matmul_scratch(a_fmt, w_fmt, m, n, k) : 0;
  return ZN_OK;
}

extern "C" zn_status zn_mx_matmul(zn_dtype a_fmt, const void *d_a, const void *d_a_scales, zn_dtype w_fmt,
                                  const void *d_w, const void *d_w_scales, uint64_t m, uint64_t n, uint64_t k,
                                  zn_dtype out_dtype, void *d_out, uint64_t out_stride, void *d_scratch,
                                  uint64_t scratch_bytes, hipStream_t stream) {
  return zn_mx_matmul2(a_fmt, d_a, d_a_scales, w_fmt, d_w, d_w_scales, m, n, k, 0, out_dtype, d_out, out_stride,
                       d_scratch, scratch_bytes, stream);
}

extern "C" zn_status zn_mx_matmul2(zn_dtype a_fmt, const void *d_a, const void *d_a_scales, zn_dtype w_fmt,
                                   const void *d_w, const void *d_w_scales, uint64_t m, uint64_t n, uint64_t k,
                                   uint32_t flags, zn_dtype out_dtype, void *d_out, uint64_t out_stride,
                                   void *d_scratch, uint64_t scratch_bytes, hipStream_t stream) {
  if (flags & ~uint32_t(ZN_MX_FAST_SUMS)) return ZN_ERR_ARG;
  if (flags && out_dtype != ZN_BF16) return ZN_ERR_ARG;
  uint64_t need;
  const zn_status st = zn_mx_matmul_scratch_bytes(a_fmt, w_fmt, m, n, k, &need);
  if (st != ZN_OK) return st;
  if (!plain(out_dtype) || !good_stride(out_stride) || (m > 1 && out_stride < n)) return ZN_ERR_ARG;
  if (m == 0 || n == 0) return ZN_OK;
  if (!at16(d_a) || !at16(d_w) || !d_a_scales || !d_w_scales || !at(d_out, out_dtype)) return ZN_ERR_ARG;
  if (need && !at16(d_scratch)) return ZN_ERR_ARG;
  if (scratch_bytes < need) return ZN_ERR_CAPACITY;
  MxMatmulArgs p;
  p.a = static_cast<const uint8_t *>(d_a);
  p.as = static_cast<const uint8_t *>(d_a_scales);
  p.w = static_cast<const uint8_t *>(d_w);
  p.ws = static_cast<const uint8_t *>(d_w_scales);
  p.m = m;
  p.n = n;
  p.k = k;
  p.out = static_cast<uint8_t *>(d_out);
  p.out_stride = out_stride;
  p.scratch = static_cast<uint8_t *>(d_scratch);
  p.scratch_bytes = at16(d_scratch) ? scratch_bytes : 0;
  return done(launch_mx_matmul(a_fmt, w_fmt, out_dtype, flags & ZN_MX_FAST_SUMS, p, stream));
}
