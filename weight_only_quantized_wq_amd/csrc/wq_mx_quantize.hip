// MXFP4 quantiser and its inverse: one pass over memory each.
//
// A lane takes eight consecutive inputs, four lanes a group: the largest magnitude
// meets over the four by two lane exchanges, one lane writes the scale byte, and the
// eight codes are four conversions.  Both kernels are bound by HBM; the loads of
// kPieces eights per lane are requested before the first is used.  28672 x 4096 from fp32:
// 94 us (5.7 TB/s in and out), back to bf16 48 us (6.2 TB/s); 5 x 8192 from bf16 2.6 and
// 2.3 us, a launch and one memory latency each.
#include <stdint.h>

#include "wq_host.hpp"
#include "wq_kv.hpp"
#include "wq_mx.hpp"

namespace wq {

constexpr int kMxThreads = 256;
constexpr int kPieces = 4;
static_assert((kMxMost / (8 * kPieces) + kMxThreads - 1) / kMxThreads * kMxThreads < (int64_t)1 << 32);

template <bool F32>
__global__ __launch_bounds__(kMxThreads) void mx_quantize_kernel(const void* w, int64_t eights, uint8_t* q, uint8_t* scale) {
  // a multiple of four eights per group, so the four lanes of a group are there together
  const int64_t first = (int64_t)blockIdx.x * (kMxThreads * kPieces) + threadIdx.x;
  u32x4 raw[kPieces][F32 ? 2 : 1];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int64_t i = first + p * kMxThreads;
    const char* from = static_cast<const char*>(w) + (i < eights ? i : 0) * (F32 ? 32 : 16);
#pragma unroll
    for (int h = 0; h < (F32 ? 2 : 1); ++h) raw[p][h] = load_stream16(from + 16 * h);
  }
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int64_t i = first + p * kMxThreads;
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (F32) {
        v[j] = __uint_as_float(raw[p][0][j]);
        v[4 + j] = __uint_as_float(raw[p][1][j]);
      } else {
        v[2 * j] = bf16lo_to_f32(raw[p][0][j]);
        v[2 * j + 1] = bf16hi_to_f32(raw[p][0][j]);
      }
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = __float_as_uint(v[j]) & 0x7FFFFFFFu;
      top = top > a ? top : a;
    }
    const uint32_t byte = mx_scale_byte(quad_max(top));
    const uint32_t codes = mx_codes(v, byte);
    if (i < eights) {
      __builtin_nontemporal_store(codes, gmem(reinterpret_cast<uint32_t*>(q) + i));
      if ((i & 3) == 0) gmem(scale)[i >> 2] = (uint8_t)byte;
    }
  }
}

template <bool F32>
__global__ __launch_bounds__(kMxThreads) void mx_dequantize_kernel(const uint8_t* q, const uint8_t* scale, int64_t eights,
                                                                   void* y) {
  const int64_t first = (int64_t)blockIdx.x * (kMxThreads * kPieces) + threadIdx.x;
  uint32_t codes[kPieces], bytes[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int64_t i = first + p * kMxThreads, at = i < eights ? i : 0;
    codes[p] = load_stream4(reinterpret_cast<const uint32_t*>(q) + at);
    bytes[p] = gmem(scale)[at >> 2];
  }
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int64_t i = first + p * kMxThreads;
    if (i >= eights) continue;
    const u32x4 pairs = __builtin_bit_cast(u32x4, mx_bf16(codes[p], mx_scale(bytes[p], 0)));
    if constexpr (F32) {
      // bf16 holds every value exactly
      u32x4 lo, hi;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        lo[2 * j] = pairs[j] << 16;
        lo[2 * j + 1] = pairs[j] & 0xFFFF0000u;
        hi[2 * j] = pairs[2 + j] << 16;
        hi[2 * j + 1] = pairs[2 + j] & 0xFFFF0000u;
      }
      u32x4* to = static_cast<u32x4*>(y) + 2 * i;
      __builtin_nontemporal_store(lo, gmem(to));
      __builtin_nontemporal_store(hi, gmem(to + 1));
    } else {
      __builtin_nontemporal_store(pairs, gmem(static_cast<u32x4*>(y) + i));
    }
  }
}

static bool mx_sizes_ok(int64_t n, int64_t k) {
  return n >= 0 && k >= 0 && k % kMxGroup == 0 && (k == 0 || n <= kMxMost / k);
}

static dim3 mx_grid(int64_t eights) {
  return dim3((unsigned)((eights + kMxThreads * kPieces - 1) / (kMxThreads * kPieces)));
}

}  // namespace wq

using namespace wq;

extern "C" int wq_quantize_mxfp4(const float* w_f32, const uint16_t* w_bf16, int64_t n, int64_t k, uint8_t* q,
                                 uint8_t* scale, void* stream) {
  const char* name = "wq_quantize_mxfp4";
  if (!w_f32 == !w_bf16) return fail(WQ_ERR_NULL, "%s: exactly one of w_f32 and w_bf16 must be given", name);
  if (!q || !scale) return fail(WQ_ERR_NULL, "%s: q and scale must be non-null", name);
  if (!mx_sizes_ok(n, k))
    return fail(WQ_ERR_SHAPE, "%s: n = %lld, k = %lld (need n, k >= 0, k %% 32 == 0, n * k <= 2^37 - 2^13)", name, (long long)n,
                (long long)k);
  const void* w = w_f32 ? (const void*)w_f32 : (const void*)w_bf16;
  if (!aligned16(w) || !aligned16(q)) return fail(WQ_ERR_ALIGN, "%s: w and q must be 16-byte aligned", name);
  const ByteRows in{w, 1, 0, n * k * (w_f32 ? 4 : 2)}, codes{q, 1, 0, n * k / 2}, bytes{scale, 1, 0, n * k / kMxGroup};
  if (rows_meet(in, codes) || rows_meet(in, bytes) || rows_meet(codes, bytes))
    return fail(WQ_ERR_SHAPE, "%s: w, q and scale must not overlap", name);
  if (n == 0 || k == 0) return WQ_OK;
  int rc = check_device();
  if (rc) return rc;
  const int64_t eights = n * k / 8;
  if (w_f32)
    hipLaunchKernelGGL(mx_quantize_kernel<true>, mx_grid(eights), dim3(kMxThreads), 0, (hipStream_t)stream, w, eights, q,
                       scale);
  else
    hipLaunchKernelGGL(mx_quantize_kernel<false>, mx_grid(eights), dim3(kMxThreads), 0, (hipStream_t)stream, w, eights, q,
                       scale);
  return launch_status(name);
}

extern "C" int wq_dequantize_mxfp4(const uint8_t* q, const uint8_t* scale, int64_t n, int64_t k, float* y_f32,
                                   uint16_t* y_bf16, void* stream) {
  const char* name = "wq_dequantize_mxfp4";
  if (!q || !scale) return fail(WQ_ERR_NULL, "%s: q and scale must be non-null", name);
  if (!y_f32 == !y_bf16) return fail(WQ_ERR_NULL, "%s: exactly one of y_f32 and y_bf16 must be given", name);
  if (!mx_sizes_ok(n, k))
    return fail(WQ_ERR_SHAPE, "%s: n = %lld, k = %lld (need n, k >= 0, k %% 32 == 0, n * k <= 2^37 - 2^13)", name, (long long)n,
                (long long)k);
  void* y = y_f32 ? (void*)y_f32 : (void*)y_bf16;
  if (!aligned16(q) || !aligned16(y)) return fail(WQ_ERR_ALIGN, "%s: q and y must be 16-byte aligned", name);
  const ByteRows out{y, 1, 0, n * k * (y_f32 ? 4 : 2)}, codes{q, 1, 0, n * k / 2}, bytes{scale, 1, 0, n * k / kMxGroup};
  if (rows_meet(out, codes) || rows_meet(out, bytes))
    return fail(WQ_ERR_SHAPE, "%s: y must not overlap q or scale", name);
  if (n == 0 || k == 0) return WQ_OK;
  int rc = check_device();
  if (rc) return rc;
  const int64_t eights = n * k / 8;
  if (y_f32)
    hipLaunchKernelGGL(mx_dequantize_kernel<true>, mx_grid(eights), dim3(kMxThreads), 0, (hipStream_t)stream, q, scale,
                       eights, y);
  else
    hipLaunchKernelGGL(mx_dequantize_kernel<false>, mx_grid(eights), dim3(kMxThreads), 0, (hipStream_t)stream, q, scale,
                       eights, y);
  return launch_status(name);
}
