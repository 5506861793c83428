// What stands between two blocks, in one pass over memory:
//   h' = h + scale * act(gate) * norm(f),   u = norm(h'), in bf16 or in MXFP4.
//
// A workgroup takes a row, a thread up to CPT pieces of eight elements, which it keeps
// in registers from the first load to the last store; everything is requested before
// the first sum.  Bound by HBM: 4099 rows of 8192 (fp32 h in and out, bf16 f and gate, two
// norms, 4-bit results; 424 MB) 110 us, 3.9 TB/s, with fp64 arithmetic about two thirds of
// the time under way beside it.  One row of 4096: 3.5 us, a launch and two latencies.
//
// Sums of squares are fp64 (no row overflows or vanishes in them).  Elements are fp32
// where u is bf16; a norm's factor is applied as mantissa and exponent, so that rows of
// any size keep their digits.  Where u is rounded to 4 bits everything is fp64: codes
// then do not depend on an order of summation or on how a factor was rounded.
#include <stdint.h>

#include "wq_host.hpp"
#include "wq_kv.hpp"
#include "wq_mx.hpp"

namespace wq {

struct NormArgs {
  const float* h32;
  const uint16_t* h16;
  int64_t h_stride;
  float* o32;
  uint16_t* o16;
  int64_t o_stride;
  const float* f32;
  const uint16_t* f16;
  int64_t f_stride;
  const uint16_t* f_norm;
  const uint16_t* gate;
  int64_t gate_stride;
  const uint16_t* norm;
  uint16_t* u;
  int64_t u_stride;
  uint8_t* q;
  uint8_t* q_scale;
  int32_t dim;
  int32_t rows;
  float scale;
  float eps;
  int32_t kind;
};

struct Raw8 {
  u32x4 a, b;     // fp32, or bf16 in `a`
};

__device__ __forceinline__ Raw8 load8(const float* p32, const uint16_t* p16, int64_t at) {
  Raw8 r;
  if (p32) {
    r.a = load16(p32 + at);
    r.b = load16(p32 + at + 4);
  } else {
    r.a = load16(p16 + at);
    r.b = r.a;
  }
  return r;
}
__device__ __forceinline__ void as_f32(const u32x4& v, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = bf16lo_to_f32(v[j]);
    x[2 * j + 1] = bf16hi_to_f32(v[j]);
  }
}
__device__ __forceinline__ void as_f32(const Raw8& r, bool wide, float (&x)[8]) {
  if (wide) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = __uint_as_float(r.a[j]);
      x[4 + j] = __uint_as_float(r.b[j]);
    }
  } else {
    as_f32(r.a, x);
  }
}

// A norm's factor.
template <class A>
struct Factor;
template <>
struct Factor<double> {
  double r;
  __device__ explicit Factor(double v) : r(v) {}
  __device__ double operator()(double v) const { return v * r; }
};
template <>
struct Factor<float> {
  float m;
  int e;
  __device__ explicit Factor(double v) {
    if (v > 0. && v < (double)INFINITY) {
      m = (float)frexp(v, &e);
    } else {
      m = (float)v;
      e = 0;
    }
  }
  // the power first, which is exact: the product of a number below 2^-126 would be rounded
  // (rows are divided by their own size, so nothing overflows)
  __device__ float operator()(float v) const { return ldexpf(v, e) * m; }
};

// sigmoid of eight gates (bf16 values).
__device__ __forceinline__ void turned(const float (&x)[8], float (&g)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = 1.f / (1.f + expf(-x[j]));
}
// 1 / (1 + 2^(n + t)), |t| <= 1/2, with 2^t = sum (t ln 2)^i / i! up to i = 10 (the rest
// is below 3e-13) and two Newton steps on the hardware's reciprocal: a third of the
// instructions of exp and a division, and far finer than what is rounded to 4 bits can
// tell.  Gates past 700, infinities and NaN take exp itself.
__device__ __forceinline__ void turned(const float (&x)[8], double (&g)[8]) {
  float most = 0.f;
  bool fine = true;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    most = fmaxf(most, fabsf(x[j]));
    fine = fine && x[j] == x[j];
  }
  if (__any(!(most <= 700.f && fine))) {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 1. / (1. + exp(-(double)x[j]));
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const double y = (double)x[j] * -1.4426950408889634, n = rint(y), t = y - n;
    double p = 7.054911620801121e-09;
    p = fma(p, t, 1.0178086009239696e-07);
    p = fma(p, t, 1.3215486790144305e-06);
    p = fma(p, t, 1.5252733804059838e-05);
    p = fma(p, t, 1.5403530393381606e-04);
    p = fma(p, t, 1.3333558146428441e-03);
    p = fma(p, t, 9.618129107628477e-03);
    p = fma(p, t, 5.5504108664821576e-02);
    p = fma(p, t, 2.402265069591007e-01);
    p = fma(p, t, 6.931471805599453e-01);
    p = fma(p, t, 1.);
    const double d = 1. + ldexp(p, (int)n);
    double r = __builtin_amdgcn_rcp(d);
    r = fma(fma(-d, r, 1.), r, r);
    g[j] = fma(fma(-d, r, 1.), r, r);
  }
}

__device__ __forceinline__ void store_f32(float* to, const float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    *gmem(reinterpret_cast<u32x4*>(to) + h) = u32x4{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                                    __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])};
}
__device__ __forceinline__ void store_bf16(uint16_t* to, const float (&v)[8]) {
  u32x4 p;
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = (uint32_t)f32_to_bf16(v[2 * j]) | (uint32_t)f32_to_bf16(v[2 * j + 1]) << 16;
  *gmem(reinterpret_cast<u32x4*>(to)) = p;
}

// fp64 to fp32, rounded to odd: an inexact result keeps an odd last bit, so that a
// second rounding to fewer bits is the one rounding of the fp64 value.
__device__ __forceinline__ float to_odd(double v) {
  const float f = (float)v;
  const double d = (double)f;
  uint32_t b = __float_as_uint(f);
  if (d != v) b = (b - (fabs(d) > fabs(v) ? 1u : 0u)) | 1u;
  return __uint_as_float(b);
}
// The codes of eight fp64 values.  Rounding to fp32 first matters only where it lands on
// a border between two codes, whose 20 last bits are 0; those few are rounded to odd.
__device__ __forceinline__ uint32_t mx_codes(const double (&v)[8], uint32_t byte) {
  float o[8];
  uint32_t low = ~0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    o[j] = (float)v[j];
    const uint32_t b = __float_as_uint(o[j]) & 0xFFFFFu;
    low = low < b ? low : b;
  }
  if (__any(low == 0)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = to_odd(v[j]);
  }
  return mx_codes(o, byte);
}
// What the fp64 value is in bf16.
__device__ __forceinline__ float narrow(double v, bool to_bf16) { return to_bf16 ? to_odd(v) : (float)v; }
__device__ __forceinline__ float narrow(float v, bool) { return v; }

template <int THREADS>
__device__ __forceinline__ double group_sum(double v, double (&part)[THREADS / 64]) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  if constexpr (THREADS > 64) {
    if (lane_id() == 0) part[wave_id()] = v;
    __syncthreads();
    v = 0.;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) v += part[w];
  }
  return v;
}

template <class A, int CPT, int THREADS>
__global__ __launch_bounds__(THREADS) void block_norm_kernel(NormArgs a) {
  __shared__ double part[2][THREADS / 64];
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.rows) return;
  const int tid = (int)threadIdx.x;
  const bool has_f = a.f32 || a.f16;
  Raw8 fr[CPT], hr[CPT];
  u32x4 gr[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int at = (tid + i * THREADS) * 8;
    const u32x4 z = {0, 0, 0, 0};
    fr[i] = hr[i] = Raw8{z, z};
    gr[i] = z;
    if (at < a.dim) {
      if (has_f) fr[i] = load8(a.f32, a.f16, row * a.f_stride + at);
      hr[i] = load8(a.h32, a.h16, row * a.h_stride + at);
      if (a.gate) gr[i] = load16(a.gate + row * a.gate_stride + at);
    }
  }
  Factor<A> post(1.);
  if (a.f_norm) {
    double s = 0.;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      float x[8];
      as_f32(fr[i], a.f32, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fma((double)x[j], (double)x[j], s);
    }
    post = Factor<A>(1. / sqrt(group_sum<THREADS>(s, part[0]) / a.dim + (double)a.eps));
  }
  A v[CPT][8];
  double s = 0.;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int at = (tid + i * THREADS) * 8;
    float x[8];
    as_f32(hr[i], a.h32, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = (A)x[j];
    if (has_f) {
      as_f32(fr[i], a.f32, x);
      A t[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = (A)x[j];
      if (a.f_norm && at < a.dim) {
        as_f32(load16(a.f_norm + at), x);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = post(t[j]) * (A)x[j];
      }
      if (a.gate) {
        // the choice stands outside the loops, whose eight chains then overlap
        as_f32(gr[i], x);
        A g[8];
        if (a.kind == WQ_GATE_PLAIN) {
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = (A)x[j];
        } else {
          turned(x, g);
          if (a.kind == WQ_GATE_SILU) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] *= (A)x[j];
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] + (A)a.scale * t[j];
    }
    if (at < a.dim) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fma((double)v[i][j], (double)v[i][j], s);
      float o[8];
      if (a.o32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = narrow(v[i][j], false);
        store_f32(a.o32 + row * a.o_stride + at, o);
      }
      if (a.o16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = narrow(v[i][j], true);
        store_bf16(a.o16 + row * a.o_stride + at, o);
      }
    }
  }
  if (!a.u && !a.q) return;
  const Factor<A> pre(1. / sqrt(group_sum<THREADS>(s, part[1]) / a.dim + (double)a.eps));
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int at = (tid + i * THREADS) * 8;
    if (at >= a.dim) continue;
    float w[8];
    if (a.norm) as_f32(load16(a.norm + at), w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = pre(v[i][j]);
      if (a.norm) v[i][j] *= (A)w[j];
    }
    float o[8];
    if (a.u) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = narrow(v[i][j], true);
      store_bf16(a.u + row * a.u_stride + at, o);
    }
    if constexpr (sizeof(A) == 8) {
      // a group is four lanes' pieces (dim is a multiple of 32 here, so all four are there)
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b = (uint32_t)(__double_as_longlong(v[i][j]) >> 32) & 0x7FFFFFFFu;
        top = top > b ? top : b;
      }
      // 2^(floor(log2) - 2) as for the quantiser; past fp32's range as an infinity
      const int e = (int)(quad_max(top) >> 20) - 1023;
      const uint32_t byte = e > 127 ? 255u : e < -125 ? 0u : (uint32_t)(e + 125);
      const uint32_t codes = mx_codes(v[i], byte);
      const int64_t piece = (row * a.dim + at) / 8;
      gmem(reinterpret_cast<uint32_t*>(a.q))[piece] = codes;
      if ((piece & 3) == 0) gmem(a.q_scale)[piece >> 2] = (uint8_t)byte;
    }
  }
}

// ---------------------------------------------------------------------------
// Host side

constexpr int64_t kNormMade = 0x77715f6e6f726d31;
constexpr int64_t kNormMaxRows = 1 << 24, kNormMaxDim = 32768, kNormGridX = 1 << 20;

static int norm_check(const char* name, const wq_block_norm& a) {
  if (!a.h_f32 == !a.h_bf16) return fail(WQ_ERR_NULL, "%s: exactly one of h_f32 and h_bf16 must be given", name);
  if (a.f_f32 && a.f_bf16) return fail(WQ_ERR_NULL, "%s: at most one of f_f32 and f_bf16 may be given", name);
  if (!a.f_f32 && !a.f_bf16 && (a.f_norm || a.gate)) return fail(WQ_ERR_NULL, "%s: f_norm and gate need f", name);
  if (a.out_f32 && a.out_bf16) return fail(WQ_ERR_NULL, "%s: at most one of out_f32 and out_bf16 may be given", name);
  if (!a.q != !a.q_scale) return fail(WQ_ERR_NULL, "%s: q and q_scale go together", name);
  if (!a.out_f32 && !a.out_bf16 && !a.u && !a.q) return fail(WQ_ERR_NULL, "%s: nothing is asked for (out, u, q)", name);
  if (a.norm && !a.u && !a.q) return fail(WQ_ERR_NULL, "%s: norm needs u or q", name);
  if (a.rows < 0 || a.rows > kNormMaxRows || a.dim < 8 || a.dim > kNormMaxDim || a.dim % 8)
    return fail(WQ_ERR_SHAPE, "%s: rows = %lld (0..2^24), dim = %lld (a multiple of 8 up to 32768)", name, (long long)a.rows,
                (long long)a.dim);
  if (a.q && a.dim % kMxGroup) return fail(WQ_ERR_SHAPE, "%s: dim = %lld must be a multiple of 32 for q", name, (long long)a.dim);
  if (a.gate_kind < WQ_GATE_PLAIN || a.gate_kind > WQ_GATE_SILU)
    return fail(WQ_ERR_SHAPE, "%s: gate_kind = %d (need WQ_GATE_PLAIN, _SIGMOID or _SILU)", name, a.gate_kind);
  if (!(a.eps >= 0.f) || !(a.eps < INFINITY) || !(a.scale - a.scale == 0.f))
    return fail(WQ_ERR_SHAPE, "%s: eps must be finite and not negative, scale finite", name);
  const int64_t most = (int64_t)1 << 40;
  auto bad = [&](const void* p, int64_t stride) { return p && (stride < a.dim || stride > most || stride % 8); };
  if (bad(a.h_f32 ? (const void*)a.h_f32 : a.h_bf16, a.h_stride) || bad(a.f_f32 ? (const void*)a.f_f32 : a.f_bf16, a.f_stride) ||
      bad(a.out_f32 ? (const void*)a.out_f32 : a.out_bf16, a.out_stride) || bad(a.u, a.u_stride) ||
      (a.gate_stride && bad(a.gate, a.gate_stride)))
    return fail(WQ_ERR_SHAPE, "%s: strides must be multiples of 8 and hold a row (gate_stride 0: one row for all)", name);
  const void* all[] = {a.h_f32, a.h_bf16, a.f_f32, a.f_bf16, a.f_norm, a.gate, a.norm, a.out_f32, a.out_bf16, a.u};
  for (const void* p : all)
    if (!aligned16(p)) return fail(WQ_ERR_ALIGN, "%s: h, f, f_norm, gate, norm, out and u must be 16-byte aligned", name);
  if ((uintptr_t)a.q & 3) return fail(WQ_ERR_ALIGN, "%s: q must be 4-byte aligned", name);
  return WQ_OK;
}

static int norm_overlap(const char* name, const wq_block_norm& a) {
  auto rows = [&](const void* p32, const void* p16, int64_t stride) {
    return ByteRows{p32 ? p32 : p16, a.rows, (p32 ? 4 : 2) * stride, (p32 ? 4 : 2) * a.dim};
  };
  const ByteRows h = rows(a.h_f32, a.h_bf16, a.h_stride), f = rows(a.f_f32, a.f_bf16, a.f_stride);
  const ByteRows out[] = {rows(a.out_f32, a.out_bf16, a.out_stride),
                          {a.u, a.rows, 2 * a.u_stride, 2 * a.dim},
                          {a.q, 1, 0, a.rows * a.dim / 2},
                          {a.q_scale, 1, 0, a.rows * a.dim / kMxGroup}};
  const ByteRows gate{a.gate, a.gate_stride ? a.rows : 1, 2 * a.gate_stride, 2 * a.dim};
  const ByteRows in[] = {f, gate, {a.f_norm, 1, 0, 2 * a.dim}, {a.norm, 1, 0, 2 * a.dim}};
  // a row is read before it is written, so h may be updated in place
  const bool same = (a.out_f32 ? (const void*)a.out_f32 == a.h_f32 : a.out_bf16 && a.out_bf16 == a.h_bf16) &&
                    (a.out_stride == a.h_stride || a.rows <= 1);
  for (int i = 0; i < 4; ++i) {
    for (const ByteRows& r : in)
      if (rows_meet(out[i], r)) return fail(WQ_ERR_SHAPE, "%s: out, u and q must not overlap f, gate or the norms", name);
    if (!(i == 0 && same) && rows_meet(out[i], h))
      return fail(WQ_ERR_SHAPE, "%s: out must be h itself or overlap no input, u and q overlap none", name);
    for (int j = 0; j < i; ++j)
      if (rows_meet(out[i], out[j])) return fail(WQ_ERR_SHAPE, "%s: out, u, q and q_scale must not overlap", name);
  }
  return WQ_OK;
}

template <class A>
static void norm_launch(const NormArgs& a, int64_t rows, hipStream_t s) {
  const int pieces = a.dim / 8;
  // a grid's axis holds less than 2^32 threads
  const int64_t wide = rows < kNormGridX ? rows : kNormGridX;
  const dim3 grid((unsigned)wide, (unsigned)((rows + wide - 1) / wide));
  // Enough threads that a row's loads are all under way, few enough that several rows share
  // a CU while others sum or store: 4099 rows of 8192 in fp64 110 us with 512 threads of two
  // pieces, 120 with 256 of four, 175 with 1024 of one.
  if (pieces <= 64)
    hipLaunchKernelGGL((block_norm_kernel<A, 1, 64>), grid, dim3(64), 0, s, a);
  else if (pieces <= 256)
    hipLaunchKernelGGL((block_norm_kernel<A, 1, 256>), grid, dim3(256), 0, s, a);
  else if (pieces <= 512)
    hipLaunchKernelGGL((block_norm_kernel<A, 2, 256>), grid, dim3(256), 0, s, a);
  else if (pieces <= 1024)
    hipLaunchKernelGGL((block_norm_kernel<A, 2, 512>), grid, dim3(512), 0, s, a);
  else if (pieces <= 2048)
    hipLaunchKernelGGL((block_norm_kernel<A, 4, 512>), grid, dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((block_norm_kernel<A, 4, 1024>), grid, dim3(1024), 0, s, a);
}

}  // namespace wq

using namespace wq;

extern "C" int wq_block_norm_prepare(const wq_block_norm* a, wq_block_norm_plan* plan) {
  const char* name = "wq_block_norm_prepare";
  if (!a || !plan) return fail(WQ_ERR_NULL, "%s: a and plan must be non-null", name);
  int rc = norm_check(name, *a);
  if (rc) return rc;
  if ((rc = norm_overlap(name, *a))) return rc;
  wq_block_norm_plan p{};
  if ((rc = plan_device(name, &p.device))) return rc;
  p.made = kNormMade;
  p.a = *a;
  *plan = p;
  return WQ_OK;
}

extern "C" int wq_block_norm_run(const wq_block_norm_plan* plan, void* stream) {
  const char* name = "wq_block_norm_run";
  if (!plan) return fail(WQ_ERR_NULL, "%s: plan must be non-null", name);
  if (plan->made != kNormMade) return fail(WQ_ERR_SHAPE, "%s: the plan was not made by wq_block_norm_prepare", name);
  int rc = same_device(name, plan->device);
  if (rc) return rc;
  const wq_block_norm& n = plan->a;
  if (n.rows == 0) return WQ_OK;
  const NormArgs a{n.h_f32,     n.h_bf16, n.h_stride,    n.out_f32, n.out_bf16, n.out_stride, n.f_f32, n.f_bf16,
                   n.f_stride,  n.f_norm, n.gate,        n.gate_stride, n.norm, n.u,          n.u_stride, n.q,
                   n.q_scale,   (int32_t)n.dim, (int32_t)n.rows, n.scale, n.eps,     n.gate_kind};
  hipStream_t s = (hipStream_t)stream;
  if (n.q)
    norm_launch<double>(a, n.rows, s);
  else
    norm_launch<float>(a, n.rows, s);
  return launch_status(name);
}
