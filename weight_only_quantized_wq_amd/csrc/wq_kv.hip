// What a verify pass does to the paged key/value cache: norms, rotation and
// append behind wqkv (wq_qkv_rope), and the move of accepted rows
// (wq_kv_accept); the rotary frequencies; the checks of cache descriptions.
#include <math.h>

#include <type_traits>

#include "wq_kv.hpp"

namespace wq {

// ---------------------------------------------------------------------------
// Host checks

int check_cache_null(const char* name, const wq_kv_cache& c) {
  if (!c.k || !c.v || !c.table) return fail(WQ_ERR_NULL, "%s: cache k, v and table must be non-null", name);
  return WQ_OK;
}

int check_cache_sizes(const char* name, const wq_kv_cache& c) {
  if (c.pages < 1 || c.pages > 0x7FFFFFFF || c.page_size < 1 || c.page_size > 0x7FFFFFFF)
    return fail(WQ_ERR_SHAPE, "%s: pages = %lld, page_size = %lld must be positive", name, (long long)c.pages,
                (long long)c.page_size);
  if (c.table_width < 1 || c.table_width > 0x7FFFFFFF || c.table_stride < c.table_width ||
      c.table_width * c.page_size > kMaxPositions)
    return fail(WQ_ERR_SHAPE, "%s: table_width = %lld (stride %lld) pages of %lld positions", name,
                (long long)c.table_width, (long long)c.table_stride, (long long)c.page_size);
  if (c.kv_heads < 1 || c.kv_heads > kMaxHeads)
    return fail(WQ_ERR_SHAPE, "%s: kv_heads = %d must be in [1, %d]", name, c.kv_heads, kMaxHeads);
  if (c.head_dim < 8 || c.head_dim > 256 || c.head_dim % 8)
    return fail(WQ_ERR_SHAPE, "%s: head_dim = %d must be a multiple of 8 up to 256", name, c.head_dim);
  const int64_t most = 0xFFFFFFFFll;
  for (int64_t s : {c.page_stride, c.token_stride, c.head_stride})
    if (s < 0 || s > most || s % 8)
      return fail(WQ_ERR_SHAPE, "%s: cache strides (%lld, %lld, %lld) must be multiples of 8 in [0, 2^32)", name,
                  (long long)c.page_stride, (long long)c.token_stride, (long long)c.head_stride);
  return WQ_OK;
}

int check_cache_align(const char* name, const wq_kv_cache& c) {
  if (!aligned16(c.k) || !aligned16(c.v) || ((uintptr_t)c.table & 3))
    return fail(WQ_ERR_ALIGN, "%s: cache k and v must be 16-byte, the table 4-byte aligned", name);
  return WQ_OK;
}

int check_batch_sizes(const char* name, const wq_batch& b) {
  if (b.tokens < 0 || b.tokens > kMaxBatchTokens || b.requests < 0 || b.requests > kMaxRequests)
    return fail(WQ_ERR_SHAPE, "%s: tokens = %lld, requests = %lld must be in [0, 2^20] and [0, %lld]", name,
                (long long)b.tokens, (long long)b.requests, (long long)kMaxRequests);
  return WQ_OK;
}

KvCache device_cache(const wq_kv_cache& c) {
  KvCache d{};
  d.k = c.k;
  d.v = c.v;
  d.page_stride = (uint32_t)c.page_stride;
  d.token_stride = (uint32_t)c.token_stride;
  d.head_stride = (uint32_t)c.head_stride;
  d.table = c.table;
  d.table_stride = c.table_stride;
  if (c.page_size > 1) {
    int l = 0;
    while (((int64_t)1 << l) < c.page_size) ++l;
    d.shift = l - 1;
    d.magic = (uint32_t)(2 * ((((uint64_t)1 << (30 + l)) / (uint64_t)c.page_size) + 1));
  }
  d.pages = (uint32_t)c.pages;
  d.page_size = (uint32_t)c.page_size;
  d.limit = (uint32_t)(c.table_width * c.page_size);
  d.kv_heads = c.kv_heads;
  d.head_dim = c.head_dim;
  return d;
}

bool rows_meet(const ByteRows& a, const ByteRows& b) {
  if (!a.at || !b.at || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
  // in order of address; rows of one buffer do not overlap (stride >= width, below
  // 2^43; of a single row it may be anything)
  uint64_t x = (uint64_t)(uintptr_t)a.at, y = (uint64_t)(uintptr_t)b.at;
  const uint64_t xs = a.rows > 1 ? a.stride : a.width, ys = b.rows > 1 ? b.stride : b.width;
  const uint64_t xe = x + (a.rows - 1) * xs, ye = y + (b.rows - 1) * ys;
  if (xe + a.width <= y || ye + b.width <= x) return false;
  while (x <= xe && y <= ye) {
    if (x + a.width <= y)
      x += xs;
    else if (y + b.width <= x)
      y += ys;
    else
      return true;
  }
  return false;
}

int plan_device(const char* name, int32_t* device) {
  int rc = check_device();
  if (rc) return rc;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) {
    (void)hipGetLastError();
    return fail(WQ_ERR_DEVICE, "%s: no current HIP device", name);
  }
  *device = dev;
  return WQ_OK;
}

int same_device(const char* name, int32_t device) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev != device) {
    (void)hipGetLastError();
    return fail(WQ_ERR_DEVICE, "%s: the plan was prepared on device %d, the current one is %d", name, device, dev);
  }
  return WQ_OK;
}

// ---------------------------------------------------------------------------
// Norms, rotation, append
//
// One workgroup takes one token (with few tokens, a share of its heads).  The
// token's first heads are requested, its request is looked up and its rot_dim /
// 2 angles are reduced in fp64 and turned into (cos, sin) once, in LDS; then
// every P = pow2(head_dim / 8) lanes take a head, 8 elements a lane, so that a
// head is read and written in 16-byte pieces, its square sum is a butterfly over
// P lanes and the partner of a rotated element is in the lane itself
// (interleaved), in a lane a fixed distance away (halves of a multiple of 8) or
// fetched through LDS (other halves).
//
// Measured (MI355X): 4095 rows of 32 / 8 heads of 128 with norms, 22 us (101 MB, 4.6
// TB/s), where the vector ALU is busy most of the time and waves in plenty hide the
// rest: one head at a time and 64 registers, since four requested at once (80
// registers) took 27.0 us, two 26.4.  32 x 5 rows of 64 / 8 heads, fp32: 4.9 us, 9.8
// MB, hardly more than a launch (one row: 3.4).

struct RopeArgs {
  KvCache c;
  Batch b;
  const void* qkv;
  int64_t qkv_stride;
  uint16_t* q;
  int64_t q_stride;
  const int32_t* positions;
  const uint16_t* q_norm;
  const uint16_t* k_norm;
  const float* freq;
  float eps;
  float per_dim;       // 1 / head_dim
  float rot_scale;
  int32_t rot_dim;
  int32_t heads;
  int32_t lanes;       // lanes per head (power of two)
};

enum { kPairs = 0, kHalves = 1, kOddHalves = 2 };
constexpr int kRopeThreads = 256;

// Eight elements of a head as loaded.
template <bool F32>
struct Head8 {
  u32x4 w[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* qkv, int64_t at) {
    const u32x4* p = reinterpret_cast<const u32x4*>(F32 ? (const void*)(static_cast<const float*>(qkv) + at)
                                                        : (const void*)(static_cast<const uint16_t*>(qkv) + at));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) w[i] = load16(p + i);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = F32 ? __uint_as_float(w[F32 ? e / 4 : 0][e & 3]) : e & 1 ? bf16hi_to_f32(w[0][e / 2]) : bf16lo_to_f32(w[0][e / 2]);
  }
};

// Sum over aligned groups of `lanes` lanes (a power of two up to 32).
__device__ __forceinline__ float group_sum(float v, int lanes) {
  if (lanes >= 2) v += dpp_f<0xB1>(v);       // quad_perm [1,0,3,2]
  if (lanes >= 4) v += dpp_f<0x4E>(v);       // quad_perm [2,3,0,1]
  if (lanes >= 8) v += dpp_f<0x141>(v);      // row_half_mirror
  if (lanes >= 16) v += dpp_f<0x140>(v);     // row_mirror
  if (lanes >= 32) v += __shfl_xor(v, 16);
  return v;
}

// other[e] = x[e] of the lane `far` on (the first `far` lanes of a head) or back
// (the next `far`); without the LDS crossbar where that is an exchange of bits.
__device__ __forceinline__ void partners(const float (&x)[8], float (&other)[8], int lane, int sub, int far) {
  if (far == 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = dpp_f<0x128>(x[e]);                 // row_ror 8
  } else if (far == 4) {
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = dpp_f<0x1B>(dpp_f<0x141>(x[e]));    // 7 - i, then 3 - i in each quad
  } else if (far == 2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = dpp_f<0x4E>(x[e]);
  } else if (far == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = dpp_f<0xB1>(x[e]);
  } else {
    const int from = lane + (sub < far ? far : sub < 2 * far ? -far : 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = __shfl(x[e], from);
  }
}

// 1 / sqrt(m).  The instruction takes a subnormal m for 0.  An eps of 2^-126 or more
// rules that out; below (TINY) such an m is scaled by 2^48, and the result by 2^24.
// (An instantiation of its own: 4095 rows take 20.3 us with it, 19.6 without.)
template <bool TINY>
__device__ __forceinline__ float inverse_root(float m) {
  if (!TINY) return __builtin_amdgcn_rsqf(m);
  const bool tiny = m < 0x1p-126f;
  return __builtin_amdgcn_rsqf(tiny ? m * 0x1p48f : m) * (tiny ? 0x1p24f : 1.f);
}

template <bool F32, int LAYOUT, bool TINY>
__global__ __launch_bounds__(kRopeThreads) void qkv_rope_kernel(RopeArgs a) {
  __shared__ float2 turn[128];
  __shared__ float exch[LAYOUT == kOddHalves ? kRopeThreads * 8 : 1];
  const int t = blockIdx.x;
  const int lane = lane_id();
  const int dim = a.c.head_dim, kv = a.c.kv_heads, heads = a.heads, all = heads + 2 * kv;
  const int sub = (int)threadIdx.x & (a.lanes - 1);        // lane within the head
  const int step = (int)gridDim.y * (kRopeThreads / a.lanes);
  const bool in = sub * 8 < dim;
  const int h0 = (int)(blockIdx.y * (kRopeThreads / a.lanes) + threadIdx.x / a.lanes);
  Head8<F32> raw;
  const auto request = [&](int h) {
    if (in && h < all) raw.load(a.qkv, (int64_t)t * a.qkv_stride + (int64_t)h * dim + sub * 8);
  };
  request(h0);
  // the token's request: how many of starts[1 ..] lie at or before it
  int r = 0;
  for (int i = 1 + lane; i - lane <= a.b.requests; i += kWave)
    r += __popcll(__ballot(i <= a.b.requests && gmem(a.b.starts)[i < a.b.requests ? i : a.b.requests] <= t));
  if (r >= a.b.requests) return;
  const int s0 = gmem(a.b.starts)[r];
  if (s0 < 0 || s0 > t) return;
  const int64_t length = max(gmem(a.b.lengths)[r], 0);
  const int64_t slot = length + (t - s0);
  const int half = a.rot_dim >> 1;
  if ((int)threadIdx.x < half) {
    const double pos = a.positions ? (double)gmem(a.positions)[t] : (double)slot;
    // turns of the circle; the fraction is exact to 2^-52 of the angle
    const double turns = pos * (double)gmem(a.freq)[threadIdx.x] * 0.15915494309189533577;
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    turn[threadIdx.x] = make_float2(c * a.rot_scale, s * a.rot_scale);
  }
  const int64_t cache_row = position_offset(a.c, r, slot);
  Head8<false> weight[2];              // q_norm, k_norm
  if (in && a.q_norm) weight[0].load(a.q_norm, sub * 8);
  if (in && a.k_norm) weight[1].load(a.k_norm, sub * 8);
  __syncthreads();
  // the lane's factors are the same for every head: o = x * cs + partner * sn
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int at = sub * 8 + e;
    const bool first = LAYOUT == kPairs ? !(e & 1) : at < half;
    const int i = LAYOUT == kPairs ? at / 2 : first ? at : at - half;
    const float2 f = at < 2 * half ? turn[i] : make_float2(1.f, 0.f);
    cs[e] = f.x;
    sn[e] = first ? -f.y : f.y;
  }

  const int first = h0 - (int)threadIdx.x / a.lanes;        // the workgroup's first head
  for (int from = first, h = h0; from < all; from += step, h += step) {       // the same trips for the whole workgroup
    const bool on = in && h < all;
    if (h != h0) request(h);
    if (!F32 && __builtin_amdgcn_readfirstlane(h) >= heads + kv) {
      // a wave of nothing but values only copies
      if (on && cache_row >= 0)
        *gmem(reinterpret_cast<u32x4*>(a.c.v + cache_row + (int64_t)(h - heads - kv) * a.c.head_stride + sub * 8)) = raw.w[0];
      continue;
    }
    float x[8];
    if (on) {
      raw.values(x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
    const bool key = h >= heads, value = h >= heads + kv;
    if (a.q_norm || a.k_norm) {
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
      sq = group_sum(sq, a.lanes);
      if (!value && (key ? a.k_norm : a.q_norm)) {
        const float f = inverse_root<TINY>(fmaf(sq, a.per_dim, a.eps));
        Head8<false> ws;
#pragma unroll
        for (int i = 0; i < 4; ++i) ws.w[0][i] = key ? weight[1].w[0][i] : weight[0].w[0][i];
        float w[8];
        ws.values(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * f * w[e];
      }
    }
    float other[8];
    if (LAYOUT == kPairs) {
#pragma unroll
      for (int e = 0; e < 8; ++e) other[e] = x[e ^ 1];
    } else if (LAYOUT == kHalves) {
      partners(x, other, lane, sub, half / 8);
    } else {
      // a wave reads only what it wrote itself
      float* row = exch + ((int)threadIdx.x - sub) * 8;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int e = 0; e < 8; ++e) row[sub * 8 + e] = x[e];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = sub * 8 + e;
        other[e] = row[i < half ? i + half : i < 2 * half ? i - half : i];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    if (!on) continue;
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float o[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = 2 * e + i;
        // elements past rot_dim, and values, stay as they are (whatever the partner is)
        const bool turns = !value && sub * 8 + k < 2 * half;
        o[i] = turns ? fmaf(other[k], sn[k], x[k] * cs[k]) : x[k];
      }
      const bf16x2 two = {(__bf16)o[0], (__bf16)o[1]};
      w[e] = __builtin_bit_cast(uint32_t, two);
    }
    uint16_t* to;
    if (!key) {
      to = a.q + (int64_t)t * a.q_stride + (int64_t)h * dim;
    } else {
      if (cache_row < 0) continue;
      to = (value ? a.c.v : a.c.k) + cache_row + (int64_t)(h - heads - (value ? kv : 0)) * a.c.head_stride;
    }
    *gmem(reinterpret_cast<u32x4*>(to + sub * 8)) = w;
  }
}

constexpr int64_t kRopeMade = 0x77715f726f706531;

static int rope_check(const char* name, const wq_qkv_rope& a) {
  int rc = check_cache_null(name, a.cache);
  if (rc) return rc;
  if (!a.batch.starts || !a.batch.lengths || !a.q) return fail(WQ_ERR_NULL, "%s: starts, lengths and q must be non-null", name);
  if (!a.qkv_f32 == !a.qkv_bf16) return fail(WQ_ERR_NULL, "%s: exactly one of qkv_f32 and qkv_bf16 must be given", name);
  if (!a.freq && a.rot_dim != 0) return fail(WQ_ERR_NULL, "%s: freq must be non-null where rot_dim is not 0", name);
  if ((rc = check_cache_sizes(name, a.cache)) || (rc = check_batch_sizes(name, a.batch))) return rc;
  const int64_t dim = a.cache.head_dim, kv = a.cache.kv_heads;
  if (a.heads < 1 || a.heads > kMaxHeads || a.heads % kv)
    return fail(WQ_ERR_SHAPE, "%s: heads = %d must be a multiple of kv_heads = %lld up to %d", name, a.heads,
                (long long)kv, kMaxHeads);
  if (a.rot_dim < 0 || a.rot_dim > dim || a.rot_dim % 2)
    return fail(WQ_ERR_SHAPE, "%s: rot_dim = %d must be even and at most head_dim", name, a.rot_dim);
  const int64_t most = (int64_t)1 << 40, unit = a.qkv_f32 ? 4 : 8;
  if (a.qkv_stride < (a.heads + 2 * kv) * dim || a.qkv_stride > most || a.qkv_stride % unit)
    return fail(WQ_ERR_SHAPE, "%s: qkv_stride = %lld must be a multiple of %lld and hold a row", name,
                (long long)a.qkv_stride, (long long)unit);
  if (a.q_stride < a.heads * dim || a.q_stride > most || a.q_stride % 8)
    return fail(WQ_ERR_SHAPE, "%s: q_stride = %lld must be a multiple of 8 and hold a row", name, (long long)a.q_stride);
  if (!(a.eps >= 0.f) || !(fabsf(a.rot_scale) < INFINITY))
    return fail(WQ_ERR_SHAPE, "%s: eps must not be negative, rot_scale must be finite", name);
  if ((rc = check_cache_align(name, a.cache))) return rc;
  if (!aligned16(a.qkv_f32) || !aligned16(a.qkv_bf16) || !aligned16(a.q) || !aligned16(a.q_norm) || !aligned16(a.k_norm))
    return fail(WQ_ERR_ALIGN, "%s: qkv, q and the norm weights must be 16-byte aligned", name);
  return WQ_OK;
}

template <bool F32, bool TINY>
static void rope_launch(const RopeArgs& r, int layout, dim3 grid, hipStream_t s) {
  if (layout == kPairs)
    hipLaunchKernelGGL((qkv_rope_kernel<F32, kPairs, TINY>), grid, dim3(kRopeThreads), 0, s, r);
  else if (layout == kHalves)
    hipLaunchKernelGGL((qkv_rope_kernel<F32, kHalves, TINY>), grid, dim3(kRopeThreads), 0, s, r);
  else
    hipLaunchKernelGGL((qkv_rope_kernel<F32, kOddHalves, TINY>), grid, dim3(kRopeThreads), 0, s, r);
}

// ---------------------------------------------------------------------------
// Accepted rows
//
// Thread (request, layer, 16-byte column of a K or V row) copies its column of
// every accepted row in order.  The path increases, so path[i] >= i: target i
// is never the source of a later row, and copying in order by one thread needs
// no second buffer.  32 layers x 32 requests, 26 MB moved: 7.9 us (3.3 TB/s); one
// layer of one request: a launch.

struct AcceptArgs {
  KvCache c;
  int64_t layer_stride;
  const int32_t* lengths;
  const int32_t* path;
  const int32_t* accepted;
  int64_t path_stride;
  int32_t path_width;
};

constexpr int kAcceptThreads = 256;
constexpr int kAcceptBatch = 8;

__global__ __launch_bounds__(kAcceptThreads) void kv_accept_kernel(AcceptArgs a) {
  const int r = blockIdx.x, lane = lane_id();
  // all of the path, however much is accepted: one round of loads
  const int listed = lane < a.path_width ? gmem(a.path)[(int64_t)r * a.path_stride + lane] : 0;
  const int64_t length = max(gmem(a.lengths)[r], 0);
  const int n = min(max(gmem(a.accepted)[r], 0), a.path_width);
  const int step = lane < n ? listed : 0x7FFFFFFF;
  const int before = __shfl_up(step, 1);
  const bool bad = lane < n && (lane == 0 ? step < 0 : step <= before);
  if (__any(bad)) return;
  int64_t from = -1, to = -1;
  if (lane < n && step != lane) {
    from = position_offset(a.c, r, length + step);
    to = position_offset(a.c, r, length + lane);
  }
  uint64_t moves = __ballot(from >= 0 && to >= 0);
  const int cols = a.c.head_dim / 8;
  const int per_head = 2 * cols;
  const int at = (int)(blockIdx.z * kAcceptThreads + threadIdx.x);
  const bool on = at < a.c.kv_heads * per_head;
  const int head = at / per_head, col = at % per_head;
  uint16_t* base = (col < cols ? a.c.k : a.c.v) + (int64_t)blockIdx.y * a.layer_stride +
                   (int64_t)head * a.c.head_stride + (int64_t)(col % cols) * 8;
  while (moves) {
    u32x4 x[kAcceptBatch];
    int64_t target[kAcceptBatch];
    int m = 0;
#pragma unroll
    for (int i = 0; i < kAcceptBatch; ++i) {
      target[i] = -1;
      if (moves) {
        const int src = __builtin_ctzll(moves);
        moves &= moves - 1;
        const int64_t f = __shfl(from, src);
        target[i] = __shfl(to, src);
        if (on) x[i] = load16(base + f);
        ++m;
      }
    }
#pragma unroll
    for (int i = 0; i < kAcceptBatch; ++i)
      if (on && i < m) *gmem(reinterpret_cast<u32x4*>(base + target[i])) = x[i];
  }
}

constexpr int64_t kAcceptMade = 0x77715f61636331;

static int accept_check(const char* name, const wq_kv_accept& a) {
  int rc = check_cache_null(name, a.cache);
  if (rc) return rc;
  if (!a.lengths || !a.path || !a.accepted)
    return fail(WQ_ERR_NULL, "%s: lengths, path and accepted must be non-null", name);
  if ((rc = check_cache_sizes(name, a.cache))) return rc;
  if (a.layers < 1 || a.layers > 4096 || a.layer_stride < 0 || a.layer_stride > (int64_t)1 << 40 ||
      a.layer_stride % 8 || (a.layers > 1 && a.layer_stride == 0))
    return fail(WQ_ERR_SHAPE, "%s: layers = %lld (1..4096), layer_stride = %lld (a positive multiple of 8)", name,
                (long long)a.layers, (long long)a.layer_stride);
  if (a.requests < 0 || a.requests > kMaxRequests)
    return fail(WQ_ERR_SHAPE, "%s: requests = %lld must be in [0, %lld]", name, (long long)a.requests,
                (long long)kMaxRequests);
  if (a.path_width < 1 || a.path_width > 64 || a.path_stride < a.path_width)
    return fail(WQ_ERR_SHAPE, "%s: path_width = %lld must be in [1, 64] and path_stride hold it", name,
                (long long)a.path_width);
  return check_cache_align(name, a.cache);
}

}  // namespace wq

using namespace wq;

extern "C" int wq_rope_frequencies(int32_t kind, int32_t rot_dim, double base, double factor, double low, double high,
                                   double original, float* freq_host, float* rot_scale) {
  const char* name = "wq_rope_frequencies";
  if (!freq_host) return fail(WQ_ERR_NULL, "%s: freq_host must be non-null", name);
  if (kind < WQ_ROPE_PLAIN || kind > WQ_ROPE_RAMP) return fail(WQ_ERR_SHAPE, "%s: kind = %d is unknown", name, kind);
  if (rot_dim < 2 || rot_dim > 256 || rot_dim % 2 || !(base > 1.0) || !(base < 1e300))
    return fail(WQ_ERR_SHAPE, "%s: rot_dim = %d must be even in [2, 256], base = %g above 1", name, rot_dim, base);
  if (kind != WQ_ROPE_PLAIN && (!(factor >= 1.0) || !(factor < 1e300)))
    return fail(WQ_ERR_SHAPE, "%s: factor = %g must be at least 1", name, factor);
  if (kind >= WQ_ROPE_BANDS && !(low > 0.0 && low < high && high < 1e300 && original >= 1.0 && original < 1e300))
    return fail(WQ_ERR_SHAPE, "%s: 0 < low = %g < high = %g and original = %g >= 1 are needed", name, low, high, original);
  const double two_pi = 6.283185307179586477;
  double first = 0.0, last = 0.0;
  if (kind == WQ_ROPE_RAMP) {
    const double per = rot_dim / (2.0 * log(base));
    first = fmin(fmax(floor(per * log(original / (two_pi * high))), 0.0), rot_dim - 1.0);
    last = fmin(fmax(ceil(per * log(original / (two_pi * low))), 0.0), rot_dim - 1.0);
    if (last <= first) last = first + 0.001;      // a step instead of a slope
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rot_dim);
    if (kind == WQ_ROPE_LINEAR) {
      f /= factor;
    } else if (kind == WQ_ROPE_BANDS) {
      const double t = (original * f / two_pi - low) / (high - low);
      const double share = fmin(fmax(t, 0.0), 1.0);
      f *= (1.0 - share) / factor + share;
    } else if (kind == WQ_ROPE_RAMP) {
      const double share = fmin(fmax((i - first) / (last - first), 0.0), 1.0);
      f *= share / factor + (1.0 - share);
    }
    freq_host[i] = (float)f;
  }
  if (rot_scale) *rot_scale = kind == WQ_ROPE_RAMP ? (float)(0.1 * log(factor) + 1.0) : 1.f;
  return WQ_OK;
}

extern "C" int wq_qkv_rope_prepare(const wq_qkv_rope* a, wq_qkv_rope_plan* plan) {
  const char* name = "wq_qkv_rope_prepare";
  if (!a || !plan) return fail(WQ_ERR_NULL, "%s: a and plan must be non-null", name);
  int rc = rope_check(name, *a);
  if (rc) return rc;
  // the workgroups of a row read and write its heads in no order
  const int64_t dim = a->cache.head_dim, heads = a->heads, all = heads + 2 * a->cache.kv_heads;
  const int64_t unit = a->qkv_f32 ? 4 : 2;
  const void* qkv = a->qkv_f32 ? (const void*)a->qkv_f32 : (const void*)a->qkv_bf16;
  if (rows_meet({a->q, a->batch.tokens, 2 * a->q_stride, 2 * heads * dim},
                {qkv, a->batch.tokens, unit * a->qkv_stride, unit * all * dim}))
    return fail(WQ_ERR_SHAPE, "%s: q must not overlap qkv", name);
  wq_qkv_rope_plan p{};
  if ((rc = plan_device(name, &p.device))) return rc;
  p.made = kRopeMade;
  p.a = *a;
  *plan = p;
  return WQ_OK;
}

extern "C" int wq_qkv_rope_run(const wq_qkv_rope_plan* plan, void* stream) {
  const char* name = "wq_qkv_rope_run";
  if (!plan) return fail(WQ_ERR_NULL, "%s: plan must be non-null", name);
  if (plan->made != kRopeMade) return fail(WQ_ERR_SHAPE, "%s: the plan was not made by wq_qkv_rope_prepare", name);
  int rc = same_device(name, plan->device);
  if (rc) return rc;
  const wq_qkv_rope& a = plan->a;
  if (a.batch.tokens == 0 || a.batch.requests == 0) return WQ_OK;
  RopeArgs r{};
  r.c = device_cache(a.cache);
  r.b = device_batch(a.batch);
  r.qkv = a.qkv_f32 ? (const void*)a.qkv_f32 : (const void*)a.qkv_bf16;
  r.qkv_stride = a.qkv_stride;
  r.q = a.q;
  r.q_stride = a.q_stride;
  r.positions = a.positions;
  r.q_norm = a.q_norm;
  r.k_norm = a.k_norm;
  r.freq = a.freq;
  r.eps = a.eps;
  r.per_dim = 1.f / (float)a.cache.head_dim;
  r.rot_scale = a.rot_scale;
  r.rot_dim = a.rot_dim;
  r.heads = a.heads;
  r.lanes = 1;
  while (r.lanes * 8 < a.cache.head_dim) r.lanes *= 2;
  // few tokens: their heads are shared out to fill the chip.  Measured, one / about
  // 512 workgroups: one row of 32 heads 4.9 / 3.4 us, 160 rows of 64 / 8 heads 6.9 / 4.9.
  const int64_t per_block = kRopeThreads / r.lanes;
  const int64_t most = (a.heads + 2 * a.cache.kv_heads + per_block - 1) / per_block;
  int64_t split = 512 / a.batch.tokens;
  split = split < 1 ? 1 : split > most ? most : split;
  const dim3 grid((unsigned)a.batch.tokens, (unsigned)split);
  const int layout = a.interleaved ? kPairs : a.rot_dim % 16 == 0 ? kHalves : kOddHalves;
  const bool tiny = a.eps < 0x1p-126f && (a.q_norm || a.k_norm);
  const auto launch = a.qkv_f32 ? (tiny ? rope_launch<true, true> : rope_launch<true, false>)
                                : (tiny ? rope_launch<false, true> : rope_launch<false, false>);
  launch(r, layout, grid, (hipStream_t)stream);
  return launch_status(name);
}

extern "C" int wq_kv_accept_prepare(const wq_kv_accept* a, wq_kv_accept_plan* plan) {
  const char* name = "wq_kv_accept_prepare";
  if (!a || !plan) return fail(WQ_ERR_NULL, "%s: a and plan must be non-null", name);
  int rc = accept_check(name, *a);
  if (rc) return rc;
  wq_kv_accept_plan p{};
  if ((rc = plan_device(name, &p.device))) return rc;
  p.made = kAcceptMade;
  p.a = *a;
  *plan = p;
  return WQ_OK;
}

extern "C" int wq_kv_accept_run(const wq_kv_accept_plan* plan, void* stream) {
  const char* name = "wq_kv_accept_run";
  if (!plan) return fail(WQ_ERR_NULL, "%s: plan must be non-null", name);
  if (plan->made != kAcceptMade) return fail(WQ_ERR_SHAPE, "%s: the plan was not made by wq_kv_accept_prepare", name);
  int rc = same_device(name, plan->device);
  if (rc) return rc;
  const wq_kv_accept& a = plan->a;
  if (a.requests == 0) return WQ_OK;
  AcceptArgs r{};
  r.c = device_cache(a.cache);
  r.layer_stride = a.layer_stride;
  r.lengths = a.lengths;
  r.path = a.path;
  r.accepted = a.accepted;
  r.path_stride = a.path_stride;
  r.path_width = (int32_t)a.path_width;
  const int pieces = a.cache.kv_heads * (a.cache.head_dim / 4);
  const dim3 grid((unsigned)a.requests, (unsigned)a.layers, (unsigned)((pieces + kAcceptThreads - 1) / kAcceptThreads));
  hipLaunchKernelGGL(kv_accept_kernel, grid, dim3(kAcceptThreads), 0, (hipStream_t)stream, r);
  return launch_status(name);
}
