// Paged key/value cache and batch descriptions on the device, and their
// host-side checks (wq_kv_cache, wq_batch); wave sums and maxima of the calls
// between the linears.
#pragma once

#include <stdint.h>

#include <type_traits>

#include "wq_device.hpp"
#include "wq_host.hpp"

namespace wq {

struct KvCache {
  uint16_t* k;
  uint16_t* v;
  const int32_t* table;
  int64_t table_stride;
  uint32_t page_stride;
  uint32_t token_stride;
  uint32_t head_stride;
  uint32_t magic;      // page of a position, see page_of
  int32_t shift;
  uint32_t pages;
  uint32_t page_size;
  uint32_t limit;      // positions the table covers
  int32_t kv_heads;
  int32_t head_dim;
};

struct Batch {
  const int32_t* starts;
  const int32_t* lengths;
  int32_t tokens;
  int32_t requests;
};

// Sum over the lanes up to and with this one (DPP, lanes a step does not reach add 0).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr 1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast31 into rows 2 and 3
  return v;
}

// Wave-wide maximum (lanes a step does not reach see -inf).
__device__ __forceinline__ float wave_max(float v) {
  const auto step = [](float x, auto ctrl, auto rows) {
    return fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp((int)0xFF800000, __float_as_int(x), decltype(ctrl)::value,
                                                               decltype(rows)::value, 0xF, false)));
  };
  using std::integral_constant;
  v = step(v, integral_constant<int, 0xB1>{}, integral_constant<int, 0xF>{});
  v = step(v, integral_constant<int, 0x4E>{}, integral_constant<int, 0xF>{});
  v = step(v, integral_constant<int, 0x141>{}, integral_constant<int, 0xF>{});
  v = step(v, integral_constant<int, 0x140>{}, integral_constant<int, 0xF>{});
  v = step(v, integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});
  v = step(v, integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Page index of a position below 2^30.  With l = ceil(log2(page_size)) >= 1,
// magic = 2 (floor(2^(30 + l) / page_size) + 1) and shift = l - 1 the quotient
// position * magic / 2^(31 + l) exceeds the true one by less than position /
// 2^(30 + l) < 1 / page_size, so its integer part is exact.  (Pages of one
// position: magic 0.)
__device__ __forceinline__ uint32_t page_of(const KvCache& c, uint32_t p) {
  return c.magic ? __umulhi(p, c.magic) >> c.shift : p;
}

// Element offset of row `row` of page `pid` (head 0).
__device__ __forceinline__ uint64_t row_offset(const KvCache& c, uint32_t pid, uint32_t row) {
  return (uint64_t)pid * c.page_stride + (uint64_t)row * c.token_stride;
}

// Element offset of request r's position p (head 0), or -1 if it holds nothing.
__device__ __forceinline__ int64_t position_offset(const KvCache& c, int r, int64_t p) {
  if (p < 0 || p >= (int64_t)c.limit) return -1;
  const uint32_t pg = page_of(c, (uint32_t)p);
  const uint32_t pid = (uint32_t)gmem(c.table)[(int64_t)r * c.table_stride + pg];
  if (pid >= c.pages) return -1;
  return (int64_t)row_offset(c, pid, (uint32_t)p - pg * c.page_size);
}

// Host: checks (sizes, then alignment) and the device view.
int check_cache_null(const char* name, const wq_kv_cache& c);
int check_cache_sizes(const char* name, const wq_kv_cache& c);
int check_cache_align(const char* name, const wq_kv_cache& c);
int check_batch_sizes(const char* name, const wq_batch& b);
KvCache device_cache(const wq_kv_cache& c);

inline Batch device_batch(const wq_batch& b) {
  return Batch{b.starts, b.lengths, (int32_t)b.tokens, (int32_t)b.requests};
}

// Rows of a buffer, in bytes; whether two such buffers share any (columns of one
// wider buffer side by side do not).
struct ByteRows {
  const void* at;
  int64_t rows, stride, width;
};
bool rows_meet(const ByteRows& a, const ByteRows& b);

// The device a plan is bound to: recorded by prepare, compared by run.
int plan_device(const char* name, int32_t* device);
int same_device(const char* name, int32_t device);

constexpr int64_t kMaxBatchTokens = 1 << 20;
constexpr int64_t kMaxRequests = 4096;
constexpr int64_t kMaxPositions = 1 << 30;      // of one request: positions and tiles stay in 32 bits
constexpr int32_t kMaxHeads = 1024;

}  // namespace wq
