// Attention of drafted tokens over a paged cache and their tree: the joining
// launch and the host side.  The kernel is in wq_attention_stream.hpp.
#include <float.h>

#include "wq_attention_stream.hpp"

namespace wq {

// Joins the parts of groups that shares cut.  A wave takes one row: 16-byte
// pieces of the parts' rows, as many parts side by side as fit the wave and 8
// deep, and meanwhile, a lane per part, their maxima and sums.
template <int D, int ROWS, int TILE>
__global__ __launch_bounds__(kAttnThreads) void attention_join_kernel(AttnArgs a, int grid) {
  constexpr int LP = D / 4 <= 16 ? 16 : D / 4 <= 32 ? 32 : 64;    // lanes per part
  constexpr int SIDE = kWave / LP;                               // parts side by side
  constexpr int BATCH = 8;
  extern __shared__ __align__(16) char lds[];
  const Deal d = deal_at(lds, a.b.requests);
  deal<ROWS, TILE>(a, d);
  const int total = d.before[a.b.requests];
  if (total == 0) return;
  const int per = share_of(total, grid);
  const int lane = lane_id();
  const int quads = (a.heads + kAttnWaves - 1) / kAttnWaves, units = a.b.tokens * quads;
#pragma unroll 1
  for (int u = (int)blockIdx.x; u < units; u += (int)gridDim.x) {
    const int token = (int)((uint32_t)u / (uint32_t)quads);
    const int r = __builtin_amdgcn_readfirstlane(request_of(d, a.b.requests, token));
    const int n = d.count(r), tok = token - d.start(r);
    const int qh = (u - token * quads) * kAttnWaves + wave_id();
    if (tok < 0 || tok >= n || qh >= a.heads) continue;
    const int rows = n * a.group, blocks = (rows + ROWS - 1) / ROWS;
    const int tiles = tiles_of<TILE>(a, d.length[r], n);
    if (tiles <= a.uncut) continue;
    const int head = token_of(a, qh), row = tok * a.group + qh - head * a.group;
    const int first = d.before[r] + (head * blocks + row / ROWS) * (tiles + kGroupCost) + kGroupCost;
    const int s0 = first / per, s1 = (first + tiles - 1) / per;
    if (s0 == s1) continue;
    const int in = row % ROWS;
    const auto part_of = [&](int s) { return a.parts + ((int64_t)s * 2 + (s == s0)) * (ROWS * (D + 2)); };
    const int side = lane / LP, piece = lane % LP;
    const bool has = piece * 4 < D;
    float top = -INFINITY, sum = 0.f;
    f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
    const int last = s1 - s0;
    f32x4 x[BATCH];
    const auto request = [&](int from) {
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const float* part = part_of(s0 + min(from + b * SIDE + side, last)) + in * D + piece * 4;
        x[b] = has ? *gmem(reinterpret_cast<const f32x4*>(part)) : f32x4{0.f, 0.f, 0.f, 0.f};
      }
    };
    for (int base = 0; base <= last; base += kWave) {
      float m = -INFINITY, l = 0.f;
      if (base + lane <= last) {
        const float* part = part_of(s0 + base + lane);
        m = gmem(part)[ROWS * D + in];
        l = gmem(part)[ROWS * (D + 1) + in];
      }
      request(base);
      const float now = fmaxf(wave_max(m), top);
      const float ref = now == -INFINITY ? 0.f : now;
      const float fo = __builtin_amdgcn_exp2f(top - ref), f = __builtin_amdgcn_exp2f(m - ref);
      top = now;
      sum = sum * fo + wave_sum(l * f);
      o *= fo;
      const int count = min(kWave, last - base + 1);
      for (int i = 0; i < count; i += BATCH * SIDE) {
        if (i) request(base + i);
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          const int s = i + b * SIDE + side;
          const float fb = __shfl(f, min(s, kWave - 1));
          if (s < count) o += x[b] * fb;
        }
      }
    }
#pragma unroll
    for (int s = LP; s < kWave; s <<= 1)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], s);
    const float f = sum == 0.f ? 0.f : 1.f / sum;
    if (side == 0 && has) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      uint32_t w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[e] = sum == 0.f ? 0u : (uint32_t)f32_to_bf16(o[2 * e] * f) | (uint32_t)f32_to_bf16(o[2 * e + 1] * f) << 16;
      *gmem(reinterpret_cast<u32x2*>(a.y + (int64_t)token * a.y_stride + qh * D + piece * 4)) = u32x2{w[0], w[1]};
    }
  }
}

// ---------------------------------------------------------------------------
// Host side

constexpr int64_t kAttnMade = 0x77715f6174746e31;

// Which kernel, by the rows per key head that max_tokens can make: up to 16 in at
// most 256 (request, key head) groups, one for each of its workgroups; up to 64 (or
// more groups, or less work than fills the third); more.  With more than 2048
// requests the deal does not fit LDS beside the last one's ring; blocks of 64 rows
// take any number.  (head_dim 256: these for all, as its buffers and accumulators
// fill LDS and the registers.)
// Measured, heads of 128, first / second kernel: one token over 500 positions, 32
// key heads, 12.9 / 18.4 us; 16 requests of 500, 64 / 8 heads, 15.2 / 19.9; 8 of up
// to 4088, 32 key heads, 57 / 53, all of 4088 104 / 114; but with 8 key heads 48
// requests of 120 positions 16.4 / 11.7, 128 of 1016 117 / 108.  Above 64 rows, third /
// second, 32 / 8 heads: 64 tokens over 1984 positions 26.3 / 21.4, over 8128 34.8 /
// 35.0; 4 x 64 over 448 32.2 / 26.9, over 1984 36.7 / 37.3, over 8128 68 / 88; 16 x 64
// over 448 33 / 28, over 1984 83 / 88, over 8128 208 / 291.
// The positions are those that the table covers, since the lengths are known on the
// device only: short contexts in a wide table take the third kernel where the second
// is faster (4 x 64 over 448, 32 / 8 heads: 27.0 us with a table of 512 positions,
// 30.2 with 1024 to 2048, where the second kernel has a joining launch, 35.2 from 4096
// on; 16 x 64 over 448 28.4 and 38.7 from 1024 on; 64 over 1984 23.2 and 27.7 with
// 32768).
enum { kRows16 = 0, kRows64 = 1, kRowsMany = 2 };
constexpr int64_t kGroups16 = 256;
constexpr int64_t kRequestsMany = 2048;
constexpr int64_t kLeastMany = 1 << 24;      // rows * positions

static int attn_variant(int64_t requests, int heads, int kv_heads, int head_dim, int max_tokens, int64_t positions) {
  const int rows = heads / kv_heads * max_tokens;
  if (head_dim == 256) return kRows64;
  if (rows <= 16 && requests * kv_heads <= kGroups16) return kRows16;
  const bool small = requests * heads * max_tokens * positions <= kLeastMany;
  return rows <= 64 || small || requests > kRequestsMany ? kRows64 : kRowsMany;
}

// Workgroups of a launch: as many as are resident while two (with WK = 1 and 4
// waves) fit a CU's 160 KB of LDS.  Each holds the deal, 12 bytes per request, behind
// its ring: up to about 480 requests with heads of 96, 1250 with 128, 3980 with 64.
// With more the 512 run in two rounds.
static int attn_grid(int variant, int head_dim) {
  return variant == kRows16 || (variant == kRowsMany && head_dim != 96) || head_dim == 256 ? 256 : 512;
}
// Rows of a block.
static int attn_rows(int variant, int head_dim) {
  return variant == kRows16 ? 16 : variant == kRows64 ? 64 : head_dim == 96 ? 128 : 256;
}

// Positions of a group that is not cut.  Where all are shorter no joining launch is
// needed.  Measured, 256 / 512 / 1024 positions, heads of 128: one token over 500
// positions, 32 key heads, 11.7 / 12.1 / 12.1 us; 16 requests of 500, 8 key heads,
// 17.6 / 15.2 / 15.2; 5 tokens over 700, 8 key heads, 13.5 / 13.5 / 25.6; 64 such
// requests 55.2 / 55.2 / 48.9.  The joining launch is left out by the table's width,
// not by the lengths: with a table of more than 512 positions a run over short contexts
// pays 2.4 us for a launch that joins nothing (one token over 500 12.2 / 14.6, 8 x 5
// over 500, 8 key heads, 18.6 / 21.1).
constexpr int kUncutPositions = 512;
// Workgroups of the joining launch, each of which computes the deal once.  Measured,
// 512 / 1024 / one per four rows: 32 x 32 tokens over 500 positions 39.1 / 37.8 / 46.4
// us, 8 x 5 over 700 19.8 / 19.1 / 19.1.
constexpr int kJoinGroups = 1024;

static bool attn_dims_ok(int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t max_tokens) {
  return heads >= 1 && heads <= kMaxHeads && kv_heads >= 1 && heads % kv_heads == 0 && heads / kv_heads <= 64 &&
         (head_dim == 64 || head_dim == 96 || head_dim == 128 || head_dim == 256) && max_tokens >= 1 && max_tokens <= 64;
}

static int attn_check(const char* name, const wq_tree_attention& a) {
  int rc = check_cache_null(name, a.cache);
  if (rc) return rc;
  if (!a.batch.starts || !a.batch.lengths || !a.q || !a.y)
    return fail(WQ_ERR_NULL, "%s: starts, lengths, q and y must be non-null", name);
  if ((rc = check_cache_sizes(name, a.cache)) || (rc = check_batch_sizes(name, a.batch))) return rc;
  if (!attn_dims_ok(a.heads, a.cache.kv_heads, a.cache.head_dim, a.max_tokens))
    return fail(WQ_ERR_SHAPE,
                "%s: heads = %d (a multiple of kv_heads = %d, at most 64 times, up to %d), head_dim = %d (64, 96, 128, "
                "256), max_tokens = %d (1..64)",
                name, a.heads, a.cache.kv_heads, kMaxHeads, a.cache.head_dim, a.max_tokens);
  const int64_t row = (int64_t)a.heads * a.cache.head_dim, most = (int64_t)1 << 40;
  if (a.q_stride < row || a.q_stride > most || a.q_stride % 8 || a.y_stride < row || a.y_stride > most || a.y_stride % 8)
    return fail(WQ_ERR_SHAPE, "%s: q_stride = %lld, y_stride = %lld must be multiples of 8 and hold a row", name,
                (long long)a.q_stride, (long long)a.y_stride);
  if (!(fabsf(a.scale) < INFINITY)) return fail(WQ_ERR_SHAPE, "%s: scale must be finite", name);
  if (a.q == a.y && a.batch.tokens > 0) return fail(WQ_ERR_SHAPE, "%s: y must not be q", name);
  const int64_t blocks = ((int64_t)(a.heads / a.cache.kv_heads) * a.max_tokens + 63) / 64;
  // the deal's costs (and a group past their end) are 32-bit sums
  const int64_t tiles = (a.cache.table_width * a.cache.page_size + 31) / 32 + kGroupCost;
  if (a.batch.requests * a.cache.kv_heads * blocks * tiles + tiles + 1024 > 0x7FFFFFFF)
    return fail(WQ_ERR_SHAPE, "%s: %lld requests of %lld positions are more than 2^31 tiles", name,
                (long long)a.batch.requests, (long long)(a.cache.table_width * a.cache.page_size));
  if ((rc = check_cache_align(name, a.cache))) return rc;
  if (!aligned16(a.q) || !aligned16(a.y) || ((uintptr_t)a.tree & 7))
    return fail(WQ_ERR_ALIGN, "%s: q and y must be 16-byte, tree 8-byte aligned", name);
  return WQ_OK;
}

template <int D, int R, int WK, int W>
static int attn_launch(const char* name, AttnArgs a, int grid, hipStream_t s) {
  constexpr int ROWS = 16 * R * (W / WK);
  constexpr int TILE = Shape<D, WK, W>::TILE;
  constexpr size_t ring = sizeof(StreamLds<D, WK, W>) + (WK > 1 ? sizeof(MeetLds<D>) : 0);
  constexpr int64_t most = WK > 1 ? kGroups16 : R > 1 ? kRequestsMany : kMaxRequests;
  static_assert(ring + deal_bytes(most) + 512 <= 160 * 1024, "ring and deal do not fit LDS");
  const size_t deal = deal_bytes(a.b.requests);
  const size_t lds = ring + deal;
  a.uncut = kUncutPositions / TILE;
  // lane offsets within 8 rows are 32-bit byte offsets
  const bool page8 = a.c.page_size % 8 == 0 && a.c.token_stride < (1u << 28);
  if constexpr (D != 96) {
    if (page8)
      hipLaunchKernelGGL((attention_stream_kernel<D, R, WK, W, true>), dim3(grid), dim3(W * kWave), lds, s, a);
  }
  if (D == 96 || !page8)
    hipLaunchKernelGGL((attention_stream_kernel<D, R, WK, W, false>), dim3(grid), dim3(W * kWave), lds, s, a);
  // a table that covers no more than an uncut group leaves nothing to join
  const int64_t units = (int64_t)a.b.tokens * ((a.heads + kAttnWaves - 1) / kAttnWaves);
  if ((int64_t)a.c.limit > kUncutPositions)
    hipLaunchKernelGGL((attention_join_kernel<D, ROWS, TILE>),
                       dim3((unsigned)(units < kJoinGroups ? units : kJoinGroups)), dim3(kAttnThreads), deal, s, a, grid);
  return launch_status(name);
}

template <int D>
static int attn_launch_d(const char* name, const AttnArgs& a, int variant, hipStream_t s) {
  const int grid = attn_grid(variant, D);
  if (variant == kRows64) return attn_launch<D, 1, 1, 4>(name, a, grid, s);
  if constexpr (D <= 128) {
    if (variant == kRows16) return attn_launch<D, 1, 4, 4>(name, a, grid, s);
    if (variant == kRowsMany) return attn_launch<D, 2, 1, D == 96 ? 4 : 8>(name, a, grid, s);
  }
  return fail(WQ_ERR_SHAPE, "%s: no kernel for this plan", name);
}

}  // namespace wq

using namespace wq;

extern "C" int64_t wq_tree_attention_workspace_bytes(int64_t requests, int32_t heads, int32_t kv_heads,
                                                     int32_t head_dim, int32_t max_tokens) {
  if (requests < 0 || requests > kMaxRequests || !attn_dims_ok(heads, kv_heads, head_dim, max_tokens)) return 0;
  // the most that a table can cover: blocks of more rows need more
  const int variant = attn_variant(requests, heads, kv_heads, head_dim, max_tokens, kMaxPositions);
  return (int64_t)attn_grid(variant, head_dim) * 2 * attn_rows(variant, head_dim) * (head_dim + 2) * 4;
}

extern "C" int wq_tree_attention_prepare(const wq_tree_attention* a, void* workspace, int64_t workspace_bytes,
                                         wq_tree_attention_plan* plan) {
  const char* name = "wq_tree_attention_prepare";
  if (!a || !plan || !workspace) return fail(WQ_ERR_NULL, "%s: a, workspace and plan must be non-null", name);
  int rc = attn_check(name, *a);
  if (rc) return rc;
  const int64_t need = wq_tree_attention_workspace_bytes(a->batch.requests, a->heads, a->cache.kv_heads,
                                                         a->cache.head_dim, a->max_tokens);
  if (workspace_bytes < need)
    return fail(WQ_ERR_SHAPE, "%s: workspace_bytes = %lld, %lld are needed", name, (long long)workspace_bytes,
                (long long)need);
  if (!aligned16(workspace)) return fail(WQ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", name);
  // a group's queries are read by every workgroup that has a share of it
  const int64_t row = 2 * (int64_t)a->heads * a->cache.head_dim;
  if (rows_meet({a->q, a->batch.tokens, 2 * a->q_stride, row}, {a->y, a->batch.tokens, 2 * a->y_stride, row}))
    return fail(WQ_ERR_SHAPE, "%s: y must not overlap q", name);
  wq_tree_attention_plan p{};
  if ((rc = plan_device(name, &p.device))) return rc;
  p.made = kAttnMade;
  p.variant = attn_variant(a->batch.requests, a->heads, a->cache.kv_heads, a->cache.head_dim, a->max_tokens,
                           a->cache.table_width * a->cache.page_size);
  p.workspace = workspace;
  p.a = *a;
  *plan = p;
  return WQ_OK;
}

extern "C" int wq_tree_attention_run(const wq_tree_attention_plan* plan, void* stream) {
  const char* name = "wq_tree_attention_run";
  if (!plan) return fail(WQ_ERR_NULL, "%s: plan must be non-null", name);
  if (plan->made != kAttnMade)
    return fail(WQ_ERR_SHAPE, "%s: the plan was not made by wq_tree_attention_prepare", name);
  int rc = same_device(name, plan->device);
  if (rc) return rc;
  const wq_tree_attention& t = plan->a;
  if (t.batch.tokens == 0 || t.batch.requests == 0) return WQ_OK;
  AttnArgs a{};
  a.c = device_cache(t.cache);
  a.b = device_batch(t.batch);
  a.q = t.q;
  a.q_stride = t.q_stride;
  a.y = t.y;
  a.y_stride = t.y_stride;
  a.tree = t.tree;
  a.parts = static_cast<float*>(plan->workspace);
  // a negative scale turns the queries over; a zero one leaves equal weights (2^-149
  // keeps a hidden score at minus infinity and is far below a step of any weight)
  a.scale2 = fmaxf(fabsf(t.scale) * 1.44269504088896340736f, FLT_TRUE_MIN);
  a.q_flip = t.scale < 0.f ? 0x80008000u : 0u;
  a.heads = t.heads;
  a.group = t.heads / t.cache.kv_heads;
  a.group_magic = ((1u << 20) + a.group - 1) / a.group;
  a.max_tokens = t.max_tokens;
  hipStream_t s = (hipStream_t)stream;
  switch (t.cache.head_dim) {
    case 64: return attn_launch_d<64>(name, a, plan->variant, s);
    case 96: return attn_launch_d<96>(name, a, plan->variant, s);
    case 128: return attn_launch_d<128>(name, a, plan->variant, s);
    default: return attn_launch_d<256>(name, a, plan->variant, s);
  }
}
