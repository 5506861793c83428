// y = x W^T with W in MXFP4 and x in bf16 or MXFP4.
//
// Few rows (mx_rows_kernel) are bound by W's bytes: a workgroup takes a block of 16-row
// tiles, its waves split the row's spans (and, for short rows, the tiles), and their
// sums meet in LDS in a fixed order.  5 rows x 57344 x 8192 (251 MB) 47.1 us, 5.3 TB/s;
// 1 row x 12288 x 4096 (26.8 MB) 7.3 us, of which the start of a launch and of the loads
// is about half.  More rows (mx_tile_kernel, mx_split_kernel) are bound by the matrix
// pipe and what feeds it; tile_plan chooses.
#include <stdint.h>

#include <algorithm>

#include "wq_host.hpp"
#include "wq_kv.hpp"
#include "wq_mx_split.hpp"
#include "wq_mx_tile.hpp"
#include "wq_row_stream.hpp"

namespace wq {

struct MxRowsArgs {
  StreamWeights w;
  const char* x;          // bf16 rows, or codes
  const uint8_t* xscale;
  int64_t x_stride;       // bytes
  uint32_t x_bytes;       // of a row
  float* y32;
  uint16_t* y16;
  int64_t y_stride;
  int64_t m;
  int32_t tiles;          // of 16 rows of W
  int32_t per;            // tiles of a workgroup
  int32_t ways;           // waves that share a tile's spans
  int32_t spans;
};

constexpr int row_tiles(bool xq) { return xq ? 8 : 16; }      // at most, of a wave

template <bool XQ, bool ODD, int COLS, int WAVES, int P>
__global__ __launch_bounds__(WAVES * 64) void mx_rows_kernel(MxRowsArgs a) {
  using S = RowStream<true, XQ, ODD, COLS, P>;
  constexpr int kRowTiles = row_tiles(XQ);
  constexpr int kRed = WAVES * kRowTiles * 1024, kAll = WAVES * S::kBytes;
  __shared__ __align__(1024) char lds[kAll > kRed ? kAll : kRed];
  const int wave = wave_id(), ways = a.ways, kw = wave % ways, tw = wave / ways, teams = WAVES / ways;
  const S s(lds + wave * S::kBytes);
  const int first = (int)blockIdx.x * a.per, mine = min(a.per, a.tiles - first);
  const int cols = (int)a.m;                       // at most COLS
  f32x4 acc[kRowTiles];
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int tiles = (mine - tw + teams - 1) / teams;
  s.template run<kRowTiles>(
      a.w, tiles, kw, ways, a.spans, (int)a.w.srow,
      [&](int t, int64_t& row0, int& left) {
        row0 = (int64_t)(first + tw + t * teams) * 16;
        left = (int)min((int64_t)16, a.w.rows - row0);
      },
      [&](int col) { return a.x + min(col, cols - 1) * a.x_stride; }, a.x_bytes, a.xscale, cols, acc, (int)blockIdx.x);
  // the waves' sums of a tile, lane by lane
  __syncthreads();
  for_tiles<kRowTiles>(tiles, [&](auto at) __attribute__((always_inline)) {
    *reinterpret_cast<f32x4*>(lds + (wave * kRowTiles + at.value) * 1024 + s.lane * 16) = acc[at.value];
  });
  __syncthreads();
  for (int o = (int)threadIdx.x; o < mine * 16 * cols; o += WAVES * 64) {
    const int row = o & 15, col = (o >> 4) % cols, tile = (o >> 4) / cols;
    const char* from = lds + ((tile % teams) * ways * kRowTiles + tile / teams) * 1024 + ((row >> 2) * 16 + col) * 16 + (row & 3) * 4;
    float v = 0.f;
    for (int w = 0; w < ways; ++w) v += *reinterpret_cast<const float*>(from + w * kRowTiles * 1024);
    const int64_t r = (int64_t)(first + tile) * 16 + row;
    if (r >= a.w.rows) continue;
    const int64_t at = col * a.y_stride + r;
    if (a.y32) gmem(a.y32)[at] = v;
    if (a.y16) gmem(a.y16)[at] = f32_to_bf16(v);
  }
}

// ---------------------------------------------------------------------------
// Host side

constexpr int64_t kGemmMade = 0x77715f6d78676d31;
constexpr int64_t kGemmMaxM = 1 << 20, kGemmMaxN = 1 << 24, kGemmMaxK = 1 << 18;

// Tiles per workgroup and waves per tile: the fewest units in the longest chain, with
// two units' worth for what a workgroup costs besides.
static void rows_plan(MxRowsArgs& a, int waves, int most) {
  double best = 1e300;
  for (int ways = 1; ways <= waves; ++ways) {
    if (waves % ways) continue;
    const int teams = waves / ways;
    for (int t = 1; t <= most; ++t) {
      const int per = t * teams;
      const int groups = (a.tiles + per - 1) / per, rounds = (groups + 255) / 256;
      const double cost = (double)rounds * ((double)t * ((a.spans + ways - 1) / ways) + 2.0);
      if (cost < best) {
        best = cost;
        a.per = per;
        a.ways = ways;
      }
    }
  }
}

template <bool XQ, int COLS, int WAVES, int P>
static int rows_launch(const char* name, MxRowsArgs a, hipStream_t s) {
  rows_plan(a, WAVES, row_tiles(XQ));
  const dim3 grid((unsigned)((a.tiles + a.per - 1) / a.per));
  if (a.w.srow % 4)
    hipLaunchKernelGGL((mx_rows_kernel<XQ, true, COLS, WAVES, P>), grid, dim3(WAVES * 64), 0, s, a);
  else
    hipLaunchKernelGGL((mx_rows_kernel<XQ, false, COLS, WAVES, P>), grid, dim3(WAVES * 64), 0, s, a);
  return launch_status(name);
}

// Bytes of a padded row of scales, and whether rows need padding.
static uint32_t pad_stride(int64_t k) { return (uint32_t)((k / kMxGroup + 7) / 8 * 8); }
static bool needs_pad(int64_t k) { return k / kMxGroup % 8 != 0; }

constexpr int64_t kRowsMost = 16;                // rows of x that mx_rows_kernel takes


// How a product of many rows is cut: tiles of `rows` of W x 16 tmt of x over `splits`
// shares of k.
struct TilePlan {
  int rows, tn, tm, tmt, splits, share;
  double us;
};
static int stages_of(int64_t k, bool xq) { return (int)(xq ? (k + 255) / 256 : (k + 63) / 64); }

// A kind of tile: what a workgroup pays for a stage of 16 x 16 of it and for its start and
// end, in us (from the times of one to seven rounds over 4096 x 14336, 4096 x 4096 and
// 28672 x 4096), and the fewest stages of a share.
struct TileKind {
  int rows, tmt;
  double rate, start;
  int least;
};

static void try_kind(TilePlan& best, int64_t m, int64_t n, int64_t k, bool xq, const TileKind& t) {
  TilePlan p{};
  p.rows = t.rows;
  p.tmt = t.tmt;
  p.tn = (int)((n + t.rows - 1) / t.rows);
  p.tm = (int)((m + 16 * t.tmt - 1) / (16 * t.tmt));
  const int stages = stages_of(k, xq);
  const int64_t tiles = (int64_t)p.tn * p.tm;
  for (int splits = 1; splits == 1 || (splits <= 16 && splits * t.least <= stages && tiles * (splits - 1) < 256); ++splits) {
    p.share = (stages + splits - 1) / splits;
    p.splits = (stages + p.share - 1) / p.share;
    // rounds over the 256 CUs; shares cost a second launch, which reads what they write
    const double rounds = (double)((tiles * p.splits + 255) / 256);
    p.us = rounds * (p.share * t.rate * (t.rows / 16 * t.tmt) * 1e-3 + t.start) + (p.splits > 1 ? 3.5 + (double)p.splits * m * n * 8 / 5.3e6 : 0.);
    if (p.us < best.us) best = p;
  }
}

// The plan of the shortest estimate.  What each kind is for (us, the others in brackets):
//   256 x 256 fills the chip: 4096 rows x 4096 x 14336 346 (256 x 128 401), and half of it
//     with two shares of k: 2048 rows 198 (without shares 287)
//   256 x 128 (bf16): 500 rows x 4096 x 14336 over four shares 67 (128 x 64 83)
//   128 x 64 (bf16) by four waves: 256 rows x 4096 x 4096 17.5 (256 x 128 28)
//   64 x 32, 48, 64 (mx_split_kernel by as many waves as have rings in LDS) where few
//     tiles must fill the chip: 47 rows x 4096 x 14336 16.4 (128 x 64 20.2)
static TilePlan tile_plan(int64_t m, int64_t n, int64_t k, bool xq) {
  TilePlan best{};
  best.us = 1e300;
  auto tiles_of = [&](int t) { return (int)((m + 16 * t - 1) / (16 * t)); };
  if (xq) {
    try_kind(best, m, n, k, xq, {256, 16, 7.2, 5., 6});
    try_kind(best, m, n, k, xq, {64, m <= 32 ? 2 : 4, 29., 1.5, 8});
  } else {
    try_kind(best, m, n, k, xq, {256, 16, 5.9, 6.5, 8});
    try_kind(best, m, n, k, xq, {256, 8, 6.8, 5., 8});
    try_kind(best, m, n, k, xq, {128, 4, 11.2, 2., 8});
    // the fewest rows of padding
    const int tmt = m <= 32 ? 2 : tiles_of(4) * 4 <= tiles_of(3) * 3 ? 4 : 3;
    try_kind(best, m, n, k, xq, {64, tmt, 13.6, 2., tmt == 4 ? 12 : 16});
  }
  return best;
}

template <bool XQ, int TN, int TM, int WN, int WM>
static void tile_launch(const MxTileArgs& a, const TilePlan& p, hipStream_t s) {
  const dim3 grid((unsigned)((a.tn * a.tm + 7) / 8 * 8), (unsigned)p.splits), block(WN * WM * 64);
  // a row ends inside a stage
  if (a.x_bytes % 128)
    hipLaunchKernelGGL((mx_tile_kernel<XQ, true, TN, TM, WN, WM>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((mx_tile_kernel<XQ, false, TN, TM, WN, WM>), grid, block, 0, s, a);
}

template <bool XQ, int TN, int TM, int P, int WAVES>
static void split_launch(const MxTileArgs& a, const TilePlan& p, hipStream_t s) {
  hipLaunchKernelGGL((mx_split_kernel<XQ, TN, TM, P, WAVES>), dim3((unsigned)(a.tn * a.tm), (unsigned)p.splits), dim3(WAVES * 64), 0, s,
                     a);
}

static int tiles_launch(const char* name, MxTileArgs a, const TilePlan& p, bool xq, hipStream_t s) {
  a.tn = p.tn;
  a.tm = p.tm;
  a.share = p.share;
  if (p.splits == 1) a.part = nullptr;
  if (p.rows == 256) {
    if (xq)
      tile_launch<true, 8, 4, 2, 4>(a, p, s);
    else if (p.tmt == 8)
      tile_launch<false, 4, 4, 4, 2>(a, p, s);
    else
      tile_launch<false, 4, 8, 4, 2>(a, p, s);
  } else if (xq) {
    if (p.tmt == 2)
      split_launch<true, 4, 2, 2, 4>(a, p, s);
    else
      split_launch<true, 4, 4, 2, 4>(a, p, s);
  } else if (p.rows == 128) {
    split_launch<false, 8, 4, 3, 4>(a, p, s);
  } else if (p.tmt == 2) {
    split_launch<false, 4, 2, 3, 8>(a, p, s);
  } else if (p.tmt == 3) {
    split_launch<false, 4, 3, 2, 8>(a, p, s);
  } else {
    split_launch<false, 4, 4, 2, 6>(a, p, s);
  }
  if (p.splits > 1) {
    const int64_t quads = (int64_t)a.m * ((a.n + 3) / 4);
    hipLaunchKernelGGL(mx_join_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, s, a, p.splits);
  }
  return launch_status(name);
}

static int gemm_check(const char* name, const wq_gemm_mxfp4& a) {
  if (!a.x == !a.xq) return fail(WQ_ERR_NULL, "%s: exactly one of x and xq must be given", name);
  if (a.xq && !a.x_scale) return fail(WQ_ERR_NULL, "%s: xq needs x_scale", name);
  if (!a.q || !a.scale) return fail(WQ_ERR_NULL, "%s: q and scale must be non-null", name);
  if (!a.y_f32 && !a.y_bf16) return fail(WQ_ERR_NULL, "%s: at least one of y_f32 / y_bf16 must be non-null", name);
  if (a.m < 0 || a.m > kGemmMaxM || a.n < 0 || a.n > kGemmMaxN || a.k < kMxGroup || a.k > kGemmMaxK || a.k % kMxGroup)
    return fail(WQ_ERR_SHAPE, "%s: m = %lld (0..2^20), n = %lld (0..2^24), k = %lld (a multiple of 32 up to 2^18)", name,
                (long long)a.m, (long long)a.n, (long long)a.k);
  const int64_t most = (int64_t)1 << 40;
  // (offsets inside a tile of 256 rows are 32 bits)
  if (a.x && (a.x_stride < a.k || a.x_stride > (1 << 22) || a.x_stride % 8))
    return fail(WQ_ERR_SHAPE, "%s: x_stride = %lld must be a multiple of 8 up to 2^22 and hold a row", name, (long long)a.x_stride);
  if (a.y_stride < a.n || a.y_stride > most)
    return fail(WQ_ERR_SHAPE, "%s: y_stride = %lld must hold a row", name, (long long)a.y_stride);
  if (!aligned16(a.x) || !aligned16(a.xq) || !aligned16(a.q))
    return fail(WQ_ERR_ALIGN, "%s: x, xq and q must be 16-byte aligned", name);
  if (((uintptr_t)a.x_scale & 3) || ((uintptr_t)a.scale & 3) || ((uintptr_t)a.y_f32 & 3) || ((uintptr_t)a.y_bf16 & 1))
    return fail(WQ_ERR_ALIGN, "%s: scales must be 4-byte aligned and y to its elements", name);
  return WQ_OK;
}

static int gemm_overlap(const char* name, const wq_gemm_mxfp4& a) {
  const ByteRows y32{a.y_f32, a.m, 4 * a.y_stride, 4 * a.n}, y16{a.y_bf16, a.m, 2 * a.y_stride, 2 * a.n};
  const ByteRows in[] = {{a.x, a.m, 2 * a.x_stride, 2 * a.k},
                         {a.xq, 1, 0, a.m * a.k / 2},
                         {a.xq ? a.x_scale : nullptr, 1, 0, a.m * a.k / kMxGroup},
                         {a.q, 1, 0, a.n * a.k / 2},
                         {a.scale, 1, 0, a.n * a.k / kMxGroup}};
  for (const ByteRows& i : in)
    if (rows_meet(y32, i) || rows_meet(y16, i)) return fail(WQ_ERR_SHAPE, "%s: y must overlap no input", name);
  if (rows_meet(y32, y16)) return fail(WQ_ERR_SHAPE, "%s: y_f32 must not overlap y_bf16", name);
  return WQ_OK;
}

}  // namespace wq

using namespace wq;

extern "C" int64_t wq_gemm_mxfp4_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || m > kGemmMaxM || n < 0 || n > kGemmMaxN || k < kMxGroup || k > kGemmMaxK || k % kMxGroup) return 0;
  int64_t bytes = 16;
  if (m <= kRowsMost) return bytes;
  // padded scales, then shares of k (of either kind of activations)
  if (needs_pad(k)) bytes += ((m + n) * pad_stride(k) + 15) / 16 * 16;
  int64_t most = 1;
  for (bool xq : {false, true}) most = std::max<int64_t>(most, tile_plan(m, n, k, xq).splits);
  if (most > 1) bytes += most * m * ((n + 3) / 4 * 4) * 4;
  return bytes;
}

extern "C" int wq_gemm_mxfp4_prepare(const wq_gemm_mxfp4* a, void* workspace, int64_t workspace_bytes,
                                     wq_gemm_mxfp4_plan* plan) {
  const char* name = "wq_gemm_mxfp4_prepare";
  if (!a || !plan || !workspace) return fail(WQ_ERR_NULL, "%s: a, workspace and plan must be non-null", name);
  int rc = gemm_check(name, *a);
  if (rc) return rc;
  const int64_t need = wq_gemm_mxfp4_workspace_bytes(a->m, a->n, a->k);
  if (workspace_bytes < need)
    return fail(WQ_ERR_SHAPE, "%s: workspace_bytes = %lld, %lld are needed", name, (long long)workspace_bytes,
                (long long)need);
  if (!aligned16(workspace)) return fail(WQ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", name);
  if ((rc = gemm_overlap(name, *a))) return rc;
  wq_gemm_mxfp4_plan p{};
  if ((rc = plan_device(name, &p.device))) return rc;
  p.made = kGemmMade;
  p.workspace = workspace;
  p.a = *a;
  *plan = p;
  return WQ_OK;
}

extern "C" int wq_gemm_mxfp4_run(const wq_gemm_mxfp4_plan* plan, void* stream) {
  const char* name = "wq_gemm_mxfp4_run";
  if (!plan) return fail(WQ_ERR_NULL, "%s: plan must be non-null", name);
  if (plan->made != kGemmMade) return fail(WQ_ERR_SHAPE, "%s: the plan was not made by wq_gemm_mxfp4_prepare", name);
  int rc = same_device(name, plan->device);
  if (rc) return rc;
  const wq_gemm_mxfp4& g = plan->a;
  if (g.m == 0 || g.n == 0) return WQ_OK;
  MxRowsArgs a{};
  a.w = {g.q, g.scale, g.n, (uint32_t)(g.k / 2), (uint32_t)(g.k / kMxGroup)};
  a.x = g.x ? reinterpret_cast<const char*>(g.x) : reinterpret_cast<const char*>(g.xq);
  a.xscale = g.x_scale;
  a.x_stride = g.x ? 2 * g.x_stride : g.k / 2;
  a.x_bytes = (uint32_t)(g.x ? 2 * g.k : g.k / 2);
  a.y32 = g.y_f32;
  a.y16 = g.y_bf16;
  a.y_stride = g.y_stride;
  a.m = g.m;
  a.tiles = (int32_t)((g.n + 15) / 16);
  a.spans = (int32_t)((g.k + 511) / 512);
  hipStream_t s = (hipStream_t)stream;
  if (g.m > kRowsMost) {
    MxTileArgs t{};
    t.w = g.q;
    t.wscale = g.scale;
    t.x = a.x;
    t.xscale = g.x_scale;
    t.x_stride = a.x_stride;
    t.y32 = g.y_f32;
    t.y16 = g.y_bf16;
    t.y_stride = g.y_stride;
    t.m = (int32_t)g.m;
    t.n = (int32_t)g.n;
    t.w_bytes = a.w.row_bytes;
    t.x_bytes = a.x_bytes;
    t.sstride = pad_stride(g.k);
    t.stages = stages_of(g.k, g.xq);
    t.vec = g.y_stride % 4 == 0 && aligned16(g.y_f32) && !((uintptr_t)g.y_bf16 & 7);
    if (needs_pad(g.k)) {
      uint8_t* to = static_cast<uint8_t*>(plan->workspace);
      auto pad = [&](const uint8_t* from, int64_t rows) {
        const int64_t blocks = std::min<int64_t>((rows * (t.sstride / 4) + 255) / 256, 2048);
        hipLaunchKernelGGL(mx_pad_kernel, dim3((unsigned)blocks), dim3(256), 0, s, from, rows, a.w.srow, t.sstride, to);
        const uint8_t* padded = to;
        to += rows * t.sstride;
        return padded;
      };
      t.wscale = pad(g.scale, g.n);
      if (g.xq) t.xscale = pad(g.x_scale, g.m);
    }
    const TilePlan p = tile_plan(g.m, g.n, g.k, g.xq);
    t.part = reinterpret_cast<float*>(static_cast<char*>(plan->workspace) +
                                      (needs_pad(g.k) ? ((g.m + g.n) * t.sstride + 15) / 16 * 16 : 0));
    return tiles_launch(name, t, p, g.xq, s);
  }
  // as many columns as there are rows of x, since their LDS comes off the ring's: eight
  // waves have three slots beside 4 columns, two beside 8; 16 columns leave room for four
  // waves (of four slots), or six of two, which were no faster (4 waves with 4 or 8 columns
  // are up to 10 % slower than eight)
  if (g.xq) return rows_launch<true, 16, 8, 3>(name, a, s);
  if (g.m <= 4) return rows_launch<false, 4, 8, 3>(name, a, s);
  if (g.m <= 8) return rows_launch<false, 8, 8, 2>(name, a, s);
  return rows_launch<false, 16, 4, 4>(name, a, s);
}
