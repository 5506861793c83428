// Low-rank adapters of many requests beside a shared projection:
//   y[t] = base[t] + scale[c] * B[c] (A[c] x[t]),  c = adapter[t].
//
// Rows of one adapter are put together on the device, wherever they stand in
// the batch: a tile is up to 32 rows of one adapter (ranked by row index), found
// from a histogram of adapter[], so no host pass and no extra launch are
// needed.  Two launches:
//   1. lora_shrink_kernel: finds its tile, then h = A x over a share of k, as
//      matrix products (16 adapter rows x 16 token rows,
//      v_mfma_f32_16x16x32_bf16); the waves' sums meet in LDS, the shares' in
//      the second launch.  The tile's rows are left in the workspace for it.
//   2. lora_expand_kernel: adds the shares in order, scales, splits h into
//      bf16 parts -- three for fp32 results (together all 24 bits, so that only
//      fp32 sums round), two for bf16 ones (16 bits) -- and multiplies 64 rows
//      of B at a time with them; base is added and the result stored from the
//      accumulators.
// lora_one_kernel does both for few rows and a small A.
//
// Weights are read once per tile.  Measured (MI355X): 32 x 5 rows of 28 adapters,
// rank 32, k = 8192, n = 10240: 18.1 us, 43 MB, of which the two launches' own
// cost and the search are about 8; 8 x 128 rows of 4 adapters, rank 64, k = 4096, n =
// 22016: 48.9 us, 157 MB (of it the second launch 39 us, 135 MB, 3.5 TB/s under the
// registers' two waves per SIMD); one row: launches.
#include <math.h>

#include "wq_kv.hpp"

namespace wq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kLoraThreads = 256;
constexpr int kLoraWaves = 4;
constexpr int kLoraRows = 32;              // rows of a tile, two halves of 16
constexpr int kLoraStep = 128;             // inputs a wave takes at a time
constexpr int64_t kLoraMaxTokens = 4096;
constexpr int64_t kLoraMaxAdapters = 4096;

// A tile as the first launch leaves it for the second.
struct alignas(16) TileRows {
  int32_t adapter;      // == adapters: rows without one
  int32_t rows;         // 0: the batch has no such tile
  int32_t unused[2];
  int32_t row[kLoraRows];
};

struct LoraArgs {
  const uint16_t* x;
  int64_t x_stride;
  const float* base;
  int64_t base_stride;
  float* y32;
  uint16_t* y16;
  int64_t y_stride;
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* adapter;
  const int32_t* ranks;
  const float* scale;
  TileRows* found;      // [tiles]
  float* part;          // [splits][tiles][32][rank16]
  int32_t tokens;
  int32_t k;
  int32_t n;
  int32_t adapters;
  int32_t rank;
  int32_t tiles;        // most tiles the batch can have
  int32_t splits;       // shares of k (shrink)
  int32_t shares;       // of n (expand)
  int32_t chunk;        // inputs per split (shrink), B rows per workgroup (expand)
  int32_t vec;          // base and y rows take 16-byte (8-byte bf16) accesses
};

// LDS of the search: counts [adapters + 1], ids as 16 bits, padded to 512.
__device__ __host__ inline size_t search_counts(int64_t adapters) { return (size_t)((adapters + 1) * 4 + 15) / 16 * 16; }
static size_t search_bytes(int64_t tokens, int64_t adapters) {
  return search_counts(adapters) + (size_t)((tokens + 511) / 512 * 512) * 2;
}

// Tile `want` of the batch into LDS.  Tiles are ordered by adapter (rows without
// one last), then by row; with up to 32 rows by the adapter's first row.  Every
// thread takes part.
__device__ void find_tile(const LoraArgs& a, int want, char* lds, TileRows& tile) {
  const int lane = lane_id(), wave = wave_id(), me = (int)threadIdx.x;
  if (a.tokens <= kLoraRows) {
    if (wave == 0) {
      const int c = lane < a.tokens ? gmem(a.adapter)[lane] : 0;
      const int id = (uint32_t)c < (uint32_t)a.adapters ? c : a.adapters;
      uint32_t left = a.tokens == 32 ? ~0u : (1u << a.tokens) - 1u, mine = 0;
      int adapter = 0;
      for (int i = 0; i <= want && left; ++i) {
        adapter = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
        mine = (uint32_t)__ballot(lane < a.tokens && id == adapter);
        left &= ~mine;
        if (i < want) mine = 0;
      }
      if (lane == 0) {
        tile.adapter = adapter;
        tile.rows = __popc(mine);
      }
      if (lane < kLoraRows && mine >> lane & 1) tile.row[__popc(mine & ((1u << lane) - 1u))] = lane;
    }
    __syncthreads();
    return;
  }
  int* count = reinterpret_cast<int*>(lds);
  uint16_t* id = reinterpret_cast<uint16_t*>(lds + search_counts(a.adapters));
  // the workgroup builds the histogram (rows of a request stand together: the
  // first of a run counts for all of it) ...
  constexpr int kBatch = 4;
  const int padded = (a.tokens + 511) / 512 * 512;
  for (int first = 0; first < padded; first += kBatch * kLoraThreads) {
    int c[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int t = first + b * kLoraThreads + me;
      c[b] = t < a.tokens ? gmem(a.adapter)[t] : -1;
    }
    if (first == 0) {
      for (int i = me; i <= a.adapters; i += kLoraThreads) count[i] = 0;
      __syncthreads();
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int t = first + b * kLoraThreads + me;
      if (t - lane >= padded) break;
      const int i = (uint32_t)c[b] < (uint32_t)a.adapters ? c[b] : a.adapters;
      id[t] = (uint16_t)(t < a.tokens ? i : 0xFFFF);
      const int before = __builtin_amdgcn_update_dpp(0, i, 0x138, 0xF, 0xF, false);     // wave_shr 1
      const uint64_t heads = __ballot(t < a.tokens && (lane == 0 || before != i));
      if (heads >> lane & 1) {
        const uint64_t later = lane == kWave - 1 ? 0 : heads >> (lane + 1);
        const int run = min(later ? __builtin_ctzll(later) + 1 : kWave - lane, a.tokens - t);
        atomicAdd(&count[i], run);
      }
    }
  }
  __syncthreads();
  // ... and every wave reads it for itself: which adapter has the tile,
  const auto tiles_of = [](int n) { return (n + kLoraRows - 1) / kLoraRows; };
  const int each = a.adapters / kWave + 1;
  int mine = 0;
  for (int i = lane * each; i < min((lane + 1) * each, a.adapters + 1); ++i) mine += tiles_of(count[i]);
  int before = wave_scan(mine) - mine;
  const uint64_t holder = __ballot(want >= before && want < before + mine);
  if (!holder) {
    if (lane == 0) tile.rows = 0;
    __syncthreads();
    return;
  }
  int adapter = 0, skip = 0, rows = 0;
  if (holder >> lane & 1) {
    for (int i = lane * each;; ++i) {
      const int tiles = tiles_of(count[i]);
      if (want < before + tiles) {
        adapter = i;
        skip = (want - before) * kLoraRows;
        rows = min(kLoraRows, count[i] - skip);
        break;
      }
      before += tiles;
    }
  }
  const int from = __builtin_ctzll(holder);
  adapter = __builtin_amdgcn_readlane(adapter, from);
  skip = __builtin_amdgcn_readlane(skip, from);
  rows = __builtin_amdgcn_readlane(rows, from);
  // and which rows, 8 ids a lane at a time (the waves write the same values)
  for (int base = 0; base < padded; base += kWave * 8) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(id + base + lane * 8);
    uint32_t hits = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) hits |= ((w[e / 2] >> (e & 1 ? 16 : 0) & 0xFFFFu) == (uint32_t)adapter ? 1u : 0u) << e;
    const int n = __popc(hits), upto = wave_scan(n);
    int at = upto - n - skip;
    for (; hits; hits &= hits - 1, ++at)
      if (at >= 0 && at < kLoraRows) tile.row[at] = base + lane * 8 + __builtin_ctz(hits);
    skip -= __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  if (lane == 0) {
    tile.adapter = adapter;
    tile.rows = rows;
  }
  __syncthreads();
}

// Workgroup -> (tile, share of the outputs or inputs).  Workgroups are dispatched
// round robin over the 8 XCDs; an XCD takes a contiguous run of the units in
// share-major order, so that tiles of one adapter read a share of its weights
// through one L2 (1024 rows of 4 adapters, rank 64, n = 22016: 48.5 us; with tiles
// dealt round robin, every XCD reading all of B, 53.7).
struct Unit {
  int tile, share;
};
__device__ __forceinline__ Unit unit_of(const LoraArgs& a, int shares) {
  const int total = a.tiles * shares, each = (total + 7) >> 3, block = (int)blockIdx.x;
  const int u = (block & 7) * each + (block >> 3);
  if (u >= total) return Unit{-1, 0};
  const int share = (int)((uint32_t)u / (uint32_t)a.tiles);
  return Unit{u - share * a.tiles, share};
}
static dim3 unit_grid(int tiles, int shares) { return dim3((unsigned)((tiles * shares + 7) / 8 * 8)); }

__device__ __forceinline__ int rank_of(const LoraArgs& a, int adapter) {
  return a.ranks ? min(max(gmem(a.ranks)[adapter], 0), a.rank) : a.rank;
}

// h = A x of a tile over inputs [k0, k1), this wave's steps of it (every W-th):
// acc[half][r] holds ranks 16 r + 4 g + i of token row 16 half + c.
template <int RT, int W>
__device__ __forceinline__ void shrink_products(const LoraArgs& a, const TileRows& tile, int rank, int k0, int k1,
                                                f32x4 (&acc)[2][RT]) {
  const int lane = lane_id(), wave = wave_id(), g = lane >> 4, c = lane & 15;
  const int halves = tile.rows > 16 ? 2 : 1;
  const uint16_t* xp[2];
  bool has[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    has[h] = 16 * h + c < tile.rows;
    xp[h] = a.x + (int64_t)tile.row[has[h] ? 16 * h + c : 0] * a.x_stride;
  }
  const uint16_t* ap = a.a + (int64_t)tile.adapter * a.rank * a.k;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[h][r] = f32x4{0.f, 0.f, 0.f, 0.f};
  // of each 32 inputs lane group g takes 8: a row's 64 bytes are one run
  for (int kb = k0 + wave * kLoraStep; kb < k1; kb += W * kLoraStep) {
    u32x4 xv[2][4], av[RT][4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int kk = kb + s * 32 + g * 8;
      const bool in = kk < k1;
#pragma unroll
      for (int r = 0; r < RT; ++r)
        av[r][s] = in && 16 * r + c < a.rank ? load16(ap + (int64_t)(16 * r + c) * a.k + kk) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) xv[h][s] = has[h] && in ? load16(xp[h] + kk) : u32x4{0, 0, 0, 0};
    }
    // rows past the adapter's own rank do not count, whatever they hold
    if (rank < a.rank) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
        if (16 * r + c >= rank) {
#pragma unroll
          for (int s = 0; s < 4; ++s) av[r][s] = u32x4{0, 0, 0, 0};
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == halves) break;
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int r = 0; r < RT; ++r)
          acc[h][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av[r][s]),
                                                              __builtin_bit_cast(bf16x8, xv[h][s]), acc[h][r], 0, 0, 0);
    }
  }
}

// The waves' sums of one half added up in wave order: use(t, j, sum) for token
// row t of the half and rank j, shared out over the workgroup.
template <int RT, int W, class Use>
__device__ __forceinline__ void shrink_sums(float (&sum)[W][RT * 16][17], const f32x4 (&acc)[RT], Use use) {
  const int lane = lane_id(), wave = wave_id(), g = lane >> 4, c = lane & 15;
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[wave][16 * r + 4 * g + i][c] = acc[r][i];
  __syncthreads();
  for (int i = (int)threadIdx.x; i < 16 * RT * 16; i += W * kWave) {
    const int t = i / (RT * 16), j = i % (RT * 16);
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += sum[w][j][t];
    use(t, j, v);
  }
}

template <int RT>
__global__ __launch_bounds__(kLoraThreads) void lora_shrink_kernel(LoraArgs a) {
  extern __shared__ __align__(16) char lds[];
  __shared__ TileRows tile;
  __shared__ float sum[kLoraWaves][RT * 16][17];
  const Unit u = unit_of(a, a.splits);
  if (u.tile < 0) return;
  find_tile(a, u.tile, lds, tile);
  if (u.share == 0 && threadIdx.x < sizeof(TileRows) / 4)
    gmem(reinterpret_cast<int32_t*>(a.found + u.tile))[threadIdx.x] = reinterpret_cast<const int32_t*>(&tile)[threadIdx.x];
  if (tile.rows == 0 || tile.adapter == a.adapters) return;
  const int rank = rank_of(a, tile.adapter);
  const int k0 = u.share * a.chunk, k1 = min(k0 + a.chunk, a.k);
  f32x4 acc[2][RT];
  shrink_products<RT, kLoraWaves>(a, tile, rank, k0, k1, acc);
  float* out = a.part + ((int64_t)u.share * a.tiles + u.tile) * (kLoraRows * RT * 16);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h && tile.rows <= 16) break;
    if (h) __syncthreads();
    shrink_sums<RT, kLoraWaves>(sum, acc[h], [&](int t, int j, float v) { gmem(out)[(h * 16 + t) * (RT * 16) + j] = v; });
  }
}

// h as the second product takes it: [half][product of 32 ranks][part][lane][8].
template <int RT, int PARTS>
struct SplitH {
  static constexpr int KS = (RT + 1) / 2;
  __bf16 at[2][KS][PARTS][kWave][8];
  // Rank j of token row t, as PARTS bf16 parts.  What would round to infinity is cut
  // off instead (the rest follows in the next part); infinity has no rest.
  __device__ __forceinline__ void put(int t, int j, float v) {
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
      __bf16 part = (__bf16)v;
      if (fabsf((float)part) == INFINITY) part = (__bf16)__uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
      at[t >> 4][j >> 5][q][(j >> 3 & 3) * 16 + (t & 15)][j & 7] = part;
      v = (float)part == v ? 0.f : v - (float)part;
    }
  }
};

// A pair of bf16 with 0 for what is infinite or NaN.
__device__ __forceinline__ uint32_t bf16_finite(uint32_t w) {
  return ((w & 0x7F80u) == 0x7F80u ? 0u : w & 0xFFFFu) | ((w & 0x7F800000u) == 0x7F800000u ? 0u : w & 0xFFFF0000u);
}

// y of a tile's rows, outputs [n0, n1).  B rows of 64 outputs go to four products
// of 16, output 4 c + j of the 64 to column c of product j: lane (g, c) ends with
// four consecutive outputs of each of the token rows 4 g .. 4 g + 3 of a half, and
// the 16 lanes of a row read base and write y in one contiguous run.  What
// bounds it is the latency of those reads, so 32 rows share the weights of 64
// outputs: twice the bytes of base in flight for the same weights.
template <int RT, int PARTS, int W>
struct Expand {
  static constexpr int KS = (RT + 1) / 2;
  const LoraArgs& a;
  const uint16_t* bp;
  int rank, halves, n1, nb;
  bool bare;
  int row[2][4];
  bool has[2][4];
  u32x4 bv[4][KS];
  f32x4 v[2][4];

  template <class T>
  __device__ __forceinline__ Expand(const LoraArgs& args, const T& tile, int rank_, int n0, int n1_)
      : a(args), rank(rank_), n1(n1_) {
    const int lane = lane_id(), g = lane >> 4;
    bare = tile.adapter == a.adapters;
    bp = a.b + (int64_t)(bare ? 0 : tile.adapter) * a.n * a.rank;
    halves = tile.rows > 16 ? 2 : 1;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        has[h][i] = 16 * h + 4 * g + i < tile.rows;
        row[h][i] = tile.row[has[h][i] ? 16 * h + 4 * g + i : 0];
      }
    nb = n0 + wave_id() * 64;
    if (nb < n1) request(nb);
  }

  // Weights and base of outputs first .. first + 63, all requested before any is used.
  __device__ __forceinline__ void request(int first) {
    const int lane = lane_id(), g = lane >> 4, c = lane & 15, o = first + 4 * c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[h][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (has[h][i] && a.base) {
          const float* base = a.base + (int64_t)row[h][i] * a.base_stride + o;
          if (a.vec && o + 4 <= n1) {
            v[h][i] = __builtin_bit_cast(f32x4, load_stream16(base));
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (o + j < n1) v[h][i][j] = gmem(base)[j];
          }
        }
      }
      if (halves == 1) break;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int s = 0; s < KS; ++s)
        bv[j][s] = !bare && o + j < n1 && s * 32 + g * 8 < a.rank ? load16(bp + (int64_t)(o + j) * a.rank + s * 32 + g * 8)
                                                                : u32x4{0, 0, 0, 0};
  }

  __device__ __forceinline__ void run(const SplitH<RT, PARTS>& hs) {
    const int lane = lane_id(), g = lane >> 4, c = lane & 15;
    for (; nb < n1; nb += W * 64) {
      if (rank < a.rank) {
        // columns of B past the adapter's own rank do not count
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int left = rank - (s * 32 + g * 8 + 2 * i);
            const uint32_t keep = left <= 0 ? 0u : left == 1 ? 0xFFFFu : ~0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) bv[j][s][i] &= keep;
          }
      }
      const int o = nb + 4 * c;
      const bool full = a.vec && o + 4 <= n1;
      f32x4 y[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == halves) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[h][i] = v[h][i];
        if (bare) continue;
        bf16x8 hv[KS][PARTS];
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int q = 0; q < PARTS; ++q) hv[s][q] = *reinterpret_cast<const bf16x8*>(hs.at[h][s][q][lane]);
        f32x4 all = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
              acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hv[s][q], __builtin_bit_cast(bf16x8, bv[j][s]), acc, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[h][i][j] += acc[i];
          all += acc;
        }
        // An infinity of B meets h as a whole: the first part alone has h's sign, the
        // others may be 0 or have another.  Where it met all of them the sum is NaN.
        const float one = (all[0] + all[1]) + (all[2] + all[3]);
        if (__builtin_expect(__any(one != one), 0)) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              u32x4 fine;
#pragma unroll
              for (int i = 0; i < 4; ++i) fine[i] = bf16_finite(bv[j][s][i]);
#pragma unroll
              for (int q = 0; q < PARTS; ++q)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hv[s][q], __builtin_bit_cast(bf16x8, q ? fine : bv[j][s]), acc,
                                                              0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) y[h][i][j] = v[h][i][j] + acc[i];
          }
        }
      }
      if (nb + W * 64 < n1) request(nb + W * 64);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == halves) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!has[h][i]) continue;
          const int64_t at = (int64_t)row[h][i] * a.y_stride + o;
          if (a.y32) {
            float* to = a.y32 + at;
            if (full) {
              __builtin_nontemporal_store(__builtin_bit_cast(u32x4, y[h][i]), gmem(reinterpret_cast<u32x4*>(to)));
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (o + j < n1) gmem(to)[j] = y[h][i][j];
            }
          }
          if (a.y16) {
            uint16_t* to = a.y16 + at;
            if (full) {
              const bf16x4 w = {(__bf16)y[h][i][0], (__bf16)y[h][i][1], (__bf16)y[h][i][2], (__bf16)y[h][i][3]};
              __builtin_nontemporal_store(__builtin_bit_cast(u32x2, w), gmem(reinterpret_cast<u32x2*>(to)));
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (o + j < n1) gmem(to)[j] = f32_to_bf16(y[h][i][j]);
            }
          }
        }
      }
    }
  }
};

// (Two waves per SIMD also where the special cases' code would need more registers;
// the smaller ranks are slower with three: 160 rows of 64 adapters 19.2 against 18.1 us.)
template <int RT, int PARTS>
__global__ __launch_bounds__(kLoraThreads, RT == 8 ? 2 : 1) void lora_expand_kernel(LoraArgs a) {
  constexpr int KS = (RT + 1) / 2;          // products of 32 ranks
  constexpr int R16 = RT * 16;
  __shared__ __align__(16) SplitH<RT, PARTS> hs;
  const Unit u = unit_of(a, a.shares);
  if (u.tile < 0) return;
  const auto& tile = *gmem(a.found + u.tile);
  const int rows = tile.rows, adapter = tile.adapter;
  if (rows == 0) return;
  const bool bare = adapter == a.adapters;
  const int rank = bare ? a.rank : rank_of(a, adapter);
  const int n0 = u.share * a.chunk, n1 = min(n0 + a.chunk, a.n);
  Expand<RT, PARTS, kLoraWaves> expand(a, tile, rank, n0, n1);
  if (!bare) {
    const float scale = a.scale ? gmem(a.scale)[adapter] : 1.f;
    for (int i = (int)threadIdx.x; i < expand.halves * 16 * KS * 32; i += kLoraThreads) {
      const int t = i / (KS * 32), j = i % (KS * 32);
      float sum = 0.f;
      if (j < R16 && t < rows) {
        const float* from = a.part + (int64_t)u.tile * (kLoraRows * R16) + t * R16 + j;
        const int64_t stride = (int64_t)a.tiles * (kLoraRows * R16);
        for (int s = 0; s < a.splits; s += 8) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = gmem(from)[min(s + e, a.splits - 1) * stride];
#pragma unroll
          for (int e = 0; e < 8; ++e) sum += s + e < a.splits ? x[e] : 0.f;
        }
      }
      hs.put(t, j, j < rank ? sum * scale : 0.f);
    }
  }
  __syncthreads();
  expand.run(hs);
}

// Both steps in one launch, for few rows and a small A: every workgroup of a tile
// computes the whole h again (from L2) rather than wait for a second launch.
constexpr int kOneWaves = 8;
template <int RT, int PARTS>
__global__ __launch_bounds__(kOneWaves * kWave) void lora_one_kernel(LoraArgs a) {
  __shared__ TileRows tile;
  __shared__ float sum[kOneWaves][RT * 16][17];
  __shared__ __align__(16) SplitH<RT, PARTS> hs;
  find_tile(a, (int)blockIdx.x, nullptr, tile);
  if (tile.rows == 0) return;
  const bool bare = tile.adapter == a.adapters;
  const int rank = bare ? a.rank : rank_of(a, tile.adapter);
  const int n0 = (int)blockIdx.y * a.chunk, n1 = min(n0 + a.chunk, a.n);
  Expand<RT, PARTS, kOneWaves> expand(a, tile, rank, n0, n1);
  if (!bare) {
    const float scale = a.scale ? gmem(a.scale)[tile.adapter] : 1.f;
    f32x4 acc[2][RT];
    shrink_products<RT, kOneWaves>(a, tile, rank, 0, a.k, acc);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h && tile.rows <= 16) break;
      if (h) __syncthreads();
      shrink_sums<RT, kOneWaves>(sum, acc[h], [&](int t, int j, float v) {
        hs.put(h * 16 + t, j, j < rank ? v * scale : 0.f);
        if (RT == 1) hs.put(h * 16 + t, 16 + j, 0.f);
      });
    }
  }
  __syncthreads();
  expand.run(hs);
}

// ---------------------------------------------------------------------------
// Host side

constexpr int64_t kLoraMade = 0x77715f6c6f726131;

static bool lora_sizes_ok(int64_t tokens, int64_t k, int64_t adapters, int32_t rank) {
  return tokens >= 0 && tokens <= kLoraMaxTokens && k >= 8 && k <= 65536 && k % 8 == 0 && adapters >= 1 &&
         adapters <= kLoraMaxAdapters && rank >= 8 && rank <= 128 && rank % 8 == 0;
}

static int lora_tiles(int64_t tokens, int64_t adapters) {
  // at most one unfilled tile per adapter in use and one for rows without
  const int64_t partly = adapters + 1 < tokens ? adapters + 1 : tokens;
  const int64_t most = partly + (tokens - partly) / kLoraRows;
  return (int)(most < 1 ? 1 : most);
}

// Shares of k: enough workgroups for the chip, each wave at least one step.
static int lora_splits(int tiles, int64_t k) {
  const int64_t most = (k + kLoraWaves * kLoraStep - 1) / (kLoraWaves * kLoraStep);
  const int64_t want = (1024 + tiles - 1) / tiles;
  return (int)(want < most ? want : most);
}

// One launch instead of two: up to 32 rows, and an A of up to 64 KB, which a
// workgroup reads in less time than a second launch takes.  Measured, one / two
// launches, rank 16, n = 4096: one row k = 1024 5.4 / 7.3 us, k = 2048 6.6 / 7.4,
// k = 4096 8.7 / 7.6; 32 rows of 32 adapters k = 1024 7.5 / 9.1.
static bool lora_in_one(int64_t tokens, int64_t k, int32_t rank) { return tokens <= kLoraRows && rank <= 32 && rank * k <= 32768; }

static int rank16(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

static int lora_check(const char* name, const wq_lora& a) {
  if (!a.x || !a.a || !a.b || !a.adapter) return fail(WQ_ERR_NULL, "%s: x, a, b and adapter must be non-null", name);
  if (!a.y_f32 && !a.y_bf16) return fail(WQ_ERR_NULL, "%s: at least one of y_f32 / y_bf16 must be non-null", name);
  if (!lora_sizes_ok(a.tokens, a.k, a.adapters, a.rank) || a.n < 0 || a.n > (1 << 20))
    return fail(WQ_ERR_SHAPE,
                "%s: tokens = %lld (0..4096), k = %lld (a multiple of 8 up to 65536), n = %lld (0..2^20), adapters = "
                "%lld (1..4096), rank = %d (a multiple of 8 up to 128)",
                name, (long long)a.tokens, (long long)a.k, (long long)a.n, (long long)a.adapters, a.rank);
  const int64_t most = (int64_t)1 << 40;
  if (a.x_stride < a.k || a.x_stride > most || a.x_stride % 8)
    return fail(WQ_ERR_SHAPE, "%s: x_stride = %lld must be a multiple of 8 and hold a row", name, (long long)a.x_stride);
  if (a.y_stride < a.n || a.y_stride > most || (a.base && (a.base_stride < a.n || a.base_stride > most)))
    return fail(WQ_ERR_SHAPE, "%s: y_stride = %lld, base_stride = %lld must hold a row", name, (long long)a.y_stride,
                (long long)a.base_stride);
  if (a.base && a.base == a.y_f32 && a.base_stride != a.y_stride)
    return fail(WQ_ERR_SHAPE, "%s: base is y_f32 but has another stride", name);
  if (!aligned16(a.x) || !aligned16(a.a) || !aligned16(a.b))
    return fail(WQ_ERR_ALIGN, "%s: x, a and b must be 16-byte aligned", name);
  if (((uintptr_t)a.base & 3) || ((uintptr_t)a.y_f32 & 3) || ((uintptr_t)a.y_bf16 & 1) || ((uintptr_t)a.adapter & 3) ||
      ((uintptr_t)a.ranks & 3) || ((uintptr_t)a.scale & 3))
    return fail(WQ_ERR_ALIGN, "%s: base, y, adapter, ranks and scale must be aligned to their elements", name);
  return WQ_OK;
}

// Results that lie on each other or on what other workgroups may still read (x and
// the weights, throughout; base, but for the very elements that it is added to).
static int lora_overlap(const char* name, const wq_lora& a) {
  const ByteRows y32{a.y_f32, a.tokens, 4 * a.y_stride, 4 * a.n}, y16{a.y_bf16, a.tokens, 2 * a.y_stride, 2 * a.n};
  const ByteRows base{a.base, a.tokens, 4 * a.base_stride, 4 * a.n};
  const ByteRows in[] = {{a.x, a.tokens, 2 * a.x_stride, 2 * a.k},
                         {a.a, 1, 0, 2 * a.adapters * a.rank * a.k},
                         {a.b, 1, 0, 2 * a.adapters * a.n * a.rank},
                         {a.adapter, 1, 0, 4 * a.tokens},
                         {a.ranks, 1, 0, 4 * a.adapters},
                         {a.scale, 1, 0, 4 * a.adapters}};
  for (const ByteRows& i : in)
    if (rows_meet(y32, i) || rows_meet(y16, i))
      return fail(WQ_ERR_SHAPE, "%s: y must not overlap x, a, b, adapter, ranks or scale", name);
  if (rows_meet(y32, y16)) return fail(WQ_ERR_SHAPE, "%s: y_f32 must not overlap y_bf16", name);
  if ((a.base != a.y_f32 && rows_meet(y32, base)) || rows_meet(y16, base))
    return fail(WQ_ERR_SHAPE, "%s: base must be y_f32 or overlap no result", name);
  return WQ_OK;
}

template <int RT>
static int lora_launch(const char* name, LoraArgs a, hipStream_t s) {
  if constexpr (RT <= 2) {
    if (lora_in_one(a.tokens, a.k, a.rank)) {
      // 64 outputs per wave at a time, about 256 workgroups in all
      const int most = (a.n + kOneWaves * 64 - 1) / (kOneWaves * 64);
      int parts = 256 / a.tiles;
      parts = parts < 1 ? 1 : parts < most ? parts : most;
      a.chunk = (most + parts - 1) / parts * kOneWaves * 64;
      const dim3 grid((unsigned)a.tiles, (unsigned)((a.n + a.chunk - 1) / a.chunk));
      if (a.y32)
        hipLaunchKernelGGL((lora_one_kernel<RT, 3>), grid, dim3(kOneWaves * kWave), 0, s, a);
      else
        hipLaunchKernelGGL((lora_one_kernel<RT, 2>), grid, dim3(kOneWaves * kWave), 0, s, a);
      return launch_status(name);
    }
  }
  const size_t lds = search_bytes(a.tokens, a.adapters);
  const int steps = (a.k + kLoraStep - 1) / kLoraStep;
  a.chunk = (steps + a.splits - 1) / a.splits * kLoraStep;
  hipLaunchKernelGGL((lora_shrink_kernel<RT>), unit_grid(a.tiles, a.splits), dim3(kLoraThreads), lds, s, a);
  // expand: 64 outputs per wave at a time, as many workgroups as are resident (two
  // per CU), so that each reads its tile's h once; twice as many where most tiles
  // may be empty (few rows for each of many adapters).  Measured, 512 / 1024: 1024
  // rows of 4 adapters 48.5 / 54.5 us, 160 rows of 64 adapters 22.0 / 19.4.
  const int rows = (a.n + 63) / 64;
  const int target = a.tiles > 2 * ((a.tokens + kLoraRows - 1) / kLoraRows) ? 1024 : 512;
  int64_t parts = (target + a.tiles - 1) / a.tiles;
  const int64_t most = (rows + kLoraWaves - 1) / kLoraWaves;
  parts = parts < most ? parts : most;
  a.chunk = (int)((most + parts - 1) / parts) * kLoraWaves * 64;
  a.shares = (a.n + a.chunk - 1) / a.chunk;
  const dim3 grid = unit_grid(a.tiles, a.shares);
  if (a.y32)
    hipLaunchKernelGGL((lora_expand_kernel<RT, 3>), grid, dim3(kLoraThreads), 0, s, a);
  else
    hipLaunchKernelGGL((lora_expand_kernel<RT, 2>), grid, dim3(kLoraThreads), 0, s, a);
  return launch_status(name);
}

}  // namespace wq

using namespace wq;

extern "C" int64_t wq_lora_workspace_bytes(int64_t tokens, int64_t k, int64_t adapters, int32_t rank) {
  if (!lora_sizes_ok(tokens, k, adapters, rank)) return 0;
  const int tiles = lora_tiles(tokens, adapters);
  return (int64_t)tiles * sizeof(TileRows) + (int64_t)lora_splits(tiles, k) * tiles * kLoraRows * rank16(rank) * 4;
}

extern "C" int wq_lora_prepare(const wq_lora* a, void* workspace, int64_t workspace_bytes, wq_lora_plan* plan) {
  const char* name = "wq_lora_prepare";
  if (!a || !plan || !workspace) return fail(WQ_ERR_NULL, "%s: a, workspace and plan must be non-null", name);
  int rc = lora_check(name, *a);
  if (rc) return rc;
  const int64_t need = wq_lora_workspace_bytes(a->tokens, a->k, a->adapters, a->rank);
  if (workspace_bytes < need)
    return fail(WQ_ERR_SHAPE, "%s: workspace_bytes = %lld, %lld are needed", name, (long long)workspace_bytes,
                (long long)need);
  if (!aligned16(workspace)) return fail(WQ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", name);
  if ((rc = lora_overlap(name, *a))) return rc;
  wq_lora_plan p{};
  if ((rc = plan_device(name, &p.device))) return rc;
  p.made = kLoraMade;
  p.tiles = lora_tiles(a->tokens, a->adapters);
  p.splits = lora_splits(p.tiles, a->k);
  p.workspace = workspace;
  p.a = *a;
  *plan = p;
  return WQ_OK;
}

extern "C" int wq_lora_run(const wq_lora_plan* plan, void* stream) {
  const char* name = "wq_lora_run";
  if (!plan) return fail(WQ_ERR_NULL, "%s: plan must be non-null", name);
  if (plan->made != kLoraMade) return fail(WQ_ERR_SHAPE, "%s: the plan was not made by wq_lora_prepare", name);
  int rc = same_device(name, plan->device);
  if (rc) return rc;
  const wq_lora& l = plan->a;
  if (l.tokens == 0 || l.n == 0) return WQ_OK;
  LoraArgs a{};
  a.x = l.x;
  a.x_stride = l.x_stride;
  a.base = l.base;
  a.base_stride = l.base_stride;
  a.y32 = l.y_f32;
  a.y16 = l.y_bf16;
  a.y_stride = l.y_stride;
  a.a = l.a;
  a.b = l.b;
  a.adapter = l.adapter;
  a.ranks = l.ranks;
  a.scale = l.scale;
  a.found = static_cast<TileRows*>(plan->workspace);
  a.part = reinterpret_cast<float*>(a.found + plan->tiles);
  a.tokens = (int32_t)l.tokens;
  a.k = (int32_t)l.k;
  a.n = (int32_t)l.n;
  a.adapters = (int32_t)l.adapters;
  a.rank = l.rank;
  a.tiles = plan->tiles;
  a.splits = plan->splits;
  a.vec = l.y_stride % 4 == 0 && (!l.y_f32 || aligned16(l.y_f32)) && (!l.y_bf16 || !((uintptr_t)l.y_bf16 & 7)) &&
          (!l.base || (l.base_stride % 4 == 0 && aligned16(l.base)));
  hipStream_t s = (hipStream_t)stream;
  switch (rank16(l.rank)) {
    case 16: return lora_launch<1>(name, a, s);
    case 32: return lora_launch<2>(name, a, s);
    case 64: return lora_launch<4>(name, a, s);
    default: return lora_launch<8>(name, a, s);
  }
}
