// Attention of drafted tokens over a paged cache and their tree.
//
// With G = heads / kv_heads query heads per key head, the n tokens of a
// request make n * G rows that read the same keys: the rows of one (request,
// key head) are cut into blocks of 16 * R, the positions into tiles of 128, and
// the tiles of all (request, key head, row block) groups, in that order, are
// dealt out to the launch's workgroups in equal contiguous shares (the lengths
// are known on the device only, so every workgroup computes the deal itself).
// A group that one workgroup covers is finished there; the parts of a group
// cut by shares go to the workspace as (running maximum, sum, unnormalised
// output) and are joined, in share order, by a second launch.
//
// Within a tile each of the 4 waves takes 32 positions and keeps its own
// running softmax; the four meet in LDS at the end of a share of a group.  A
// wave holds everything in registers (no staging through LDS), by choosing
// which position stands in which matrix slot:
//   * S^T = K Q^T (v_mfma_f32_16x16x32_bf16): A row m of sub-tile t is position
//     8 (m / 4) + 4 t + m % 4; lane l = 16 g + c loads A row c, D/4 contiguous
//     elements from g D/4 on (the contraction order is free as long as Q has
//     the same).  D gives lane (g, c) the scores of query row c against
//     positions 8 g .. 8 g + 7: eight in a row, so a mask is one byte.
//   * O = P V: A wants lane (g, c) to hold row c's weights of slots 8 g .. 8 g +
//     7, which is what it has.  B wants, for output column c, the same eight
//     positions of V: lane (g, c) loads D/16 contiguous elements of each of
//     them (a row of V is one contiguous run over the 16 lanes), and output
//     column c of product j is element c D/16 + j, gathered from the eight rows
//     by v_perm.  O ends with D/16 contiguous elements of a row per lane.
//   * The maximum used for the exponents is raised only when some score
//     exceeds it by more than 2^8 (its exact value cancels in the quotient),
//     so the usual tile needs no exchange between lanes.
#include <math.h>

#include "wq_kv.hpp"

namespace wq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = 4;
constexpr int kTile = 128;            // positions of a tile, 32 per wave
constexpr float kLazy = 8.f;          // powers of two the running maximum may lag behind

// Workgroups per CU: two where queries and accumulators leave the registers for it.
constexpr int attn_groups_per_cu(int row_tiles, int head_dim) { return row_tiles * head_dim <= 128 ? 2 : 1; }

struct AttnArgs {
  KvCache c;
  Batch b;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* y;
  int64_t y_stride;
  const uint64_t* tree;
  float* parts;          // [grid][2][16 R][D + 2]
  float scale2;          // scale * log2(e)
  int32_t heads;
  int32_t group;         // heads / kv_heads
  int32_t max_tokens;
};

// The deal: per request its rows, length and the tiles of all groups before it.
struct Deal {
  int64_t* before;       // [requests + 1]
  int32_t* start;
  int32_t* count;
  int32_t* length;
};

__device__ __forceinline__ Deal deal_at(char* lds, int requests) {
  Deal d;
  d.before = reinterpret_cast<int64_t*>(lds);
  d.start = reinterpret_cast<int32_t*>(d.before + requests + 1);
  d.count = d.start + requests;
  d.length = d.count + requests;
  return d;
}
static size_t deal_bytes(int64_t requests) { return (size_t)((requests + 1) * 8 + requests * 12 + 15) / 16 * 16; }

// Every thread of the workgroup; ends with a barrier.
template <int ROWS>
__device__ void deal(const AttnArgs& a, const Deal& d) {
  __shared__ int64_t wave_sum_of[kAttnThreads / kWave];
  const int n = a.b.requests;
  const int each = (n + kAttnThreads - 1) / kAttnThreads;
  const int first = (int)threadIdx.x * each;
  int64_t mine = 0;
  for (int r = first; r < min(first + each, n); ++r) {
    const int s0 = gmem(a.b.starts)[r], s1 = gmem(a.b.starts)[r + 1];
    const int len = min(max(gmem(a.b.lengths)[r], 0), (int)a.c.limit);
    const bool ok = s0 >= 0 && s1 >= s0 && s1 <= a.b.tokens && s1 - s0 <= a.max_tokens;
    const int cnt = ok ? s1 - s0 : 0;
    d.start[r] = s0;
    d.count[r] = cnt;
    d.length[r] = len;
    const int blocks = (cnt * a.group + ROWS - 1) / ROWS;
    const int tiles = (int)(((int64_t)len + cnt + kTile - 1) / kTile);
    mine += (int64_t)a.c.kv_heads * blocks * tiles;
    d.before[r] = mine;                    // within the thread; shifted below
  }
  int64_t run = mine;
  const int lane = lane_id(), wave = wave_id();
  for (int s = 1; s < kWave; s <<= 1) {
    const int64_t up = __shfl_up(run, s);
    if (lane >= s) run += up;
  }
  if (lane == kWave - 1) wave_sum_of[wave] = run;
  __syncthreads();
  int64_t base = run - mine;
  for (int w = 0; w < wave; ++w) base += wave_sum_of[w];
  // before[r + 1] = base + (sum up to and with r)
  int64_t prev = 0;
  for (int r = first; r < min(first + each, n); ++r) {
    const int64_t upto = d.before[r];
    d.before[r] = base + prev;
    prev = upto;
  }
  if (first < n && first + each >= n) d.before[n] = base + mine;
  __syncthreads();
}

// Shares: `per` tiles for each of the launch's workgroups.
__device__ __forceinline__ int64_t share_of(int64_t total, int grid) { return (total + grid - 1) / grid; }

// Workgroups are dispatched round robin over the 8 XCDs; consecutive shares go
// to one XCD, so row blocks and cut groups that read the same keys share its L2.
__device__ __forceinline__ int share_index(int block, int grid) { return (block & 7) * (grid >> 3) + (block >> 3); }

// The lane's rows of one 32-position step: element offsets of its two K rows
// and eight V rows, and which of the eight V positions hold something.  With
// pages of a multiple of 8 positions the eight are rows of one page.
template <bool P8>
struct StepRows {
  int32_t pid[P8 ? 2 : 10];
  uint32_t pos[2];               // first V position (8 g on), first K position

  static __device__ __forceinline__ int32_t look(const KvCache& c, const int32_t* table, uint32_t p) {
    return p < c.limit ? gmem(table)[page_of(c, p)] : -1;
  }
  __device__ __forceinline__ void fetch(const KvCache& c, const int32_t* table, uint32_t base, int g, int m) {
    pos[0] = base + 8 * g;
    pos[1] = base + 8 * (m >> 2);
    if (P8) {
      pid[0] = look(c, table, pos[0]);
      pid[1] = look(c, table, pos[1]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) pid[e] = look(c, table, pos[0] + e);
#pragma unroll
      for (int t = 0; t < 2; ++t) pid[P8 ? 1 : 8 + t] = look(c, table, pos[1] + 4 * t + (m & 3));
    }
  }
  __device__ __forceinline__ int64_t at(const KvCache& c, int32_t id, uint32_t p) const {
    return (uint32_t)id < c.pages ? row_offset(c, (uint32_t)id, p - page_of(c, p) * c.page_size) : 0;
  }
  __device__ __forceinline__ uint32_t v_live(const KvCache& c) const {
    if (P8) return (uint32_t)pid[0] < c.pages ? 0xFFu : 0u;
    uint32_t live = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) live |= ((uint32_t)pid[P8 ? 0 : e] < c.pages ? 1u : 0u) << e;
    return live;
  }
};

// WORDS consecutive dwords as the widest loads their alignment allows.
template <int WORDS>
__device__ __forceinline__ void load_words(const uint16_t* p, uint32_t (&w)[WORDS]) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
  typedef u32x3 u32x3a __attribute__((aligned(4)));
  if constexpr (WORDS == 2) {
    const u32x2 x = *gmem(reinterpret_cast<const u32x2*>(p));
    w[0] = x[0], w[1] = x[1];
  } else if constexpr (WORDS == 3) {
    const u32x3a x = *(const __attribute__((address_space(1))) u32x3a*)p;
    w[0] = x[0], w[1] = x[1], w[2] = x[2];
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) {
      const u32x4 x = load16(p + 2 * i);
      w[i] = x[0], w[i + 1] = x[1], w[i + 2] = x[2], w[i + 3] = x[3];
    }
  }
}

__device__ __forceinline__ bool bf16_special(uint32_t bits) { return (bits & 0x7F80u) == 0x7F80u; }

template <int D, int R>
struct AttnLds {
  float o[2][R * 16][D];
  float m[kAttnWaves][R * 16];
  float l[kAttnWaves][R * 16];
  int special[kAttnWaves];
};

template <int D, int R, bool P8>
__global__ __launch_bounds__(kAttnThreads, attn_groups_per_cu(R, D)) void tree_attention_kernel(AttnArgs a) {
  constexpr int KS = D / 32;           // products per K sub-tile
  constexpr int CW = D / 16;           // output columns (V elements) per lane
  constexpr int VW = CW / 2;           // their dwords
  constexpr int ROWS = 16 * R;
  extern __shared__ __align__(16) char lds[];
  AttnLds<D, R>& sh = *reinterpret_cast<AttnLds<D, R>*>(lds);
  const Deal d = deal_at(lds + sizeof(AttnLds<D, R>), a.b.requests);
  deal<ROWS>(a, d);
  const int64_t total = d.before[a.b.requests];
  const int64_t per = share_of(total, (int)gridDim.x);
  const int share = share_index((int)blockIdx.x, (int)gridDim.x);
  int64_t at = (int64_t)share * per;
  const int64_t stop = min(at + per, total);
  const int lane = lane_id(), wave = wave_id();
  const int g = lane >> 4, c = lane & 15;

  while (at < stop) {
    // the request of tile `at`, then its (head, row block, tile)
    int lo = 0, hi = a.b.requests - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (d.before[mid] <= at) lo = mid; else hi = mid - 1;
    }
    const int r = __builtin_amdgcn_readfirstlane(lo);
    const int n = d.count[r], length = d.length[r], start = d.start[r];
    const int rows = n * a.group;
    const int blocks = (rows + ROWS - 1) / ROWS;
    const int end = length + n;
    const int tiles = (int)(((int64_t)length + n + kTile - 1) / kTile);
    const int64_t in_request = at - d.before[r];
    const int hb = (int)(in_request / tiles);
    const int head = hb / blocks, block = hb % blocks;
    const int t0 = (int)(in_request - (int64_t)hb * tiles);
    const int t1 = (int)min((int64_t)tiles, t0 + (stop - at));
    const int row0 = block * ROWS;
    const int32_t* table = a.c.table + (int64_t)r * a.c.table_stride;
    const uint16_t* kbase = a.c.k + (int64_t)head * a.c.head_stride + g * (D / 4);
    const uint16_t* vbase = a.c.v + (int64_t)head * a.c.head_stride + c * CW;

    // queries of row c of each row tile, and the drafts its token sees
    bf16x8 q[R][KS];
    uint64_t seen[R];
#pragma unroll
    for (int t = 0; t < R; ++t) {
      const int row = row0 + 16 * t + c;
      const bool on = row < rows;
      const int tok = on ? row / a.group : 0;
      const int h = head * a.group + (on ? row - tok * a.group : 0);
      const uint16_t* p = a.q + (int64_t)(start + tok) * a.q_stride + h * D + g * (D / 4);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        u32x4 w = load16(p + 8 * s);
        if (!on) w = u32x4{0, 0, 0, 0};
        q[t][s] = __builtin_bit_cast(bf16x8, w);
      }
      const uint64_t all = n >= 64 ? ~0ull : (1ull << n) - 1;
      seen[t] = !on ? 0 : (a.tree ? gmem(a.tree)[start + tok] : (tok >= 63 ? ~0ull : (2ull << tok) - 1)) & all;
    }

    f32x4 o[R][CW];
    float top[R], sum[R];
#pragma unroll
    for (int t = 0; t < R; ++t) {
      top[t] = -INFINITY;
      sum[t] = 0.f;
#pragma unroll
      for (int j = 0; j < CW; ++j) o[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    StepRows<P8> rows_now, rows_next;
    uint32_t kw[2][KS][4], vw[8][VW];
    uint32_t live_v;
    const auto load_k = [&](const StepRows<P8>& s) {
      if constexpr (P8) {
        const int64_t off = s.at(a.c, s.pid[1], s.pos[1]) + (c & 3) * a.c.token_stride;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < KS; ++i) load_words<4>(kbase + off + 4 * t * a.c.token_stride + 8 * i, kw[t][i]);
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int64_t off = s.at(a.c, s.pid[8 + t], s.pos[1] + 4 * t + (c & 3));
#pragma unroll
          for (int i = 0; i < KS; ++i) load_words<4>(kbase + off + 8 * i, kw[t][i]);
        }
      }
    };
    const auto load_v = [&](const StepRows<P8>& s) {
      live_v = s.v_live(a.c);
      if constexpr (P8) {
        const int64_t off = s.at(a.c, s.pid[0], s.pos[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) load_words<VW>(vbase + off + e * a.c.token_stride, vw[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) load_words<VW>(vbase + s.at(a.c, s.pid[e], s.pos[0] + e), vw[e]);
      }
    };

    bool special = false;
    const int base0 = t0 * kTile + wave * 32;
    int steps = t1 - t0;
    // the last tile may end before this wave's positions
    while (steps > 0 && base0 + (steps - 1) * kTile >= end) --steps;
    if (steps > 0) {
      rows_now.fetch(a.c, table, (uint32_t)base0, g, c);
      rows_next.fetch(a.c, table, (uint32_t)(base0 + kTile), g, c);
      load_k(rows_now);
      load_v(rows_now);
    }
    for (int it = 0; it < steps; ++it) {
      const int base = base0 + it * kTile;
      f32x4 s[R][2];
#pragma unroll
      for (int t = 0; t < R; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            const u32x4 w = {kw[u][i][0], kw[u][i][1], kw[u][i][2], kw[u][i][3]};
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), q[t][i], acc, 0, 0, 0);
          }
          s[t][u] = acc;
        }
      const uint32_t live = live_v;
      // the last step's request falls past the share: it reads row 0 of the pool or rows not used
      const StepRows<P8> coming = rows_next;
      load_k(coming);
      rows_next.fetch(a.c, table, (uint32_t)(base + 2 * kTile), g, c);

      float p[R][8];
      const bool whole = __all(live == 0xFFu && base + 32 <= length);
#pragma unroll
      for (int t = 0; t < R; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) p[t][e] = s[t][e >> 2][e & 3] * a.scale2;
      uint32_t dead = 0;
      if (!whole) {
        // lane's positions start at `past` drafts behind the context
        const int past = base + 8 * g - length;
        const uint32_t context = past >= 0 ? 0u : past <= -8 ? 0xFFu : (1u << -past) - 1u;
        const int have = n - past;                        // drafts from the lane's first position on
        const uint32_t filled = have <= 0 ? 0u : have >= 8 ? 0xFFu : (1u << have) - 1u;
        dead = ~(live & filled) & 0xFFu;
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const uint32_t draft = past >= 64 ? 0u : past >= 0 ? (uint32_t)(seen[t] >> past) & 0xFFu
                                 : past > -8 ? (uint32_t)(seen[t] << -past) & 0xFFu : 0u;
          const uint32_t sees = (context | draft) & live;
#pragma unroll
          for (int e = 0; e < 8; ++e) p[t][e] = sees >> e & 1 ? p[t][e] : -INFINITY;
        }
      }
      bool raise = false;
#pragma unroll
      for (int t = 0; t < R; ++t) {
        float most = fmaxf(fmaxf(fmaxf(p[t][0], p[t][1]), fmaxf(p[t][2], p[t][3])),
                           fmaxf(fmaxf(p[t][4], p[t][5]), fmaxf(p[t][6], p[t][7])));
        raise |= most > top[t] + kLazy;
      }
      if (__any(raise)) {
#pragma unroll
        for (int t = 0; t < R; ++t) {
          float most = fmaxf(fmaxf(fmaxf(p[t][0], p[t][1]), fmaxf(p[t][2], p[t][3])),
                             fmaxf(fmaxf(p[t][4], p[t][5]), fmaxf(p[t][6], p[t][7])));
          most = fmaxf(most, __shfl_xor(most, 16));
          most = fmaxf(most, __shfl_xor(most, 32));
          const float now = fmaxf(top[t], most);
          const float f = now == -INFINITY || now == top[t] ? 1.f : __builtin_amdgcn_exp2f(top[t] - now);
          top[t] = now;
          sum[t] *= f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float fr = __shfl(f, 4 * g + i);
#pragma unroll
            for (int j = 0; j < CW; ++j) o[t][j][i] *= fr;
          }
        }
      }
      bf16x8 w[R];
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const float ref = top[t] == -INFINITY ? 0.f : top[t];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[t][e] = __builtin_amdgcn_exp2f(p[t][e] - ref);
          sum[t] += p[t][e];
          w[t][e] = (__bf16)p[t][e];
        }
      }
      if (!whole) {
        // positions that hold nothing weigh nothing, whatever memory has there;
        // a draft's infinities and NaN must reach only the rows that see it, so
        // they leave the product (0 * inf is NaN) and are added at the end
        const int past = base + 8 * g - length;
        const uint32_t drafts = past >= 0 ? 0xFFu : past <= -8 ? 0u : 0xFFu << -past & 0xFFu;
        bool found = false;
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            const uint32_t x = dead >> e & 1 ? 0u : vw[e][i];
            const uint32_t fine = (bf16_special(x) ? 0u : x & 0xFFFFu) | (bf16_special(x >> 16) ? 0u : x & 0xFFFF0000u);
            const bool odd = (drafts >> e & 1) && fine != x;
            vw[e][i] = odd ? fine : x;
            found |= odd;
          }
        if (__any(found)) special = true;
      }
#pragma unroll
      for (int j = 0; j < CW; ++j) {
        const uint32_t pick = j & 1 ? 0x07060302u : 0x05040100u;
        u32x4 b;
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __builtin_amdgcn_perm(vw[2 * i + 1][j / 2], vw[2 * i][j / 2], pick);
#pragma unroll
        for (int t = 0; t < R; ++t)
          o[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[t], __builtin_bit_cast(bf16x8, b), o[t][j], 0, 0, 0);
      }
      load_v(coming);
    }

    // the four waves meet: a common maximum, then (2, 3) -> (0, 1) -> 0
#pragma unroll
    for (int t = 0; t < R; ++t) {
      sum[t] += __shfl_xor(sum[t], 16);
      sum[t] += __shfl_xor(sum[t], 32);
      if (g == 0) {
        sh.m[wave][16 * t + c] = top[t];
        sh.l[wave][16 * t + c] = sum[t];
      }
    }
    if (lane == 0) sh.special[wave] = special;
    __syncthreads();
    const bool any_special = (sh.special[0] | sh.special[1] | sh.special[2] | sh.special[3]) != 0;
    float most[R][4], all[R][4];
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 16 * t + 4 * g + i;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) m = fmaxf(m, sh.m[w][row]);
        const float ref = m == -INFINITY ? 0.f : m;
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) l += sh.l[w][row] * __builtin_amdgcn_exp2f(sh.m[w][row] - ref);
        const float f = __builtin_amdgcn_exp2f(sh.m[wave][row] - ref);
        most[t][i] = m;
        all[t][i] = l;
#pragma unroll
        for (int j = 0; j < CW; ++j) o[t][j][i] *= f;
      }
#pragma unroll
    for (int half = 2; half >= 1; half >>= 1) {
      if (wave >= half && wave < 2 * half) {
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < CW; ++j) sh.o[wave - half][16 * t + 4 * g + i][c * CW + j] = o[t][j][i];
      }
      __syncthreads();
      if (wave < half) {
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < CW; ++j) o[t][j][i] += sh.o[wave][16 * t + 4 * g + i][c * CW + j];
      }
      __syncthreads();
    }
    if (wave == 0) {
      const bool done = t0 == 0 && t1 == tiles;
      float* part = a.parts + ((int64_t)share * 2 + (t0 == 0)) * (ROWS * (D + 2));
#pragma unroll
      for (int t = 0; t < R; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int in = 16 * t + 4 * g + i, row = row0 + in;
          if (row >= rows) continue;
          if (done) {
            const int tok = row / a.group;
            const float f = all[t][i] == 0.f ? 0.f : 1.f / all[t][i];
            uint16_t* to = a.y + (int64_t)(start + tok) * a.y_stride + (head * a.group + row - tok * a.group) * D + c * CW;
#pragma unroll
            for (int j = 0; j < CW; j += 2) {
              const float x = all[t][i] == 0.f ? 0.f : o[t][j][i] * f, y = all[t][i] == 0.f ? 0.f : o[t][j + 1][i] * f;
              *gmem(reinterpret_cast<uint32_t*>(to + j)) = (uint32_t)f32_to_bf16(x) | (uint32_t)f32_to_bf16(y) << 16;
            }
          } else {
#pragma unroll
            for (int j = 0; j < CW; ++j) gmem(part)[in * D + c * CW + j] = o[t][j][i];
            if (c == 0) {
              gmem(part)[ROWS * D + in] = most[t][i];
              gmem(part)[ROWS * (D + 1) + in] = all[t][i];
            }
          }
        }
      if (any_special) {
        // infinities and NaN of this share's drafts, to the rows that see them: a
        // positive weight does not change them, so they are added as they are to
        // what this lane has just written
        for (int j = max(0, t0 * kTile - length); j < n && length + j < t1 * kTile; ++j) {
          const int64_t off = position_offset(a.c, r, (int64_t)length + j);
          if (off < 0) continue;
          for (int e = 0; e < CW; ++e) {
            const uint32_t bits = gmem(a.c.v)[off + (int64_t)head * a.c.head_stride + c * CW + e];
            if (!bf16_special(bits)) continue;
            for (int k = 0; k < 4 * R; ++k) {
              const int in = 16 * (k >> 2) + 4 * g + (k & 3), row = row0 + in, tok = row / a.group;
              if (row >= rows || (a.tree ? !(gmem(a.tree)[start + tok] >> j & 1) : j > tok)) continue;
              uint16_t* to = a.y + (int64_t)(start + tok) * a.y_stride + (head * a.group + row - tok * a.group) * D + c * CW + e;
              if (done)
                *gmem(to) = f32_to_bf16(__uint_as_float((uint32_t)*gmem(to) << 16) + __uint_as_float(bits << 16));
              else
                gmem(part)[in * D + c * CW + e] += __uint_as_float(bits << 16);
            }
          }
        }
      }
    }
    at += t1 - t0;
  }
}

// Joins the parts of groups that shares cut: a wave takes one row of a group.
template <int D, int R>
__global__ __launch_bounds__(kAttnThreads) void tree_attention_join_kernel(AttnArgs a, int grid) {
  constexpr int ROWS = 16 * R;
  constexpr int E = (D + kWave - 1) / kWave;      // elements per lane (D = 96: half the lanes have one less)
  extern __shared__ __align__(16) char lds[];
  const Deal d = deal_at(lds, a.b.requests);
  deal<ROWS>(a, d);
  const int64_t total = d.before[a.b.requests];
  const int64_t per = share_of(total, grid);
  const int lane = lane_id();
  // blockIdx.x: row of the batch (token); waves and blockIdx.y: heads
  int lo = 0, hi = a.b.requests - 1;
  const int token = (int)blockIdx.x;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (d.start[mid] <= token) lo = mid; else hi = mid - 1;
  }
  const int r = lo;
  const int n = d.count[r], tok = token - d.start[r];
  const int qh = (int)blockIdx.y * kAttnWaves + wave_id();
  if (tok < 0 || tok >= n || qh >= a.heads) return;
  const int rows = n * a.group, blocks = (rows + ROWS - 1) / ROWS;
  const int tiles = (int)(((int64_t)d.length[r] + n + kTile - 1) / kTile);
  const int head = qh / a.group, row = tok * a.group + qh - head * a.group;
  const int64_t first = d.before[r] + ((int64_t)head * blocks + row / ROWS) * tiles;
  const int64_t s0 = first / per, s1 = (first + tiles - 1) / per;
  if (s0 == s1) return;
  const int in = row % ROWS;
  float top = -INFINITY, sum = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int64_t s = s0; s <= s1; ++s) {
    const float* part = a.parts + (s * 2 + (s == s0)) * (ROWS * (D + 2));
    const float m = gmem(part)[ROWS * D + in], l = gmem(part)[ROWS * (D + 1) + in];
    const float now = fmaxf(top, m);
    const float ref = now == -INFINITY ? 0.f : now;
    const float fo = __builtin_amdgcn_exp2f(top - ref), fn = __builtin_amdgcn_exp2f(m - ref);
    top = now;
    sum = sum * fo + l * fn;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int at = e * kWave + lane;
      if (at < D) o[e] = o[e] * fo + gmem(part)[in * D + at] * fn;
    }
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int at = e * kWave + lane;
    if (at < D) gmem(a.y)[(int64_t)token * a.y_stride + qh * D + at] = f32_to_bf16(sum == 0.f ? 0.f : o[e] * f);
  }
}

// ---------------------------------------------------------------------------
// Host side

constexpr int64_t kAttnMade = 0x77715f6174746e31;

// Row tiles per block: the fewest of 1, 2, 4 that hold max_tokens rows per key
// head (head_dim 256: at most 2, its accumulators fill the registers).
static int attn_row_tiles(int group, int head_dim, int max_tokens) {
  const int rows = group * max_tokens;
  return rows <= 16 ? 1 : rows <= 32 || head_dim > 128 ? 2 : 4;
}
static int attn_grid(int row_tiles, int head_dim) { return 256 * attn_groups_per_cu(row_tiles, head_dim); }

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
  if ((rc = check_cache_align(name, a.cache))) return rc;
  if (!aligned16(a.q) || !aligned16(a.y) || ((uintptr_t)a.tree & 7))
    return fail(WQ_ERR_ALIGN, "%s: q and y must be 16-byte, tree 8-byte aligned", name);
  return WQ_OK;
}

template <int D, int R, bool P8>
static int attn_launch(const char* name, const AttnArgs& a, hipStream_t s) {
  const size_t deal = deal_bytes(a.b.requests);
  const size_t lds = sizeof(AttnLds<D, R>) + deal;
  const int grid = attn_grid(R, D);
  hipLaunchKernelGGL((tree_attention_kernel<D, R, P8>), dim3(grid), dim3(kAttnThreads), lds, s, a);
  hipLaunchKernelGGL((tree_attention_join_kernel<D, R>),
                     dim3((unsigned)a.b.tokens, (unsigned)((a.heads + kAttnWaves - 1) / kAttnWaves)),
                     dim3(kAttnThreads), deal, s, a, grid);
  return launch_status(name);
}

template <int D>
static int attn_launch_d(const char* name, const AttnArgs& a, int tiles, hipStream_t s) {
  const bool p8 = a.c.page_size % 8 == 0;
  if (tiles == 1) return p8 ? attn_launch<D, 1, true>(name, a, s) : attn_launch<D, 1, false>(name, a, s);
  if (tiles == 2) return p8 ? attn_launch<D, 2, true>(name, a, s) : attn_launch<D, 2, false>(name, a, s);
  if constexpr (D <= 128) return p8 ? attn_launch<D, 4, true>(name, a, s) : attn_launch<D, 4, false>(name, a, s);
  return fail(WQ_ERR_SHAPE, "%s: no kernel for this plan", name);
}

}  // namespace wq

using namespace wq;

extern "C" int64_t wq_tree_attention_workspace_bytes(int32_t heads, int32_t kv_heads, int32_t head_dim,
                                                     int32_t max_tokens) {
  if (!attn_dims_ok(heads, kv_heads, head_dim, max_tokens)) return 0;
  const int tiles = attn_row_tiles(heads / kv_heads, head_dim, max_tokens);
  return (int64_t)attn_grid(tiles, head_dim) * 2 * (16 * tiles) * (head_dim + 2) * 4;
}

extern "C" int wq_tree_attention_prepare(const wq_tree_attention* a, void* workspace, int64_t workspace_bytes,
                                         wq_tree_attention_plan* plan) {
  const char* name = "wq_tree_attention_prepare";
  if (!a || !plan || !workspace) return fail(WQ_ERR_NULL, "%s: a, workspace and plan must be non-null", name);
  int rc = attn_check(name, *a);
  if (rc) return rc;
  const int64_t need = wq_tree_attention_workspace_bytes(a->heads, a->cache.kv_heads, a->cache.head_dim, a->max_tokens);
  if (workspace_bytes < need)
    return fail(WQ_ERR_SHAPE, "%s: workspace_bytes = %lld, %lld are needed", name, (long long)workspace_bytes,
                (long long)need);
  if (!aligned16(workspace)) return fail(WQ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", name);
  wq_tree_attention_plan p{};
  if ((rc = plan_device(name, &p.device))) return rc;
  p.made = kAttnMade;
  p.variant = attn_row_tiles(a->heads / a->cache.kv_heads, a->cache.head_dim, a->max_tokens);
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
  a.scale2 = t.scale * 1.44269504088896340736f;
  a.heads = t.heads;
  a.group = t.heads / t.cache.kv_heads;
  a.max_tokens = t.max_tokens;
  hipStream_t s = (hipStream_t)stream;
  switch (t.cache.head_dim) {
    case 64: return attn_launch_d<64>(name, a, plan->variant, s);
    case 96: return attn_launch_d<96>(name, a, plan->variant, s);
    case 128: return attn_launch_d<128>(name, a, plan->variant, s);
    default: return attn_launch_d<256>(name, a, plan->variant, s);
  }
}
