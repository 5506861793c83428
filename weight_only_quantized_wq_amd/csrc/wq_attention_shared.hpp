// What attention is made of: arguments, the deal of the positions to
// workgroups, one step of the running softmax, and how results leave.
//
// With G = heads / kv_heads query heads per key head, the n tokens of a
// request make n * G rows that read the same keys.  The rows of one (request,
// key head) are cut into blocks of ROWS, the positions into tiles of TILE, and
// the tiles of all (request, key head, row block) groups, in that order, are
// dealt out to the launch's workgroups in equal contiguous shares (the lengths
// are known on the device only, so every workgroup computes the deal itself).
// A group that one workgroup covers is finished there; short groups are never
// cut.  The parts of a group cut by shares go to the workspace as (running
// maximum, sum, unnormalised output) and are joined, in share order, by a
// second launch.
//
// Matrix slots (v_mfma_f32_16x16x32_bf16, lane l = 16 g + c) are filled so that
// nothing moves between lanes in a step of 32 positions:
//   * S^T = K Q^T: A row m of sub-tile t is position 8 (m / 4) + 4 t + m % 4;
//     lane (g, c) supplies D/4 contiguous elements of A row c, from g D/4 on
//     (the contraction order is free as long as Q has the same).  The result
//     gives lane (g, c) the scores of query row c against positions 8 g .. 8 g +
//     7: eight in a row, so what a row sees of them is one byte.
//   * O = P V: A wants lane (g, c) to hold row c's weights of slots 8 g .. 8 g +
//     7, which is what it has.  B wants, for output column c, the same eight
//     positions of V: lane (g, c) holds D/16 contiguous elements of each of
//     them, and output column c of product j is element c D/16 + j, gathered
//     from the eight by v_perm.  O ends with D/16 contiguous elements of rows
//     4 g .. 4 g + 3 per lane.
#pragma once

#include <math.h>

#include "wq_kv.hpp"

namespace wq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = 4;
constexpr float kLazy = 8.f;          // powers of two the running maximum may lag behind
constexpr float kFar = 4194304.f;     // 2^22: from here on a maximum's own rounding moves weights (softmax_step)

struct AttnArgs {
  KvCache c;
  Batch b;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* y;
  int64_t y_stride;
  const uint64_t* tree;
  float* parts;          // [grid][2][ROWS][D + 2]
  float scale2;          // |scale| * log2(e), positive
  uint32_t q_flip;       // sign bits of a negative scale, for a pair of bf16
  int32_t heads;
  int32_t group;         // heads / kv_heads
  uint32_t group_magic;  // ceil(2^20 / group)
  int32_t max_tokens;
  int32_t uncut;         // groups of so many tiles are not cut
};

// What a group costs besides its tiles, in tiles: queries in, results out (about
// 9000 clocks a piece; 32 trees of 8 over up to 16384 positions, 0 / 4: 65 / 61 us).
constexpr int kGroupCost = 4;

// The deal: per request its rows, length and the cost of all groups before it.
struct Deal {
  int32_t* before;       // [requests + 1]
  uint32_t* where;       // first row + (rows << 24)
  int32_t* length;
  __device__ __forceinline__ int start(int r) const { return (int)(where[r] & 0xFFFFFFu); }
  __device__ __forceinline__ int count(int r) const { return (int)(where[r] >> 24); }
};

__device__ __forceinline__ Deal deal_at(char* lds, int requests) {
  Deal d;
  d.before = reinterpret_cast<int32_t*>(lds);
  d.where = reinterpret_cast<uint32_t*>(d.before + requests + 1);
  d.length = reinterpret_cast<int32_t*>(d.where + requests);
  return d;
}
constexpr size_t deal_bytes(int64_t requests) { return (size_t)((3 * requests + 1) * 4 + 15) / 16 * 16; }

// Tiles of a group: positions past the table hold nothing.
template <int TILE>
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int length, int count) {
  return (min(length + count, (int)a.c.limit) + TILE - 1) / TILE;
}

// Every thread of the workgroup; ends with a barrier.  A wave takes 64 requests
// at a time; with more than 64, sums of the chunks before are added in a second
// pass.
template <int ROWS, int TILE>
__device__ __forceinline__ void deal(const AttnArgs& a, const Deal& d) {
  __shared__ int chunk_sum[kMaxRequests / kWave];
  const int n = a.b.requests, lane = lane_id(), wave = wave_id();
  for (int base = wave * kWave; base < n; base += (int)blockDim.x) {
    const int r = base + lane;
    int cost = 0;
    if (r < n) {
      const int s0 = gmem(a.b.starts)[r], s1 = gmem(a.b.starts)[r + 1];
      const int len = min(max(gmem(a.b.lengths)[r], 0), (int)a.c.limit);
      const bool ok = s0 >= 0 && s1 >= s0 && s1 <= a.b.tokens && s1 - s0 <= a.max_tokens;
      const int cnt = ok ? s1 - s0 : 0;
      d.where[r] = ((uint32_t)max(s0, 0) & 0xFFFFFFu) | (uint32_t)cnt << 24;
      d.length[r] = len;
      const int blocks = (cnt * a.group + ROWS - 1) / ROWS;
      cost = a.c.kv_heads * blocks * (tiles_of<TILE>(a, len, cnt) + kGroupCost);
    }
    const int upto = wave_scan(cost);
    if (r < n) d.before[r] = upto - cost;
    if (lane == kWave - 1) {
      chunk_sum[base / kWave] = upto;
      if (n <= kWave) d.before[n] = upto;
    }
  }
  __syncthreads();
  if (n > kWave) {
    const int chunks = (n + kWave - 1) / kWave;
    const int sum = lane < chunks ? chunk_sum[lane] : 0;
    const int upto = wave_scan(sum);
    for (int base = wave * kWave; base < n; base += (int)blockDim.x) {
      const int add = __shfl(upto - sum, base / kWave);
      if (base + lane < n) d.before[base + lane] += add;
    }
    if (wave == 0 && lane == kWave - 1) d.before[n] = upto;
    __syncthreads();
  }
}

// The last request whose groups start at or before cost `at` (one with groups,
// if `at` lies below the total).
__device__ __forceinline__ int request_at(const Deal& d, int requests, int at) {
  const int lane = lane_id();
  int chunk = 0;
  if (requests > kWave) {
    const int r = lane * kWave;
    chunk = __popcll(__ballot(r < requests && d.before[min(r, requests)] <= at)) - 1;
  }
  const int r = chunk * kWave + lane;
  return chunk * kWave + __popcll(__ballot(r < requests && d.before[min(r, requests)] <= at)) - 1;
}

// The last request whose rows start at or before `token` (the first, if none).
__device__ __forceinline__ int request_of(const Deal& d, int requests, int token) {
  const int lane = lane_id();
  int chunk = 0;
  if (requests > kWave) {
    const int r = lane * kWave;
    chunk = max(__popcll(__ballot(r < requests && d.start(min(r, requests - 1)) <= token)) - 1, 0);
  }
  const int r = chunk * kWave + lane;
  return chunk * kWave + max(__popcll(__ballot(r < requests && d.start(min(r, requests - 1)) <= token)) - 1, 0);
}

// Cost of a share: equal for the launch's workgroups (a power of two of them),
// however small.  Measured, at least 256 positions / any: 5 tokens over 700
// positions, 64 / 8 heads of 128, 18.0 / 13.5 us; 8 such requests 23.1 / 19.0.
__device__ __forceinline__ int share_of(int total, int grid) { return (total + grid - 1) >> (31 - __builtin_clz(grid)); }

// Workgroups are dispatched round robin over the 8 XCDs; consecutive shares go
// to one XCD, so row blocks and cut groups that read the same keys share its L2.
__device__ __forceinline__ int share_index(int block, int grid) { return (block & 7) * (grid >> 3) + (block >> 3); }

__device__ __forceinline__ bool bf16_special(uint32_t bits) { return (bits & 0x7F80u) == 0x7F80u; }

// Token of a row of a request's rows per key head (row < 4096, group <= 64: the
// rounding of the factor adds less than 4096 / 2^20 < 1 / 64).
__device__ __forceinline__ int token_of(const AttnArgs& a, int row) { return (int)(((uint32_t)row * a.group_magic) >> 20); }

// A share's part of one group: which rows, positions and cache it covers.
struct Piece {
  int r, n, length, start;     // the request
  int rows, blocks;            // its rows per key head, their blocks
  int head, block;
  int tiles, t0, t1;           // tiles of the group, this share's (t0 == t1: none left)
  int after;                   // cost before the group's first tile
};

template <int ROWS, int TILE>
__device__ __forceinline__ void piece_request(const AttnArgs& a, const Deal& d, int r, Piece& p) {
  p.r = r;
  const uint32_t where = __builtin_amdgcn_readfirstlane(d.where[r]);
  p.n = (int)(where >> 24);
  p.start = (int)(where & 0xFFFFFFu);
  p.length = __builtin_amdgcn_readfirstlane(d.length[r]);
  p.rows = p.n * a.group;
  p.blocks = (p.rows + ROWS - 1) / ROWS;
  p.tiles = tiles_of<TILE>(a, p.length, p.n);
}

// The share's next piece (t0 == t1: none).
template <int ROWS, int TILE>
__device__ __forceinline__ void next_piece(const AttnArgs& a, const Deal& d, int stop, Piece& p) {
  p.after += p.tiles + kGroupCost;
  p.t0 = p.t1 = 0;
  if (p.after >= stop) return;
  if (++p.block == p.blocks) {
    p.block = 0;
    if (++p.head == a.c.kv_heads) {
      p.head = 0;
      int r = p.r + 1;
      while (__builtin_amdgcn_readfirstlane(d.where[r]) >> 24 == 0) ++r;     // a later request has tiles: after < stop
      piece_request<ROWS, TILE>(a, d, r, p);
    }
  }
  p.t1 = p.tiles <= a.uncut ? p.tiles : min(p.tiles, stop - p.after);
}

// The first piece of the share of cost [at, stop).
template <int ROWS, int TILE>
__device__ __forceinline__ Piece first_piece(const AttnArgs& a, const Deal& d, int at, int stop) {
  Piece p{};
  const int r = __builtin_amdgcn_readfirstlane(request_at(d, a.b.requests, at));
  piece_request<ROWS, TILE>(a, d, r, p);
  const int before = __builtin_amdgcn_readfirstlane(d.before[r]);
  const int each = p.tiles + kGroupCost;
  // quotients below 2^16 from a reciprocal of 24 bits: off by one at most
  int hb = (int)((float)(at - before) * __builtin_amdgcn_rcpf((float)each));
  hb += (int64_t)hb * each > at - before ? -1 : (int64_t)(hb + 1) * each <= at - before ? 1 : 0;
  hb = __builtin_amdgcn_readfirstlane(hb);
  p.head = p.blocks == 1 ? hb : (int)((uint32_t)hb / (uint32_t)p.blocks);
  p.block = hb - p.head * p.blocks;
  p.after = before + hb * each + kGroupCost;
  if (p.after >= stop) return p;
  if (p.tiles > a.uncut) {
    p.t0 = max(0, at - p.after);
    p.t1 = min(p.tiles, stop - p.after);
  } else if (at <= p.after) {
    p.t1 = p.tiles;
  } else {
    next_piece<ROWS, TILE>(a, d, stop, p);        // the group is another share's
  }
  return p;
}

// Queries of row `row` of the block, this lane's part, and the drafts that its
// token sees (none past the request's rows).
template <int D>
__device__ __forceinline__ void load_query(const AttnArgs& a, const Piece& p, int row, int g, bf16x8 (&q)[D / 32],
                                           uint64_t& seen) {
  const bool on = row < p.rows;
  const int tok = on ? token_of(a, row) : 0;
  const int h = p.head * a.group + (on ? row - tok * a.group : 0);
  const uint16_t* from = a.q + (int64_t)(p.start + tok) * a.q_stride + h * D + g * (D / 4);
#pragma unroll
  for (int s = 0; s < D / 32; ++s) {
    u32x4 w = load16(from + 8 * s);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = on ? w[i] ^ a.q_flip : 0u;
    q[s] = __builtin_bit_cast(bf16x8, w);
  }
  const uint64_t all = p.n >= 64 ? ~0ull : (1ull << p.n) - 1;
  seen = !on ? 0 : (a.tree ? gmem(a.tree)[p.start + tok] : (tok >= 63 ? ~0ull : (2ull << tok) - 1)) & all;
}

// Of the eight positions from `past` drafts behind the context on, those that
// belong to the context and those a row with `seen` sees (drafts it has).
__device__ __forceinline__ uint32_t sees_of(int past, uint64_t seen) {
  const uint32_t context = past >= 0 ? 0u : past <= -8 ? 0xFFu : (1u << -past) - 1u;
  const uint32_t draft = past >= 64 ? 0u : past >= 0 ? (uint32_t)(seen >> past) & 0xFFu
                         : past > -8 ? (uint32_t)(seen << -past) & 0xFFu : 0u;
  return context | draft;
}

__device__ __forceinline__ bf16x8 ones() {
  const __bf16 one = (__bf16)1.f;
  return bf16x8{one, one, one, one, one, one, one, one};
}

// x * scale rounded as the running maximum is: not fused with what follows.
__device__ __forceinline__ float scaled(float x, float scale) {
#pragma clang fp contract(off)
  return x * scale;
}

// One step of the running softmax over 32 positions: raw scores s in, weights w
// (bf16, relative to 2^top) out; sums and outputs are rescaled where the
// running maximum is raised.  That happens only when some score exceeds it by
// more than 2^kLazy (its exact value cancels in the quotient), so the usual
// step needs no exchange between lanes.  `sees` is used unless `whole`.
// The weights are rounded to bf16 for the matrix product (2^-8 of each at most).
// They are summed by one more product, with a column of ones: so the sum has the
// weights that the output has (a row that sees one position gets its value
// exactly), in the layout of the output's rows.  All else is fp32.
// The maximum is a rounded product.  One fma for score * scale - maximum keeps
// that rounding, up to half a step of the maximum, as a common factor of all the
// row's weights; below 2^22 that is less than 2^0.5 and cancels in the quotient, but
// from 2^31 on it leaves the range of fp32 (all weights 0, or infinite).  Where a row
// of the wave has such a maximum (`far`, kept from step to step: it changes only
// where a maximum does) the product is rounded first.
template <int R, int CW>
__device__ __forceinline__ void softmax_step(const f32x4 (&s)[R][2], float scale2, bool whole,
                                             const uint32_t (&sees)[R], int g, float (&top)[R], bool& far,
                                             f32x4 (&sum)[R], f32x4 (&o)[R][CW], bf16x8 (&w)[R]) {
  float x[R][8], most[R];
#pragma unroll
  for (int t = 0; t < R; ++t)
#pragma unroll
    for (int e = 0; e < 8; ++e) x[t][e] = s[t][e >> 2][e & 3];
  if (!whole) {
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[t][e] = sees[t] >> e & 1 ? x[t][e] : -INFINITY;
  }
  bool raise = false;
#pragma unroll
  for (int t = 0; t < R; ++t) {
    most[t] = fmaxf(fmaxf(fmaxf(x[t][0], x[t][1]), fmaxf(x[t][2], x[t][3])),
                    fmaxf(fmaxf(x[t][4], x[t][5]), fmaxf(x[t][6], x[t][7]))) * scale2;
    raise |= most[t] > top[t] + kLazy;
  }
  if (__any(raise)) {
    bool past = false;
#pragma unroll
    for (int t = 0; t < R; ++t) {
      float m = fmaxf(most[t], __shfl_xor(most[t], 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float now = fmaxf(top[t], m);
      const float f = now == -INFINITY || now == top[t] ? 1.f : __builtin_amdgcn_exp2f(top[t] - now);
      top[t] = now;
      past |= fabsf(now) >= kFar && now != -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float fr = __shfl(f, 4 * g + i);
        sum[t][i] *= fr;
#pragma unroll
        for (int j = 0; j < CW; ++j) o[t][j][i] *= fr;
      }
    }
    far = __any(past);
  }
  if (__builtin_expect(far, 0)) {
#pragma unroll
    for (int t = 0; t < R; ++t) {
      const float ref = top[t] == -INFINITY ? 0.f : top[t];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[t][e] = scaled(x[t][e], scale2) - ref;
    }
  }
  const float factor = far ? 1.f : scale2;
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const float ref = far || top[t] == -INFINITY ? 0.f : top[t];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[t][e] = (__bf16)__builtin_amdgcn_exp2f(fmaf(x[t][e], factor, -ref));
    }
    sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[t], ones(), sum[t], 0, 0, 0);
  }
}

// Operand B of output column j: element j of the lane's part of eight V rows.
template <int VW>
__device__ __forceinline__ bf16x8 v_column(const uint32_t (&v)[8][VW], int j) {
  const uint32_t pick = j & 1 ? 0x07060302u : 0x05040100u;
  u32x4 b;
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __builtin_amdgcn_perm(v[2 * i + 1][j / 2], v[2 * i][j / 2], pick);
  return __builtin_bit_cast(bf16x8, b);
}

// Results of rows 4 g .. 4 g + 3 of row tile t of the block leave: to y if the
// share covers the group, else to the share's part.  Part 1 of a share is a
// group that starts in it, part 0 one that does not.
template <int D, int ROWS>
__device__ __forceinline__ void write_rows(const AttnArgs& a, const Piece& p, int share, int in, int g, int c,
                                           const f32x4 (&o)[D / 16], const float (&top)[4], const float (&sum)[4]) {
  constexpr int CW = D / 16;
  const bool done = p.t0 == 0 && p.t1 == p.tiles;
  float* part = a.parts + ((int64_t)share * 2 + (p.t0 == 0)) * (ROWS * (D + 2));
  const int head = p.head, row0 = p.block * ROWS;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = in + 4 * g + i, row = row0 + at;
    if (row >= p.rows) continue;
    if (done) {
      const int tok = token_of(a, row);
      const float f = sum[i] == 0.f ? 0.f : 1.f / sum[i];
      uint16_t* to = a.y + (int64_t)(p.start + tok) * a.y_stride + (head * a.group + row - tok * a.group) * D + c * CW;
      uint32_t w[CW / 2];
#pragma unroll
      for (int j = 0; j < CW; j += 2) {
        const float x = sum[i] == 0.f ? 0.f : o[j][i] * f, y = sum[i] == 0.f ? 0.f : o[j + 1][i] * f;
        w[j / 2] = (uint32_t)f32_to_bf16(x) | (uint32_t)f32_to_bf16(y) << 16;
      }
      if constexpr (CW % 8 == 0) {
#pragma unroll
        for (int j = 0; j < CW / 2; j += 4)
          *gmem(reinterpret_cast<u32x4*>(to + 2 * j)) = u32x4{w[j], w[j + 1], w[j + 2], w[j + 3]};
      } else {
#pragma unroll
        for (int j = 0; j < CW / 2; ++j) *gmem(reinterpret_cast<uint32_t*>(to + 2 * j)) = w[j];
      }
    } else {
      if constexpr (CW % 4 == 0) {
#pragma unroll
        for (int j = 0; j < CW; j += 4)
          *gmem(reinterpret_cast<f32x4*>(part + at * D + c * CW + j)) = f32x4{o[j][i], o[j + 1][i], o[j + 2][i], o[j + 3][i]};
      } else {
#pragma unroll
        for (int j = 0; j < CW; ++j) gmem(part)[at * D + c * CW + j] = o[j][i];
      }
      if (c == 0) {
        gmem(part)[ROWS * D + at] = top[i];
        gmem(part)[ROWS * (D + 1) + at] = sum[i];
      }
    }
  }
}

// The infinities and NaN of the share's drafts were left out of the products (0
// * inf is NaN, and they must reach only the rows that see them); a positive
// weight does not change them, so they are added as they are to what this
// lane has written.
template <int D, int ROWS>
__device__ void add_special(const AttnArgs& a, const Piece& p, int share, int from, int to_pos, int in, int g, int c) {
  constexpr int CW = D / 16;
  const bool done = p.t0 == 0 && p.t1 == p.tiles;
  float* part = a.parts + ((int64_t)share * 2 + (p.t0 == 0)) * (ROWS * (D + 2));
  const int head = p.head, row0 = p.block * ROWS;
  for (int j = max(0, from - p.length); j < p.n && p.length + j < to_pos; ++j) {
    const int64_t off = position_offset(a.c, p.r, (int64_t)p.length + j);
    if (off < 0) continue;
    for (int e = 0; e < CW; ++e) {
      const uint32_t bits = gmem(a.c.v)[off + (int64_t)head * a.c.head_stride + c * CW + e];
      if (!bf16_special(bits)) continue;
      for (int i = 0; i < 4; ++i) {
        const int at = in + 4 * g + i, row = row0 + at, tok = token_of(a, row);
        if (row >= p.rows || (a.tree ? !(gmem(a.tree)[p.start + tok] >> j & 1) : j > tok)) continue;
        uint16_t* to = a.y + (int64_t)(p.start + tok) * a.y_stride + (head * a.group + row - tok * a.group) * D + c * CW + e;
        if (done)
          *gmem(to) = f32_to_bf16(__uint_as_float((uint32_t)*gmem(to) << 16) + __uint_as_float(bits << 16));
        else
          gmem(part)[at * D + c * CW + e] += __uint_as_float(bits << 16);
      }
    }
  }
}

}  // namespace wq
