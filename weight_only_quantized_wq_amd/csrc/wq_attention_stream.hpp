// The attention kernel: keys and values stream through LDS.
//
// A workgroup's share is a sequence of tiles, piece after piece.  Tiles travel
// from memory to a ring of STAGES buffers in LDS without passing through
// registers (global_load_lds: 64 lanes x 16 bytes to 1 KB of consecutive LDS),
// STAGES of them under way before the first product and, across the borders of
// pieces, one more requested into each buffer as it is done with.  Each wave
// requests its share of every tile's rows and counts its own requests: before
// the barrier that opens a tile it waits until all but the (STAGES - 2) newest
// tiles' requests are done.  (Ordinary loads and stores
// in between only make that wait longer.)
//
// With pages of a multiple of 8 positions (PAGE8) every 8 rows of a tile share a
// page: its number is a scalar load, all address arithmetic is scalar, and a
// request's lanes add offsets fixed for the whole launch.  Other pages look up
// every row (and have their page numbers come through LDS like the tiles).
//
// The waves share the tile in two ways, by the rows a launch can have per key
// head:
//   * WK = 1, blocks of 16 R W rows: every wave owns 16 R rows from the first
//     position of a piece to the last and reads the whole tile; nothing is
//     joined inside the workgroup.  Two workgroups of W = 4 waves share a CU (while
//     the deal leaves room for both, see attn_grid), or one of 8 waves with R = 2,
//     whose blocks of 256 rows pay half as much for each tile's way to LDS.
//   * WK = 4, up to 16 rows: all waves have the same rows and take 32 positions
//     of a tile of 128 each, so that a short context is a few steps long; they
//     meet in LDS at the end of a piece.
// Measured (MI355X, heads of 128), with the joining launch: 5 tokens over 32763
// positions, 64 / 8 heads, 39.7 us (134 MB, 3.4 TB/s; about 5 us until the ring runs
// and 6.5 to join); 32 trees of 8 over up to 16384, 32 / 8 heads, 61 us (231 MB, 3.8
// TB/s; what pieces cost between their tiles, and the join); one token over 500, 32 /
// 32 heads, 12.3 us (32 workgroups at the 33 bytes a clock that the direct loads
// reach on a CU, and a launch); 2 x 64 tokens over 16000, 64 / 8 heads, 103 us (656
// TFLOP/s: vector ALU 48 % and matrix pipe 33 % of the cycles, LDS 25 %, and too
// little of each beside the other).  For such trees 4 waves of 32 rows, two
// workgroups per CU, take 136 us.
// Page numbers of 8 rows against every row's: 32 trees of 8 65 / 87 us, 2 x 64 tokens
// 105 / 110, one token 12.9 / 14.2.
// K rows are stored with their 16-byte pieces exchanged by row (piece p of A
// row m at p ^ m), so that the 16 lanes reading one piece of 16 rows hit
// different banks; V rows are read along the row.
#pragma once

#include "wq_attention_shared.hpp"

namespace wq {

// Shape of a launch: positions of a tile, buffers of the ring, workgroups per
// CU.  The ring holds up to 64 KB (two workgroups share a CU's 160 KB), 96 KB with
// room for the deal of 4096 requests behind it, or 128 KB for fewer; a wave's share
// of a tile must be whole requests of 1 KB.
template <int D, int WK, int W>
struct Shape {
  static constexpr int TILE = WK == 4 ? 128 : D == 96 || W == 8 ? 64 : 32;
  static constexpr int STAGES = WK == 4 ? 2 : D == 96 || D == 256 ? 3 : 4;
  static constexpr int GROUPS = WK == 4 || W == 8 || D == 256 ? 1 : 2;
};

constexpr int kIdSlots = 8;           // page numbers: requested STAGES tiles before the tile's own requests

template <int D, int WK, int W>
struct StreamLds {
  using S = Shape<D, WK, W>;
  alignas(16) uint16_t k[S::STAGES][S::TILE][D];
  alignas(16) uint16_t v[S::STAGES][S::TILE][D];
  alignas(16) uint32_t ids[W][kIdSlots][S::TILE / W];
  uint32_t live[S::STAGES][W];      // which of a wave's rows are in use and have a page
};
// Where the waves of WK = 4 meet.
template <int D>
struct MeetLds {
  alignas(16) float o[2][16][D];
  float m[kAttnWaves][16];
  float l[kAttnWaves][16];
  int special[kAttnWaves];
};

// Which piece of a K row stands at piece `p` (an involution).
template <int D>
__device__ __forceinline__ int k_piece(int p, int m) {
  return D % 128 == 0 ? p ^ m : D == 64 ? p ^ (m >> 1) : p;
}

// Offset in LDS of a __shared__ object.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// Lane l's 16 (4) bytes at `from` to LDS at `to` + 16 (4) l.  In assembly so that
// no wait is placed for it but those below; `to` is an operand in m0, so that the
// compiler itself writes that register (one wait state before its use).
__device__ __forceinline__ void request16(const void* from, uint32_t to) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(to), "v"(from) : "memory");
}
// The same from lane offsets to a uniform address, which scalar additions make: a
// vector write of `base` would need five wait states before the load (a test reads the
// listing for that; with them in place one token takes 12.4 us instead of 12.3, wide
// trees 103 instead of 102).
__device__ __forceinline__ void request16(const void* base, uint32_t off, uint32_t to) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(to), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void request4(const void* from, uint32_t to) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, off" ::"{m0}"(to), "v"(from) : "memory");
}
// All but the N newest requests of this wave are done, its LDS accesses too.
template <int N>
__device__ __forceinline__ void wait_requests() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void meet() { asm volatile("s_barrier" ::: "memory"); }

template <int D, int R, int WK, int W, bool PAGE8>
__global__ __launch_bounds__(W * kWave, (Shape<D, WK, W>::GROUPS)) void attention_stream_kernel(AttnArgs a) {
  using S = Shape<D, WK, W>;
  constexpr int TILE = S::TILE, STAGES = S::STAGES;
  constexpr int ROWS = 16 * R * (W / WK);
  constexpr int KS = D / 32, CW = D / 16, VW = CW / 2;
  constexpr int CH = D / 8;                              // 16-byte pieces of a row
  constexpr int TR = TILE / W;                  // a wave's rows of a tile
  constexpr int NP = TR * CH / kWave;                    // its requests, each for keys and for values
  constexpr int STEPS = TILE / 32 / WK;
  static_assert(NP * kWave == TR * CH && STEPS >= 1 && (WK == 1 || (R == 1 && W == WK)), "tile does not divide");
  static_assert(!PAGE8 || D != 96, "8 rows are no whole number of requests");
  extern __shared__ __align__(16) char lds[];
  StreamLds<D, WK, W>& sh = *reinterpret_cast<StreamLds<D, WK, W>*>(lds);
  constexpr int MEET = sizeof(StreamLds<D, WK, W>);
  MeetLds<D>& mt = *reinterpret_cast<MeetLds<D>*>(lds + MEET);
  const Deal d = deal_at(lds + MEET + (WK > 1 ? sizeof(MeetLds<D>) : 0), a.b.requests);
  deal<ROWS, TILE>(a, d);
  const int total = __builtin_amdgcn_readfirstlane(d.before[a.b.requests]);
  const int per = share_of(total, (int)gridDim.x);
  const int share = share_index((int)blockIdx.x, (int)gridDim.x);
  if ((int64_t)share * per >= total) return;
  const int at = share * per;
  const int stop = (int)min((int64_t)at + per, (int64_t)total);
  const int lane = lane_id(), wave = wave_id();
  const int g = lane >> 4, c = lane & 15;
  const int wr = wave / WK, wk = wave % WK;

  Piece p = first_piece<ROWS, TILE>(a, d, at, stop);     // the products' piece
  if (p.t0 >= p.t1) return;
  Piece pi = p, pt = p;                                  // the page numbers', the tiles'
  int ti = p.t0, tt = p.t0;

  // PAGE8: lane offsets in bytes within 8 rows, keys (by the rows' place in a
  // step) and values, and the page numbers of this wave's rows of tile tt
  constexpr int GP = TR / 8;                             // a wave's groups of 8 rows
  constexpr int N8 = 8 * CH / kWave;                     // requests of 8 rows
  uint32_t koff[PAGE8 ? GP : 1][PAGE8 ? N8 : 1], voff[PAGE8 ? N8 : 1];
  uint32_t id8[GP];
  if constexpr (PAGE8) {
#pragma unroll
    for (int i = 0; i < N8; ++i) {
      const int row = (i * kWave + lane) / CH, ch = (i * kWave + lane) % CH;
      voff[i] = 2u * ((uint32_t)row * a.c.token_stride + 8 * ch);
#pragma unroll
      for (int j = 0; j < GP; ++j) {
        const int m = (row & 3) | (GP == 1 ? wave & 3 : GP == 2 ? (2 * wave + j) & 3 : j) << 2;
        koff[j][i] = 2u * ((uint32_t)row * a.c.token_stride + 8 * k_piece<D>(ch, m));
      }
    }
  }
  // the page numbers the next request_tile needs (scalar loads)
  const auto look_ahead = [&]() {
    if constexpr (PAGE8) {
      if (pt.t0 >= pt.t1) return;
      const int32_t* table = a.c.table + (int64_t)pt.r * a.c.table_stride;
#pragma unroll
      for (int j = 0; j < GP; ++j) {
        const uint32_t pos = (uint32_t)(tt * TILE + wave * TR + 8 * j);
        const int32_t* from = table + (pos < a.c.limit ? page_of(a.c, pos) : 0u);
        id8[j] = (uint32_t)*(const __attribute__((address_space(4))) int32_t*)from;
      }
    }
  };
  // other pages: page numbers of this wave's rows of the next tile
  int slot_i = 0;
  const auto request_ids = [&]() {
    if (PAGE8 || pi.t0 >= pi.t1) return;
    if (lane < TR) {
      const uint32_t pos = (uint32_t)(ti * TILE + wave * TR + lane);
      const int32_t* from = a.c.table + (int64_t)pi.r * a.c.table_stride + (pos < a.c.limit ? page_of(a.c, pos) : 0u);
      request4(from, lds_offset(&sh.ids[wave][slot_i][0]));
    }
    slot_i = (slot_i + 1) & (kIdSlots - 1);
    if (++ti == pi.t1) {
      next_piece<ROWS, TILE>(a, d, stop, pi);
      ti = pi.t0;
    }
  };
  // this wave's rows of the next tile; false where no tile is left
  int slot_t = 0, stage_t = 0;
  const auto request_tile = [&]() -> bool {
    if (pt.t0 >= pt.t1) return false;
    if constexpr (PAGE8) {
      const uint32_t kto = lds_offset(&sh.k[stage_t][wave * TR][0]), vto = lds_offset(&sh.v[stage_t][wave * TR][0]);
      const uint64_t head = (uint64_t)pt.head * a.c.head_stride;
      const uint32_t end = min((uint32_t)(pt.length + pt.n), a.c.limit);
      uint32_t live = 0;
#pragma unroll
      for (int j = 0; j < GP; ++j) {
        const uint32_t pos = (uint32_t)(tt * TILE + wave * TR + 8 * j);
        const bool has = pos < end && id8[j] < a.c.pages;
        // of rows that hold nothing: the pool's first, never used
        const uint64_t off = head + (has ? row_offset(a.c, id8[j], pos - page_of(a.c, pos) * a.c.page_size) : 0);
        live |= (has ? end - pos >= 8 ? 0xFFu : (1u << (end - pos)) - 1u : 0u) << (8 * j);
        const uint16_t* kp = (const uint16_t*)uniform_i64((int64_t)(a.c.k + off));
        const uint16_t* vp = (const uint16_t*)uniform_i64((int64_t)(a.c.v + off));
#pragma unroll
        for (int i = 0; i < N8; ++i) {
          request16(kp, koff[j][i], __builtin_amdgcn_readfirstlane(kto + (j * N8 + i) * (kWave * 16)));
          request16(vp, voff[i], __builtin_amdgcn_readfirstlane(vto + (j * N8 + i) * (kWave * 16)));
        }
      }
      if (lane == 0) sh.live[stage_t][wave] = live;
      stage_t = stage_t + 1 == STAGES ? 0 : stage_t + 1;
      if (++tt == pt.t1) {
        next_piece<ROWS, TILE>(a, d, stop, pt);
        tt = pt.t0;
      }
      look_ahead();
      return true;
    }
    const int pl = lane & (TR - 1);
    const uint32_t pos = (uint32_t)(tt * TILE + wave * TR + pl);
    const uint32_t id = sh.ids[wave][slot_t][pl];
    const bool has = pos < (uint32_t)(pt.length + pt.n) && pos < a.c.limit && id < a.c.pages;
    // of a position that holds nothing: row 0 of the pool, never used
    const uint64_t off = has ? row_offset(a.c, id, pos - page_of(a.c, pos) * a.c.page_size) : 0;
    const uint32_t live = (uint32_t)__ballot(has);
    if (lane == 0) sh.live[stage_t][wave] = live;
    const uint64_t head = (uint64_t)pt.head * a.c.head_stride;
    const uint16_t* from[NP][2];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int row = (i * kWave + lane) / CH, ch = (i * kWave + lane) % CH;
      const int m = (row + wave * TR) & 31;              // its place in a step of 32
      const uint64_t ro = __shfl(off, row) + head;
      from[i][0] = a.c.k + ro + 8 * k_piece<D>(ch, (m & 3) | (m >> 3) << 2);
      from[i][1] = a.c.v + ro + 8 * ch;
    }
    const uint32_t kto = lds_offset(&sh.k[stage_t][wave * TR][0]), vto = lds_offset(&sh.v[stage_t][wave * TR][0]);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      request16(from[i][0], __builtin_amdgcn_readfirstlane(kto + i * (kWave * 16)));
      request16(from[i][1], __builtin_amdgcn_readfirstlane(vto + i * (kWave * 16)));
    }
    slot_t = (slot_t + 1) & (kIdSlots - 1);
    stage_t = stage_t + 1 == STAGES ? 0 : stage_t + 1;
    if (++tt == pt.t1) {
      next_piece<ROWS, TILE>(a, d, stop, pt);
      tt = pt.t0;
    }
    return true;
  };

  const int in0 = wr * 16 * R;                           // the wave's first row of a block
  bf16x8 q[R][KS];
  uint64_t seen[R];
#pragma unroll
  for (int t = 0; t < R; ++t) load_query<D>(a, p, p.block * ROWS + in0 + 16 * t + c, g, q[t], seen[t]);
  if constexpr (PAGE8) {
    look_ahead();
  } else {
#pragma unroll 1
    for (int i = 0; i < 2 * STAGES; ++i) request_ids();
    wait_requests<0>();
  }
  bool more = true;
#pragma unroll 1
  for (int i = 0; i < STAGES; ++i) more = request_tile();
  // opens the share's first tile (fewer than STAGES may be left to request)
  if (more)
    wait_requests<(STAGES - 1) * 2 * NP>();
  else
    wait_requests<0>();
  meet();

  int stage = 0;
  while (p.t0 < p.t1) {
    const bool busy = p.block * ROWS + in0 < p.rows;     // else the wave only moves data
    f32x4 o[R][CW];
    float top[R];
    f32x4 sum[R];
#pragma unroll
    for (int t = 0; t < R; ++t) {
      top[t] = -INFINITY;
      sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < CW; ++j) o[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    bool special = false, far = false;
#pragma unroll 1
    for (int tile = p.t0; tile < p.t1; ++tile) {
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const int first = 32 * (wk + WK * st);           // the step's first position in the tile
        const int base = tile * TILE + first;
        if (busy && base < p.length + p.n) {
          uint32_t live_step;
          if constexpr (TR == 32) {
            live_step = sh.live[stage][wk];
          } else {
            const uint32_t* lv = &sh.live[stage][first / TR];
            live_step = 0;
#pragma unroll
            for (int i = 0; i < 32 / TR; ++i) live_step |= (lv[i] & ((1u << TR) - 1u)) << (TR * i);
          }
          live_step = __builtin_amdgcn_readfirstlane(live_step);
          const bool whole = live_step == ~0u && base + 32 <= p.length;
          // all of the step's reads from LDS first, so that the products wait once
          bf16x8 kf[2][KS];
          uint32_t vw[8][VW];
#pragma unroll
          for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint16_t* row = sh.k[stage][first + 8 * (c >> 2) + 4 * u + (c & 3)];
              kf[u][i] = *reinterpret_cast<const bf16x8*>(row + 8 * k_piece<D>(g * KS + i, c));
            }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t* row = reinterpret_cast<const uint32_t*>(&sh.v[stage][first + 8 * g + e][c * CW]);
#pragma unroll
            for (int i = 0; i < VW; ++i) vw[e][i] = row[i];
          }
          if constexpr (R == 1) __builtin_amdgcn_sched_barrier(0);
          f32x4 s[R][2];
#pragma unroll
          for (int t = 0; t < R; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) s[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int t = 0; t < R; ++t)
#pragma unroll
              for (int u = 0; u < 2; ++u)
                s[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[u][i], q[t][i], s[t][u], 0, 0, 0);
          uint32_t sees[R] = {};
          if (!whole) {
            const int past = base + 8 * g - p.length;    // drafts behind the context
            const uint32_t live = live_step >> (8 * g) & 0xFFu;
#pragma unroll
            for (int t = 0; t < R; ++t) sees[t] = sees_of(past, seen[t]) & live;
            // positions that hold nothing weigh nothing, whatever memory has
            // there; a draft's infinities and NaN are added at the end
            const uint32_t drafts = past >= 0 ? 0xFFu : past <= -8 ? 0u : 0xFFu << -past & 0xFFu;
            bool found = false;
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
              for (int i = 0; i < VW; ++i) {
                const uint32_t x = live >> e & 1 ? vw[e][i] : 0u;
                const uint32_t fine = (bf16_special(x) ? 0u : x & 0xFFFFu) | (bf16_special(x >> 16) ? 0u : x & 0xFFFF0000u);
                const bool odd = (drafts >> e & 1) && fine != x;
                vw[e][i] = odd ? fine : x;
                found |= odd;
              }
            if (__any(found)) special = true;
          }
          bf16x8 w[R];
          softmax_step<R, CW>(s, a.scale2, whole, sees, g, top, far, sum, o, w);
#pragma unroll
          for (int j = 0; j < CW; ++j) {
            const bf16x8 b = v_column<VW>(vw, j);
#pragma unroll
            for (int t = 0; t < R; ++t) o[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[t], b, o[t][j], 0, 0, 0);
          }
        }
      }
      stage = stage + 1 == STAGES ? 0 : stage + 1;
      // opens the next tile: its requests are done, and everyone is through with this one's buffer
      if (more)
        wait_requests<(STAGES - 2) * 2 * NP>();
      else
        wait_requests<0>();
      meet();
      more = request_tile();
      request_ids();
    }

    // the next piece's queries are under way while this one's results leave
    const Piece now = p;
    next_piece<ROWS, TILE>(a, d, stop, p);
    if (p.t0 < p.t1) {
#pragma unroll
      for (int t = 0; t < R; ++t) load_query<D>(a, p, p.block * ROWS + in0 + 16 * t + c, g, q[t], seen[t]);
    }
    if constexpr (WK == 1) {
#pragma unroll
      for (int t = 0; t < R; ++t) {
        float most[4], all[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          most[i] = __shfl(top[t], 4 * g + i);
          all[i] = sum[t][i];
        }
        if (busy) {
          write_rows<D, ROWS>(a, now, share, in0 + 16 * t, g, c, o[t], most, all);
          if (special) add_special<D, ROWS>(a, now, share, now.t0 * TILE, now.t1 * TILE, in0 + 16 * t, g, c);
        }
      }
    } else {
      // the four waves meet: a common maximum, then (2, 3) -> (0, 1) -> 0
      if (g == 0) mt.m[wave][c] = top[0];
      if (c < 4) mt.l[wave][4 * g + c] = c == 0 ? sum[0][0] : c == 1 ? sum[0][1] : c == 2 ? sum[0][2] : sum[0][3];
      if (lane == 0) mt.special[wave] = special;
      __syncthreads();
      const bool any_special = (mt.special[0] | mt.special[1] | mt.special[2] | mt.special[3]) != 0;
      float most[4], all[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * g + i;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) m = fmaxf(m, mt.m[w][row]);
        const float ref = m == -INFINITY ? 0.f : m;
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) l += mt.l[w][row] * __builtin_amdgcn_exp2f(mt.m[w][row] - ref);
        const float f = __builtin_amdgcn_exp2f(mt.m[wave][row] - ref);
        most[i] = m;
        all[i] = l;
#pragma unroll
        for (int j = 0; j < CW; ++j) o[0][j][i] *= f;
      }
#pragma unroll
      for (int half = 2; half >= 1; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < CW; ++j) mt.o[wave - half][4 * g + i][c * CW + j] = o[0][j][i];
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < CW; ++j) o[0][j][i] += mt.o[wave][4 * g + i][c * CW + j];
        }
        __syncthreads();
      }
      if (wave == 0) {
        write_rows<D, ROWS>(a, now, share, 0, g, c, o[0], most, all);
        if (any_special) add_special<D, ROWS>(a, now, share, now.t0 * TILE, now.t1 * TILE, 0, g, c);
      }
    }
  }
}

}  // namespace wq
