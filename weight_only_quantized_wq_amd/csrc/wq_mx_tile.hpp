// Product of many rows with MXFP4 weights: a workgroup of WN x WM waves computes a tile
// of BN weight rows x BM activation rows over a range of k, both operands staged through
// a ring of `kStages` buffers in LDS by direct loads, one barrier a stage.
//
// bf16 activations (XQ = false): stages of 64 inputs.  W stays in 4 bits up to the
// registers (8 bytes of a row a lane) and is converted there, four instructions for the
// A operand of a v_mfma_f32_16x16x32_bf16.  A lane's inputs are 16 g .. 16 g + 15 of the
// stage (g = lane / 16), so it needs one scale.
// MXFP4 activations (XQ): stages of 256 inputs and v_mfma_scale_f32_16x16x128_f8f6f4,
// which takes codes and scale bytes as they are.  A lane's groups are 2 g and 2 g + 1.
//
// Scale rows are multiples of 8 bytes here (windows of 256 inputs); others are padded
// beforehand (mx_pad_kernel).
//
// bf16, 2000 rows x 28672 x 4096: 393 us, 1.19 PFLOP/s (a library's bf16 product of this
// shape, with W in bf16, 332); with zeros for data the same kernel runs a third faster, so
// what is left is the chip's power, and conversions, which are 5 %.
// Both in 4 bits, 4096 rows x 10240 x 8192: 217 us, 3.2 PFLOP/s, half of what the matrix
// pipe gives.  Without the matrix instructions it takes 165, though its loads are 14 bytes
// per CU and clock only: with two buffers one stage is under way while one is multiplied,
// and its latency is what bounds it (matrix pipe busy 33 % of the time, LDS 16 %), besides
// 2.5 rounds of 256 tiles.  Stages of 128 inputs in four buffers are not built.
#pragma once

#include <stdint.h>

#include <type_traits>

#include "wq_direct.hpp"
#include "wq_mx.hpp"

namespace wq {

struct MxTileArgs {
  const uint8_t* w;
  const uint8_t* wscale;    // rows of sstride bytes
  const char* x;
  const uint8_t* xscale;
  int64_t x_stride;         // bytes
  float* y32;
  uint16_t* y16;
  int64_t y_stride;
  float* part;              // [shares][m][n] sums of shares of k, or null
  int32_t m, n;
  uint32_t w_bytes, x_bytes, sstride;
  int32_t stages, share;    // of a row; of a workgroup
  int32_t tn, tm;           // tiles
  int32_t vec;              // y takes 4 elements at once
};

// Four consecutive results of a row; past its end none.
__device__ __forceinline__ void store_quad(const MxTileArgs& a, int row, int col, f32x4 v) {
  const int64_t to = (int64_t)row * a.y_stride + col;
  if (a.vec && col + 4 <= a.n) {
    if (a.y32) *gmem(reinterpret_cast<f32x4*>(a.y32 + to)) = v;
    if (a.y16)
      *gmem(reinterpret_cast<uint64_t*>(a.y16 + to)) =
          (uint64_t)((uint32_t)f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16) |
          (uint64_t)((uint32_t)f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16) << 32;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < a.n) {
        if (a.y32) gmem(a.y32)[to + i] = v[i];
        if (a.y16) gmem(a.y16)[to + i] = f32_to_bf16(v[i]);
      }
  }
}

// The same of a share of k, in rows of a multiple of 4.
__device__ __forceinline__ void store_part(const MxTileArgs& a, int row, int col, f32x4 v) {
  const int64_t width = (a.n + 3) / 4 * 4;
  if (col < a.n) *gmem(reinterpret_cast<f32x4*>(a.part + ((int64_t)blockIdx.y * a.m + row) * width + col)) = v;
}

template <bool XQ, int TN, int TM, int WN, int WM>
struct TileShape {
  static constexpr int kWaves = WN * WM, BN = WN * TN * 16, BM = WM * TM * 16;
  static constexpr int kWRow = XQ ? 128 : 32;                    // bytes of W per row and stage
  static constexpr int kX = BM * 128, kW = BN * kWRow;
  static constexpr int kSW = BN * 8, kSX = XQ ? BM * 8 : 0;      // scales of a window
  static constexpr int kStages = XQ ? 2 : 3;
  // requests of a wave for a stage
  static constexpr int kXOps = kX / 1024 / kWaves, kWOps = kW / 1024 / kWaves, kSWOps = kSW / 256 / kWaves,
                       kSXOps = kSX / 256 / kWaves;
  static constexpr int kOps = kXOps + kWOps + kSWOps + kSXOps;
  static constexpr int kLds = kStages * (kX + kW) + 2 * (kSW + kSX);
  static_assert(kXOps * kWaves * 1024 == kX && kWOps * kWaves * 1024 == kW && kSWOps * kWaves * 256 == kSW &&
                kSXOps * kWaves * 256 == kSX);
};

// Where 16-byte piece `p` of row `r` stands among the eight of a 128-byte row in LDS: XOR
// by a permutation of the row's number.  A ds_read_b128 is served 16 lanes at a time, of
// which eight read piece p of rows {0-3, 12-15} and eight piece p ^ 2 of rows {4-11} of a
// tile (or the other way round), so the permutation keeps those halves' pieces apart
// (4 cycles a read; with r / 2 itself 8).
__device__ __forceinline__ int tile_piece(int p, int r) {
  const int q = (r >> 1) & 7;
  return p ^ (((q ^ (q << 1)) & 4) | ((q >> 1) & 2) | (q & 1));
}

template <int N, int I = 0, class F>
__device__ __forceinline__ void for_parts(F step) {
  if constexpr (I < N) {
    step(At<I>{});
    for_parts<N, I + 1>(step);
  }
}

template <bool XQ, bool TAIL, int TN, int TM, int WN, int WM>
__global__ __launch_bounds__(WN * WM * 64) void mx_tile_kernel(MxTileArgs a) {
  using T = TileShape<XQ, TN, TM, WN, WM>;
  constexpr int S = T::kStages;
  __shared__ __align__(1024) char lds[T::kLds];
  const int lane = lane_id(), wave = wave_id(), g = lane >> 4, c = lane & 15;
  // Workgroups go to the eight XCDs in turn: each XCD takes a contiguous range of tiles,
  // eight m tiles for one n tile before the next, so that its L2 serves neighbours.
  const int tiles = a.tn * a.tm, per = (tiles + 7) / 8;
  const int tile = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  if (((int)blockIdx.x >> 3) >= per || tile >= tiles) return;
  const int panel = tile / (8 * a.tn), rest = tile - panel * 8 * a.tn, high = min(8, a.tm - panel * 8);
  const int n0 = rest / high * T::BN, m0 = (panel * 8 + rest % high) * T::BM;

  char* const xs = lds;
  char* const ws = lds + S * T::kX;
  char* const sw = ws + S * T::kW;
  char* const sx = sw + 2 * T::kSW;
  const int rows_w = a.n - 1 - n0, rows_x = a.m - 1 - m0;        // last row of the tile that is there

  // where this wave's pieces come from: offsets to a scalar base that moves with the
  // stage, rows past the end as the last
  uint32_t xo[T::kXOps], xp[T::kXOps], wo[T::kWOps], wp[T::kWOps], swo[T::kSWOps], sxo[T::kSXOps > 0 ? T::kSXOps : 1];
#pragma unroll
  for (int i = 0; i < T::kXOps; ++i) {
    const int r = (i * T::kWaves + wave) * 8 + (lane >> 3);
    xp[i] = (uint32_t)tile_piece(lane & 7, r) * 16u;
    xo[i] = (uint32_t)min(r, rows_x) * (uint32_t)a.x_stride + xp[i];
  }
#pragma unroll
  for (int i = 0; i < T::kWOps; ++i) {
    // of 32-byte rows the halves change places from eight rows to the next, for ds_read_b32
    const int r = XQ ? (i * T::kWaves + wave) * 8 + (lane >> 3) : (i * T::kWaves + wave) * 32 + (lane >> 1);
    wp[i] = XQ ? (uint32_t)tile_piece(lane & 7, r) * 16u : (uint32_t)((lane ^ (r >> 3)) & 1) * 16u;
    wo[i] = (uint32_t)min(r, rows_w) * a.w_bytes + wp[i];
  }
#pragma unroll
  for (int i = 0; i < T::kSWOps; ++i)
    swo[i] = (uint32_t)min((i * T::kWaves + wave) * 32 + (lane >> 1), rows_w) * a.sstride + (lane & 1) * 4;
#pragma unroll
  for (int i = 0; i < T::kSXOps; ++i)
    sxo[i] = (uint32_t)min((i * T::kWaves + wave) * 32 + (lane >> 1), rows_x) * a.sstride + (lane & 1) * 4;
  const char* const xbase = a.x + m0 * a.x_stride;
  const uint8_t* const wbase = a.w + (int64_t)n0 * a.w_bytes;
  const uint8_t* const swbase = a.wscale + (int64_t)n0 * a.sstride;
  const uint8_t* const sxbase = XQ ? a.xscale + (int64_t)m0 * a.sstride : nullptr;

  // Request `op` of stage s, to the buffer of stage `to`.  In a row's last stage pieces
  // past its end read its first instead (what they meet is 0 or cleared).
  auto request_op = [&](int s, int to, auto op) __attribute__((always_inline)) {
    constexpr int o = decltype(op)::value;
    const int at = to % S, window = XQ ? s : s >> 2;
    if constexpr (o < T::kXOps) {
      const uint32_t k = (uint32_t)s * 128u;
      uint32_t off = xo[o];
      if (TAIL && k + xp[o] >= a.x_bytes) off -= xp[o];
      request16(xbase + k, off, lds_offset(xs + at * T::kX + (o * T::kWaves + wave) * 1024));
    } else if constexpr (o < T::kXOps + T::kWOps) {
      constexpr int i = o - T::kXOps;
      const uint32_t k = (uint32_t)s * T::kWRow;
      uint32_t off = wo[i];
      if (TAIL && k + wp[i] >= a.w_bytes) off -= wp[i];
      request16(wbase + k, off, lds_offset(ws + at * T::kW + (i * T::kWaves + wave) * 1024));
    } else if constexpr (o < T::kXOps + T::kWOps + T::kSWOps) {
      constexpr int i = o - T::kXOps - T::kWOps;
      request4(swbase + window * 8, swo[i], lds_offset(sw + (window & 1) * T::kSW + (i * T::kWaves + wave) * 256));
    } else {
      constexpr int i = o - T::kXOps - T::kWOps - T::kSWOps;
      request4(sxbase + window * 8, sxo[i], lds_offset(sx + (window & 1) * T::kSX + (i * T::kWaves + wave) * 256));
    }
  };
  const int rn = wave / WM * TN * 16 + c, rm = wave % WM * TM * 16 + c;   // this lane's first rows in the tile
  // A stage is multiplied in parts: half h of its inputs with TN / RS of the row tiles.
  constexpr int RS = XQ ? 2 : 1, TR = TN / RS, kParts = 2 * RS;
  u32x4 bx[2][TM];                                       // of the two halves
  typename std::conditional<XQ, u32x4, uint32_t>::type bw[2][TR];   // of even and odd parts
  uint32_t fw[TN], fx[XQ ? TM : 1];                      // scales, of a whole stage
  auto read = [&](int s, auto part) __attribute__((always_inline)) {
    constexpr int p = decltype(part)::value, h = p / RS, rs = p % RS;
    const char* const x = xs + s % S * T::kX;
    const char* const w = ws + s % S * T::kW;
    const int at = tile_piece(2 * g + h, c) << 4;
    if constexpr (rs == 0) {
#pragma unroll
      for (int t = 0; t < TM; ++t) bx[h][t] = *reinterpret_cast<const u32x4*>(x + (rm + t * 16) * 128 + at);
    }
#pragma unroll
    for (int r = 0; r < TR; ++r) {
      const int row = rn + (rs * TR + r) * 16;
      if constexpr (XQ)
        bw[p & 1][r] = *reinterpret_cast<const u32x4*>(w + row * 128 + at);
      else
        bw[p & 1][r] = *reinterpret_cast<const uint32_t*>(w + row * 32 + (((g >> 1) ^ (c >> 3)) & 1) * 16 + (g & 1) * 8 + h * 4);
    }
  };
  auto read_scales = [&](int s) __attribute__((always_inline)) {
    const int window = XQ ? s : s >> 2;
    const char* const f = sw + (window & 1) * T::kSW;
#pragma unroll
    for (int r = 0; r < TN; ++r) {
      if constexpr (XQ)
        fw[r] = *reinterpret_cast<const uint16_t*>(f + (rn + r * 16) * 8 + 2 * g);
      else
        fw[r] = *reinterpret_cast<const uint8_t*>(f + (rn + r * 16) * 8 + (s & 3) * 2 + (g >> 1));
    }
    if constexpr (XQ) {
#pragma unroll
      for (int t = 0; t < TM; ++t) fx[t] = *reinterpret_cast<const uint16_t*>(sx + (s & 1) * T::kSX + (rm + t * 16) * 8 + 2 * g);
    }
  };

  f32x4 acc[TN][TM];
#pragma unroll
  for (int r = 0; r < TN; ++r)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](auto part, auto then) __attribute__((always_inline)) {
    constexpr int p = decltype(part)::value, h = p / RS, rs = p % RS;
    for_parts<TR>([&](auto at) __attribute__((always_inline)) {
      constexpr int r = decltype(at)::value, r0 = rs * TR;
      if constexpr (XQ) {
        const i32x8 q = mx_operand(bw[p & 1][r]);
#pragma unroll
        for (int t = 0; t < TM; ++t)
          acc[r0 + r][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q, mx_operand(bx[h][t]), acc[r0 + r][t], 4, 4, h, (int)fw[r0 + r], h, (int)fx[t]);
      } else {
        const bf16x8 q = mx_bf16(bw[p & 1][r], __uint_as_float(fw[r0 + r] << 23));
#pragma unroll
        for (int t = 0; t < TM; ++t)
          acc[r0 + r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q, __builtin_bit_cast(bf16x8, bx[h][t]), acc[r0 + r][t], 0, 0, 0);
      }
      then(at);
    });
  };
  auto nothing = [](auto) __attribute__((always_inline)) {};
  // half a stage past the end: the scales are 0 there, bf16 activations anything
  auto clear = [&](int s, auto half) __attribute__((always_inline)) {
    if constexpr (TAIL && !XQ) {
      const uint32_t keep = (uint32_t)(s + 1) * 128u > a.x_bytes && g >= 2 ? 0u : ~0u;
#pragma unroll
      for (int t = 0; t < TM; ++t) bx[decltype(half)::value][t] &= u32x4{keep, keep, keep, keep};
    }
  };

  // Operands of a part are read while the part before is multiplied.  The wait and the
  // barrier stand before a stage's last part: the next stage has arrived then, and this
  // one's buffer has been read by all.  The loop has no branch: past the end the last
  // stage is requested again, to buffers that nobody reads any more (its scales over
  // themselves), and what lies there is read but not multiplied.  (With branches the
  // compiler moves the products behind them, and their operands to memory.)
  const int begin = (int)blockIdx.y * a.share, end = min(begin + a.share, a.stages);
#pragma unroll
  for (int i = 0; i < S; ++i)
    for_parts<T::kOps>([&](auto op) __attribute__((always_inline)) { request_op(min(begin + i, end - 1), begin + i, op); });
  wait_requests<(S - 1) * T::kOps>();
  meet();
  read(begin, At<0>{});
  read_scales(begin);
  for (int s = begin; s < end; ++s) {
    clear(s, At<0>{});
    for_parts<kParts - 1>([&](auto part) __attribute__((always_inline)) {
      read(s, At<decltype(part)::value + 1>{});
      multiply(part, nothing);
      __builtin_amdgcn_sched_barrier(0);          // no reads from further ahead: registers
    });
    wait_requests<(S - 2) * T::kOps>();
    meet();
    clear(s, At<1>{});
    read(s + 1, At<0>{});
    // the requests of a stage between the products, so that the matrix pipe does not wait
    // for all waves to have made theirs
    multiply(At<kParts - 1>{}, [&](auto at) __attribute__((always_inline)) {
      constexpr int r = decltype(at)::value, from = r * T::kOps / TR, to = (r + 1) * T::kOps / TR;
      for_parts<to - from>([&](auto op) __attribute__((always_inline)) {
        request_op(min(s + S, end - 1), s, At<from + decltype(op)::value>{});
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    read_scales(min(s + 1, end - 1));
  }
  wait_requests<0>();

  // lane: rows 4 g + i of W's 16, one activation row
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const int row = m0 + wave % WM * TM * 16 + t * 16 + c;
    if (row >= a.m) continue;
#pragma unroll
    for (int r = 0; r < TN; ++r) {
      const int col = n0 + wave / WM * TN * 16 + r * 16 + 4 * g;
      if (a.part)
        store_part(a, row, col, acc[r][t]);
      else
        store_quad(a, row, col, acc[r][t]);
    }
  }
}

// Rows of scales padded to multiples of 8 bytes, zeros (2^-127) behind the last.
__global__ __launch_bounds__(256) void mx_pad_kernel(const uint8_t* from, int64_t rows, uint32_t srow, uint32_t sstride, uint8_t* to) {
  const int64_t words = rows * (sstride / 4);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / (sstride / 4);
    const uint32_t at = (uint32_t)(i - r * (sstride / 4)) * 4u;
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (at + j < srow) v |= (uint32_t)gmem(from)[r * srow + at + j] << (8 * j);
    gmem(reinterpret_cast<uint32_t*>(to))[i] = v;
  }
}

}  // namespace wq
