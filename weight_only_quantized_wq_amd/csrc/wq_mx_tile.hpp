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
// 128-byte rows lie XOR-permuted by pieces of 16 bytes, so that 16 rows read at one
// piece meet no bank twice.  Scale rows are multiples of 8 bytes here (windows of 256
// inputs); others are padded beforehand (mx_pad_kernel).
#pragma once

#include <stdint.h>

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
  int32_t stages, share;    // of a row; of a workgroup of mx_split_kernel
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

template <bool XQ, int TN, int TM, int WN, int WM>
__global__ __launch_bounds__(WN * WM * 64) void mx_tile_kernel(MxTileArgs a) {
  using T = TileShape<XQ, TN, TM, WN, WM>;
  __shared__ __align__(1024) char lds[T::kLds];
  const int lane = lane_id(), wave = wave_id(), g = lane >> 4, c = lane & 15;
  // Workgroups go to the eight XCDs in turn: each XCD takes a contiguous range of tiles,
  // eight m tiles for one n tile before the next, so that its L2 serves neighbours.
  const int tiles = a.tn * a.tm, per = (tiles + 7) / 8;
  const int tile = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  if (((int)blockIdx.x >> 3) >= per || tile >= tiles) return;
  const int panel = tile / (8 * a.tn), rest = tile - panel * 8 * a.tn, high = min(8, a.tm - panel * 8);
  const int n0 = rest / high * T::BN, m0 = (panel * 8 + rest % high) * T::BM;
  const int count = a.stages;

  char* const xs = lds;
  char* const ws = lds + T::kStages * T::kX;
  char* const sw = ws + T::kStages * T::kW;
  char* const sx = sw + 2 * T::kSW;
  const int rows_w = a.n - 1 - n0, rows_x = a.m - 1 - m0;        // last row of the tile that is there

  // offsets of this wave's pieces, rows past the end as the last
  uint32_t xo[T::kXOps], wo[T::kWOps], swo[T::kSWOps], sxo[T::kSXOps > 0 ? T::kSXOps : 1];
  uint32_t xp[T::kXOps], wp[T::kWOps];
#pragma unroll
  for (int i = 0; i < T::kXOps; ++i) {
    const int r = (i * T::kWaves + wave) * 8 + (lane >> 3);
    xp[i] = (uint32_t)((lane & 7) ^ ((r >> 1) & 7)) * 16u;
    xo[i] = (uint32_t)(min(r, rows_x));
  }
#pragma unroll
  for (int i = 0; i < T::kWOps; ++i) {
    const int r = XQ ? (i * T::kWaves + wave) * 8 + (lane >> 3) : (i * T::kWaves + wave) * 32 + (lane >> 1);
    wp[i] = XQ ? (uint32_t)((lane & 7) ^ ((r >> 1) & 7)) * 16u : (uint32_t)(lane & 1) * 16u;
    wo[i] = (uint32_t)min(r, rows_w) * a.w_bytes;
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

  auto request = [&](int s) {
    const int at = s % T::kStages, window = XQ ? s : s >> 2;
    const uint32_t xk = (uint32_t)s * 128u, wk = (uint32_t)s * T::kWRow;
#pragma unroll
    for (int i = 0; i < T::kXOps; ++i)
      request16(xbase + xo[i] * a.x_stride + min(xk + xp[i], a.x_bytes - 16u),
                lds_offset(xs + at * T::kX + (i * T::kWaves + wave) * 1024));
#pragma unroll
    for (int i = 0; i < T::kWOps; ++i)
      request16_late(wbase, wo[i] + min(wk + wp[i], a.w_bytes - 16u),
                     lds_offset(ws + at * T::kW + (i * T::kWaves + wave) * 1024));
#pragma unroll
    for (int i = 0; i < T::kSWOps; ++i)
      request4_late(swbase + window * 8, swo[i], lds_offset(sw + (window & 1) * T::kSW + (i * T::kWaves + wave) * 256));
#pragma unroll
    for (int i = 0; i < T::kSXOps; ++i)
      request4_late(sxbase + window * 8, sxo[i], lds_offset(sx + (window & 1) * T::kSX + (i * T::kWaves + wave) * 256));
  };

  f32x4 acc[TN][TM];
#pragma unroll
  for (int r = 0; r < TN; ++r)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int rn = wave / WM * TN * 16 + c, rm = wave % WM * TM * 16 + c;   // this lane's first rows in the tile

#pragma unroll
  for (int i = 0; i < T::kStages - 1; ++i)
    if (i < count) request(i);
  for (int s = 0; s < count; ++s) {
    const int at = s % T::kStages;
    if (T::kStages > 2 && s + 1 < count)
      wait_requests<(T::kStages - 2) * T::kOps>();
    else
      wait_requests<0>();
    meet();
    if (s + T::kStages - 1 < count) request(s + T::kStages - 1);
    const char* const x = xs + at * T::kX;
    const char* const w = ws + at * T::kW;
    if constexpr (XQ) {
      const char* const fw = sw + (s & 1) * T::kSW;
      const char* const fx = sx + (s & 1) * T::kSX;
      uint32_t ps[TM];
#pragma unroll
      for (int t = 0; t < TM; ++t) ps[t] = *reinterpret_cast<const uint16_t*>(fx + (rm + t * 16) * 8 + 2 * g);
      auto step = [&](auto at) __attribute__((always_inline)) {
        constexpr int ks = decltype(at)::value;
        i32x8 b[TM];
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(x + (rm + t * 16) * 128 + (((2 * g + ks) ^ ((c >> 1) & 7)) << 4));
          b[t] = i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
        }
#pragma unroll
        for (int r = 0; r < TN; ++r) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(w + (rn + r * 16) * 128 + (((2 * g + ks) ^ ((c >> 1) & 7)) << 4));
          const i32x8 q = {(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
          const int sc = *reinterpret_cast<const uint16_t*>(fw + (rn + r * 16) * 8 + 2 * g);
#pragma unroll
          for (int t = 0; t < TM; ++t)
            acc[r][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q, b[t], acc[r][t], 4, 4, ks, sc, ks, (int)ps[t]);
        }
      };
      step(At<0>{});
      step(At<1>{});
    } else {
      const uint8_t* const fw = reinterpret_cast<const uint8_t*>(sw + ((s >> 2) & 1) * T::kSW) + (s & 3) * 2 + (g >> 1);
      u32x4 b[TM][2];
#pragma unroll
      for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          b[t][h] = *reinterpret_cast<const u32x4*>(x + (rm + t * 16) * 128 + (((2 * g + h) ^ ((c >> 1) & 7)) << 4));
      if ((uint32_t)(s + 1) * 128u > a.x_bytes && g >= 2) {
        // half a stage past the end: the scales are 0 there, the activations anything
#pragma unroll
        for (int t = 0; t < TM; ++t) b[t][0] = b[t][1] = u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int r = 0; r < TN; ++r) {
        const uint64_t v = *reinterpret_cast<const uint64_t*>(w + (rn + r * 16) * 32 + g * 8);
        const float sc = __uint_as_float((uint32_t)fw[(rn + r * 16) * 8] << 23);
        const bf16x8 lo = mx_bf16((uint32_t)v, sc), hi = mx_bf16((uint32_t)(v >> 32), sc);
#pragma unroll
        for (int t = 0; t < TM; ++t)
          acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, __builtin_bit_cast(bf16x8, b[t][0]), acc[r][t], 0, 0, 0);
#pragma unroll
        for (int t = 0; t < TM; ++t)
          acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, __builtin_bit_cast(bf16x8, b[t][1]), acc[r][t], 0, 0, 0);
      }
    }
  }

  // lane: rows 4 g + i of W's 16, one activation row
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const int row = m0 + wave % WM * TM * 16 + t * 16 + c;
    if (row >= a.m) continue;
#pragma unroll
    for (int r = 0; r < TN; ++r) {
      const int col = n0 + wave / WM * TN * 16 + r * 16 + 4 * g;
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
