// Product of a middling number of rows with MXFP4 weights, where tiles of 256 x 256 do
// not fill the chip: a workgroup takes 16 TN weight rows x 16 TM activation rows over a
// share of k, and its waves take the share's stages in turn, each with a ring of P stages
// of its own (no barrier until the end; a wave's operands meet the whole tile, so little
// LDS is read per product).  The waves' sums meet in LDS, the shares' in a second launch,
// both in a fixed order.
//
// Stages, operands and lanes are those of mx_tile_kernel.  47 rows x 4096 x 14336 (tiles
// of 64 x 48, four shares): 16.4 us, about 13 in this launch and 3.5 in the second.  It is
// bound by latencies: the start of both launches, and seven stages a wave of which two are
// under way.
#pragma once

#include <stdint.h>

#include "wq_mx_tile.hpp"

namespace wq {

template <bool XQ, int TN, int TM, int P, int WAVES>
struct SplitShape {
  static constexpr int BN = TN * 16, BM = TM * 16;
  static constexpr int kWRow = XQ ? 128 : 32;
  static constexpr int kX = BM * 128, kW = BN * kWRow;
  // scale bytes of a row and stage: 8 (256 inputs), or the word that holds 64 inputs' two
  static constexpr int kScale = XQ ? 8 : 4;
  static constexpr int kSW = BN * kScale, kSX = XQ ? BM * kScale : 0;
  static constexpr int kSlot = kX + kW + kSW + kSX;
  static constexpr int kXOps = kX / 1024, kWOps = kW / 1024, kSWOps = kSW / 256, kSXOps = kSX / 256;
  static constexpr int kOps = kXOps + kWOps + kSWOps + kSXOps;
  static constexpr int kRing = WAVES * P * kSlot, kSums = WAVES * BN * BM * 4;
  static constexpr int kLds = kRing > kSums ? kRing : kSums;
  static_assert(kXOps * 1024 == kX && kWOps * 1024 == kW && kSWOps * 256 == kSW && kSXOps * 256 == kSX && (P - 1) * kOps < 64);
};

template <bool XQ, int TN, int TM, int P, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void mx_split_kernel(MxTileArgs a) {
  using T = SplitShape<XQ, TN, TM, P, WAVES>;
  __shared__ __align__(1024) char lds[T::kLds];
  const int lane = lane_id(), wave = wave_id(), g = lane >> 4, c = lane & 15;
  // the m tiles of one n tile and share next to each other
  const int m0 = (int)blockIdx.x % a.tm * T::BM, n0 = (int)blockIdx.x / a.tm * T::BN;
  const int s0 = (int)blockIdx.y * a.share, s1 = min(s0 + a.share, a.stages);
  const int rows_w = a.n - 1 - n0, rows_x = a.m - 1 - m0;
  char* const ring = lds + wave * P * T::kSlot;
  const char* const xbase = a.x + m0 * a.x_stride;
  const uint8_t* const wbase = a.w + (int64_t)n0 * a.w_bytes;
  const uint8_t* const swbase = a.wscale + (int64_t)n0 * a.sstride;
  const uint8_t* const sxbase = XQ ? a.xscale + (int64_t)m0 * a.sstride : nullptr;

  auto request = [&](int s, int slot) {
    char* const to = ring + slot * T::kSlot;
    const uint32_t xk = (uint32_t)s * 128u, wk = (uint32_t)s * T::kWRow;
    const uint32_t sk = XQ ? (uint32_t)s * 8u : (uint32_t)(s >> 1) * 4u;
#pragma unroll
    for (int i = 0; i < T::kXOps; ++i) {
      const int r = i * 8 + (lane >> 3);
      const uint32_t p = (uint32_t)tile_piece(lane & 7, r) * 16u;
      request16(xbase + min(r, rows_x) * a.x_stride + min(xk + p, a.x_bytes - 16u), lds_offset(to + i * 1024));
    }
#pragma unroll
    for (int i = 0; i < T::kWOps; ++i) {
      const int r = XQ ? i * 8 + (lane >> 3) : i * 32 + (lane >> 1);
      const uint32_t p = XQ ? (uint32_t)tile_piece(lane & 7, r) * 16u : (uint32_t)((lane ^ (r >> 3)) & 1) * 16u;
      request16_late(wbase, (uint32_t)min(r, rows_w) * a.w_bytes + min(wk + p, a.w_bytes - 16u), lds_offset(to + T::kX + i * 1024));
    }
    constexpr int words = T::kScale / 4;
#pragma unroll
    for (int i = 0; i < T::kSWOps; ++i) {
      const int r = i * (64 / words) + lane / words;
      request4_late(swbase + sk, (uint32_t)min(r, rows_w) * a.sstride + lane % words * 4, lds_offset(to + T::kX + T::kW + i * 256));
    }
#pragma unroll
    for (int i = 0; i < T::kSXOps; ++i) {
      const int r = i * 32 + (lane >> 1);
      request4_late(sxbase + sk, (uint32_t)min(r, rows_x) * a.sstride + (lane & 1) * 4,
                    lds_offset(to + T::kX + T::kW + T::kSW + i * 256));
    }
  };

  f32x4 acc[TN][TM];
#pragma unroll
  for (int r = 0; r < TN; ++r)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int first = s0 + wave, count = first < s1 ? (s1 - first + WAVES - 1) / WAVES : 0;
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (p < count) request(first + p * WAVES, p);
  for (int i = 0; i < count; ++i) {
    const int s = first + i * WAVES;
    if (count - i >= P)
      wait_requests<(P - 1) * T::kOps>();
    else if (P > 2 && count - i == 2)
      wait_requests<T::kOps>();
    else
      wait_requests<0>();
    const char* const x = ring + i % P * T::kSlot;
    const char* const w = x + T::kX;
    if constexpr (XQ) {
      const char* const fw = w + T::kW;
      const char* const fx = fw + T::kSW;
      i32x8 b[2][TM], q[2][TN];
      int pw[TN], px[TM];
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        px[t] = *reinterpret_cast<const uint16_t*>(fx + (c + t * 16) * 8 + 2 * g);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(x + (c + t * 16) * 128 + (tile_piece(2 * g + h, c) << 4));
          b[h][t] = mx_operand(v);
        }
      }
#pragma unroll
      for (int r = 0; r < TN; ++r) {
        pw[r] = *reinterpret_cast<const uint16_t*>(fw + (c + r * 16) * 8 + 2 * g);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(w + (c + r * 16) * 128 + (tile_piece(2 * g + h, c) << 4));
          q[h][r] = mx_operand(v);
        }
      }
      wait_lds();
      if (i + P < count) request(s + P * WAVES, i % P);
#pragma unroll
      for (int r = 0; r < TN; ++r)
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          acc[r][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q[0][r], b[0][t], acc[r][t], 4, 4, 0, pw[r], 0, px[t]);
          acc[r][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q[1][r], b[1][t], acc[r][t], 4, 4, 1, pw[r], 1, px[t]);
        }
    } else {
      u32x4 b[TM][2];
      uint64_t q[TN];
      uint32_t sc[TN];
#pragma unroll
      for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          b[t][h] = *reinterpret_cast<const u32x4*>(x + (c + t * 16) * 128 + (tile_piece(2 * g + h, c) << 4));
#pragma unroll
      for (int r = 0; r < TN; ++r) {
        q[r] = *reinterpret_cast<const uint64_t*>(w + (c + r * 16) * 32 + (((g >> 1) ^ (c >> 3)) & 1) * 16 + (g & 1) * 8);
        sc[r] = *reinterpret_cast<const uint8_t*>(w + T::kW + (c + r * 16) * 4 + (s & 1) * 2 + (g >> 1));
      }
      wait_lds();
      if (i + P < count) request(s + P * WAVES, i % P);
      if ((uint32_t)(s + 1) * 128u > a.x_bytes && g >= 2) {
        // half a stage past the end: the scales are 0 there, the activations anything
#pragma unroll
        for (int t = 0; t < TM; ++t) b[t][0] = b[t][1] = u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int r = 0; r < TN; ++r) {
        const float f = __uint_as_float(sc[r] << 23);
        const bf16x8 lo = mx_bf16((uint32_t)q[r], f), hi = mx_bf16((uint32_t)(q[r] >> 32), f);
#pragma unroll
        for (int t = 0; t < TM; ++t)
          acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, __builtin_bit_cast(bf16x8, b[t][0]), acc[r][t], 0, 0, 0);
#pragma unroll
        for (int t = 0; t < TM; ++t)
          acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, __builtin_bit_cast(bf16x8, b[t][1]), acc[r][t], 0, 0, 0);
      }
    }
  }
  // the waves' sums, lane by lane, then 4 consecutive weight rows of an activation row
  __syncthreads();
#pragma unroll
  for (int r = 0; r < TN; ++r)
#pragma unroll
    for (int t = 0; t < TM; ++t) *reinterpret_cast<f32x4*>(lds + ((wave * TN + r) * TM + t) * 1024 + lane * 16) = acc[r][t];
  __syncthreads();
  for (int o = (int)threadIdx.x; o < T::BN / 4 * T::BM; o += WAVES * 64) {
    const int quad = o % (T::BN / 4), row = o / (T::BN / 4);          // rows 4 quad .. of W, row `row` of x
    if (m0 + row >= a.m) break;
    const char* from = lds + ((quad >> 2) * TM + (row >> 4)) * 1024 + ((quad & 3) * 16 + (row & 15)) * 16;
    f32x4 v = *reinterpret_cast<const f32x4*>(from);
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += *reinterpret_cast<const f32x4*>(from + w * TN * TM * 1024);
    const int col = n0 + 4 * quad;
    if (a.part)
      store_part(a, m0 + row, col, v);
    else
      store_quad(a, m0 + row, col, v);
  }
}

// Shares of k summed in order.
__global__ __launch_bounds__(256) void mx_join_kernel(MxTileArgs a, int splits) {
  const int quads = (a.n + 3) / 4;
  const int64_t all = (int64_t)a.m * quads, step = all * 4;
  const int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (o >= all) return;
  const float* from = a.part + o * 4;
  f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; s += 8) {
    f32x4 p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = *gmem(reinterpret_cast<const f32x4*>(from + min(s + i, splits - 1) * step));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s + i < splits) v += p[i];
  }
  store_quad(a, (int)(o / quads), (int)(o % quads) * 4, v);
}

}  // namespace wq
