// Products of quantized weight rows with a few activation rows: how one wave streams
// its share.  Used by the MXFP4 product of few rows and by the expert layer.
//
// A unit is 16 weight rows x 256 bytes (512 MXFP4 or 256 int8 inputs, a "span" of the
// row).  Units come by direct loads into a ring of P slots in LDS that belongs to the
// wave alone, so no barrier is needed: each load takes 8 rows x 128 contiguous bytes,
// whole cache lines, with the 16-byte pieces of a row XOR-permuted so that the reads
// below meet no bank twice.  From the slot a lane reads the A operand of
// v_mfma_f32_16x16x32_bf16: row l % 16, and of the span's 16 pieces the four that start
// at 4 (l / 16), so that its four scale bytes are one word.  The order of inputs inside
// a span is free as long as the activations follow it.
//
// Activations (up to COLS rows) of a span come by direct loads too, and stay in
// registers while the units of the wave's row tiles go by: RT tiles share one read.
// D: lane l holds rows 4 (l / 16) + r of column l % 16.
#pragma once

#include <stdint.h>

#include "wq_direct.hpp"
#include "wq_mx.hpp"

namespace wq {

// What a stream reads: `rows` weight rows of row_bytes, and for MXFP4 their scale bytes
// (srow = inputs / 32 of a row; base 4-byte aligned).
struct StreamWeights {
  const uint8_t* w;
  const uint8_t* scale;
  int64_t rows;
  uint32_t row_bytes;
  uint32_t srow;
};

// step(0), step(1), ... below `count`, at most RT of them, with the index a constant (so
// that registers can be indexed by it).
template <int RT, int T = 0, class F>
__device__ __forceinline__ void for_tiles(int count, F step) {
  if constexpr (T < RT) {
    if (T < count) {
      step(At<T>{});
      for_tiles<RT, T + 1>(count, step);
    }
  }
}

// MX: MXFP4 weights, else int8.  XQ: activations in MXFP4 (MX only), else bf16.  ODD:
// rows of scales are no multiple of 4 bytes.
template <bool MX, bool XQ, bool ODD, int COLS, int P>
struct RowStream {
  static_assert(MX || !XQ, "4-bit activations meet 4-bit weights only");
  static constexpr int kSpan = MX ? 512 : 256;
  static constexpr int kXRow = XQ ? 256 : 2 * kSpan;                 // bytes of a span of an activation row
  static constexpr int kXBytes = (COLS * kXRow + 1023) / 1024 * 1024;
  static constexpr int kWords = !MX ? 0 : ODD ? 2 : 1;               // scale words of a lane
  static constexpr int kXWords = XQ ? kWords : 0;
  static constexpr int kXOps = kXBytes / 1024 + kXWords;
  static constexpr int kOps = 4 + kWords;
  static constexpr int kSlot = 4096 + 256 * kWords;
  static constexpr int kBytes = kXBytes + 256 * kXWords + P * kSlot; // LDS of a wave
  static constexpr int kFrags = XQ ? 4 : kSpan / 32;                 // 16-byte pieces of activations per lane

  char* lds;
  int lane, g, c;

  __device__ __forceinline__ RowStream(char* at) : lds(at), lane(lane_id()) {
    g = lane >> 4;
    c = lane & 15;
  }

  // Offset of lane (row, quarter)'s scale word in rows that follow `row0`, from that
  // row's own word.
  __device__ __forceinline__ uint32_t scale_shift(const StreamWeights& a, int64_t row0, int left) const {
    return (uint32_t)((row0 + min(c, left - 1)) * a.srow) & 3u;
  }

  __device__ __forceinline__ void request_scales(const uint8_t* scale, uint32_t srow, int64_t rows, int64_t row0, int left,
                                                 int span, uint32_t to) const {
    const int64_t first = row0 * srow;
    const uint32_t low = (uint32_t)first & 3u;
    const uint8_t* base = scale + (first - low);
    // pieces past the row's end stand for nothing: any byte of the row will do
    const uint32_t at = low + (uint32_t)min(c, left - 1) * srow + min((uint32_t)span * 16u + 4u * g, srow - 1);
    request4_late(base, at & ~3u, to);
    if constexpr (ODD) {
      // the word after it, or the last that holds a scale
      const int64_t most = ((rows * srow - 1) & ~(int64_t)3) - (first - low);
      const uint32_t last = (uint32_t)(most < 0x7FFFFFFF ? most : 0x7FFFFFFF);
      request4_late(base, min((at & ~3u) + 4u, last), to + 256);
    }
  }

  // Requests span `span` of rows row0 .. row0 + 15 (the first `left` of them are there).
  __device__ __forceinline__ void request_unit(const StreamWeights& a, int64_t row0, int left, int span, int slot) const {
    const uint8_t* base = a.w + row0 * a.row_bytes + (uint32_t)span * 256u;
    const uint32_t to = lds_offset(lds + kXBytes + 256 * kXWords + slot * kSlot);
    const uint32_t last = a.row_bytes - 16u - (uint32_t)span * 256u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (i & 1) * 8 + (lane >> 3);
      const uint32_t piece = (i >> 1) * 8 + ((lane & 7) ^ ((r >> 1) & 7));
      const uint32_t off = __umul24(min(r, left - 1), a.row_bytes) + min(piece * 16u, last);
      request16_late(base, off, to + i * 1024);
    }
    if constexpr (MX) request_scales(a.scale, a.srow, a.rows, row0, left, span, to + 4096);
  }

  // Requests a span of the activation rows: row(column) is where each starts, x_bytes
  // its length.
  template <class Row>
  __device__ __forceinline__ void request_x(Row row, uint32_t x_bytes, int span) const {
    const uint32_t to = lds_offset(lds);
    constexpr int per = kXRow / 16;
#pragma unroll
    for (int i = 0; i < kXBytes / 1024; ++i) {
      const int p = i * 64 + lane, col = p / per;
      const uint32_t piece = (uint32_t)((p % per) ^ (col & 15));
      request16(row(min(col, COLS - 1)) + min((uint32_t)span * kXRow + piece * 16u, x_bytes - 16u), to + i * 1024);
    }
  }

  // The activations of a span in registers, zeros past the end (`pieces` in all).
  __device__ __forceinline__ void read_x(u32x4 (&x)[kFrags], int span, int pieces) const {
    constexpr int per = kFrags / 4;                                   // of one weight piece
    const int col = min(c, COLS - 1);
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      const int piece = (4 * g + f / per) * per + f % per;
      x[f] = *reinterpret_cast<const u32x4*>(lds + col * kXRow + ((piece ^ col) << 4));
    }
    if ((span + 1) * 16 > pieces) {
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
        if (span * 16 + 4 * g + f / per >= pieces) x[f] = u32x4{0, 0, 0, 0};
    }
  }

  // A lane's four scales from its words; those past the row's end as 0 (2^-127).
  __device__ __forceinline__ uint32_t scales(const char* at, uint32_t shift, int span, int pieces) const {
    uint32_t s = *reinterpret_cast<const uint32_t*>(at + 4 * lane);
    if constexpr (ODD) s = __builtin_amdgcn_alignbyte(*reinterpret_cast<const uint32_t*>(at + 256 + 4 * lane), s, shift);
    if ((span + 1) * 16 > pieces) {
      const int have = pieces - (span * 16 + 4 * g);
      s &= have >= 4 ? ~0u : have <= 0 ? 0u : (1u << (8 * have)) - 1u;
    }
    return s;
  }

  struct Unit {
    u32x4 w[4];
    uint32_t s;
  };
  __device__ __forceinline__ Unit read_unit(const StreamWeights& a, int64_t row0, int left, int span, int pieces,
                                            int slot) const {
    const char* at = lds + kXBytes + 256 * kXWords + slot * kSlot;
    Unit u;
    const char* row = at + ((g >> 1) * 2 + (c >> 3)) * 1024 + (c & 7) * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j) u.w[j] = *reinterpret_cast<const u32x4*>(row + (((4 * (g & 1) + j) ^ ((c >> 1) & 7)) << 4));
    u.s = 0;
    if constexpr (MX) u.s = scales(at + 4096, ODD ? scale_shift(a, row0, left) : 0u, span, pieces);
    return u;
  }

  // Eight int8 weights as bf16 (exact).
  __device__ static __forceinline__ bf16x8 i8_bf16(uint32_t lo, uint32_t hi) {
    bf16x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = (__bf16)(float)(int8_t)(lo >> (8 * i));
      r[4 + i] = (__bf16)(float)(int8_t)(hi >> (8 * i));
    }
    return r;
  }

  template <int J>
  __device__ __forceinline__ static f32x4 multiply4(const Unit& u, const u32x4 (&x)[kFrags], uint32_t xs, f32x4 acc) {
    // both operands as they are: 16 bytes of codes, scale byte J of either word
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(u.w[J]), mx_operand(x[J]), acc, 4, 4, J, (int)u.s, J, (int)xs);
  }

  __device__ __forceinline__ static f32x4 multiply(const Unit& u, const u32x4 (&x)[kFrags], uint32_t xs, f32x4 acc) {
    if constexpr (XQ) {
      acc = multiply4<0>(u, x, xs, acc);
      acc = multiply4<1>(u, x, xs, acc);
      acc = multiply4<2>(u, x, xs, acc);
      acc = multiply4<3>(u, x, xs, acc);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (MX) {
          const float s = mx_scale(u.s, j);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_bf16(u.w[j][i], s), __builtin_bit_cast(bf16x8, x[4 * j + i]), acc, 0, 0, 0);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(i8_bf16(u.w[j][2 * i], u.w[j][2 * i + 1]),
                                                          __builtin_bit_cast(bf16x8, x[2 * j + i]), acc, 0, 0, 0);
        }
      }
    }
    return acc;
  }

  template <int K>
  __device__ __forceinline__ static void wait_later(int k) {
    if constexpr (K == 0)
      wait_requests<0>();
    else if (k >= K)
      wait_requests<K * kOps>();
    else
      wait_later<K - 1>(k);
  }

  // Adds to acc[t] the products of tile(t)'s rows with the activations over spans
  // first, first + step, ... below `spans`, for t < tiles.  tile(t, row0, left) tells a
  // tile's rows; the loop waits for a unit by the number of requests made after it.
  template <int RT, class Tile, class Row>
  __device__ __forceinline__ void run(const StreamWeights& a, int tiles, int first, int step, int spans, int pieces, Tile tile,
                                      Row row, uint32_t x_bytes, const uint8_t* xscale, int xrows,
                                      f32x4 (&acc)[RT], int turn = 0) const {
    const int mine = first < spans ? (spans - first + step - 1) / step : 0;
    const int total = mine * tiles;
    if (total == 0) return;
    int made = 0, at_span = 0, at_tile = 0;
    // Long chains start at different spans, so that the chip's workgroups do not walk all
    // rows in step: 128256 x 8192 (rows of 4 KB, four spans at a time) 112 -> 107.5 us.
    turn = mine >= 4 ? turn % mine : 0;
    auto span_at = [&](int i) {
      i += turn;
      return first + (i < mine ? i : i - mine) * step;
    };
    auto request = [&] {
      if (made < total) {
        int64_t row0;
        int left;
        tile(at_tile, row0, left);
        request_unit(a, row0, left, span_at(at_span), made % P);
        ++made;
        if (++at_tile == tiles) {
          at_tile = 0;
          ++at_span;
        }
      }
    };
    auto request_span = [&](int span) {
      request_x(row, x_bytes, span);
      if constexpr (XQ) request_scales(xscale, a.srow, xrows, 0, xrows, span, lds_offset(lds + kXBytes));
    };
    request_span(span_at(0));
#pragma unroll
    for (int p = 0; p < P; ++p) request();
    int u = 0, before = 0;                       // units requested before the span's activations
    for (int si = 0; si < mine; ++si) {
      const int span = span_at(si);
      u32x4 x[kFrags];
      uint32_t xs = 0;
      for_tiles<RT>(tiles, [&](auto at) __attribute__((always_inline)) {
        constexpr int t = decltype(at)::value;
        int64_t row0;
        int left;
        tile(t, row0, left);
        if constexpr (t == 0) {
          wait_later<P - 1>(min(made - u - 1, made - before));
          read_x(x, span, pieces);
          if constexpr (XQ) xs = scales(lds + kXBytes, ODD ? (uint32_t)min(c, xrows - 1) * a.srow & 3u : 0u, span, pieces);
        } else if (t < P && si + 1 < mine && made - u == P) {
          wait_requests<(P - 1) * kOps + kXOps>();    // the next span's activations come after this unit
        } else {
          wait_later<P - 1>(made - u - 1);
        }
        const Unit unit = read_unit(a, row0, left, span, pieces, u % P);
        wait_lds();
        if (t == 0 && si + 1 < mine) {
          before = made;
          request_span(span_at(si + 1));
        }
        request();
        acc[t] = multiply(unit, x, xs, acc[t]);
        ++u;
      });
    }
  }
};

}  // namespace wq
