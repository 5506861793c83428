// A whole mixture-of-experts layer for a few tokens: router, selected experts (SwiGLU)
// and their weighted sum.  Bound by the bytes of the experts in use: W1 and W3 are read once
// for up to 4, 8 or 16 tokens of an expert (by the number of tokens), W2 for up to 2, 3 or 5,
// and again for as many more.
//
//   scores   x router^T in fp64, every expert's sum in the same order, so that equal
//            router rows score the same; where the caller gives logits, none
//   route    the `top` largest scores of each token and their gates
//   up       a workgroup takes a block of rows of W1 and W3 of one expert over the
//            tokens that chose it: h1, h3 meet in LDS, silu(h1) h3 goes to the workspace
//   down     the same for rows of W2; results go to the workspace, weighted by the gate
//   join     a token's experts are added in the order of its selection
//
// A token's experts are distinct and there are at most 64 tokens, so the tokens of an
// expert are a 64-bit mask, which every workgroup builds itself from the selections.
// The second product takes silu(h1) h3 in three bf16 parts (24 bits, an fp32 value's), as
// further columns of the matrix instruction.
//
// Measured (dim 4096, f 14336): one token of two int8 experts (352 MB) 73 us, 4.8 TB/s;
// 6 tokens of 8 experts in MXFP4 (616 MB) 134 us, 64 tokens (749 MB) 300.  61 tokens of 128
// experts (dim 2048, f 768, 316 MB) 99 us, five dependent launches and many starts of short
// streams.
#include <stdint.h>

#include <math.h>

#include <algorithm>

#include "wq_host.hpp"
#include "wq_kv.hpp"
#include "wq_row_stream.hpp"

namespace wq {

constexpr int kMoeTokens = 64, kMoeExperts = 256, kMoeTop = 16;
constexpr int kParts = 3;                        // of silu(h1) h3

struct MoeArgs {
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* router;
  const float* logits;
  double* scores;          // [tokens][e], or null where logits are given
  int32_t* sel;            // [tokens][top]
  float* gates;
  int32_t* user_sel;       // the caller's copies, or null
  float* user_gates;
  uint16_t* act;           // [tokens * top][kParts][f], in the order of experts
  float* sums;             // [tokens * top][dim], in the order of selection, weighted
  StreamWeights w13, w2;
  const uint16_t* s13;     // int8: row scales
  const uint16_t* s2;
  float* y32;
  uint16_t* y16;
  int64_t y_stride;
  int32_t tokens, dim, f, e, top, renormalize;
  int32_t here;            // the selection is made by the up launch itself
  int32_t spans, spans2;   // of a row of W1, of W2
  // of a launch: pairs of row tiles (up) or tiles (down) of a workgroup, workgroups of an
  // expert's rows, waves that share a tile's spans
  int32_t pairs, per, blocks, ways;
};

// ---------------------------------------------------------------------------
// Scores and selection

constexpr int kScoreWaves = 16, kScoreBatch = 4;
constexpr int kScoreParts = 16;                  // at most, of k

// Wave-wide sums of four values; lane 16 i ends with that of v[i] (halves of the wave
// keep two each, quarters one, so seven exchanges do for four sums).
__device__ __forceinline__ double wave_sum4(const double (&v)[4]) {
  const int lane = lane_id();
  const bool high = lane & 32, odd = lane & 16;
  const double a = (high ? v[2] : v[0]) + __shfl_xor(high ? v[0] : v[2], 32);
  const double b = (high ? v[3] : v[1]) + __shfl_xor(high ? v[1] : v[3], 32);
  double s = (odd ? b : a) + __shfl_xor(odd ? a : b, 16);
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) s += __shfl_xor(s, d);
  return s;
}

// Sums of experts first .. last - 1 of token t over `parts` shares of k: the waves of a
// workgroup take (four experts, share) units, part[share][expert - first].
__device__ __forceinline__ void score_experts(const MoeArgs& a, int t, int first, int last, int parts,
                                              double (&part)[kScoreParts][kMoeExperts]) {
  const int lane = lane_id(), units = (last - first + kScoreBatch - 1) / kScoreBatch * parts;
  const int share = (a.dim / 8 + parts * 64 - 1) / (parts * 64) * 512;
  const uint16_t* x = a.x + t * a.x_stride;
  for (int u = wave_id(); u < units; u += kScoreWaves) {
    const int e = first + u / parts * kScoreBatch, p = u % parts, end = min((p + 1) * share, a.dim);
    double sum[kScoreBatch] = {0., 0., 0., 0.};
    for (int i = p * share + lane * 8; i < end; i += 512) {
      const u32x4 xv = load16(x + i);
      u32x4 wv[kScoreBatch];
#pragma unroll
      for (int b = 0; b < kScoreBatch; ++b) wv[b] = load16(a.router + (int64_t)min(e + b, last - 1) * a.dim + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double lo = bf16lo_to_f32(xv[j]), hi = bf16hi_to_f32(xv[j]);
#pragma unroll
        for (int b = 0; b < kScoreBatch; ++b) {
          sum[b] = fma(lo, (double)bf16lo_to_f32(wv[b][j]), sum[b]);
          sum[b] = fma(hi, (double)bf16hi_to_f32(wv[b][j]), sum[b]);
        }
      }
    }
    const double v = wave_sum4(sum);
    if ((lane & 15) == 0 && e + (lane >> 4) < last) part[p][e + (lane >> 4) - first] = v;
  }
}

template <int CTRL, int MASK = 0xF>
__device__ __forceinline__ int32_t dpp_max(int32_t v) {
  const int32_t o = __builtin_amdgcn_update_dpp((int)0x80000000, v, CTRL, MASK, 0xF, false);
  return v > o ? v : o;
}
__device__ __forceinline__ int32_t wave_max_i32(int32_t v) {
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  v = dpp_max<0x141>(v);
  v = dpp_max<0x140>(v);
  v = dpp_max<0x142, 0xA>(v);
  v = dpp_max<0x143, 0xC>(v);
  return __builtin_amdgcn_readlane(v, 63);
}

// The selection of one token by one wave: score(e) of e < a.e, the largest `top` in
// order, equal ones by index, NaN after all others.  out(j, expert, gate) is called in
// one lane.
template <class Score, class Out>
__device__ __forceinline__ void select_experts(const MoeArgs& a, Score score, Out out) {
  const int lane = lane_id();
  constexpr int N = kMoeExperts / kWave;
  int64_t key[N];
  double s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 64 * i;
    s[i] = e < a.e ? score(e) + 0.0 : 0.0;      // -0 counts as 0
    const int64_t b = __double_as_longlong(s[i]);
    key[i] = b ^ ((b >> 63) & 0x7FFFFFFFFFFFFFFFll);   // ordered as the values are
    if (s[i] != s[i]) key[i] = INT64_MIN + 1;
    if (e >= a.e) key[i] = INT64_MIN;
  }
  int mine = -1;                                // lane j: the j-th expert and its score
  double value = 0.;
  for (int j = 0; j < a.top; ++j) {
    int64_t k = key[0];
#pragma unroll
    for (int i = 1; i < N; ++i) k = k > key[i] ? k : key[i];
    const int32_t hi = wave_max_i32((int32_t)(k >> 32));
    // the low half as it compares unsigned, among the lanes with this high half
    const int32_t lo = wave_max_i32((int32_t)(k >> 32) == hi ? (int32_t)((uint32_t)k ^ 0x80000000u) : INT32_MIN);
    const int64_t best = (int64_t)(((uint64_t)(uint32_t)hi << 32) | ((uint32_t)lo ^ 0x80000000u));
    int found = 0;
    bool done = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint64_t at = __ballot(key[i] == best);
      if (!done && at) {
        done = true;
        const int l = __ffsll((unsigned long long)at) - 1;
        found = l + 64 * i;
        const double v = __shfl(s[i], l);
        if (lane == j) {
          mine = found;
          value = v;
        }
        if (lane == l) key[i] = INT64_MIN;
      }
    }
  }
  const double top = __shfl(value, 0);
  float w = lane < a.top ? expf((float)(value - top)) : 0.f;
  float total;
  if (a.renormalize) {
    total = wave_sum(w);
  } else {
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane + 64 * i < a.e) all += expf((float)(s[i] - top));
    total = wave_sum(all);
  }
  if (lane < a.top) out(lane, mine, w / total);
}

__device__ __forceinline__ void put_selection(const MoeArgs& a, int t, int j, int e, float gate) {
  const int at = t * a.top + j;
  a.sel[at] = e;
  a.gates[at] = gate;
  if (a.user_sel) a.user_sel[at] = e;
  if (a.user_gates) a.user_gates[at] = gate;
}

// Scores of a token's experts by one workgroup, which selects at once; or of a share of
// them (gridDim.y > 1), for moe_route_kernel.
__global__ __launch_bounds__(kScoreWaves * 64) void moe_score_kernel(MoeArgs a) {
  __shared__ double part[kScoreParts][kMoeExperts];
  const int t = (int)blockIdx.x, share = (a.e + (int)gridDim.y - 1) / (int)gridDim.y;
  const int first = (int)blockIdx.y * share, last = min(first + share, a.e);
  // enough units for the waves, each at least 512 inputs; of a whole share in the last one
  // too, or its experts' sums would be split in another way
  const int batches = (share + kScoreBatch - 1) / kScoreBatch;
  const int parts = max(1, min(min(kScoreParts, (kScoreWaves + batches - 1) / batches), (a.dim + 511) / 512));
  score_experts(a, t, first, last, parts, part);
  __syncthreads();
  auto score = [&](int e) {
    double v = part[0][e - first];
    for (int p = 1; p < parts; ++p) v += part[p][e - first];
    return v;
  };
  if (gridDim.y > 1) {
    for (int e = first + (int)threadIdx.x; e < last; e += kScoreWaves * 64) a.scores[t * a.e + e] = score(e);
  } else if (wave_id() == 0) {
    select_experts(a, score, [&](int j, int e, float g) { put_selection(a, t, j, e, g); });
  }
}

__global__ __launch_bounds__(64) void moe_route_kernel(MoeArgs a) {
  const int t = (int)blockIdx.x;
  select_experts(
      a, [&](int e) { return a.logits ? (double)a.logits[t * a.e + e] : a.scores[t * a.e + e]; },
      [&](int j, int e, float g) { put_selection(a, t, j, e, g); });
}

// ---------------------------------------------------------------------------
// The experts' tokens

struct MoeTokens {
  uint64_t mask[kMoeExperts];
  int32_t sel[kMoeTokens * kMoeTop];
  float gate[kMoeTokens * kMoeTop];
};

// Fills `all` from the selections (a barrier at the end).
template <int WAVES>
__device__ __forceinline__ void find_tokens(const MoeArgs& a, MoeTokens& all) {
  const int tid = (int)threadIdx.x, n = a.tokens * a.top;
  for (int e = tid; e < kMoeExperts; e += WAVES * 64) all.mask[e] = 0;
  if (!a.here) {
    for (int i = tid; i < n; i += WAVES * 64) {
      all.sel[i] = a.sel[i];
      all.gate[i] = a.gates[i];
    }
  } else {
    for (int t = wave_id(); t < a.tokens; t += WAVES)
      select_experts(
          a, [&](int e) { return a.logits ? (double)a.logits[t * a.e + e] : a.scores[t * a.e + e]; },
          [&](int j, int e, float g) {
            all.sel[t * a.top + j] = e;
            if (blockIdx.x == 0) put_selection(a, t, j, e, g);
          });
  }
  __syncthreads();
  for (int i = tid; i < n; i += WAVES * 64) atomicOr((unsigned long long*)&all.mask[all.sel[i]], 1ull << (i / a.top));
  __syncthreads();
}

// Item `item` of the experts in use, `chunk` tokens an item: its expert, the first of
// its tokens among the expert's, and the expert's first row of `act`; false past the
// last item.
__device__ __forceinline__ bool find_item(const MoeTokens& all, int item, int chunk, int& expert, int& begin, int& slot) {
  const int lane = lane_id();
  constexpr int N = kMoeExperts / kWave;
  int items = 0, rows = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = __popcll(all.mask[lane * N + i]);
    items += (c + chunk - 1) / chunk;
    rows += c;
  }
  const int before = wave_scan(items) - items, row0 = wave_scan(rows) - rows;
  const uint64_t at = __ballot(item >= before && item < before + items);
  if (!at) return false;
  const int l = __ffsll((unsigned long long)at) - 1;
  int left = item - __shfl(before, l), row = __shfl(row0, l);
  expert = l * N;
  for (int i = 0; i < N; ++i) {
    const int c = __popcll(all.mask[l * N + i]), n = (c + chunk - 1) / chunk;
    expert = l * N + i;
    if (left < n) break;
    left -= n;
    row += c;
  }
  expert = __builtin_amdgcn_readfirstlane(expert);
  begin = __builtin_amdgcn_readfirstlane(left * chunk);
  slot = __builtin_amdgcn_readfirstlane(row);
  return true;
}

// bf16 parts of v, whose sum is v (but for what lies below 2^-133).  Truncated, so that
// none overflows; infinities and NaN are the first part alone.
__device__ __forceinline__ void bf16_parts(float v, uint16_t (&p)[kParts]) {
  p[1] = p[2] = 0;
  if (!(fabsf(v) < INFINITY)) {
    p[0] = f32_to_bf16(v);
    return;
  }
  const uint32_t b = __float_as_uint(v);
  p[0] = (uint16_t)(b >> 16);
  const float rest = v - __uint_as_float(b & 0xFFFF0000u);
  const uint32_t m = __float_as_uint(rest);
  p[1] = (uint16_t)(m >> 16);
  p[2] = f32_to_bf16(rest - __uint_as_float(m & 0xFFFF0000u));
}

// ---------------------------------------------------------------------------
// First products and the gate

constexpr int kUpTiles = 16;

// TWO: two workgroups share a CU, and with it its registers.
template <bool MX, bool ODD, int COLS, int WAVES, int P, bool TWO>
__global__ __launch_bounds__(WAVES * 64, TWO ? 2 : 1) void moe_up_kernel(MoeArgs a) {
  using S = RowStream<MX, false, ODD, COLS, P>;
  constexpr int kRed = WAVES * kUpTiles * 1024, kAll = WAVES * S::kBytes;
  __shared__ __align__(1024) char lds[kAll > kRed ? kAll : kRed];
  __shared__ int list[COLS];
  MoeTokens& all = *reinterpret_cast<MoeTokens*>(lds);
  static_assert(sizeof(MoeTokens) <= sizeof(lds));
  find_tokens<WAVES>(a, all);
  int expert, begin, slot;
  if (!find_item(all, (int)blockIdx.x / a.blocks, COLS, expert, begin, slot)) return;
  const uint64_t mask = all.mask[expert];
  const int cols = min(COLS, __popcll(mask) - begin);
  if (wave_id() == 0) {
    const int lane = lane_id(), rank = __popcll(mask & ((1ull << lane) - 1)) - begin;
    if ((mask >> lane & 1) && rank >= 0 && rank < COLS) list[rank] = lane;
  }
  __syncthreads();
  const int wave = wave_id(), ways = a.ways, kw = wave % ways, tw = wave / ways, teams = WAVES / ways;
  const S s(lds + wave * S::kBytes);
  const int first = (int)blockIdx.x % a.blocks * a.per, mine = min(a.per, a.pairs - first);
  const int pairs = (mine - tw + teams - 1) / teams;
  f32x4 acc[kUpTiles];
#pragma unroll
  for (int t = 0; t < kUpTiles; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t rows0 = (int64_t)expert * 2 * a.f;
  // a tile of W1, then the same rows of W3
  s.template run<kUpTiles>(
      a.w13, 2 * pairs, kw, ways, a.spans, (int)(a.w13.row_bytes / 16),
      [&](int t, int64_t& row0, int& left) {
        row0 = rows0 + (t & 1) * a.f + (int64_t)(first + tw + (t >> 1) * teams) * 16;
        left = 16;
      },
      [&](int col) { return reinterpret_cast<const char*>(a.x + list[min(col, cols - 1)] * a.x_stride); }, 2u * a.dim, nullptr, 0,
      acc);
  __syncthreads();
  for_tiles<kUpTiles>(2 * pairs, [&](auto at) __attribute__((always_inline)) {
    *reinterpret_cast<f32x4*>(lds + (wave * kUpTiles + at.value) * 1024 + s.lane * 16) = acc[at.value];
  });
  __syncthreads();
  for (int o = (int)threadIdx.x; o < mine * 16 * cols; o += WAVES * 64) {
    const int row = o & 15, col = (o >> 4) % cols, pair = (o >> 4) / cols;
    const char* from = lds + ((pair % teams) * ways * kUpTiles + 2 * (pair / teams)) * 1024 + ((row >> 2) * 16 + col) * 16 + (row & 3) * 4;
    float h1 = 0.f, h3 = 0.f;
    for (int w = 0; w < ways; ++w) {
      h1 += *reinterpret_cast<const float*>(from + w * kUpTiles * 1024);
      h3 += *reinterpret_cast<const float*>(from + w * kUpTiles * 1024 + 1024);
    }
    const int r = (first + pair) * 16 + row;
    if constexpr (!MX) {
      h1 *= __uint_as_float((uint32_t)gmem(a.s13)[rows0 + r] << 16);
      h3 *= __uint_as_float((uint32_t)gmem(a.s13)[rows0 + a.f + r] << 16);
    }
    const float v = h1 / (1.f + expf(-h1)) * h3;
    uint16_t p[kParts];
    bf16_parts(v, p);
    uint16_t* to = a.act + (int64_t)(slot + begin + col) * kParts * a.f + r;
#pragma unroll
    for (int q = 0; q < kParts; ++q) gmem(to)[q * a.f] = p[q];
  }
}

// ---------------------------------------------------------------------------
// Second products, and the sum over a token's experts

template <bool MX, bool ODD, int COLS, int WAVES, int P, bool TWO>
__global__ __launch_bounds__(WAVES * 64, TWO ? 2 : 1) void moe_down_kernel(MoeArgs a) {
  using S = RowStream<MX, false, ODD, COLS, P>;
  constexpr int kRed = WAVES * kUpTiles * 1024, kAll = WAVES * S::kBytes;
  __shared__ __align__(1024) char lds[kAll > kRed ? kAll : kRed];
  MoeTokens& all = *reinterpret_cast<MoeTokens*>(lds);
  static_assert(sizeof(MoeTokens) <= sizeof(lds));
  __shared__ float gate[COLS];
  __shared__ int pick[COLS];
  find_tokens<WAVES>(a, all);
  constexpr int chunk = COLS / kParts;              // tokens; a column for each of their parts
  int expert, begin, slot;
  if (!find_item(all, (int)blockIdx.x / a.blocks, chunk, expert, begin, slot)) return;
  const uint64_t mask = all.mask[expert];
  const int have = min(chunk, __popcll(mask) - begin);
  if (wave_id() == 0) {
    const int lane = lane_id(), rank = __popcll(mask & ((1ull << lane) - 1)) - begin;
    if ((mask >> lane & 1) && rank >= 0 && rank < chunk)
      for (int j = 0; j < a.top; ++j)
        if (all.sel[lane * a.top + j] == expert) {
          gate[rank] = all.gate[lane * a.top + j];
          pick[rank] = lane * a.top + j;
        }
  }
  __syncthreads();
  const int wave = wave_id(), ways = a.ways, kw = wave % ways, tw = wave / ways, teams = WAVES / ways;
  const S s(lds + wave * S::kBytes);
  const int first = (int)blockIdx.x % a.blocks * a.per, mine = min(a.per, a.dim / 16 - first);
  const int tiles = (mine - tw + teams - 1) / teams;
  f32x4 acc[kUpTiles];
#pragma unroll
  for (int t = 0; t < kUpTiles; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t rows0 = (int64_t)expert * a.dim;
  const uint16_t* act = a.act + (int64_t)(slot + begin) * kParts * a.f;
  s.template run<kUpTiles>(
      a.w2, tiles, kw, ways, a.spans2, (int)(a.w2.row_bytes / 16),
      [&](int t, int64_t& row0, int& left) {
        row0 = rows0 + (int64_t)(first + tw + t * teams) * 16;
        left = 16;
      },
      // columns: part after part, `chunk` tokens each
      [&](int col) {
        const int part = min(col / chunk, kParts - 1), tok = min(col % chunk, have - 1);
        return reinterpret_cast<const char*>(act + (int64_t)(tok * kParts + part) * a.f);
      },
      2u * a.f, nullptr, 0, acc);
  __syncthreads();
  for_tiles<kUpTiles>(tiles, [&](auto at) __attribute__((always_inline)) {
    *reinterpret_cast<f32x4*>(lds + (wave * kUpTiles + at.value) * 1024 + s.lane * 16) = acc[at.value];
  });
  __syncthreads();
  for (int o = (int)threadIdx.x; o < mine * 16 * have; o += WAVES * 64) {
    const int row = o & 15, tok = (o >> 4) % have, tile = (o >> 4) / have;
    const char* from = lds + ((tile % teams) * ways * kUpTiles + tile / teams) * 1024 + ((row >> 2) * 16 + tok) * 16 + (row & 3) * 4;
    float v = 0.f;
#pragma unroll
    for (int q = kParts - 1; q >= 0; --q)
      for (int w = 0; w < ways; ++w) v += *reinterpret_cast<const float*>(from + w * kUpTiles * 1024 + q * chunk * 16);
    const int r = (first + tile) * 16 + row;
    if constexpr (!MX) v *= __uint_as_float((uint32_t)gmem(a.s2)[rows0 + r] << 16);
    gmem(a.sums)[(int64_t)pick[tok] * a.dim + r] = gate[tok] * v;
  }
}

// A token's experts summed in the order of selection.
__global__ __launch_bounds__(256) void moe_join_kernel(MoeArgs a) {
  const int o = (int)(blockIdx.x * 256 + threadIdx.x), quads = a.dim / 4;
  if (o >= a.tokens * quads) return;
  const int t = o / quads, col = o % quads * 4;
  const float* from = a.sums + (int64_t)t * a.top * a.dim + col;
  f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < a.top; j += 4) {
    f32x4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *gmem(reinterpret_cast<const f32x4*>(from + (int64_t)min(j + i, a.top - 1) * a.dim));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j + i < a.top) v += p[i];
  }
  const int64_t at = t * a.y_stride + col;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (a.y32) gmem(a.y32)[at + i] = v[i];
    if (a.y16) gmem(a.y16)[at + i] = f32_to_bf16(v[i]);
  }
}

// One token, or two: a workgroup takes 16 rows of W2 of every expert in use, so that the
// sum over experts stays inside it and nothing is joined; its waves take (expert, span)
// pairs in turn, each with the activations that meet it.  (One token of Mixtral's int8
// layer: 25.4 us, where moe_down_kernel and the join took 26.9 and 4.7.)

// The experts in use, in order.
struct MoeDown {
  int32_t expert[kMoeExperts];
  int32_t slot[kMoeExperts];
  int32_t used;
};

// TOKENS: of the call, so that an expert has no more.
template <bool MX, bool ODD, int TOKENS, int WAVES, int P>
__global__ __launch_bounds__(WAVES * 64) void moe_few_kernel(MoeArgs a) {
  using S = RowStream<MX, false, ODD, TOKENS * kParts, P>;
  // a unit is a span of W2's rows and of the activations that meet it; both have P slots
  constexpr int kWave0 = S::kXBytes * (P - 1) + S::kBytes;
  __shared__ __align__(1024) char lds[WAVES * kWave0];
  __shared__ __align__(16) float sums[WAVES][TOKENS * 16];
  __shared__ MoeTokens all;
  __shared__ MoeDown down;
  find_tokens<WAVES>(a, all);
  const int wave = wave_id(), lane = lane_id();
  if (wave == 0) {
    constexpr int N = kMoeExperts / kWave;
    int used = 0, rows = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = __popcll(all.mask[lane * N + i]);
      used += c > 0;
      rows += c;
    }
    int at = wave_scan(used) - used, row = wave_scan(rows) - rows;
    for (int i = 0; i < N; ++i) {
      const int c = __popcll(all.mask[lane * N + i]);
      if (c) {
        down.expert[at] = lane * N + i;
        down.slot[at++] = row;
      }
      row += c;
    }
    if (lane == 63) down.used = at;
  }
  for (int i = lane; i < TOKENS * 16; i += 64) sums[wave][i] = 0.f;
  __syncthreads();
  const int64_t tile = (int64_t)blockIdx.x * 16;
  char* const base = lds + wave * kWave0;
  const int g = lane >> 4, c = lane & 15;

  // this wave's units: (expert in use, span) pairs wave, wave + WAVES, ...; slots of
  // weights lie behind those of activations
  const int pairs = down.used * a.spans2;
  auto request = [&](int pair, int slot) {
    const int u = pair / a.spans2, span = pair % a.spans2;
    const int expert = __builtin_amdgcn_readfirstlane(down.expert[u]), row = __builtin_amdgcn_readfirstlane(down.slot[u]);
    const int have = TOKENS == 1 ? 1 : __builtin_amdgcn_readfirstlane(__popcll(all.mask[expert]));
    const uint16_t* act = a.act + (int64_t)row * kParts * a.f;
    // columns: part after part, TOKENS each
    const S x(base + slot * S::kXBytes);
    x.request_x(
        [&](int col) {
          const int part = min(col / TOKENS, kParts - 1), tok = min(col % TOKENS, have - 1);
          return reinterpret_cast<const char*>(act + (int64_t)(tok * kParts + part) * a.f);
        },
        2u * a.f, span);
    const S w(base + (P - 1) * S::kXBytes);
    w.request_unit(a.w2, (int64_t)expert * a.dim + tile, 16, span, slot);
  };
  int made = 0;
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (wave + made * WAVES < pairs) {
      request(wave + made * WAVES, p);
      ++made;
    }
  f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int kOps = S::kOps + S::kXOps;
  const int pieces = (int)(a.w2.row_bytes / 16);
  for (int done = 0, pair = wave; pair < pairs; ++done, pair += WAVES) {
    const int u = pair / a.spans2, span = pair % a.spans2;
    const int expert = __builtin_amdgcn_readfirstlane(down.expert[u]);
    const int slot = done % P;
    if (made - done == P)
      wait_requests<(P - 1) * kOps>();
    else
      wait_requests<0>();
    u32x4 x[S::kFrags];
    S(base + slot * S::kXBytes).read_x(x, span, pieces);
    const auto unit = S(base + (P - 1) * S::kXBytes).read_unit(a.w2, (int64_t)expert * a.dim + tile, 16, span, pieces, slot);
    wait_lds();
    if (wave + made * WAVES < pairs) {
      request(wave + made * WAVES, slot);
      ++made;
    }
    acc = S::multiply(unit, x, 0u, acc);
    if (pair + WAVES >= pairs || (pair + WAVES) / a.spans2 != u) {
      // columns of a token's parts meet, then go to its row of this wave's sums
      f32x4 v = acc;
#pragma unroll
      for (int q = 1; q < kParts; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += __shfl(acc[i], lane + q * TOKENS);
      uint64_t m = all.mask[expert];
      if (c < __popcll(m)) {
        // the c-th token of the mask
        for (int i = 0; i < c; ++i) m &= m - 1;
        const int t = __ffsll((unsigned long long)m) - 1;
        float gate = 0.f;
        for (int j = 0; j < a.top; ++j)
          if (all.sel[t * a.top + j] == expert) gate = all.gate[t * a.top + j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float o = v[i];
          if constexpr (!MX) o *= __uint_as_float((uint32_t)gmem(a.s2)[(int64_t)expert * a.dim + tile + 4 * g + i] << 16);
          sums[wave][t * 16 + 4 * g + i] += gate * o;
        }
      }
      acc = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  __syncthreads();
  for (int o = (int)threadIdx.x; o < a.tokens * 16; o += WAVES * 64) {
    float v = 0.f;
    for (int w = 0; w < WAVES; ++w) v += sums[w][o];
    const int64_t at = (o >> 4) * a.y_stride + tile + (o & 15);
    if (a.y32) gmem(a.y32)[at] = v;
    if (a.y16) gmem(a.y16)[at] = f32_to_bf16(v);
  }
}

// ---------------------------------------------------------------------------
// Host side

constexpr int64_t kScoreMost = 1 << 16;
constexpr int64_t kMoeMade = 0x77715f6d6f656631;

static bool moe_sizes_ok(int64_t tokens, int64_t dim, int64_t f, int64_t e, int32_t top) {
  return tokens >= 0 && tokens <= kMoeTokens && dim >= 16 && dim <= 32768 && dim % 16 == 0 && f >= 16 && f <= 32768 && f % 16 == 0 &&
         e >= 1 && e <= kMoeExperts && top >= 1 && top <= kMoeTop && top <= e;
}

// Workspace: selections, gates, scores, activations, weighted results.
struct MoeSpace {
  int64_t sel, gates, scores, act, sums, all;
};
static MoeSpace moe_space(int64_t tokens, int64_t dim, int64_t f, int64_t e, int32_t top) {
  auto up = [](int64_t b) { return (b + 255) / 256 * 256; };
  MoeSpace s;
  s.sel = 0;
  s.gates = s.sel + up(4 * tokens * top);
  s.scores = s.gates + up(4 * tokens * top);
  s.act = s.scores + up(8 * tokens * e);
  s.sums = s.act + up(tokens * top * 3 * f * 2);
  s.all = s.sums + up(tokens * top * dim * 4);
  return s;
}

static int moe_check(const char* name, const wq_moe_ffn& a) {
  if (!a.x || !a.w13 || !a.s13 || !a.w2 || !a.s2) return fail(WQ_ERR_NULL, "%s: x, w13, s13, w2 and s2 must be non-null", name);
  if (!a.router == !a.logits) return fail(WQ_ERR_NULL, "%s: exactly one of router and logits must be given", name);
  if (!a.y_f32 && !a.y_bf16) return fail(WQ_ERR_NULL, "%s: at least one of y_f32 / y_bf16 must be non-null", name);
  if (a.format != WQ_FORMAT_INT8 && a.format != WQ_FORMAT_MXFP4)
    return fail(WQ_ERR_SHAPE, "%s: format = %d (need WQ_FORMAT_INT8 or WQ_FORMAT_MXFP4)", name, a.format);
  if (!moe_sizes_ok(a.tokens, a.dim, a.f, a.e, a.top))
    return fail(WQ_ERR_SHAPE,
                "%s: tokens = %lld (0..64), dim = %lld, f = %lld (multiples of 16 up to 32768), e = %lld (1..256), top = %d "
                "(1..16, at most e)",
                name, (long long)a.tokens, (long long)a.dim, (long long)a.f, (long long)a.e, a.top);
  if (a.format == WQ_FORMAT_MXFP4 && (a.dim % kMxGroup || a.f % kMxGroup))
    return fail(WQ_ERR_SHAPE, "%s: dim = %lld, f = %lld must be multiples of 32 for MXFP4", name, (long long)a.dim, (long long)a.f);
  const int64_t most = (int64_t)1 << 40;
  if (a.x_stride < a.dim || a.x_stride > most || a.x_stride % 8)
    return fail(WQ_ERR_SHAPE, "%s: x_stride = %lld must be a multiple of 8 and hold a row", name, (long long)a.x_stride);
  if (a.y_stride < a.dim || a.y_stride > most)
    return fail(WQ_ERR_SHAPE, "%s: y_stride = %lld must hold a row", name, (long long)a.y_stride);
  if (!aligned16(a.x) || !aligned16(a.w13) || !aligned16(a.w2) || !aligned16(a.router))
    return fail(WQ_ERR_ALIGN, "%s: x, w13, w2 and router must be 16-byte aligned", name);
  // int8 scales are read one by one, MXFP4 ones in words
  const uintptr_t part = a.format == WQ_FORMAT_INT8 ? 1 : 3;
  if (((uintptr_t)a.s13 & part) || ((uintptr_t)a.s2 & part) || ((uintptr_t)a.logits & 3) || ((uintptr_t)a.y_f32 & 3) ||
      ((uintptr_t)a.y_bf16 & 1) || ((uintptr_t)a.sel & 3) || ((uintptr_t)a.gates & 3))
    return fail(WQ_ERR_ALIGN, "%s: s13 and s2 must be %d-byte aligned, logits, y, sel and gates to their elements", name, (int)part + 1);
  return WQ_OK;
}

static int moe_overlap(const char* name, const wq_moe_ffn& a) {
  const bool mx = a.format == WQ_FORMAT_MXFP4;
  const int64_t up = a.e * 2 * a.f, down = a.e * a.dim;
  const ByteRows out[] = {{a.y_f32, a.tokens, 4 * a.y_stride, 4 * a.dim},
                          {a.y_bf16, a.tokens, 2 * a.y_stride, 2 * a.dim},
                          {a.sel, 1, 0, 4 * a.tokens * a.top},
                          {a.gates, 1, 0, 4 * a.tokens * a.top}};
  const ByteRows in[] = {{a.x, a.tokens, 2 * a.x_stride, 2 * a.dim},
                         {a.router, 1, 0, 2 * a.e * a.dim},
                         {a.logits, 1, 0, 4 * a.tokens * a.e},
                         {a.w13, 1, 0, mx ? up * a.dim / 2 : up * a.dim},
                         {a.s13, 1, 0, mx ? up * a.dim / kMxGroup : up * 2},
                         {a.w2, 1, 0, mx ? down * a.f / 2 : down * a.f},
                         {a.s2, 1, 0, mx ? down * a.f / kMxGroup : down * 2}};
  for (int i = 0; i < 4; ++i) {
    for (const ByteRows& r : in)
      if (rows_meet(out[i], r)) return fail(WQ_ERR_SHAPE, "%s: y, sel and gates must overlap no input", name);
    for (int j = 0; j < i; ++j)
      if (rows_meet(out[i], out[j])) return fail(WQ_ERR_SHAPE, "%s: y, sel and gates must not overlap each other", name);
  }
  return WQ_OK;
}

// Row tiles of a workgroup (`each` streams at once, of `tiles` such) and waves per tile,
// for `items` experts in use: the fewest units in the longest chain of a CU, which holds
// one workgroup of eight waves or two of four.
static void rows_plan(MoeArgs& a, int waves, int items, int tiles, int each, int spans, int64_t slots) {
  double best = 1e300;
  for (int ways = 1; ways <= waves; ways *= 2) {
    const int teams = waves / ways;
    for (int t = 1; t <= kUpTiles / each; ++t) {
      const int per = t * teams, blocks = (tiles + per - 1) / per;
      const int64_t rounds = ((int64_t)blocks * items + slots - 1) / slots;
      const double cost = (double)rounds * ((double)each * t * ((spans + ways - 1) / ways) + 2.0);
      if (cost < best) {
        best = cost;
        a.per = per;
        a.ways = ways;
        a.blocks = blocks;
      }
    }
  }
}

// Items of `chunk` tokens over all experts, as expected where a token picks any of them
// alike, and a tenth more: an item too many for one round of workgroups costs a second
// (MXFP4 layers of 4 to 60 experts, 6 to 64 tokens: 1 % shorter in the mean than without the
// tenth, 10 % instead of 20 behind the best plan at the worst).
static int expected_items(int tokens, int top, int e, int chunk) {
  if (top == e) return e * ((tokens + chunk - 1) / chunk);
  const double odds = (double)top / (e - top);
  double p = pow(1. - (double)top / e, tokens), items = 0.;   // p: that an expert has c tokens
  for (int c = 1; c <= tokens; ++c) {
    p *= odds * (tokens - c + 1) / c;
    items += p * ((c + chunk - 1) / chunk);
  }
  return (int)ceil(1.1 * e * items);
}

template <bool MX, int COLS, int WAVES, int P, bool TWO = false>
static void up_launch(MoeArgs a, hipStream_t s) {
  const int picks = a.tokens * a.top, used = std::min(a.e, picks);
  a.pairs = a.f / 16;
  rows_plan(a, WAVES, used, a.pairs, 2, a.spans, TWO ? 512 : 256);
  const dim3 grid((unsigned)((used + picks / COLS) * a.blocks));
  if (MX && a.w13.srow % 4)
    hipLaunchKernelGGL((moe_up_kernel<MX, MX, COLS, WAVES, P, TWO>), grid, dim3(WAVES * 64), 0, s, a);
  else
    hipLaunchKernelGGL((moe_up_kernel<MX, false, COLS, WAVES, P, TWO>), grid, dim3(WAVES * 64), 0, s, a);
}

template <bool MX, int COLS, int WAVES, int P, bool TWO = false>
static void down_launch(MoeArgs a, hipStream_t s) {
  constexpr int chunk = COLS / kParts;
  const int picks = a.tokens * a.top, used = std::min(a.e, picks);
  rows_plan(a, WAVES, std::max(used, expected_items(a.tokens, a.top, a.e, chunk)), a.dim / 16, 1, a.spans2, TWO ? 512 : 256);
  const dim3 grid((unsigned)((used + picks / chunk) * a.blocks));
  if (MX && a.w2.srow % 4)
    hipLaunchKernelGGL((moe_down_kernel<MX, MX, COLS, WAVES, P, TWO>), grid, dim3(WAVES * 64), 0, s, a);
  else
    hipLaunchKernelGGL((moe_down_kernel<MX, false, COLS, WAVES, P, TWO>), grid, dim3(WAVES * 64), 0, s, a);
}

template <bool MX, int TOKENS, int WAVES>
static void few_launch(const MoeArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.dim / 16)), block(WAVES * 64);
  if (MX && a.w2.srow % 4)
    hipLaunchKernelGGL((moe_few_kernel<MX, MX, TOKENS, WAVES, 2>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((moe_few_kernel<MX, false, TOKENS, WAVES, 2>), grid, block, 0, s, a);
}

template <bool MX>
static void experts_launch(MoeArgs a, hipStream_t s) {
  const int mean = (a.tokens * a.top + a.e - 1) / a.e;      // tokens of an expert
  // Many experts of a few tokens each: two workgroups of four waves on a CU, whose starts
  // (the search for an expert's tokens, the first loads) and ends lie beside the other's
  // streams.  61 tokens of 128 experts: 104 us, with one workgroup 116; but 16 tokens of
  // Mixtral's eight 182 and 166, its int8 layer for one token 79 and 75, and 10 to 32 tokens
  // of 16 to 60 experts the same in the mean (16 of 16 150 and 139, 16 of 32 115 and 117).
  const bool many = a.tokens > 8 && a.e >= 64 && mean <= 4;
  if (a.tokens <= 4)
    up_launch<MX, 4, 8, 3>(a, s);
  else if (many)
    up_launch<MX, 8, 4, 2, true>(a, s);
  else if (a.tokens <= 8 || 2 * mean <= 8)
    up_launch<MX, 8, 8, 2>(a, s);
  else
    up_launch<MX, 16, 4, 4>(a, s);
  a.here = 0;
  // Nothing to join, where LDS holds a token's three parts beside enough weights: two tokens
  // in seven waves (of Mixtral's experts in MXFP4 69 us, with moe_down_kernel and the join
  // 77; but of 6 of 64 small experts 34 and 32, of Mixtral's in int8 151 and 141).
  if (a.tokens == 1) return few_launch<MX, 1, 8>(a, s);
  if constexpr (MX) {
    if (a.tokens == 2 && a.top <= 4) return few_launch<MX, 2, 7>(a, s);
  }
  // Columns are three for a token.  Two tokens at once leave room for eight waves of three
  // slots (8 tokens of 128 experts 46 us, five at once 49).  (Seven or eight at once, as two
  // products of the same weights, need 21 KB a wave for a span's activations in MXFP4:
  // Mixtral, 24 tokens 218 to 307 us, five at once 206 to 211; in int8, where that is 12, the
  // same within 1 % over 42 layers.)
  if (many)
    down_launch<MX, 9, 4, 2, true>(a, s);
  else if (mean <= 1)
    down_launch<MX, 6, 8, 3>(a, s);
  else
    down_launch<MX, 15, 4, 4>(a, s);
  hipLaunchKernelGGL(moe_join_kernel, dim3((unsigned)((a.tokens * (a.dim / 4) + 255) / 256)), dim3(256), 0, s, a);
}

}  // namespace wq

using namespace wq;

extern "C" int64_t wq_moe_ffn_workspace_bytes(int64_t tokens, int64_t dim, int64_t f, int64_t e, int32_t top) {
  if (!moe_sizes_ok(tokens, dim, f, e, top)) return 0;
  return moe_space(tokens, dim, f, e, top).all + 16;
}

extern "C" int wq_moe_ffn_prepare(const wq_moe_ffn* a, void* workspace, int64_t workspace_bytes, wq_moe_ffn_plan* plan) {
  const char* name = "wq_moe_ffn_prepare";
  if (!a || !plan || !workspace) return fail(WQ_ERR_NULL, "%s: a, workspace and plan must be non-null", name);
  int rc = moe_check(name, *a);
  if (rc) return rc;
  const int64_t need = wq_moe_ffn_workspace_bytes(a->tokens, a->dim, a->f, a->e, a->top);
  if (workspace_bytes < need)
    return fail(WQ_ERR_SHAPE, "%s: workspace_bytes = %lld, %lld are needed", name, (long long)workspace_bytes,
                (long long)need);
  if (!aligned16(workspace)) return fail(WQ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", name);
  if ((rc = moe_overlap(name, *a))) return rc;
  wq_moe_ffn_plan p{};
  if ((rc = plan_device(name, &p.device))) return rc;
  p.made = kMoeMade;
  p.workspace = workspace;
  p.a = *a;
  *plan = p;
  return WQ_OK;
}

extern "C" int wq_moe_ffn_run(const wq_moe_ffn_plan* plan, void* stream) {
  const char* name = "wq_moe_ffn_run";
  if (!plan) return fail(WQ_ERR_NULL, "%s: plan must be non-null", name);
  if (plan->made != kMoeMade) return fail(WQ_ERR_SHAPE, "%s: the plan was not made by wq_moe_ffn_prepare", name);
  int rc = same_device(name, plan->device);
  if (rc) return rc;
  const wq_moe_ffn& m = plan->a;
  if (m.tokens == 0) return WQ_OK;
  const bool mx = m.format == WQ_FORMAT_MXFP4;
  const MoeSpace at = moe_space(m.tokens, m.dim, m.f, m.e, m.top);
  char* ws = static_cast<char*>(plan->workspace);
  MoeArgs a{};
  a.x = m.x;
  a.x_stride = m.x_stride;
  a.router = m.router;
  a.logits = m.logits;
  a.sel = reinterpret_cast<int32_t*>(ws + at.sel);
  a.gates = reinterpret_cast<float*>(ws + at.gates);
  a.scores = m.router ? reinterpret_cast<double*>(ws + at.scores) : nullptr;
  a.act = reinterpret_cast<uint16_t*>(ws + at.act);
  a.sums = reinterpret_cast<float*>(ws + at.sums);
  a.user_sel = m.sel;
  a.user_gates = m.gates;
  const uint32_t up = (uint32_t)(mx ? m.dim / 2 : m.dim), down = (uint32_t)(mx ? m.f / 2 : m.f);
  a.w13 = {static_cast<const uint8_t*>(m.w13), static_cast<const uint8_t*>(m.s13), m.e * 2 * m.f, up, (uint32_t)(m.dim / kMxGroup)};
  a.w2 = {static_cast<const uint8_t*>(m.w2), static_cast<const uint8_t*>(m.s2), m.e * m.dim, down, (uint32_t)(m.f / kMxGroup)};
  a.s13 = static_cast<const uint16_t*>(m.s13);
  a.s2 = static_cast<const uint16_t*>(m.s2);
  a.y32 = m.y_f32;
  a.y16 = m.y_bf16;
  a.y_stride = m.y_stride;
  a.tokens = (int32_t)m.tokens;
  a.dim = (int32_t)m.dim;
  a.f = (int32_t)m.f;
  a.e = (int32_t)m.e;
  a.top = m.top;
  a.renormalize = m.renormalize;
  a.spans = (int32_t)((up + 255) / 256);
  a.spans2 = (int32_t)((down + 255) / 256);
  hipStream_t s = (hipStream_t)stream;
  // a workgroup reads up to 128 KB of router rows; where it reads a token's all, it selects
  const int shares = m.router ? (int)std::min<int64_t>(m.e, (m.e * m.dim + kScoreMost - 1) / kScoreMost) : 0;
  if (m.router)
    hipLaunchKernelGGL(moe_score_kernel, dim3((unsigned)m.tokens, (unsigned)shares), dim3(kScoreWaves * 64), 0, s, a);
  // Otherwise every workgroup of the next launch selects for itself where that is one
  // token a wave (8 tokens of 128 experts: 47.5 us, with a launch of its own 48.9).
  a.here = shares != 1 && m.tokens <= 8;
  if (shares != 1 && !a.here) hipLaunchKernelGGL(moe_route_kernel, dim3((unsigned)m.tokens), dim3(64), 0, s, a);
  if (mx)
    experts_launch<true>(a, s);
  else
    experts_launch<false>(a, s);
  return launch_status(name);
}
