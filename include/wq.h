/*
 * wq.h -- C ABI of libwq: weight-only quantized decode matvecs on AMD MI355X
 * (gfx950).
 *
 * The operation is the batch-1 decode product y = x . W^T of a linear layer
 * whose weight W [N_out][K_in] is stored quantized: it is applied once per
 * generated token, so its cost is the bytes of W it streams.  Sources, by
 * page title and section:
 *
 *   [README]   gittoolsai.com "gpt-fast" (Chinese mirror of the project
 *              README): "量化" (quantization) with "Int8 仅权重量化" and
 *              "Int4 仅权重量化" (int8 / int4 weight-only, group size 32);
 *              "基准测试" (batch-1 benchmark table: tokens/s and GB/s per
 *              format); "推测采样" (speculative sampling); "Mixtral 8x7B".
 *   [GUIDE]    onegen.ai "Efficiently implementing the Mixtral 8x7B model
 *              with gpt-fast": "Key Features" (int8/int4 weight-only
 *              quantization; a draft model's tokens verified by the larger
 *              model).
 *   [TAGS]     awesome-repositories.com "meta-pytorch/gpt-fast": tag
 *              "Grouped Quantization".
 *
 * Conventions shared by every call
 * --------------------------------
 * - Every buffer is DEVICE memory owned by the caller.  The library allocates
 *   nothing.  Its only state: a thread-local error text, per-device host
 *   caches (device check, occupancy; safe across host threads) and the
 *   static device scratch of moe_top2_gemv_noalloc.  Passing a host pointer
 *   is outside the contract (the kernel would fault).
 * - Row-major layouts; bf16 values are passed as their uint16 bit patterns.
 * - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Work
 *   is enqueued and the call returns without synchronising.
 * - Outputs must not alias inputs.  Where both `y_f32` and `y_bf16` are
 *   accepted, either may be NULL but not both; y_bf16 is the fp32 result
 *   rounded to nearest-even.
 * - Return value: a wq_status.  Arguments are checked on the host before
 *   anything is launched; a non-OK return launched nothing, except
 *   WQ_ERR_LAUNCH, which reports a failed launch.  No call aborts or prints;
 *   wq_last_error() gives the detail of the calling thread's last failure.
 * - Weights must be finite.  This is not checked; the result of a
 *   non-finite weight is unspecified.
 * - Alignment: x, weight and code pointers 16-byte aligned (WQ_ERR_ALIGN).
 * - Sizes: n >= 0, k >= 0 (n == 0 is a no-op).  K limits per format are
 *   stated at each call; a larger K returns WQ_ERR_SHAPE.
 * - Only gfx950 devices are supported (WQ_ERR_DEVICE otherwise).
 * - Results are deterministic: the same inputs give bitwise the same
 *   outputs (fixed reduction order, no atomics).
 */
#ifndef WQ_H
#define WQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  WQ_OK = 0,
  WQ_ERR_NULL = 1,   /* a required pointer is NULL                       */
  WQ_ERR_SHAPE = 2,  /* a size is negative, unsupported or inconsistent  */
  WQ_ERR_ALIGN = 3,  /* a pointer is not 16-byte aligned                 */
  WQ_ERR_DEVICE = 4, /* no current HIP device, or it is not gfx950       */
  WQ_ERR_LAUNCH = 5  /* the HIP runtime reported a launch failure        */
} wq_status;

/* ------------------------------------------------------------------------ */
/* Quantizers (offline: once per weight, not per token) -- [README] "Int8   */
/* 仅权重量化", "Int4 仅权重量化"; [TAGS] "Grouped Quantization".            */
/* ------------------------------------------------------------------------ */

/*
 * int8 weight-only, per output row (symmetric).
 *   in : w      fp32 [n][k], k % 4 == 0 (16-byte aligned)
 *   out: q      int8 [n][k]    codes in [-127, 127]
 *        scale  bf16 [n]       s = bf16(fp32(max_k |w[r][k]| / 127))
 * q[r][k] = round-half-even of the exact quotient w[r][k] / s (the stored
 * bf16 s), clamped to [-127, 127]; a zero scale gives zero codes.  Hence
 * |w - q s| <= s / 2.  Codes are bit-identical to the CPU oracle's.
 * q 4-byte and scale 2-byte aligned; no upper limit on k.
 */
int wq_quantize_int8(const float* w, int64_t n, int64_t k, int8_t* q, uint16_t* scale,
                     void* stream);

/*
 * int4 weight-only, groups of 32 consecutive inputs of one row (asymmetric).
 *   in : w        fp32 [n][k], k % 32 == 0 (w, qpacked 16-byte aligned,
 *                  sz 4-byte aligned)
 *   out: qpacked  u8   [n][k/2]    byte j = code(2j) | code(2j+1) << 4
 *        sz       bf16 [n][k/32][2] = (scale s, zero z) per group
 * z = bf16(min of the group) is what code 0 decodes to; t = fp32(max - z);
 * s = bf16(fp32(t / 15)) if t > 0 else 0.  code = round-half-even of the
 * exact quotient (w - z) / s clamped to [0, 15] (0 when s == 0); the value a
 * code stands for is z + code * s.  0.625 byte per weight.  Bit-identical to
 * the CPU oracle.
 */
int wq_quantize_int4g32(const float* w, int64_t n, int64_t k, uint8_t* qpacked, uint16_t* sz,
                        void* stream);

/*
 * int4 with a chosen group size -- [README] "Int4 仅权重量化" (the int4
 * quantizer takes a group size; the benchmark rows show 32);
 * [TAGS] "Grouped Quantization".  As wq_quantize_int4g32 with groups of
 * `group` consecutive inputs, group one of 32, 64, 128, 256, or group == k
 * (one group per output row, "per-channel"; k a positive multiple of 32):
 *   sz bf16 [n][k/group][2]; 0.5 + 4/group bytes per weight.
 * k % group == 0.  Errors: WQ_ERR_SHAPE for another group size.
 */
int wq_quantize_int4(const float* w, int64_t n, int64_t k, int32_t group, uint8_t* qpacked, uint16_t* sz,
                     void* stream);

/* ------------------------------------------------------------------------ */
/* Decode matvecs, batch 1 -- [README] "基准测试" (Base / 8-bit / 4-bit     */
/* (G=32) rows: the per-token linear layers of batch-1 generation).         */
/* Accumulation is fp32.                                                    */
/* ------------------------------------------------------------------------ */

/*
 * Unquantized baseline.  x bf16 [k]; w bf16 [n][k];
 * y[r] = sum_k x[k] * w[r][k].   k % 8 == 0, k <= 65536.
 */
int wq_gemv_bf16(const uint16_t* x, const uint16_t* w, int64_t n, int64_t k, float* y_f32,
                 uint16_t* y_bf16, void* stream);

/*
 * int8 per-row.  x bf16 [k]; q int8 [n][k]; scale bf16 [n] (as written by
 * wq_quantize_int8); y[r] = scale[r] * sum_k x[k] * q[r][k].
 * k % 16 == 0, k <= 65536.
 */
int wq_gemv_int8(const uint16_t* x, const int8_t* q, const uint16_t* scale, int64_t n, int64_t k,
                 float* y_f32, uint16_t* y_bf16, void* stream);

/*
 * int4 G=32.  x bf16 [k]; qpacked, sz as written by wq_quantize_int4g32;
 * y[r] = sum_g ( s[r][g] * sum_{k in g} x[k] code[r][k] + z[r][g] * sum_{k in g} x[k] ).
 * k % 32 == 0, k <= 131072.
 */
int wq_gemv_int4g32(const uint16_t* x, const uint8_t* qpacked, const uint16_t* sz, int64_t n,
                    int64_t k, float* y_f32, uint16_t* y_bf16, void* stream);

/*
 * int4 with groups of `group` inputs (32, 64, 128, 256, or k: one group per
 * row), qpacked and sz as written by wq_quantize_int4 with that group; the
 * same sum over groups of `group`.  k % group == 0 (k % 32 == 0 for a
 * per-row group), k <= 131072.  group == 32 is wq_gemv_int4g32.
 * Errors: WQ_ERR_SHAPE for another group size.
 */
int wq_gemv_int4(const uint16_t* x, const uint8_t* qpacked, const uint16_t* sz, int64_t n, int64_t k,
                 int32_t group, float* y_f32, uint16_t* y_bf16, void* stream);

/*
 * Speculative-decoding verify -- [GUIDE] "Key Features" (the larger model
 * checks the draft's tokens), [README] "推测采样".  The m draft tokens go
 * through one int4 G=32 linear in one pass, each weight read once:
 *   x bf16 [m][k], 1 <= m <= 8; y [m][n]; row i of y equals
 *   wq_gemv_int4g32 applied to row i of x (to fp32 rounding).
 * k % 32 == 0, k <= 131072.  From two tokens on the matrix cores (each weight
 * decoded once for all tokens).  The environment variable
 * WQ_SMALLM_ENGINE=valu (read at each call) moves 2, 3 and 5 tokens to the
 * vector ALU where its plans reach (k <= 32768 for int4, 16384 for int8),
 * for comparison; =mfma or unset keeps the matrix cores (measured faster).
 * On the matrix cores, 2..5 tokens over large matrices (k >= 8192 within
 * one activation window, at least 1280 blocks of 32 rows) run a kernel
 * whose workgroups claim row blocks from a per-call counter in a static
 * device array of 1024 slots, each launch taking the next slot and leaving
 * it zeroed: up to 1024 such launches may be in flight on one device at
 * once.  WQ_SMALLM_KERNEL=split or =claim (read at each call) forces the
 * fixed-stride or the claiming kernel wherever a row fits one activation
 * window, for comparison; results agree to fp32 rounding and each kernel's
 * are reproducible bit for bit.
 */
int wq_gemm_smallM(const uint16_t* x, int64_t m, const uint8_t* qpacked, const uint16_t* sz,
                   int64_t n, int64_t k, float* y_f32, uint16_t* y_bf16, void* stream);

/*
 * The same verify product through int4 weights with groups of `group`
 * inputs (32, 64, 128, 256, or k: one group per row), qpacked and sz as
 * written by wq_quantize_int4 with that group -- [TAGS] "Grouped
 * Quantization".  k % group == 0 (k % 32 == 0 for a per-row group); limits
 * as wq_gemm_smallM.  group == 32 is wq_gemm_smallM.
 */
int wq_gemm_smallM_int4(const uint16_t* x, int64_t m, const uint8_t* qpacked, const uint16_t* sz, int64_t n,
                        int64_t k, int32_t group, float* y_f32, uint16_t* y_bf16, void* stream);

/*
 * Speculative-decoding verify through an int8 linear -- [GUIDE] "Key
 * Features", [README] "推测采样" (the verify pass), with the int8 weights of
 * [README] "Int8 仅权重量化".  x bf16 [m][k], 1 <= m <= 8; q, scale as written
 * by wq_quantize_int8; y [m][n] with y[t][r] = scale[r] * sum_k x[t][k] q[r][k];
 * row t of y equals wq_gemv_int8 applied to row t of x (to fp32 rounding).
 * Each weight is read once (m >= 2: on the matrix cores; WQ_SMALLM_ENGINE and
 * WQ_SMALLM_KERNEL as for wq_gemm_smallM, the claiming kernel taken by
 * default from 98304 rows on, for k from 8192 to 32768, with the same
 * per-call slots).  k % 16 == 0; k <= 65536 for m == 1 (the one-token
 * matvec), k <= 2^24 and n * k <= 0xFFFFFF00 for m >= 2.  scale 2-byte
 * aligned.
 */
int wq_gemm_smallM_int8(const uint16_t* x, int64_t m, const int8_t* q, const uint16_t* scale, int64_t n,
                        int64_t k, float* y_f32, uint16_t* y_bf16, void* stream);

/*
 * Top-2 mixture-of-experts decode step for one token, int8 per-row experts
 * -- [README] "Mixtral 8x7B" (sparse MoE, int8 on one GPU).
 *   x       bf16 [dim]
 *   logits  fp32 [e]                 router logits (e == 8)
 *   w13     int8 [e][2f][dim], s13 bf16 [e][2f]   rows 0..f-1: W1 (gate),
 *                                                 rows f..2f-1: W3 (up)
 *   w2      int8 [e][dim][f],  s2  bf16 [e][dim]
 *   work    fp32 [2][f]          caller-provided scratch (overwritten)
 *   sel     int32 [2] or NULL    selected experts, larger gate first
 *   gates   fp32 [2] or NULL     their renormalised gates
 * Routing: softmax over the e logits, keep the two largest (equal logits:
 * lower index first), renormalise the pair (g_a = 1 / (1 + exp(l_b - l_a))).
 * Each selected expert computes a = silu(W1 x) * (W3 x) in fp32 and
 * o = W2 a; y = g_a o_a + g_b o_b.  Only the two selected experts' weights
 * are read; routing happens on the device (no host synchronisation).
 * dim % 16 == 0, f % 16 == 0, 16 <= dim <= 32768, 16 <= f <= 32768; x, w13,
 * w2 and work 16-byte aligned.
 */
int moe_top2_gemv(const uint16_t* x, const float* logits, int64_t e, const int8_t* w13,
                  const uint16_t* s13, const int8_t* w2, const uint16_t* s2, int64_t dim,
                  int64_t f, float* work, float* y_f32, uint16_t* y_bf16, int32_t* sel,
                  float* gates, void* stream);

/*
 * moe_top2_gemv without the caller's workspace, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  Same arguments as moe_top2_gemv minus
 * `work`, same results (bitwise: the same kernels run); the fp32 [2][f]
 * SwiGLU intermediate lives in a static device array of the library (one per
 * device, 128 KiB, held until the process ends), so f <= 16384
 * (WQ_ERR_SHAPE beyond).  Allocates nothing and calls no allocating routine.
 * Every call on one device shares that device's array: calls that overlap on
 * one device (different streams, or host threads without ordering) race and
 * give unspecified results; calls ordered on one stream are safe.  The first
 * call on a device looks the array's address up once (with that device
 * current).  The W13 launch writes the whole intermediate before the W2
 * launch reads it, so no contents carry over from an earlier call.
 */
int moe_top2_gemv_noalloc(const uint16_t* x, const float* logits, int64_t e, const int8_t* w13,
                          const uint16_t* s13, const int8_t* w2, const uint16_t* s2, int64_t dim,
                          int64_t f, float* y_f32, uint16_t* y_bf16, int32_t* sel, float* gates,
                          void* stream);

/* ------------------------------------------------------------------------ */
/* A whole decode step in one launch -- [README] "基准测试" (tokens/s of a  */
/* batch-1 step is the time to stream every linear layer once).             */
/* ------------------------------------------------------------------------ */

enum {
  WQ_FORMAT_BF16 = 1,
  WQ_FORMAT_INT8 = 2,
  WQ_FORMAT_INT4G32 = 3,
  /* int4 with larger groups (wq_quantize_int4) */
  WQ_FORMAT_INT4G64 = 4,
  WQ_FORMAT_INT4G128 = 5,
  WQ_FORMAT_INT4G256 = 6,
  /* int4 with one group per row (wq_quantize_int4 with group == k): each
     matrix's sz is [n][1][2]; k % 32 == 0 */
  WQ_FORMAT_INT4PC = 7
};

/* One linear layer of a step, in the layout of the single-matrix calls:
 *   x    bf16 [m][k]   (16-byte aligned)
 *   w    bf16 [n][k] | int8 [n][k] | int4 packed [n][k/2]   (16-byte aligned)
 *   aux  NULL (bf16) | bf16 scale [n] (int8) | sz [n][k/G][2] (int4 with groups of G, G = k per row;
 *        4-byte aligned)
 *   y_f32 / y_bf16  [m][n], either may be NULL but not both. */
typedef struct {
  const void* x;
  const void* w;
  const void* aux;
  int64_t n;
  int64_t k;
  float* y_f32;
  uint16_t* y_bf16;
} wq_matrix;

/* Filled by wq_decode_step_prepare; pass it unchanged to wq_decode_step_run. */
typedef struct {
  int32_t format;
  int32_t m;
  int32_t count;
  int32_t groups;
  int64_t total_batches;
  const void* workspace;
} wq_step_plan;

/* Upper bound of the device workspace a plan of `count` matrices needs. */
int64_t wq_decode_step_workspace_bytes(int32_t count);

/*
 * Plans `count` independent matvecs of one format (m token rows each: m = 1
 * for bf16, 1 <= m <= 8 for int8 and for int4 with any group size) as ONE
 * persistent launch: every
 * workgroup streams an equal share of the step's weight bytes as a contiguous
 * range of row batches across the matrices, so no matrix pays its own
 * launch, ramp-up and drain.  Results equal the single-matrix calls' to fp32
 * rounding (the per-row reduction order may differ).
 * Validates every matrix on the host (null -> sizes -> alignment; k must be a
 * positive multiple of 8 / 16 / G per format (32 for a per-row group) and within the kernel's row
 * limit: with one token row the activations are staged whole in LDS, so
 * k <= 80896 (bf16), 36864 (int8), 73728 (int4); int4 with 2..8 token rows
 * k <= 131072; int8 with 2..8 token rows k <= 2^24 and n * k <= 0xFFFFFF00),
 * then writes the launch description into `workspace` (device
 * memory, 16-byte aligned, `workspace_bytes` long, caller-owned; it must
 * stay allocated and unmodified while the plan is used).  This copy is
 * synchronous: prepare once, outside any graph capture.  The matrices'
 * buffers must stay where they are for as long as the plan is run.
 */
int wq_decode_step_prepare(int32_t format, int32_t m, const wq_matrix* mats, int32_t count,
                           void* workspace, int64_t workspace_bytes, wq_step_plan* plan);

/* Launches a prepared step on `stream` (asynchronous; may be captured into a
 * HIP graph).  Runs of one plan must not overlap (they share its workspace,
 * which carries balance state that each run measures and the next run uses
 * to cut the step into per-CU ranges: the measured speed of each workgroup,
 * and for int4 with 2..8 token rows the relative cost of rows longer than
 * one activation window); runs of plans that share output buffers race. */
int wq_decode_step_run(const wq_step_plan* plan, void* stream);

/* ------------------------------------------------------------------------ */
/* Top-2 MoE decode over many layers in two launches -- [README] "Mixtral   */
/* 8x7B" (a token's MoE layers are streamed once per decode step).          */
/* ------------------------------------------------------------------------ */

/* One MoE layer, with the buffers and layouts of moe_top2_gemv. */
typedef struct {
  const void* x;          /* bf16 [dim], 16-byte aligned */
  const float* logits;    /* fp32 [e] */
  const int8_t* w13;      /* int8 [e][2f][dim], 16-byte aligned */
  const uint16_t* s13;    /* bf16 [e][2f] */
  const int8_t* w2;       /* int8 [e][dim][f], 16-byte aligned */
  const uint16_t* s2;     /* bf16 [e][dim] */
  float* work;            /* fp32 [2][f], 16-byte aligned; caller scratch (overwritten) */
  float* y_f32;           /* [dim] or NULL */
  uint16_t* y_bf16;       /* [dim] or NULL (not both NULL) */
  int32_t* sel;           /* [2] or NULL */
  float* gates;           /* [2] or NULL */
} wq_moe_layer;

/* Filled by wq_moe_step_prepare; pass it unchanged to wq_moe_step_run. */
typedef struct {
  int64_t dim;
  int64_t f;
  int32_t e;
  int32_t count;
  int32_t grid13;
  int32_t grid2;
  const void* workspace;
} wq_moe_plan;

/* Device workspace a plan of `count` layers needs (bytes). */
int64_t wq_moe_step_workspace_bytes(int32_t count);

/*
 * Plans `count` independent MoE layers (each its own token, logits, experts,
 * work buffer and output; every layer computes exactly what moe_top2_gemv
 * computes for it, to fp32 rounding) as two persistent launches: the W13
 * pass of every layer, then the W2 pass of every layer.  All layers share
 * e == 8, dim and f, with dim % 16 == 0, f % 16 == 0, 16 <= dim <= 14336 and
 * 16 <= f <= 16384 (a layer's activations are staged whole in LDS).
 * Validates every layer on the host (null -> sizes -> alignment), then copies
 * the layer descriptors and the two launches' initial balance state into
 * `workspace` (device memory, 16-byte aligned, caller-owned, unmodified
 * while the plan is used).  The copy is synchronous: prepare once, outside
 * any graph capture.
 */
int wq_moe_step_prepare(int64_t e, int64_t dim, int64_t f, const wq_moe_layer* layers, int32_t count,
                        void* workspace, int64_t workspace_bytes, wq_moe_plan* plan);

/* Launches a prepared MoE step on `stream` (asynchronous; may be captured
 * into a HIP graph).  Runs of one plan must not overlap (each run measures
 * its workgroups' speeds into the workspace and later runs cut their per-CU
 * ranges from them); runs of plans that share buffers must not overlap
 * either. */
int wq_moe_step_run(const wq_moe_plan* plan, void* stream);

/* ------------------------------------------------------------------------ */
/* Between the linears of a verify pass -- [GUIDE] "Key Features" (the      */
/* larger model checks the draft's tokens), [README] "推测采样".  A request */
/* has a context in a paged cache and brings a few drafted tokens (a tree,  */
/* a chain, or the one token of an ordinary decode step).  wqkv's product   */
/* goes through wq_qkv_rope (norms, rotation, append), the drafted tokens   */
/* attend through wq_tree_attention, and after the judgement wq_kv_accept   */
/* moves the accepted tokens' rows next to the context.                     */
/*                                                                          */
/* Each call is a prepare, which checks every argument on the host and      */
/* fills a plan (caller-owned host memory, passed on unchanged), and a run, */
/* which enqueues on `stream` and may be captured into a HIP graph.  A plan */
/* holds addresses and sizes only: the buffers' contents (lengths, tables,  */
/* masks, ...) are read by each run on the device, so they may change       */
/* between runs, and the buffers must stay where they are.  A plan is run   */
/* on the device that was current when it was prepared (WQ_ERR_DEVICE       */
/* otherwise).  Indexes that the device reads are bounds-checked there, as  */
/* stated at each call; nothing outside the described buffers is touched.   */
/* ------------------------------------------------------------------------ */

/*
 * A layer's keys and values in pages of `page_size` positions.  Position p of
 * request r is row p % page_size of page table[r][p / page_size]; head h of
 * that row starts at k (or v) + page * page_stride + row * token_stride +
 * h * head_stride (strides in elements, any order of the axes).  A position
 * whose table entry lies past table_width, or names a page outside
 * [0, pages), holds nothing: it is not read, attended to or written.
 *   k, v bf16, 16-byte aligned, strides multiples of 8, head_dim elements of
 *   one head contiguous; table int32 [requests][table_stride].
 * 1 <= page_size, table_width * page_size <= 2^30, strides below 2^32, 1 <= kv_heads <= 1024,
 * head_dim a multiple of 8 up to 256 (wq_tree_attention: 64, 96, 128, 256).
 * Requests may share pages that no call writes; a row that a call writes must
 * be one position only.
 */
typedef struct {
  uint16_t* k;
  uint16_t* v;
  int64_t pages;
  int64_t page_size;
  int64_t page_stride;
  int64_t token_stride;
  int64_t head_stride;
  const int32_t* table;
  int64_t table_width;
  int64_t table_stride;
  int32_t kv_heads;
  int32_t head_dim;
} wq_kv_cache;

/*
 * The drafted tokens of `requests` requests in the rows of one batch:
 * request r brings rows starts[r] .. starts[r + 1] - 1 (starts int32
 * [requests + 1], non-decreasing, within [0, tokens]; a request may bring
 * none) on top of lengths[r] cached positions (int32, a negative one counts
 * as 0); its row j stands at cache position lengths[r] + j.  Rows of no
 * request are left alone.  (With starts out of order or range it is
 * unspecified which rows of the batch are written; nothing else is touched.)
 * 0 <= tokens <= 2^20, 0 <= requests <= 4096.
 */
typedef struct {
  const int32_t* starts;
  const int32_t* lengths;
  int64_t tokens;
  int64_t requests;
} wq_batch;

/*
 * Rotary frequencies, radians per position, for rot_dim / 2 rotated pairs, in
 * HOST memory (computed in fp64, rounded once): f_i = base^(-2i / rot_dim),
 * then for contexts past the `original` length that a model was trained on
 *   WQ_ROPE_PLAIN     f_i
 *   WQ_ROPE_LINEAR    f_i / factor
 *   WQ_ROPE_BANDS     by wavelength w = 2 pi / f_i: f_i below original / high,
 *                     f_i / factor above original / low, and between them
 *                     f_i * ((1 - t) / factor + t), t = (original / w - low) / (high - low)
 *   WQ_ROPE_RAMP      by pair: f_i below pair a, f_i / factor above pair b and
 *                     linear in i between, with a = floor(pair(high)), b =
 *                     ceil(pair(low)), pair(n) = rot_dim ln(original / (2 pi n))
 *                     / (2 ln base) the pair that turns n times in `original`
 *                     positions, both limited to [0, rot_dim - 1]; *rot_scale =
 *                     0.1 ln(factor) + 1 (for the other kinds 1)
 * factor >= 1; 0 < low < high and original >= 1 where they are used; base > 1;
 * rot_dim even, 2 .. 256.  rot_scale may be NULL.  Needs no device.
 */
enum { WQ_ROPE_PLAIN = 0, WQ_ROPE_LINEAR = 1, WQ_ROPE_BANDS = 2, WQ_ROPE_RAMP = 3 };
int wq_rope_frequencies(int32_t kind, int32_t rot_dim, double base, double factor, double low, double high,
                        double original, float* freq_host, float* rot_scale);

/*
 * What stands between wqkv and attention, in one pass over the product:
 *   qkv   [tokens][qkv_stride]: a row is heads query heads, kv_heads key
 *         heads, kv_heads value heads of head_dim; exactly one of qkv_f32
 *         (stride a multiple of 4) and qkv_bf16 (of 8) is given
 *   u     = x / sqrt(mean(x^2) + eps) * norm  for each query and key head
 *         (q_norm, k_norm bf16 [head_dim], each may be NULL: u = x)
 *   q, k  the first rot_dim elements of u turned in pairs by the angle
 *         positions[t] * freq[i]: (a, b) -> rot_scale * (a cos - b sin,
 *         b cos + a sin), pairs (2i, 2i + 1) if interleaved, else
 *         (i, i + rot_dim / 2); the others as they are
 *   q     bf16 [tokens][q_stride] out; keys and values (bf16) go to the
 *         cache rows of the tokens
 * positions int32 [tokens], or NULL: cache positions, lengths[r] + j (right for
 * one token and for a chain; a draft of a tree stands at lengths[r] + its depth
 * in the tree, which is not its place in the cache).  freq fp32
 * [rot_dim / 2] on the device; angles are reduced in fp64, all else is fp32,
 * each result rounded to nearest-even once.  rot_dim even, 0 .. head_dim (0:
 * freq may be NULL).  heads a multiple of kv_heads, up to 1024; q and qkv
 * 16-byte aligned, their rows not overlapping (WQ_ERR_SHAPE), q_stride a
 * multiple of 8; strides at least a row.
 */
typedef struct {
  wq_kv_cache cache;
  wq_batch batch;
  const float* qkv_f32;
  const uint16_t* qkv_bf16;
  int64_t qkv_stride;
  uint16_t* q;
  int64_t q_stride;
  const int32_t* positions;
  const uint16_t* q_norm;
  const uint16_t* k_norm;
  const float* freq;
  float eps;
  float rot_scale;
  int32_t rot_dim;
  int32_t interleaved;
  int32_t heads;
} wq_qkv_rope;

typedef struct {
  int64_t made;        /* set by prepare */
  int32_t device;
  int32_t reserved;
  wq_qkv_rope a;
} wq_qkv_rope_plan;

int wq_qkv_rope_prepare(const wq_qkv_rope* a, wq_qkv_rope_plan* plan);
int wq_qkv_rope_run(const wq_qkv_rope_plan* plan, void* stream);

/*
 * Attention of each request's drafted tokens over its context and its tree:
 *   y[t][h] = sum_p w_p v[p], w = softmax over the visible p of
 *             scale * q[t][h] . k[p], key head h / (heads / kv_heads)
 * Every position < lengths[r] is visible; position lengths[r] + j is visible
 * to the request's row i if bit j of tree[starts[r] + i] is set (tree uint64
 * [tokens]: normally the token's ancestors and itself), and with tree == NULL
 * if j <= i (a chain; one token: ordinary decode attention).  The drafts' own
 * keys and values must be in the cache (wq_qkv_rope).  A row that sees
 * nothing gets zeros; what a row does not see (NaN and infinities too) does
 * not change it.
 *   q, y  bf16 [tokens][q_stride / y_stride], rows of heads * head_dim,
 *         16-byte aligned, strides multiples of 8; rows of y must not overlap
 *         rows of q (WQ_ERR_SHAPE)
 * A request brings at most max_tokens rows, 1 <= max_tokens <= 64; one that
 * brings more is left alone.  heads / kv_heads <= 64.  scale finite.  requests
 * * kv_heads * row blocks (of 64 rows per key head) * (positions / 32 + 4)
 * stays below 2^31, with the positions that the table covers.
 * Scores and sums are fp32 (any finite score, before and after scaling); the
 * weights enter the second product as bf16.  The weighted values are summed
 * before the division, with weights of at most 2^8: a row's positions times its
 * largest value must stay below 2^119.
 *
 * The positions of all requests are cut into equal shares for the launch's
 * workgroups and partial results joined in a fixed order: results are
 * bitwise reproducible.  `workspace` (device, 16-byte aligned,
 * wq_tree_attention_workspace_bytes long) holds the partial results between
 * the launches of a run; nothing in it is kept from run to run.  Runs that
 * share a workspace must not overlap.
 */
typedef struct {
  wq_kv_cache cache;
  wq_batch batch;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* y;
  int64_t y_stride;
  const uint64_t* tree;
  float scale;
  int32_t heads;
  int32_t max_tokens;
} wq_tree_attention;

typedef struct {
  int64_t made;        /* set by prepare */
  int32_t device;
  int32_t variant;
  void* workspace;
  wq_tree_attention a;
} wq_tree_attention_plan;

/* Workspace of a plan with these sizes (0 if they are not supported). */
int64_t wq_tree_attention_workspace_bytes(int64_t requests, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                          int32_t max_tokens);
int wq_tree_attention_prepare(const wq_tree_attention* a, void* workspace, int64_t workspace_bytes,
                              wq_tree_attention_plan* plan);
int wq_tree_attention_run(const wq_tree_attention_plan* plan, void* stream);

/*
 * After the judgement: the cache rows of each request's accepted drafts move
 * next to its context, in every layer at once.  path int32 [requests][64 or
 * less: path_width] (stride path_stride) lists the accepted drafts of a
 * request by depth, accepted[r] of them (limited to [0, path_width]); the
 * rows of draft path[r][i] (position lengths[r] + path[r][i]) are copied to
 * position lengths[r] + i for i = 0, 1, ...  path[r] must increase and start
 * at 0 or later: a request whose path does not is left alone, as is a row
 * whose source or target holds nothing.  Lengths are the caller's to advance.
 * cache describes layer 0; layer l lies l * layer_stride elements on (a
 * multiple of 8, positive where there are several; layers must not share
 * memory), 1 <= layers <= 4096.
 */
typedef struct {
  wq_kv_cache cache;
  int64_t layers;
  int64_t layer_stride;
  int64_t requests;
  const int32_t* lengths;
  const int32_t* path;
  int64_t path_width;
  int64_t path_stride;
  const int32_t* accepted;
} wq_kv_accept;

typedef struct {
  int64_t made;        /* set by prepare */
  int32_t device;
  int32_t reserved;
  wq_kv_accept a;
} wq_kv_accept_plan;

int wq_kv_accept_prepare(const wq_kv_accept* a, wq_kv_accept_plan* plan);
int wq_kv_accept_run(const wq_kv_accept_plan* plan, void* stream);

/* ------------------------------------------------------------------------ */
/* Low-rank adapters beside a shared projection (the quantized products     */
/* above), a different one for each row.                                    */
/* ------------------------------------------------------------------------ */

/*
 *   y[t] = base[t] + scale[c] * B[c] (A[c] x[t]),   c = adapter[t]
 *   x     bf16 [tokens][x_stride]
 *   base  fp32 [tokens][base_stride] (a shared product's y_f32), or NULL: 0
 *   a     bf16 [adapters][rank][k];  b  bf16 [adapters][n][rank]
 *   adapter int32 [tokens]; outside [0, adapters): no adapter, y = base
 *   ranks int32 [adapters] or NULL: only the first ranks[c] of the `rank`
 *         rows of A and columns of B count (limited to [0, rank]; the rest is
 *         not used, whatever it holds)
 *   scale fp32 [adapters] or NULL: 1
 *   y_f32 / y_bf16 [tokens][y_stride], either may be NULL but not both; base
 *         may be y_f32 itself (then with the same stride), otherwise results
 *         overlap neither each other nor an input (WQ_ERR_SHAPE)
 * Rows of one adapter share its weights, wherever they stand in the batch.
 * Sums are fp32, and A x is carried to the second product in bf16 parts: three
 * (24 bits), or two (16 bits) where only y_bf16 is asked for.  k % 8 == 0, 8 <= k <= 65536; rank % 8 == 0,
 * 8 <= rank <= 128; 0 <= n <= 2^20; 0 <= tokens <= 4096;
 * 1 <= adapters <= 4096; x, a, b 16-byte aligned, x_stride a multiple of 8.
 * `workspace` as for wq_tree_attention.
 */
typedef struct {
  const uint16_t* x;
  int64_t x_stride;
  const float* base;
  int64_t base_stride;
  float* y_f32;
  uint16_t* y_bf16;
  int64_t y_stride;
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* adapter;
  const int32_t* ranks;
  const float* scale;
  int64_t tokens;
  int64_t k;
  int64_t n;
  int64_t adapters;
  int32_t rank;
} wq_lora;

typedef struct {
  int64_t made;        /* set by prepare */
  int32_t device;
  int32_t tiles;
  int32_t splits;
  int32_t reserved;
  void* workspace;
  wq_lora a;
} wq_lora_plan;

/* Workspace of a plan with these sizes (0 if they are not supported). */
int64_t wq_lora_workspace_bytes(int64_t tokens, int64_t k, int64_t adapters, int32_t rank);
int wq_lora_prepare(const wq_lora* a, void* workspace, int64_t workspace_bytes, wq_lora_plan* plan);
int wq_lora_run(const wq_lora_plan* plan, void* stream);

/* Static text for a wq_status value ("unknown status" otherwise). */
const char* wq_status_string(int status);

/* Detail of the calling thread's last non-OK return ("" if none).  The
 * pointer stays valid until the thread's next failing call. */
const char* wq_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* WQ_H */
