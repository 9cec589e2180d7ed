/*
 * ft.h -- C ABI of libft.so: block-quantized matvec, routed-MoE vector path and
 * grouped keep-quant expert GEMM on AMD Instinct MI355X (gfx950).
 *
 * Sources the operations come from (cited by page title and section):
 *  [P1] FreeToken PR #136 "enable native GGUF kernels on ROCm (validated on RDNA4)",
 *       Summary: Q4_0 dequantization, the int8-dot matvec (mul_mat_vec with
 *       quantized activations) and the routed MoE vector kernel.
 *  [P2] FreeToken PR #260 "validate native gfx1151 serving on Strix Halo",
 *       Summary: packed Q4_K, Q5_K, Q6_K and Q8_0 weights kept quantized.
 *  [P3] vllm.cpp PR #523 "grouped + non-grouped keep-quant expert GEMM",
 *       What changed: Y = X.W^T with keep-quant W (non-grouped op) and the same
 *       grouped over expert_ids; Q8_0/Q8_K activation quantizers; per-superblock
 *       integer dots.  Review and rework: a per-format availability query in place
 *       of a boolean, refusal before the first forward, a grow-only per-stream
 *       scratch pool with no per-call malloc, free or synchronize.
 *  [P4] ds4 PR #656 "Add ROCm MXFP4 routed expert kernels", Summary: MXFP4 x Q8_K
 *       routed gate/up and down, SwiGLU between them, tiny batches (2-4 tokens)
 *       on direct kernels and larger ones on expert-sorted tiles.
 * Block byte layouts are the public GGUF (ggml) formats; the pages name the
 * formats but do not print them.
 *
 * Conventions for every call:
 *  - Pointers are device pointers unless stated.  The caller owns every input
 *    and output buffer; the library owns only its scratch pool.
 *  - Layouts are row-major, little-endian.  Weights are [rows][k/blk] blocks
 *    with rows the outputs (y = W.x).  Activations are [tokens][k/blk_a] blocks.
 *  - Weight, block and activation base pointers must be 16-byte aligned
 *    (FT_ERR_ALIGNMENT otherwise).  Kernels may read up to 15 bytes past the end
 *    of a weight buffer whose size is not a multiple of 16; such reads never
 *    cross a 4 KiB page.
 *  - Work is enqueued on `stream` (0 = the null stream) and the call returns.
 *    No call synchronizes.  After ft_scratch_reserve() has sized the pool, no
 *    call allocates, so the calls may be captured in a HIP graph.
 *  - Errors are returned as ft_status, nothing throws.  Host-checkable
 *    conditions (NULL, shapes, unsupported pairs) are refused before any work
 *    is enqueued.  Out-of-range expert ids and non-finite inputs are outside
 *    the contract (results undefined, never a memory fault: ids are clamped).
 *  - Calls on different streams may run concurrently; calls that share a
 *    stream's scratch pool are ordered by that stream, from however many host
 *    threads they come (a call holds the pool until it has enqueued its work).
 *    Scratch that a caller gives (ft_attn_opts, ft_lora_opts) is the caller's to order.
 */
#ifndef FT_H
#define FT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void* ft_stream_t; /* a hipStream_t */

/* block formats */
typedef enum {
  FT_Q4_0 = 0,  /* 32 weights: fp16 d, 16 B nibbles; w = d*(n-8)            18 B */
  FT_Q8_0 = 1,  /* 32 weights (or activations): fp16 d, 32 int8; w = d*q     34 B */
  FT_Q4_K = 2,  /* 256: fp16 d, fp16 dmin, 12 B of 6-bit scales/mins, 128 B nibbles;
                   w = d*sc_j*n - dmin*m_j per 32-element sub-block j       144 B */
  FT_Q5_K = 3,  /* 256: as Q4_K plus 32 B of fifth bits                     176 B */
  FT_Q6_K = 4,  /* 256: 128 B low nibbles, 64 B high 2-bit pairs, 16 int8 scales,
                   fp16 d; w = d*sc*(q6-32) per 16-element sub-block         210 B */
  FT_MXFP4 = 5, /* 32: E8M0 exponent e, 16 B E2M1 codes; w = E2M1*2^(e-127)   17 B */
  FT_Q8_1 = 6,  /* activation, 32: fp16 d, fp16 s = d*sum(q), 32 int8         36 B */
  FT_Q8_K = 7,  /* activation, 256: fp32 d, 256 int8, 16 int16 group sums   292 B */
  FT_Q2_K = 8,  /* 256: 16 B of 4-bit scale|min pairs, 64 B of 2-bit codes, fp16 d,
                   fp16 dmin; w = d*sc*q - dmin*m per 16 elements              84 B */
  FT_Q3_K = 9,  /* 256: 32 B third bits, 64 B of 2-bit codes, 12 B of 6-bit
                   scales (+32), fp16 d; w = d*(sc-32)*(q-4) per 16 elements 110 B */
  FT_Q4_1 = 10, /* 32: fp16 d, fp16 m, 16 B nibbles; w = d*n + m              20 B */
  FT_Q5_0 = 11, /* 32: fp16 d, 4 B fifth bits, 16 B nibbles; w = d*(q-16)     22 B */
  FT_Q5_1 = 12  /* 32: fp16 d, fp16 m, 4 B fifth bits, 16 B nibbles; w = d*q + m
                                                                            24 B */
} ft_type;

typedef enum {
  FT_OK = 0,
  FT_ERR_INVALID_ARG = 1, /* NULL pointer, negative size, bad option */
  FT_ERR_UNSUPPORTED = 2, /* (op, weight, activation) combination not provided */
  FT_ERR_SHAPE = 3,       /* k not a multiple of the block sizes, topk out of range */
  FT_ERR_ALIGNMENT = 4,   /* a base pointer is not 16-byte aligned */
  FT_ERR_NO_SCRATCH = 5,  /* the pool is too small and the stream is capturing, or the
                             caller's workspace is too small */
  FT_ERR_HIP = 6          /* a HIP runtime call or kernel launch failed */
} ft_status;

typedef enum {
  FT_OP_QUANTIZE = 0, FT_OP_DEQUANT = 1, FT_OP_MMVQ = 2, FT_OP_MOE_VEC = 3,
  FT_OP_GROUPED = 4, FT_OP_BLOCK_DOTS = 5,
  FT_OP_KV_CACHE = 6 /* w: the keys' block type, act: the values' */
} ft_op;

/* element types of the plain tensors around the key/value cache, the scored router, the
   rotation, the norm and the adapters (every other call's plain tensors are fp32) */
typedef enum { FT_F32 = 0, FT_F16 = 1, FT_BF16 = 2 } ft_float;

/* Elements per block (32 or 256) and bytes per block; 0 for an unknown type. */
int ft_block_elems(ft_type type);
size_t ft_block_bytes(ft_type type);

/* Per-format availability, answered on the host before any data exists [P3,
   review: a per-dtype query instead of a boolean].  Returns 1 if `op` runs for
   (w, act); act is ignored for FT_OP_DEQUANT and w for FT_OP_QUANTIZE.
   Every combination reported 0 makes the op return FT_ERR_UNSUPPORTED. */
int ft_supported(ft_op op, ft_type w, ft_type act);

/* Human-readable status. */
const char* ft_status_str(ft_status status);

/* Library version string (static storage). */
const char* ft_version(void);

/* Activation quantizer [P3 What changed: Q8_0/Q8_K quantizers; P4: Q8 prequant].
   x: [rows][k] fp32 with row stride ldx (elements) >= k.  xq: [rows][k/blk] blocks
   of `act` (FT_Q8_1, FT_Q8_0 or FT_Q8_K), written in full.
   Q8_1 per 32-block: d = fp16(amax/127); q = clamp(round_half_away(x/d), -127, 127)
   against the stored d (q = 0 when d is 0); s = fp16(d * sum q).
   Q8_0 per 32-block: d and q as Q8_1, no s (fp16 d at byte 0, codes from byte 2).
   Q8_K per 256-block: d = amax/127 in fp32; q as above; bsums[g] = sum of q over
   elements 16g..16g+15. */
ft_status ft_quantize_act(ft_type act, const float* x, int64_t rows, int64_t k, int64_t ldx,
                          void* xq, ft_stream_t stream);

/* Dequantization [P1 Summary: Q4_0 dequantization; P2: packed K-quants].
   blocks: [rows][k/blk] of weight type w.  out: [rows][k] fp32 -- each value is
   the exact weight rounded once to fp32 (exact for every format but the Q4_K /
   Q5_K / Q2_K difference d*sc*n - dmin*m and the Q4_1 / Q5_1 sum d*q + m, which
   round once). */
ft_status ft_dequant(ft_type w, const void* blocks, int64_t rows, int64_t k, float* out,
                     ft_stream_t stream);

/* Quantized matvec [P1 Summary: int8-dot matvec; P3 What changed: non-grouped op].
   W: [n][k/blk] blocks of w; xq: [t][k/blk_a] blocks of act;
   y: [t][ldy] fp32, ldy >= n, y[i][r] = sum_k w[r][k] * xhat[i][k], computed as exact
   integer dots per block followed by an fp32 scale combine.  Any t >= 0 (t = 0 is a
   no-op); batches beyond 8 tokens are processed 8 at a time.  Supported (w, act):
   every weight type x FT_Q8_1 and x FT_Q8_0; (Q4_K, Q5_K, Q6_K, MXFP4) x FT_Q8_K
   [P3 What changed: the non-grouped op with Q8_0 / Q8_K activations].  With
   FT_Q8_1 or FT_Q8_0, from 2-5 tokens on (the threshold depends on the format and
   on k) every format runs on the int8 matrix cores when k is a multiple of 256 (512
   for MXFP4); the result is the same integer dots either way.  FT_Q8_0 activations
   are first copied into the Q8_1 block layout (same d and codes) in the stream's
   scratch pool, so under graph capture the pool must hold t*(k/32)*36 bytes
   (FT_ERR_NO_SCRATCH otherwise).  FT_Q8_K runs on the dot4 kernels at every t. */
ft_status ft_mul_mat_vec_q(ft_type w, const void* W, int64_t n, int64_t k,
                           ft_type act, const void* xq, int64_t t,
                           float* y, int64_t ldy, ft_stream_t stream);

/* Router [P4 Summary; routing semantics as read from the pages]:
   logits [t][n_expert] fp32 -> ids [t][topk] int32 (the topk largest logits, ties
   toward the lower expert index, slot 0 the largest) and w [t][topk] fp32 = softmax
   over the selected logits.  1 <= topk <= min(8, n_expert), n_expert <= 1024. */
ft_status ft_moe_route(const float* logits, int64_t t, int64_t n_expert, int topk,
                       int32_t* ids, float* w, ft_stream_t stream);

/* Stable token->expert sort of the t*topk (token, slot) pairs [P4: expert-sorted
   tiles].  counts [n_expert], offsets [n_expert+1] (exclusive prefix sum), pairs
   [t*topk] = pair indices (token*topk + slot) ordered by expert, ascending pair index
   within an expert.  All int32. */
ft_status ft_moe_sort(const int32_t* ids, int64_t t, int topk, int64_t n_expert,
                      int32_t* counts, int32_t* offsets, int32_t* pairs, ft_stream_t stream);

/* Options of ft_moe_q_vec; pass NULL for defaults. */
typedef struct {
  int route;          /* 0 auto, 1 force the direct route ((Q4_K, Q8_1) and (MXFP4,
                         Q8_K) only), 2 force sorted tiles (every (w, Q8_K) pair);
                         a route the pair lacks gives FT_ERR_UNSUPPORTED */
  int direct_max_t;   /* auto route: direct for t <= direct_max_t (0 = default 8),
                         sorted tiles above it where supported; pairs without a
                         direct route take the tiles at every t */
  float* tap_g;       /* nullable [t*topk][inter] fp32: gate projections */
  float* tap_u;       /* nullable [t*topk][inter] fp32: up projections */
  float* tap_h;       /* nullable [t*topk][inter] fp32: silu(g)*u */
  void* tap_hq;       /* nullable [t*topk][inter/blk_a] blocks: quantized h */
  float* tap_down;    /* nullable [t*topk][hidden] fp32: per-pair down projections */
  const void* in_hq;  /* nullable: use these quantized h blocks for the down stage */
  const float* logits;/* nullable [t][n_expert] router logits (n_expert <= 1024): the layer
                         routes each token itself, as ft_moe_route, and expert_ids /
                         expert_w are not read (they may be NULL) */
  int32_t* ids_out;   /* nullable [t][topk]: receives that routing's ids ... */
  float* w_out;       /* nullable [t][topk]: ... and weights */
} ft_moe_opts;

/* Routed-MoE layer [P1: routed MoE vector kernel; P4: gate/up, SwiGLU, down].
   w_gate, w_up: [n_expert][inter][hidden/blk]; w_down: [n_expert][hidden][inter/blk],
   all of weight type w.  x: [t][hidden] fp32.  expert_ids, expert_w: [t][topk].
   For every token i and slot s with e = expert_ids[i][s]:
     g = W_gate[e].xhat_i, u = W_up[e].xhat_i (xhat = act-quantized x_i),
     h = silu(g)*u, hhat = act-quantized h, d = W_down[e].hhat,
   and y[i] = sum over s (in slot order) of expert_w[i][s] * d.  y: [t][hidden] fp32.
   The topk ids of one token must be distinct (as top-k routing makes them).
   Supported (w, act): (Q4_K, Q8_1) and (MXFP4, Q8_K) on both routes; (Q4_K, Q8_K),
   (Q5_K, Q8_K), (Q6_K, Q8_K) on the sorted tiles.  topk 1..8; n_expert <= 8192 on
   the sorted tiles.
   Routes [P4 Summary: tiny batches direct, larger ones on expert-sorted tiles;
   P3 What changed: the grouped keep-quant op over expert_ids]:
   direct = the selected experts' rows streamed once per chunk of tokens, every token
   that picked an expert served from the same bytes: for (Q4_K, Q8_1) with hidden
   and inter multiples of 256 up to 4096 (inter up to about 1536), two launches per
   4-token chunk (routing from the logits, x quantize, gate/up + SwiGLU, h quantize;
   then down and the slot-order combine), otherwise one workgroup per selected
   expert and row tile per stage, then a combine; for (MXFP4, Q8_K) the gate/up
   launch routes 1-2 tokens from the logits itself, and at 1-2 tokens down and the
   combine are one launch whose workgroups each take one token's rows (an expert
   both tokens picked is read once per token there);
   sorted tiles = token->expert sort, one fused gate/up + SwiGLU grouped MFMA GEMM,
   h quantize, grouped down GEMM, slot-order combine.  Both give the same result
   up to fp32 rounding order. */
ft_status ft_moe_q_vec(ft_type w, const void* w_gate, const void* w_up, const void* w_down,
                       int64_t n_expert, int64_t hidden, int64_t inter,
                       ft_type act, const float* x, int64_t t,
                       const int32_t* expert_ids, const float* expert_w, int topk,
                       float* y, const ft_moe_opts* opts, ft_stream_t stream);

/* The same layer for callers that cannot allocate device memory (code under HIP
   graph capture, serving loops that must not call hipMalloc, harnesses that forbid
   it).  Arguments, routes, results and errors as ft_moe_q_vec; its scratch is a
   fixed device array of FT_NOALLOC_SCRATCH_BYTES per GPU, held by the library until
   the process ends, instead of the stream's pool.  A problem whose scratch
   (ft_moe_scratch_bytes) exceeds that size is refused with FT_ERR_SHAPE before
   anything is enqueued.  Calls on one GPU share that array: calls that may overlap
   on one GPU (different streams) race and must be ordered by the caller.  Nothing
   in the array needs to start at zero.  The first call on a device looks the
   array's address up (hipGetSymbolAddress) and keeps it. */
#define FT_NOALLOC_SCRATCH_BYTES (32u << 20)
ft_status ft_moe_q_vec_noalloc(ft_type w, const void* w_gate, const void* w_up, const void* w_down,
                               int64_t n_expert, int64_t hidden, int64_t inter,
                               ft_type act, const float* x, int64_t t,
                               const int32_t* expert_ids, const float* expert_w, int topk,
                               float* y, const ft_moe_opts* opts, ft_stream_t stream);

/* Grouped keep-quant expert GEMM [P3 What changed: grouped over expert_ids].
   W: [n_expert][n][k/blk] blocks; xq: act blocks, [t][k/blk_a] when x_per_pair = 0
   (every slot of a token reads its token's row) or [t*topk][k/blk_a] when 1.
   y: [t*topk][n] fp32 in (token, slot) order: y[p] = W[ids[p]] . xhat_row(p).
   Supported (w, act): (Q5_K, Q8_K), (Q6_K, Q8_K), (MXFP4, Q8_K), (Q4_K, Q8_K). */
ft_status ft_grouped_gemm_q(ft_type w, const void* W, int64_t n_expert, int64_t n, int64_t k,
                            ft_type act, const void* xq, int x_per_pair,
                            const int32_t* expert_ids, int64_t t, int topk,
                            float* y, ft_stream_t stream);

/* Integer partials of the block dots (debug tap; [P3 What changed: bit-identical
   integer core]).  partials: [t][n][k/sub] int32, sub = 16 for Q2_K, Q3_K and Q6_K
   and 32 otherwise: the sum over each sub-block of the weight's integer code (n-8 for
   Q4_0, q for Q8_0, the 4/5-bit n for Q4_K/Q5_K, q6-32 for Q6_K, twice the E2M1 value
   for MXFP4, the 2-bit q for Q2_K, the 3-bit q-4 for Q3_K) times the activation's
   int8 code (act: FT_Q8_1, FT_Q8_0 -- through its Q8_1 layout, as the matvec --
   or FT_Q8_K).  Computed with the unpack and v_dot4 core of the dot4 matvec kernels
   (one and two tokens); the int8-MFMA matvec, the grouped GEMM and the FP4-MFMA
   MoE kernels form the same integers on the matrix cores and are checked for
   them through exactly representable outputs instead. */
ft_status ft_debug_block_dots(ft_type w, const void* W, int64_t n, int64_t k,
                              ft_type act, const void* xq, int64_t t,
                              int32_t* partials, ft_stream_t stream);

/* Measurement microkernels (not part of the method): the ceilings the hot path is
   held against, measured on the part next to its published peaks.
   which = 0: streaming read of `bytes` bytes at `buf` (device, 16-byte aligned,
   bytes a multiple of 16) with 16-byte loads; which = 1: `iters` rounds of eight
   independent int8 MFMA chains (v_mfma_i32_16x16x32_i8, 16384 ops each) per wave;
   which = 2: `iters` rounds of eight independent v_dot4_i32_i8 chains per lane
   (8 ops per lane each); which = 3: as 1 with v_mfma_i32_16x16x64_i8 (32768 ops
   each).  1-3 run 8 workgroups of 256 threads per CU and ignore buf/bytes.  out: one device uint32 that receives nothing in practice (it keeps
   the work live).  The caller times the call. */
ft_status ft_debug_ceiling(int which, const void* buf, int64_t bytes, int64_t iters, void* out,
                           ft_stream_t stream);

/* Router with scores over all experts, a bias for balance and expert groups.
   logits: [t][n_expert] of `type`, rows ld (elements) apart.  Per token:
     score_e  = softmax over all experts, or with `sigmoid` 1 / (1 + exp(-x_e));
     choice_e = score_e + bias_e;
     with n_group > 1 the experts are n_group consecutive groups of equal size; a
     group's value is its largest choice (group_top 1) or the sum of its two largest
     (group_top 2), and only the topk_group groups of largest value stay;
     ids [t][topk] = the topk largest choices left, slot 0 the largest;
     w   [t][topk] = score of ids (without the bias), divided by their sum with
     `renorm`, times scale.
   Every tie goes to the lower index.  Scores, choices and sums are held in 64 bits,
   w is rounded to fp32 once.  A logit of -inf has score 0; NaN logits count as -inf
   when experts are chosen.  t <= 2^25, 1 <= topk <= min(32, topk_group * n_expert / n_group),
   n_expert <= 1024, n_group <= 64 and a divisor of n_expert, 1 <= topk_group <=
   n_group.  opts NULL: softmax, no bias, one group, renorm, scale 1.
   The library's own calls that take ids (ft_moe_sort, ft_moe_q_vec, ft_grouped_gemm_q)
   take topk up to 8. */
typedef struct {
  int sigmoid;        /* 0 softmax, 1 sigmoid */
  const float* bias;  /* nullable [n_expert] */
  int n_group;        /* 0 = 1 */
  int topk_group;     /* 0 = n_group */
  int group_top;      /* 1 or 2 (0 = 1) */
  int no_renorm;      /* 1: the weights are not divided by their sum */
  double scale;       /* 0 = 1 */
} ft_route_opts;
ft_status ft_moe_route_ex(const void* logits, ft_float type, int64_t t, int64_t n_expert, int64_t ld, int topk,
                          const ft_route_opts* opts, int32_t* ids, float* w, ft_stream_t stream);

/* Paged key/value cache, its rows quantized in blocks of 32 along head_dim as they
   are written.  A pool of pages per side; a page holds page_size tokens of every KV
   head and is [n_kv_head] page heads; slot s is token s % page_size of page
   s / page_size.  Types FT_Q8_0 and FT_Q4_0 (each side its own), page_size 16, 32,
   64, 128 or 256, head_dim 64, 96, 128 or 256.  A page takes as many bytes as the
   same rows in GGUF blocks, in another order.  With P = page_size, NB = head_dim / 32
   and element e = 32 b + i of token j, a page head is its codes, then the scales, fp16
   [NB][P]; the code is
     K, FT_Q8_0: the byte (code + 128) at P*64*(b/2) + j*32*m + (i/8)*8*m + (b%2)*8 + i%8,
       m the number of blocks in the group b/2 (2; 1 in a last odd group);
     K, FT_Q4_0: nibble (i%8)/2 + 4*(i%2) (code + 8) of the 32-bit word at P*64*(b/4) +
       j*16*m + (i/8)*4*m + (b%4)*4, m the number of blocks in the group b/4;
     V, FT_Q8_0: the byte (code + 128) at e*P + j;
     V, FT_Q4_0: in the byte at (16*b + i%16)*P + j, low nibble for i < 16, high above.
   k_pages, v_pages: 16-byte aligned, n_pages * ft_kv_page_bytes each. */
typedef struct {
  ft_type k_type, v_type;
  void* k_pages;
  void* v_pages;
  int64_t n_pages;
  int64_t page_size, n_kv_head, head_dim;
} ft_kv_cache;
/* bytes of one page of one side; 0 for a type or size that is not provided */
size_t ft_kv_page_bytes(ft_type type, int64_t page_size, int64_t n_kv_head, int64_t head_dim);

/* Quantize t tokens' keys and values into the cache.  k, v: [t][n_kv_head][head_dim] of
   `type`, element stride 1, token and head strides in elements.  slots [t] int64: a
   negative slot, or one past the pool, writes nothing.  Per block of 32:
     FT_Q8_0: d = fp16(amax / 127), q = clamp(round_half_away(x / d), -127, 127);
     FT_Q4_0: d = fp16(m / -8) with m the first element of largest magnitude,
              q = clamp(round_half_away(x / d), -8, 7);
   against the stored d (q = 0 where it is 0); d is limited to +-65504.  The slots of
   one call must be distinct: of two tokens with one slot, each code and scale is one or
   the other's.  A NaN has no magnitude and an unspecified code.  t <= 2^24, here and in
   ft_kv_load. */
ft_status ft_kv_store(const ft_kv_cache* cache, ft_float type, const void* k, int64_t k_token, int64_t k_head,
                      const void* v, int64_t v_token, int64_t v_head, const int64_t* slots, int64_t t,
                      ft_stream_t stream);
/* The rows of t slots as plain numbers d * q, rounded once to `type`.  k or v may be
   NULL: that side is not read.  A negative slot, or one past the pool, gives zeros. */
ft_status ft_kv_load(const ft_kv_cache* cache, const int64_t* slots, int64_t t, ft_float type, void* k,
                     int64_t k_token, int64_t k_head, void* v, int64_t v_token, int64_t v_head, ft_stream_t stream);

/* Attention of n_tok query tokens over the cache.
   q, out: [n_tok][n_head][head_dim] of `type`, element stride 1, token and head strides
   in elements; n_head a multiple of the cache's n_kv_head, KV head h serves query heads
   h*G .. h*G + G-1.  Sequence i has the query tokens q_start[i] .. q_start[i+1]-1 (its
   newest, already stored) and kv_len[i] keys; its key j lies in slot j % page_size of page
   table[i][j / page_size], table rows table_ld apart, n_col pages each.  q_start is
   [n_seq+1], ascending; kv_len and table are int32.  All of it is on the device: max_kv
   is the host's bound of kv_len (lengths past it or past the table are cut to it).
   The query token at position p = kv_len - (number of query tokens) + its index sees key j
     if j < kv_len and (j <= p, unless `bidirectional`) and (j > p - window, with a window),
     or if j < kv_len and j < prefix_len[i] (a prefix that all see: prompt or sink tokens).
   score = scale * q.k; with softcap c, c * tanh(score / c); with slopes, - slopes[head] *
   |p - j|; out = softmax over the visible keys times v, zeros where there is none.  A row of
   q with a NaN or an infinity gives NaN (zeros where it sees no key), and no other row does.
   Tokens of no sequence (before q_start[0], from q_start[n_seq] on) are left as they were.
   n_shared > 0: the first n_shared keys (a multiple of page_size) of every sequence are
   the pages of table row 0, read once for all sequences.  The result is the same up to the
   roundings of its type named here; which of the kernels (few or many query tokens) reads
   the shared keys depends on the rows of all sequences together.
   fp32: products of fp16 pairs summed in fp32, about fp32 accuracy; fp16: the
   probabilities times V's scales are rounded to fp16, everything else as for fp32; bf16:
   with many query tokens the keys and the probabilities are rounded to fp16 too, and V's
   scales are held to 2^-25 of the largest of 64 keys.  With a cap
   above 512 every type is computed as fp32 is; a cap above 1e30 counts as 1e30.
   Page ids outside the pool are clamped.  Refused as too large: n_tok > 2^24, n_seq > 2^20,
   n_head > 1024, max_kv > 2^30, n_tok * G >= 2^30, and more rows than one launch takes
   (n_tok * n_head past 2^30, less where the keys are split).  opts NULL: causal, scale 1/sqrt(head_dim).
   Scratch (parts of split keys): the stream's pool, or the caller's `workspace` (16-byte
   aligned, ft_attn_kv_scratch_bytes).  Graphs captured on one stream share its pool: give
   those that may replay at the same time a workspace each. */
typedef struct {
  float scale;               /* 0 = 1/sqrt(head_dim) */
  float softcap;             /* 0 = none */
  int bidirectional;         /* 1: keys after the token are seen too */
  int64_t window;            /* 0 = none */
  const float* slopes;       /* nullable [n_head] */
  const int32_t* prefix_len; /* nullable [n_seq] */
  int64_t n_shared;          /* 0 = none */
  void* workspace;           /* nullable */
  size_t workspace_bytes;
} ft_attn_opts;
ft_status ft_attn_kv(const ft_kv_cache* cache, ft_float type, const void* q, int64_t q_token, int64_t q_head,
                     int64_t n_tok, int64_t n_head, const int32_t* q_start, const int32_t* kv_len,
                     const int32_t* table, int64_t table_ld, int64_t n_col, int64_t n_seq, int64_t max_kv, void* out,
                     int64_t out_token, int64_t out_head, const ft_attn_opts* opts, ft_stream_t stream);
/* Scratch bytes that are enough for ft_attn_kv with these sizes and options, whatever the type
   and the table's width, and with any smaller max_kv (calls of many query rows per sequence then
   split their keys as far as the scratch goes).  Another number of tokens or sequences has a size
   of its own, a smaller batch sometimes a larger one, as its keys are split further: scratch for
   several batches takes the largest of their sizes. */
size_t ft_attn_kv_scratch_bytes(const ft_kv_cache* cache, int64_t n_tok, int64_t n_head, int64_t n_seq, int64_t max_kv,
                                const ft_attn_opts* opts);

/* Rotary positions.  A pair (a, b) of a row at position p turns by the angle p * f_j:
     a' = a cos - b sin,  b' = b cos + a sin,
   pair j of rot_dim / 2 being elements (j, j + rot_dim / 2), or (2j, 2j + 1) with
   `interleaved`; elements from rot_dim on stay as they are.  cos and sin are read from a table
   [n_pos][rot_dim] fp32, row p the cosines, then the sines: ft_rope_table's, or the caller's.
   positions [t] int32; one outside the table counts as its nearest row.  Products and sums
   are single fp32 operations. */
typedef struct {
  const float* table;
  const int32_t* positions;
  int64_t n_pos;
  int64_t rot_dim;   /* even, 2 .. head_dim */
  int interleaved;
} ft_rotation;
/* Row p of the table: cos(p * f_j) * scale and sin(p * f_j) * scale, computed in 64 bits and
   rounded once.  freqs [half] double (every scaling for long contexts is a choice of f and
   scale; negative f turns back), table [n_pos][2 * half].  half <= 2^15, n_pos <= 2^30 / half. */
ft_status ft_rope_table(const double* freqs, int64_t half, int64_t n_pos, double scale, float* table, ft_stream_t stream);
/* Turn the rows of x, [t][n_head][dim] of `type`, into out (which may be x itself, with its
   strides; otherwise they must not overlap).  Element stride 1, token and head strides in
   elements; no two rows of out overlap.  With weight ([dim] fp32) each row is first x * rstd * weight, rstd = 1 / sqrt(mean x^2 + eps)
   (mean in 64 bits, rstd rounded to fp32).  dim 2 .. 512, t <= 2^24, n_head <= 1024, t * n_head <= 2^30. */
ft_status ft_rope(const ft_rotation* rot, ft_float type, const void* x, int64_t x_token, int64_t x_head, int64_t t,
                  int64_t n_head, int64_t dim, const float* weight, double eps, void* out, int64_t out_token,
                  int64_t out_head, ft_stream_t stream);
/* ft_kv_store with the keys normed (k_weight, nullable) and turned on the way, and the queries
   turned into q_out as ft_rope does, in the same launch.  q: [t][n_head][head_dim], n_head >= 0 (0:
   none, q and q_out may be NULL; otherwise n_head need not fit the cache's).  A token whose slot is
   negative or past the pool stores nothing; its query is turned all the same.  The keys' codes are
   those of ft_rope's fp32 rows given to ft_kv_store.  q_out may be q itself, and must not overlap k or v. */
typedef struct {
  const void* q;
  int64_t q_token, q_head, n_head;
  const float* q_weight;   /* nullable [head_dim] */
  void* q_out;
  int64_t out_token, out_head;
  const void* k;
  int64_t k_token, k_head;
  const float* k_weight;   /* nullable [head_dim] */
  const void* v;
  int64_t v_token, v_head;
  double eps;
} ft_qkv_rows;
ft_status ft_kv_store_rope(const ft_kv_cache* cache, const ft_rotation* rot, ft_float type, const ft_qkv_rows* rows,
                           const int64_t* slots, int64_t t, ft_stream_t stream);

/* The norm around a block.  For rows of x, [rows][width] of `type`:
     b = x;  with `post`: b = norm(b) * post_weight + post_bias;
     with gate: b = b * gate;  b = b * scale;
     r = residual + b (b without a residual);
     n = norm(r) * weight + bias
   norm(v) = v / sqrt(mean v^2 + eps), or with `layer` (v - mean) / sqrt(variance + eps).  Written are
   r, n (`out`, of `type`) and n's blocks of `act` (`xq`, [rows][width / blk], ft_quantize_act's of n in
   fp32), whichever are not NULL, at least one.  n is the norm of r before r is rounded to its type.
   Means are summed in 64 bits, 1 / sqrt is rounded to fp32, every further step is one fp32 operation.
   Weights and biases are fp32, NULL for ones and zeros.  Row strides in elements, at least width;
   ld_gate 0: one row of gates for all.  r and out may each be x or the residual itself (same
   stride).  width <= 32768, rows <= 2^24; blocks need a width of whole blocks. */
typedef struct {
  const void* residual;     /* nullable [rows][width] */
  int64_t ld_residual;
  const void* gate;         /* nullable */
  int64_t ld_gate;
  int post;                 /* 1: x is normed first */
  const float* post_weight;
  const float* post_bias;
  float scale;              /* 0 = 1 */
  int layer;                /* 0: root mean square, 1: mean and variance */
  double eps;
  const float* weight;
  const float* bias;
  void* r;
  int64_t ld_r;
  void* out;
  int64_t ld_out;
  ft_type act;              /* FT_Q8_1, FT_Q8_0 or FT_Q8_K; read with xq only */
  void* xq;
} ft_norm_opts;
ft_status ft_norm(ft_float type, const void* x, int64_t ldx, int64_t rows, int64_t width, const ft_norm_opts* opts,
                  ft_stream_t stream);

/* Low-rank adapters of many requests beside a shared projection:
     out_i = y_i + scales[a] * B[a] (A[a] x_i),  a = ids[i], i < t.
   x: [t][k] of x_type; y (nullable: zeros) and out: [t][n] fp32, row strides in elements; out may be y
   itself (same stride).  A: [n_adapter][rank][k], B: [n_adapter][n][rank], both of w_type.  ids [t] int32:
   one outside 0 .. n_adapter-1 names no adapter, and its row of out is y's.  ranks (nullable) [n_adapter]
   int32: only that many ranks of an adapter count (0: none; at most rank), what A and B hold beyond is
   not used.  scales (nullable: 1) [n_adapter] fp32.  About fp32 accuracy for every type: sums and A x are held in
   fp32, and a product with an fp32 operand (A x is one) comes out short by at most 2^-21 of itself.  A
   row of x with a NaN or an infinity gives NaN in its own row of out only.  t, k, n <= 2^20, rank 1 .. 256,
   n_adapter <= 8192.  Scratch: the stream's pool, or the caller's `workspace` (16-byte aligned,
   ft_lora_scratch_bytes). */
typedef struct {
  const int32_t* ranks;
  const float* scales;
  void* workspace;          /* nullable */
  size_t workspace_bytes;
} ft_lora_opts;
ft_status ft_lora(ft_float x_type, const void* x, int64_t ldx, int64_t t, int64_t k, ft_float w_type, const void* A,
                  const void* B, int64_t n_adapter, int64_t rank, int64_t n, const int32_t* ids, const float* y,
                  int64_t ldy, float* out, int64_t ldo, const ft_lora_opts* opts, ft_stream_t stream);
/* Scratch bytes that are enough for these sizes and any smaller t; 0 for sizes that are refused. */
size_t ft_lora_scratch_bytes(int64_t t, int64_t k, int64_t n_adapter, int64_t rank);

/* Grow the stream's scratch pool to at least `bytes` [P3 review: grow-only
   per-stream pool].  Call before capturing a graph.  The pool is never shrunk;
   retired buffers are released by ft_shutdown(). */
ft_status ft_scratch_reserve(ft_stream_t stream, size_t bytes);

/* Scratch bytes ft_moe_q_vec / ft_grouped_gemm_q need for a problem size. */
size_t ft_moe_scratch_bytes(ft_type w, ft_type act, int64_t n_expert, int64_t hidden,
                            int64_t inter, int64_t t, int topk);
size_t ft_grouped_scratch_bytes(ft_type w, int64_t n_expert, int64_t k, int64_t t, int topk, int x_per_pair);

/* Release every scratch buffer.  No call may be in flight. */
void ft_shutdown(void);

#ifdef __cplusplus
}
#endif
#endif /* FT_H */
