// ft_attn_kernels.h -- attention over the paged, block-quantized cache: device code
// and launch templates, instantiated per head dimension in ft_attn_d*.hip.
//
// For query row (token i, head h) over the keys j of its sequence:
//   s_j = scale * q . k_j, then cap * tanh(s_j / cap), then - slope_h |pos_i - j|,
//   o = sum_j exp(s_j) v_j / sum_j exp(s_j) over the visible keys, 0 if there is none.
#pragma once

#include "ft_device.h"
#include "ft_internal.h"
#include "ft_kv.h"

namespace ftk {

constexpr float LOG2E = 1.44269504088896340736f;
constexpr int ATTN_STEP = 64;    // keys per step of a wave
constexpr float NO_MAX = -1e30f; // below every score

// a value of the four lane groups (lanes l, l^16, l^32, l^48) met in all of them
__device__ __forceinline__ float groups_max(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float groups_sum(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
__device__ __forceinline__ uint32_t groups_umax(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max((uint32_t)b[0], (uint32_t)b[1]);
}
// over the 16 lanes of a row of the wave
__device__ __forceinline__ int row_min(int v) {
  v = min(v, __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, false));
  v = min(v, __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, false));
  v = min(v, __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, false));
  return min(v, __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, false));
}
__device__ __forceinline__ int row_max(int v) { return -row_min(-v); }

// c * tanh(x / c) in the units of `cap`; x comes divided by c, without EXACT times 2 log2(e).
// EXACT: an odd series below 0.35 (its next term is under 2^-26 of the result), else
// 1 - 2 / (exp(2x) + 1), within 2^-22.6 absolute; without EXACT the latter throughout,
// which takes 2^-22 c from a score: up to WIDE_CAP under a quarter of what rounding a
// probability to fp16 does.
template <bool EXACT>
__device__ __forceinline__ float capped_score(float x, float cap) {
  const float r = __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(EXACT ? x * (2.0f * LOG2E) : x) + 1.0f);
  if constexpr (EXACT) {
    const float y = fmaf(-2.0f, r, 1.0f);
    const float q = x * x;
    float p = fmaf(q, -1382.0f / 155925.0f, 62.0f / 2835.0f);
    p = fmaf(q, p, -17.0f / 315.0f);
    p = fmaf(q, p, 2.0f / 15.0f);
    p = fmaf(q, p, -1.0f / 3.0f);
    p = fmaf(x * q, p, x);
    return cap * (fabsf(x) < 0.35f ? p : y);
  }
  return fmaf(-2.0f * cap, r, cap);
}

// from a product of operands to what capped_score takes, or to the score in powers of two;
// finite, as a product may be 0, and not 0, as a masked score is -inf
template <bool EXACT>
__device__ __forceinline__ float score_factor(float c, float softcap) {
  const float f = softcap > 0.0f ? c / softcap * (EXACT ? 1.0f : 2.0f * LOG2E) : c * LOG2E;
  return fminf(fmaxf(f, 0x1p-126f), 3.0e38f);
}

// two fp16 numbers of a word (by value: a bit cast of a vector's element would read the
// vector's first)
__device__ __forceinline__ h16x2 halves(uint32_t w) { return __builtin_bit_cast(h16x2, w); }
__device__ __forceinline__ h16x8 join8(const h16x2 (&p)[4]) {
  return __builtin_shufflevector(__builtin_shufflevector(p[0], p[1], 0, 1, 2, 3), __builtin_shufflevector(p[2], p[3], 0, 1, 2, 3),
                                 0, 1, 2, 3, 4, 5, 6, 7);
}

// ---- codes to fp16 (exact) -------------------------------------------------
// 0x6400 | u is the fp16 number 1024 + u
__device__ __forceinline__ h16x2 code_pair(uint32_t biased, float off) {
  const h16x2 o = {(_Float16)off, (_Float16)off};
  return __builtin_bit_cast(h16x2, biased) - o;
}
__device__ __forceinline__ h16x8 codes8_q8(u32x2 w) {   // eight bytes, code + 128
  h16x2 p[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    p[2 * i] = code_pair(__builtin_amdgcn_perm(0x64646464u, w[i], 0x04010400u), 1152.0f);
    p[2 * i + 1] = code_pair(__builtin_amdgcn_perm(0x64646464u, w[i], 0x04030402u), 1152.0f);
  }
  return join8(p);
}
__device__ __forceinline__ h16x8 codes8_q4(uint32_t w) {   // eight nibbles, code + 8: nibbles (0, 4), (1, 5), ...
  h16x2 p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = code_pair(((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u, 1032.0f);
  return join8(p);
}
// the low (H = 0) or high nibbles of eight bytes: keys 0, 2, 1, 3, 4, 6, 5, 7
template <int H>
__device__ __forceinline__ h16x8 codes8_q4_half(u32x2 w) {
  h16x2 p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p[i] = code_pair(((w[i >> 1] >> (4 * H + 8 * (i & 1))) & 0x000F000Fu) | 0x64006400u, 1032.0f);
  return join8(p);
}

// Eight numbers as fp16, and (LO) what the rounding left as fp16 too.  The first part
// passes through a register the compiler cannot look into: it would otherwise round
// some uses of it from the product's exact value and others from the product's fp32
// one, and the remainder would belong to the other.
template <bool LO>
__device__ __forceinline__ void split8(const float (&p)[8], h16x8& hi, h16x8& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = __builtin_bit_cast(uint32_t, h16x2{(_Float16)p[2 * i], (_Float16)p[2 * i + 1]});
    if constexpr (LO) {
      asm("" : "+v"(h[i]));
      const h16x2 x = __builtin_bit_cast(h16x2, h[i]);
      l[i] = __builtin_bit_cast(uint32_t, h16x2{(_Float16)(p[2 * i] - (float)x[0]), (_Float16)(p[2 * i + 1] - (float)x[1])});
    }
  }
  hi = __builtin_bit_cast(h16x8, u32x4{h[0], h[1], h[2], h[3]});
  if constexpr (LO) lo = __builtin_bit_cast(h16x8, u32x4{l[0], l[1], l[2], l[3]});
}

// 2, 3 or 4 words, as aligned as their number allows (unrolled: `words` is known)
__device__ __forceinline__ void load_words(const uint8_t* p, int words, uint32_t* w) {
  if (words == 4) {
    const u32x4 x = *(const u32x4*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = x[i];
  } else if (words == 2) {
    const u32x2 x = *(const u32x2*)p;
    w[0] = x[0];
    w[1] = x[1];
  } else {
    for (int i = 0; i < words; ++i) w[i] = ((const uint32_t*)p)[i];
  }
}

// Key blocks (of 64 keys) that some row of a tile can see, in the part [lo, hi) of
// the keys: a first run [a, b) and a second [c, d); step i is block i + a, then on
// from c.
struct AttnSteps {
  int a, n1, c, total;
  __device__ __forceinline__ int block(int i) const { return i < n1 ? a + i : c + i - n1; }
};

__device__ __forceinline__ AttnSteps attn_steps(const AttnArgs& A, int part_lo, int part_hi, int min_pos, int max_pos,
                                                int max_len, int max_pfx) {
  AttnSteps s;
  const int end = min(part_hi, max_len);
  int hi = A.causal ? min(end, max_pos + 1) : end;
  int lo = A.window > 0 ? max(part_lo, min_pos - (int)A.window + 1) : part_lo;
  lo = max(lo, part_lo);
  const int pfx = min(end, max_pfx);
  s.a = part_lo / ATTN_STEP;
  const int b = pfx > part_lo ? (pfx + ATTN_STEP - 1) / ATTN_STEP : s.a;
  s.n1 = b - s.a;
  s.c = max(lo / ATTN_STEP, b);
  const int d = hi > part_lo ? (hi + ATTN_STEP - 1) / ATTN_STEP : s.c;
  s.total = s.n1 + max(0, d - s.c);
  return s;
}

// What a workgroup's tile belongs to: its sequence (-1: the rows of all, shared part) and
// that sequence's query tokens [q0, q1), keys and prefix.
struct AttnSeq {
  int seq, q0, q1, len, pfx;
};
__device__ __forceinline__ AttnSeq seq_facts(const AttnArgs& A, int seq) {
  AttnSeq s;
  s.seq = seq;
  s.q0 = min(max(A.q_start[seq], 0), A.n_tok);
  s.q1 = min(max(A.q_start[seq + 1], s.q0), A.n_tok);
  s.len = min(max(A.kv_len[seq], 0), A.max_kv);
  s.pfx = A.prefix_len ? min(max(A.prefix_len[seq], 0), s.len) : 0;
  return s;
}
// Sequence i's tiles start at tile q_start[i] * group / ROWS + i (floor): the starts grow
// by at least one per sequence and leave room for every sequence's last, partly filled
// tile.  A wave counts the starts at or below `tile`, 64 sequences at a time, with all
// that is to be known of them loaded at once.
template <int ROWS>
__device__ __forceinline__ AttnSeq seq_of_tile(const AttnArgs& A, int tile, int lane) {
  AttnSeq s = {0, 0, 0, 0, 0};
  for (int i0 = 0; i0 < A.n_seq; i0 += 64) {
    const int i = min(i0 + lane, A.n_seq - 1);
    const int a = A.q_start[i], b = A.q_start[i + 1], n = A.kv_len[i], p = A.prefix_len ? A.prefix_len[i] : 0;
    const int q0 = min(max(a, 0), A.n_tok);
    const uint64_t at = __ballot(i0 + lane < A.n_seq && q0 * A.group / ROWS + i <= tile);
    const int c = __popcll(at);
    if (c > 0 || i0 == 0) {
      const int w = max(c - 1, 0);
      s.seq = i0 + w;
      s.q0 = __builtin_amdgcn_readlane(q0, w);
      s.q1 = min(max(__builtin_amdgcn_readlane(b, w), s.q0), A.n_tok);
      s.len = min(max(__builtin_amdgcn_readlane(n, w), 0), A.max_kv);
      s.pfx = min(max(__builtin_amdgcn_readlane(p, w), 0), s.len);
    }
    if (c < 64) break;
  }
  return s;
}
// the sequence that token `tok` belongs to: the last i with q_start[i] <= tok
__device__ __forceinline__ int seq_of_token(const AttnArgs& A, int tok) {
  int lo = 0, hi = A.n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (A.q_start[mid] <= tok) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
// query rows of a sequence
__device__ __forceinline__ int seq_rows(const AttnArgs& A, int seq) {
  const int q0 = min(max(A.q_start[seq], 0), A.n_tok), q1 = min(max(A.q_start[seq + 1], q0), A.n_tok);
  return (q1 - q0) * A.group;
}

// One row: its token and head (within the KV head's group), its position, how many keys
// it has and how many of them everyone sees.
struct AttnRow {
  int tok, head;
  int pos, len, pfx;
  bool real;
};
// n / group: the host's multiplier is right for n < 2^30
__device__ __forceinline__ int by_group(const AttnArgs& A, int n) { return (int)(((uint64_t)(uint32_t)n * A.group_mul) >> 40); }
// Row `at` of a tile that starts at row `first`; rows past the end repeat the last one and
// are not real.
__device__ __forceinline__ AttnRow attn_row(const AttnArgs& A, const AttnSeq& s, int first, int at) {
  AttnRow r;
  const int n = (s.q1 - s.q0) * A.group;
  int i = first + at;
  r.real = i >= 0 && i < n;
  i = max(0, min(i, n - 1));
  const int t = by_group(A, i);
  r.tok = s.q0 + t;
  r.head = i - t * A.group;
  r.len = s.len;
  r.pfx = s.pfx;
  r.pos = s.len - (s.q1 - s.q0) + t;
  return r;
}
// the same of the shared part's rows, which are of many sequences: every lane looks its own up
__device__ __forceinline__ void own_seq(const AttnArgs& A, AttnRow& r) {
  const AttnSeq s = seq_facts(A, seq_of_token(A, r.tok));
  r.len = s.len;
  r.pfx = s.pfx;
  r.pos = s.len - (s.q1 - s.q0) + (r.tok - s.q0);
}
__device__ __forceinline__ AttnSeq all_rows(const AttnArgs& A) {
  return {-1, 0, min(max(A.q_start[A.n_seq], 0), A.n_tok), 0, 0};
}

// The keys a row sees of the part [lo, hi): key >= lo, and either above < key < below
// or key < pfx.
struct AttnSeen {
  int above, below, pfx;
};
__device__ __forceinline__ AttnSeen seen_by(const AttnArgs& A, const AttnRow& r, int part_hi) {
  AttnSeen s;
  s.below = min(r.len, part_hi);
  s.pfx = min(r.pfx, part_hi);
  if (A.causal) s.below = min(s.below, r.pos + 1);
  s.above = A.window > 0 ? r.pos - (int)A.window : -1;
  return s;
}
// What any row of a tile sees.  Slots outside may hold anything (no key, a page that a window
// has left behind): V's scales there count as zero, since 0 * NaN would reach every row and
// a large one would set the unit of p.  Of a sequence's rows, whose windows overlap, exactly
// the keys some row sees; of the shared keys, which are all stored, perhaps more.  The
// arguments are the same in all lanes.
__device__ __forceinline__ AttnSeen seen_by_any(const AttnArgs& A, int min_pos, int max_pos, int max_len, int max_pfx, int part_hi) {
  AttnSeen s;
  s.below = min(max_len, part_hi);
  s.pfx = min(max_pfx, s.below);
  if (A.causal) s.below = min(s.below, max_pos + 1);
  s.above = A.window > 0 ? min_pos - (int)A.window : -1;
  return {__builtin_amdgcn_readfirstlane(s.above), __builtin_amdgcn_readfirstlane(s.below), __builtin_amdgcn_readfirstlane(s.pfx)};
}
// by bits, not by branches: a select per score
__device__ __forceinline__ bool sees(const AttnSeen& s, int part_lo, int key) {
  return (key >= part_lo) & (((key > s.above) & (key < s.below)) | (key < s.pfx));
}

// eight scales of keys key .. key+7: those that `s` does not hold count as zero
__device__ __forceinline__ void only_seen(u32x4& d, const AttnSeen& s, int part_lo, int key) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    d[k] &= (sees(s, part_lo, key + 2 * k) ? 0xFFFFu : 0u) | (sees(s, part_lo, key + 2 * k + 1) ? 0xFFFF0000u : 0u);
}

__device__ __forceinline__ int page_at(const int32_t* row, int col, int cols, int n_pages) {
  const int p = row[min(col, cols - 1)];
  return min(max(p, 0), n_pages - 1);   // ids outside the pool are clamped, never followed
}

// q rows as matrix operands: a power of two brings the largest element of a row to [2^10,
// 2^11), so that an fp16 (and, for fp32 rows, a second one of the remainder) holds every
// element to 2^-24 of the largest.  A negative scale turns q's sign, so that the scores'
// factor is positive and their maximum can be taken before it.  A row with an element that is
// not finite becomes NaN throughout, and so its output, however its keys are split.
// Returns the factor (the scale and the power back).
template <int NB, bool LO>
__device__ __forceinline__ float q_operands(const AttnArgs& A, float (&x)[NB][8], h16x8 (&hi)[NB], h16x8 (&lo)[LO ? NB : 1]) {
  uint32_t most = 0;   // the largest magnitude's bits: infinity lies above the numbers, NaN above that
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(x[b][e]) & 0x7FFFFFFFu);
  most = groups_umax(most);
  const bool finite = most < 0x7F800000u;
  const int ex = most > 0 && finite ? min(max(11 - __builtin_amdgcn_frexp_expf(__uint_as_float(most)), -120), 120) : 0;
  const float up = finite ? __builtin_ldexpf(A.scale < 0.0f ? -1.0f : 1.0f, ex) : NAN;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[b][e] *= up;
    split8<LO>(x[b], hi[b], lo[LO ? b : 0]);
  }
  return fabsf(A.scale) * __builtin_ldexpf(1.0f, -ex);
}

// ---------------------------------------------------------------------------
// up to 16 query rows per workgroup, its waves taking the 64-key blocks in turn
//
// One pass with a running maximum and sum per row (in powers of two); the waves' states
// meet in LDS at the end, those of splits in attn_join_kernel.  The rows are the query
// heads of a KV head (and the few tokens of its sequence), so that each code is read once:
// bound by HBM on long contexts (32 ragged sequences of 512 to 8192 keys, 8 KV heads of
// 128 in Q8_0: 79 us with the join, 3.8 TB/s; 2 of 100000 to 131071, V in Q4_0: 84 us, 4.6
// TB/s; a large copy 5.0), by latency on short ones (777 keys: 8 us and the join's 3).  Codes
// go from memory to registers in the order of a matrix operand, one step ahead, with no
// pass through LDS: each is used by one wave only.  K's scale multiplies a block's
// product, V's the probability, so the codes are exact operands.  Where a load was issued
// by a branch the compiler spilled and waited (batch 112 -> 176 us): loads past the last
// step repeat it.
// Rows of 16 bits round p times V's scale to one fp16: half a step of 2^-11 per term, against
// the output's own (errors against 64 bits, fp16 outputs: 2.7e-4 of the root mean square, where
// products in fp32 throughout leave 2.1e-4; bf16 ones 1.7e-3 both).  A pair as fp32 rows have
// costs 5 to 10 % (batch 72.5 -> 78.4 us, head size 256 186 -> 205).
// ---------------------------------------------------------------------------
template <int TK, int TV, int NB, int NW, bool LO>
__global__ void __launch_bounds__(64 * NW, NB <= 4 || NW > 4 ? 2 : 1)
attn_step_kernel(AttnArgs A) {
  constexpr int D = NB * 32;
  using C = KvCodes<TK>;
  constexpr int NG = (NB + C::GROUP - 1) / C::GROUP;
  constexpr int VT = TV == FT_Q8_0 ? 2 * NB : NB;            // 16-row pieces of V^T
  constexpr int SC = 2 * NB * 8, SL = (SC + 63) / 64;        // 16-byte pieces of a step's scales, per lane
  __shared__ __align__(16) float s_o[NW][16][D + 4];
  __shared__ float s_m[NW][16], s_l[NW][16];
  __shared__ u32x4 s_sc[NW][SL * 64];                        // a step's scales: K's [NB][64], V's [NB][64]
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int col = lane & 15, g = lane >> 4;
  const int tile = blockIdx.x / (unsigned)A.n_kv_head, hk = blockIdx.x - tile * A.n_kv_head;
  // the part of the keys: those that all share (the first splits, where there are any of
  // them in this launch), or the sequence's own
  const bool shared = A.shared_part || (int)blockIdx.y < A.shared_splits;
  const int split = shared ? (int)blockIdx.y : (int)blockIdx.y - A.shared_splits;
  const int per_split = shared && A.shared_splits ? A.shared_steps : A.split_steps;
  if (shared && A.shared_splits && tile >= A.shared_tiles) return;

  AttnSeq sq;
  int first = tile * 16;
  if (A.step_rows) {   // beside the tile kernel: the sequences of at most step_rows rows
    const unsigned per = A.step_rows / 16;
    sq = seq_facts(A, (int)((unsigned)tile / per));
    first = (int)((unsigned)tile % per) * 16;
    if ((sq.q1 - sq.q0) * A.group > A.step_rows) return;
  } else if (shared) {
    sq = all_rows(A);
  } else {
    sq = seq_of_tile<16>(A, tile, lane);
    first = (tile - (sq.q0 * A.group / 16 + sq.seq)) * 16;
  }
  AttnRow row = attn_row(A, sq, first, col);
  if (!__ballot(row.real)) return;   // a tile past its sequence's rows
  if (shared) own_seq(A, row);

  const int min_pos = row_min(row.pos), max_pos = row_max(row.pos);
  const int min_len = row_min(row.len), max_len = row_max(row.len);
  const int min_pfx = row_min(row.pfx), max_pfx = row_max(row.pfx);
  const int part_lo = shared ? 0 : A.n_shared, part_hi = shared ? A.n_shared : A.max_kv;
  const AttnSeen seen = seen_by(A, row, part_hi);
  AttnSteps steps = attn_steps(A, part_lo, part_hi, min_pos, max_pos, max_len, max_pfx);
  // the same in all lanes: in scalar registers, which takes back what the masks of unseen keys
  // cost short calls (16 drafts 17.1 us against 17.6, head size 64 batch in Q4_0 42.0 against
  // 43.7; the other kernel spills for it: fp16 prompts 514 against 502)
  steps = {__builtin_amdgcn_readfirstlane(steps.a), __builtin_amdgcn_readfirstlane(steps.n1), __builtin_amdgcn_readfirstlane(steps.c),
           __builtin_amdgcn_readfirstlane(steps.total)};
  const int s_end = min(steps.total, (split + 1) * per_split);
  const int s0 = split * per_split + wave;
  const int s_last = s0 + (s_end - 1 - s0) / NW * NW;   // this wave's last step (where there is one)
  const int32_t* pages = A.table + (int64_t)max(sq.seq, 0) * A.table_ld;

  const int page_mask = A.page - 1;
  const int hb_k = kv_head_bytes(TK, D, A.page), hb_v = kv_head_bytes(TV, D, A.page);
  const int cb_k = kv_code_bytes(TK, D, A.page), cb_v = kv_code_bytes(TV, D, A.page);
  const uint32_t pb_k = (uint32_t)A.n_kv_head * hb_k, pb_v = (uint32_t)A.n_kv_head * hb_v;   // under 2^30
  const uint8_t *k_head = A.k_pages + (uint32_t)hk * hb_k, *v_head = A.v_pages + (uint32_t)hk * hb_v;

  // Lane row r = col holds key (r/4)*16 + 4t + r%4 of score tile t, so that the four scores
  // a lane group gets of every tile are its own 16 keys 16g .. 16g+15.  Scales: piece
  // lane + 64 i is eight keys of one block and side.
  const int my_k = (col >> 2) * 16 + (col & 3), my_v = 16 * g, my_s = 8 * (lane & 7);
  struct Ids { int k, v, s; };
  const auto ids_of = [&](int i) {
    const int key0 = steps.block(i) * ATTN_STEP;
    return Ids{page_at(pages, (key0 + my_k) >> A.page_shift, A.cols, A.n_pages),
               page_at(pages, (key0 + my_v) >> A.page_shift, A.cols, A.n_pages),
               page_at(pages, (key0 + my_s) >> A.page_shift, A.cols, A.n_pages)};
  };
  uint32_t kcode[4][NB * C::CB / 4];
  u32x4 vcode[VT], sc[SL];
  const auto load_scales = [&](int i, const Ids& id) {
    const int j = (steps.block(i) * ATTN_STEP + my_s) & page_mask;
#pragma unroll
    for (int n = 0; n < SL; ++n) {
      const int p = min(lane + 64 * n, SC - 1);   // lanes past the pieces repeat the last
      const int b = (p >> 3) % NB;
      const uint8_t* src = p < NB * 8 ? k_head + (uint64_t)(uint32_t)id.s * pb_k + cb_k : v_head + (uint64_t)(uint32_t)id.s * pb_v + cb_v;
      sc[n] = *(const u32x4*)(src + 2 * (b * A.page + j));
    }
  };
  const auto load_k = [&](int i, const Ids& id) {
    const int j = (steps.block(i) * ATTN_STEP + my_k) & page_mask;
    const uint8_t* src = k_head + (uint64_t)(uint32_t)id.k * pb_k;
#pragma unroll
    for (int p = 0; p < NG; ++p) {
      const int words = (NB - p * C::GROUP < C::GROUP ? NB - p * C::GROUP : C::GROUP) * C::CB / 4;
      const uint8_t* at = src + A.page * 64 * p + (4 * j + g) * words * 4;
#pragma unroll
      for (int t = 0; t < 4; ++t) load_words(at + 64 * t * words, words, &kcode[t][p * C::GROUP * C::CB / 4]);
    }
  };
  const auto load_v = [&](int i, const Ids& id) {
    const uint8_t* at = v_head + (uint64_t)(uint32_t)id.v * pb_v + ((steps.block(i) * ATTN_STEP + my_v) & page_mask) + col * A.page;
#pragma unroll
    for (int d = 0; d < VT; ++d) vcode[d] = *(const u32x4*)(at + 16 * d * A.page);
  };

  const int head = hk * A.group + row.head;
  float x[NB][8];
  Ids id = {0, 0, 0};
  if (s0 < s_end) id = ids_of(s0);
  kv_load_row<NB>(A.ftype, A.q, row.tok * A.q_token + head * A.q_head + 8 * g, A.q_vec, x);
  const float slope = A.slopes ? A.slopes[head] * LOG2E : 0.0f;
  if (s0 < s_end) {
    load_scales(s0, id);
    load_k(s0, id);
    load_v(s0, id);
    id = ids_of(min(s0 + NW, s_last));
  }
  h16x8 qh[NB], ql[LO ? NB : 1];
  const float c1 = q_operands<NB, LO>(A, x, qh, ql);
  const bool capped = A.softcap > 0.0f, plain = !capped && !A.slopes;
  const float c0 = score_factor<LO>(c1, A.softcap), cap = A.softcap * LOG2E;
  const float k0 = plain ? c0 : 1.0f;   // the factor can wait for the exponent

  float m = NO_MAX, l = 0.0f;
  f32x4 o[2 * NB];
#pragma unroll
  for (int i = 0; i < 2 * NB; ++i) o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const AttnSeen any = seen_by_any(A, min_pos, max_pos, max_len, max_pfx, part_hi);

  // Each load goes out as soon as its registers are free, a step (of this wave) ahead;
  // behind the last step the last one is loaded again (a branch around the loads costs
  // registers on both its sides: spills, 112 -> 176 us at 64 x 4096 keys).
  for (int i = s0; i < s_end; i += NW) {
    const int next = min(i + NW, s_last);
    const int key0 = steps.block(i) * ATTN_STEP, last = key0 + ATTN_STEP - 1;
    const int kg = key0 + 16 * g;
    const bool all = key0 >= part_lo && last < min(min_len, part_hi) &&
                     (((!A.causal || last <= min_pos) && (!A.window || key0 > max_pos - (int)A.window)) || last < min_pfx);
    // by some row; expected, so that the masks stay behind a branch (in every step: batch 83 us for 80)
    const bool all_seen = key0 >= part_lo && key0 > any.above && last < any.below;
    // scales through LDS (the wave's own); those of keys that no row sees count as zero
    uint32_t top_d = 0;
#pragma unroll
    for (int n = 0; n < SL; ++n) {
      const int p = lane + 64 * n;
      if (__builtin_expect(!all_seen, 0)) only_seen(sc[n], any, part_lo, key0 + my_s);
      if (p >= NB * 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) top_d = max(top_d, max(sc[n][k] & 0x7FFFu, (sc[n][k] >> 16) & 0x7FFFu));
      }
      s_sc[wave][p] = sc[n];
    }
    top_d = wave_umax(top_d);
    wave_lds_sync();
    const u32x4 *kd = &s_sc[wave][2 * g], *vd = &s_sc[wave][NB * 8 + 2 * g];
    load_scales(next, id);

    // scores: s[t][e] of key kg + 4t + e
    f32x4 s[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) s[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const u32x4 d[2] = {kd[8 * b], kd[8 * b + 1]};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        h16x8 a;
        if constexpr (TK == FT_Q8_0) a = codes8_q8(u32x2{kcode[t][2 * b], kcode[t][2 * b + 1]});
        else a = codes8_q4(kcode[t][b]);
        f32x4 y = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, qh[b], f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
        if constexpr (LO) y = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ql[b], y, 0, 0, 0);
        const h16x2 d0 = halves(d[t >> 1][2 * (t & 1)]), d1 = halves(d[t >> 1][2 * (t & 1) + 1]);
        s[t][0] = fmaf((float)d0[0], y[0], s[t][0]);
        s[t][1] = fmaf((float)d0[1], y[1], s[t][1]);
        s[t][2] = fmaf((float)d1[0], y[2], s[t][2]);
        s[t][3] = fmaf((float)d1[1], y[3], s[t][3]);
      }
    }
    load_k(next, id);
    if (!plain) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] *= c0;
      if (capped) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][e] = capped_score<LO>(s[t][e], cap);
      }
      if (A.slopes) {
        const float away = (float)(row.pos - kg);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][e] -= slope * fabsf(away - (float)(4 * t + e));
      }
    }
    if (!all) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] = sees(seen, part_lo, kg + 4 * t + e) ? s[t][e] : -INFINITY;
    }
    // with C = 29 - the fp16 exponent of the step's largest V scale, exp2(s - m) * d stays
    // below 2^15 where m is at least the largest score minus C
    const float lift = (float)(29 - (int)(top_d >> 10));
    float top = s[0][0];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, s[t][e]);
    top = groups_max(top) * k0;
    const float mn = fmaxf(m, top - lift);
    if (__ballot(mn != m)) {
      const float al = __builtin_amdgcn_exp2f(m - mn);
      l *= al;
#pragma unroll
      for (int n = 0; n < 2 * NB; ++n) o[n] *= al;
      m = mn;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[t][e] = __builtin_amdgcn_exp2f(fmaf(s[t][e], k0, -m));
        l += s[t][e];
      }
    // o += V^T p: p times V's scale of (key, block) as fp16 (fp32 rows: and its remainder)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {   // keys 16g + 8h .. + 7
        const u32x4 dw = vd[8 * b + h];
        float p[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = s[2 * h + (k >> 2)][k & 3] * (float)halves(dw[k >> 1])[k & 1];
        if constexpr (TV == FT_Q4_0) {   // its codes come as keys 0, 2, 1, 3
          float y = p[1]; p[1] = p[2]; p[2] = y;
          y = p[5]; p[5] = p[6]; p[6] = y;
        }
        h16x8 ph, pl;
        split8<LO>(p, ph, pl);
#pragma unroll
        for (int d2 = 0; d2 < 2; ++d2) {
          h16x8 a;
          if constexpr (TV == FT_Q8_0) a = codes8_q8(u32x2{vcode[2 * b + d2][2 * h], vcode[2 * b + d2][2 * h + 1]});
          else if (d2 == 0) a = codes8_q4_half<0>(u32x2{vcode[b][2 * h], vcode[b][2 * h + 1]});
          else a = codes8_q4_half<1>(u32x2{vcode[b][2 * h], vcode[b][2 * h + 1]});
          o[2 * b + d2] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ph, o[2 * b + d2], 0, 0, 0);
          if constexpr (LO) o[2 * b + d2] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pl, o[2 * b + d2], 0, 0, 0);
        }
      }
    }
    load_v(next, id);
    id = ids_of(min(next + NW, s_last));
    wave_lds_sync();   // the scales are read before the next step's take their place
  }

  // the waves' states meet in LDS: rows of D floats per wave, and (m, l) per wave and row
  l = groups_sum(l);
  if (g == 0) {
    s_m[wave][col] = m;
    s_l[wave][col] = l;
  }
  if (row.real) {
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) *(f32x4*)&s_o[wave][col][16 * i + 4 * g] = o[i];
  }
  lds_barrier();
  // 4 NW threads per row, four consecutive elements each at a time
  constexpr int TR = 4 * NW;
  const int r = threadIdx.x / TR, e0 = (threadIdx.x % TR) * 4;
  float M = s_m[0][r];
#pragma unroll
  for (int w = 1; w < NW; ++w) M = fmaxf(M, s_m[w][r]);
  float f[NW], L = 0.0f;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    f[w] = __builtin_amdgcn_exp2f(s_m[w][r] - M);
    L += f[w] * s_l[w][r];
  }
  const AttnRow out = attn_row(A, sq, first, r);
  if (!out.real) return;
  const int oh = hk * A.group + out.head;
  if (A.part_o) {
    const int64_t at = A.step_rows ? ((int64_t)sq.seq * A.step_rows + first + r) * A.n_kv_head + hk : (int64_t)out.tok * A.n_head + oh;
    const int64_t ps = (A.split0 + (int)blockIdx.y) * A.part_rows + at;
    if (threadIdx.x % TR == 0) {
      A.part_ml[2 * ps] = L != 0.0f ? M : NO_MAX;
      A.part_ml[2 * ps + 1] = L;
    }
    if (L == 0.0f) return;   // no key seen: the join skips it (NaN it takes)
    for (int e = e0; e < D; e += 4 * TR) {
      f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < NW; ++w) x += f[w] * *(const f32x4*)&s_o[w][r][e];
      *(f32x4*)(A.part_o + ps * D + e) = x;
    }
    return;
  }
  const float inv = L != 0.0f ? 1.0f / L : 0.0f;
  for (int e = e0; e < D; e += 4 * TR) {
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < NW; ++w) x += f[w] * *(const f32x4*)&s_o[w][r][e];
    const float y[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
    kv_store_n<4>(A.ftype, A.out, out.tok * A.out_token + oh * A.out_head + e, A.out_vec, y);
  }
}

// ---------------------------------------------------------------------------
// many query rows: NW waves of 16 * CT rows each over the same keys
//
// The same sums as above; a step's codes become fp16 operands in LDS once for all rows of
// the workgroup, double buffered, laid out as the matrix unit takes them (operand_slot).
//   fp32 rows: q and p as pairs of fp16, four products in place of two;
//   fp16 rows: K's scales on the products, p times V's scale rounded to fp16, as above (a
//     pair: prompts 513 -> 620 us, head size 256 1020 -> 1240);
//   bf16 rows: K's scales in the operand (fp16, a power of two per key apart), p and its
//     product with V's scale in fp16: no fp32 work per block, and an eighth of the output's
//     own rounding each.  V's scales are held to 2^-25 of the largest of the 64 keys.
// Bound by vector instructions, not by the matrix unit (busy a quarter to a third of the
// time): 4096 bf16 tokens over 16384 keys of 8 heads of 128 take 1290 us, 850 TFLOP/s; ragged
// causal prompts of 2239 to 4096 tokens 380 to 400 us, with a cap 475 us (two exponentials and
// a reciprocal per score); an fp32 chunk of 1000 tokens over 7000 keys 300 to 315 us, 345
// TFLOP/s of the result and twice that of fp16 products.  Figures of two forms below were
// taken in turn in one run; from run to run these kernels differ by up to 8 %.
// Two row operands per wave (CT = 2) halve the layout's share for bf16 at head size 128
// (423 us against 461); fp16 and fp32 rows then spill (1066 us against 535), other head
// sizes gain nothing.
// ---------------------------------------------------------------------------
// natural key order: the low (H = 0) or high nibbles of eight bytes
template <int H>
__device__ __forceinline__ h16x8 codes8_q4_bytes(u32x2 w) {
  h16x2 p[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = (w[i] >> (4 * H)) & 0x0F0F0F0Fu;
    p[2 * i] = code_pair(__builtin_amdgcn_perm(0x64646464u, x, 0x04010400u), 1032.0f);
    p[2 * i + 1] = code_pair(__builtin_amdgcn_perm(0x64646464u, x, 0x04030402u), 1032.0f);
  }
  return join8(p);
}
// 2^n as fp16, -15 <= n <= 15, in both halves
__device__ __forceinline__ h16x2 pow2_pair(int n) {
  const uint32_t h = n >= -14 ? (uint32_t)(n + 15) << 10 : 0x0200u;
  return __builtin_bit_cast(h16x2, h | (h << 16));
}
__device__ __forceinline__ h16x8 times(h16x8 a, h16x2 f) {   // by pairs
  return a * __builtin_shufflevector(f, f, 0, 1, 0, 1, 0, 1, 0, 1);
}

constexpr int PREC_BF16 = 0, PREC_F16 = 1, PREC_F32 = 2;
// 16-bit rows under a cap above 512 take the fp32 rows' kernels (both forms of the cap in the
// 16-bit kernels cost them registers, and all their calls 2 to 5 %: fp16 prompts 501 -> 526 us)
constexpr float WIDE_CAP = 512.0f;
inline int attn_prec(const AttnArgs& a) {
  return a.ftype == FT_F32 || a.softcap > WIDE_CAP ? PREC_F32 : a.ftype == FT_F16 ? PREC_F16 : PREC_BF16;
}

// Where lane (g, r) of an operand lies in its 1 KB.  LDS serves a 16-byte access in
// groups of 16 lanes that take quads 0, 3 of lane group 0 with quads 1, 2 of group 1
// (and so on): turning the quads of group g by 0, 3, 2, 1 keeps such reads on different
// banks, and puts the four lane groups of one row or key, which one write holds side by
// side, on different banks too (in order they would meet on one).
__device__ __forceinline__ int operand_slot(int g, int r) { return g * 16 + (r ^ (((-g) & 3) * 4)); }

template <int NB>
struct TileLds {
  u32x4 k[2][4][NB][64];          // K operands: [key tile][block][lane]
  u32x4 v[2][2 * NB][2][64];      // V operands: [16 rows of V^T][key half][lane]
  uint16_t vd[2][NB][64];         // V's scales
  uint16_t kd[2][NB][64];         // K's scales (fp16, fp32 rows)
  float kf[2][64];                // K's power of two per key (bf16 rows)
  uint32_t vmax[2];               // largest |scale| of V in the step
};

template <int TK, int TV, int NB, int NW, int CT, int PREC>
__global__ void __launch_bounds__(64 * NW, CT == 1 && (NB <= 3 || (NB == 4 && PREC != PREC_F32)) ? 4 : 2)
attn_tile_kernel(AttnArgs A) {
  constexpr int D = NB * 32, T = 64 * NW, ROWS = NW * 16 * CT;
  constexpr bool LO = PREC == PREC_F32;
  using C = KvCodes<TK>;
  constexpr int NG = (NB + C::GROUP - 1) / C::GROUP;
  constexpr int KU = (NG * 256 + T - 1) / T;                       // K units per thread
  constexpr int VR = TV == FT_Q8_0 ? D : D / 2;
  constexpr int VU = (VR * 4 + T - 1) / T;                         // V units per thread
  __shared__ TileLds<NB> L;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int col = lane & 15, g = lane >> 4;
  // the last tiles first: under the causal mask they have the most keys
  const int back = blockIdx.x / (unsigned)A.n_kv_head, hk = blockIdx.x - back * A.n_kv_head;
  const int tile = (int)A.tiles - 1 - back, split = blockIdx.y;

  AttnSeq sq;
  int first = tile * ROWS;
  if (A.shared_part) {
    sq = all_rows(A);
  } else {
    sq = seq_of_tile<ROWS>(A, tile, lane);
    first = (tile - (sq.q0 * A.group / ROWS + sq.seq)) * ROWS;
    if (A.step_rows && (sq.q1 - sq.q0) * A.group <= A.step_rows) return;   // the other kernel's
  }
  if (!attn_row(A, sq, first, 0).real) return;
  // what the whole workgroup's rows can see (row 0 and the last are the extremes of a
  // sequence; rows of many sequences are looked at one by one)
  AttnRow row[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    row[c] = attn_row(A, sq, first, (wave * CT + c) * 16 + col);
    if (A.shared_part) own_seq(A, row[c]);
  }
  int lo_pos = row[0].pos, hi_pos = row[0].pos, lo_len = row[0].len, hi_len = row[0].len, lo_pfx = row[0].pfx, hi_pfx = row[0].pfx;
#pragma unroll
  for (int c = 1; c < CT; ++c) {
    lo_pos = min(lo_pos, row[c].pos);
    hi_pos = max(hi_pos, row[c].pos);
    lo_len = min(lo_len, row[c].len);
    hi_len = max(hi_len, row[c].len);
    lo_pfx = min(lo_pfx, row[c].pfx);
    hi_pfx = max(hi_pfx, row[c].pfx);
  }
  const int min_pos = row_min(lo_pos), max_pos = row_max(hi_pos), min_len = row_min(lo_len), max_len = row_max(hi_len);
  const int min_pfx = row_min(lo_pfx), max_pfx = row_max(hi_pfx);
  __shared__ int s_ext[4][NW];
  if (lane == 0) {
    s_ext[0][wave] = min_pos;
    s_ext[1][wave] = max_pos;
    s_ext[2][wave] = max_len;
    s_ext[3][wave] = max_pfx;
  }
  __syncthreads();
  int w_min_pos = s_ext[0][0], w_max_pos = s_ext[1][0], w_max_len = s_ext[2][0], w_max_pfx = s_ext[3][0];
#pragma unroll
  for (int w = 1; w < NW; ++w) {
    w_min_pos = min(w_min_pos, s_ext[0][w]);
    w_max_pos = max(w_max_pos, s_ext[1][w]);
    w_max_len = max(w_max_len, s_ext[2][w]);
    w_max_pfx = max(w_max_pfx, s_ext[3][w]);
  }
  const int part_lo = A.shared_part ? 0 : A.n_shared, part_hi = A.shared_part ? A.n_shared : A.max_kv;
  AttnSeen seen[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) seen[c] = seen_by(A, row[c], part_hi);
  int pos[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) pos[c] = row[c].pos;
  const AttnSteps steps = attn_steps(A, part_lo, part_hi, w_min_pos, w_max_pos, w_max_len, w_max_pfx);
  const int s0 = split * A.split_steps, s_end = min(steps.total, s0 + A.split_steps);
  const int32_t* pages = A.table + (int64_t)max(sq.seq, 0) * A.table_ld;

  h16x8 qh[CT][NB];
  h16x8 ql[LO ? CT : 1][LO ? NB : 1];
  float c0[CT];
  __shared__ int s_tok[NW][CT][16], s_head[NW][CT][16];   // where the rows go; -1: nowhere
  __shared__ float s_slope[NW][CT][16];
  const bool capped = A.softcap > 0.0f;
  const float cap = A.softcap * LOG2E;
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int head = hk * A.group + row[c].head;
    float x[NB][8];
    kv_load_row<NB>(A.ftype, A.q, row[c].tok * A.q_token + head * A.q_head + 8 * g, A.q_vec, x);
    const float c1 = q_operands<NB, LO>(A, x, qh[c], ql[LO ? c : 0]);
    c0[c] = score_factor<LO>(c1, A.softcap);
    if (g == 0) {
      s_tok[wave][c][col] = row[c].real ? row[c].tok : -1;
      s_head[wave][c][col] = head;
      s_slope[wave][c][col] = A.slopes ? A.slopes[head] * LOG2E : 0.0f;
    }
  }

  float m[CT], l[CT];
  f32x4 o[CT][2 * NB];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    m[c] = NO_MAX;
    l[c] = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) o[c][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const int page_mask = A.page - 1;
  const int hb_k = kv_head_bytes(TK, D, A.page), hb_v = kv_head_bytes(TV, D, A.page);
  const int cb_k = kv_code_bytes(TK, D, A.page), cb_v = kv_code_bytes(TV, D, A.page);
  const uint32_t pb_k = (uint32_t)A.n_kv_head * hb_k, pb_v = (uint32_t)A.n_kv_head * hb_v;   // under 2^30
  const uint8_t *k_head = A.k_pages + (uint32_t)hk * hb_k, *v_head = A.v_pages + (uint32_t)hk * hb_v;
  // TIGHT, where the 128 registers of two workgroups per CU are short: the compiler must not
  // keep over the loop what follows from the thread's number, as a spilled value's reload
  // waits for every load in flight (64 bf16 prompts of 70 tokens over 1700 keys: 354 us
  // against 425; fp32 at head size 96 560 against 588; no gain elsewhere).
  // AHEAD: page ids are known a step before the loads that need them, which otherwise wait
  // for the loads before them (fp32 378 us against 407); for fp16 at head size 128 the
  // registers for it cost more (549 us against 531).
  constexpr bool TIGHT = CT == 1 && ((NB == 3 && PREC == PREC_F32) || (NB == 4 && PREC == PREC_BF16));
  constexpr bool AHEAD = !(NB == 4 && PREC == PREC_F16);
  const auto raw_page = [&](int key) { return pages[min(key >> A.page_shift, A.cols - 1)]; };
  const auto pool_page = [&](int id) { return (uint32_t)min(max(id, 0), A.n_pages - 1); };   // clamped, never followed

  const int slot = operand_slot(g, col);
  // this thread's part of a step: K units (group p of blocks, key j, lane group kg_) and V
  // units (row of V^T, 16 keys 16 * vg_ ..)
  struct Part {
    int tid, lane, j, kg, vg;
  };
  const auto my_part = [&] {
    int x = tid;
    if constexpr (TIGHT) asm volatile("" : "+v"(x));
    return Part{x, x & 63, (x >> 2) & 63, x & 3, x & 3};
  };
  uint32_t kw[KU][4];
  uint16_t ksc[PREC == PREC_BF16 ? NB : 1];
  u32x4 vw[VU], sc;
  int id_k, id_v, id_s;
  const auto fetch_ids = [&](int key0) {
    const Part my = my_part();
    id_k = raw_page(key0 + my.j);
    id_v = raw_page(key0 + 16 * my.vg);
    id_s = raw_page(key0 + 8 * (my.lane & 7));
  };
  const auto fetch = [&](int key0) {
    const auto [tid, lane, j, kg_, vg_] = my_part();
    const int key = key0 + j, keyv = key0 + 16 * vg_;
    if constexpr (!AHEAD) fetch_ids(key0);
    const uint8_t* kc = k_head + (uint64_t)pool_page(id_k) * pb_k;
    const uint8_t* vc = v_head + (uint64_t)pool_page(id_v) * pb_v;
#pragma unroll
    for (int i = 0; i < KU; ++i) {
      const int p = (tid + i * T) >> 8;   // uniform over a wave
      if (p < NG) {
        const uint8_t* src = kc + A.page * 64 * p;
        if (NB % C::GROUP == 0 || p < NG - 1) {
          constexpr int W = (NB < C::GROUP ? NB : C::GROUP) * C::CB / 4;
          load_words(src + ((key & page_mask) * 4 + kg_) * W * 4, W, kw[i]);
        } else {
          constexpr int W = (NB % C::GROUP) * C::CB / 4;
          load_words(src + ((key & page_mask) * 4 + kg_) * W * 4, W, kw[i]);
        }
      }
    }
    if constexpr (PREC == PREC_BF16) {
#pragma unroll
      for (int b = 0; b < NB; ++b) ksc[b] = *(const uint16_t*)(kc + cb_k + 2 * (b * A.page + (key & page_mask)));
    }
#pragma unroll
    for (int i = 0; i < VU; ++i) {
      const int r = (tid + i * T) >> 2;
      if (VR * 4 % T == 0 || r < VR) vw[i] = *(const u32x4*)(vc + r * A.page + (keyv & page_mask));
    }
    if (wave < (PREC == PREC_BF16 ? 1 : 2) && lane < NB * 8) {   // the scales, eight keys per lane: V's, and K's
      const int kk = key0 + 8 * (lane & 7), b = lane >> 3;
      const uint64_t pg = pool_page(id_s);
      const uint8_t* src = wave == 0 ? v_head + pg * pb_v + cb_v : k_head + pg * pb_k + cb_k;
      sc = *(const u32x4*)(src + 2 * (b * A.page + (kk & page_mask)));
    }
  };
  const AttnSeen any = seen_by_any(A, w_min_pos, w_max_pos, w_max_len, w_max_pfx, part_hi);
  const auto commit = [&](int buf, int key0) {
    const auto [tid, lane, j, kg_, vg_] = my_part();
    const int r = (j >> 4) * 4 + (j & 3), t = (j >> 2) & 3;   // key j's row and tile
    h16x2 df[PREC == PREC_BF16 ? NB : 1];
    if constexpr (PREC == PREC_BF16) {
      // the key's scales as multiples of a power of two that takes the largest to [1, 2)
      uint32_t top = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b) top = max(top, (uint32_t)ksc[b] & 0x7FFFu);
      const int e = min((int)(top >> 10), 30);
      const h16x2 f = pow2_pair(15 - e);
#pragma unroll
      for (int b = 0; b < NB; ++b) df[b] = __builtin_bit_cast(h16x2, (uint32_t)ksc[b] * 0x00010001u) * f;
      if (tid < 256 && kg_ == 0) L.kf[buf][j] = __uint_as_float((uint32_t)(e - 15 + 127) << 23);
    }
#pragma unroll
    for (int i = 0; i < KU; ++i) {
      const int p = (tid + i * T) >> 8;
      if (p < NG) {
#pragma unroll
        for (int q = 0; q < C::GROUP; ++q) {
          const int b = p * C::GROUP + q;
          if (b < NB) {
            h16x8 a;
            if constexpr (TK == FT_Q8_0) a = codes8_q8(u32x2{kw[i][2 * q], kw[i][2 * q + 1]});
            else a = codes8_q4(kw[i][q]);
            if constexpr (PREC == PREC_BF16) {
              h16x2 d = df[q];
#pragma unroll
              for (int pp = 1; pp < NG; ++pp)
                if (p == pp && pp * C::GROUP + q < NB) d = df[pp * C::GROUP + q < NB ? pp * C::GROUP + q : 0];
              a = times(a, d);
            }
            L.k[buf][t][b][operand_slot(kg_, r)] = __builtin_bit_cast(u32x4, a);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < VU; ++i) {
      const int vr = (tid + i * T) >> 2;
      if (VR * 4 % T == 0 || vr < VR) {
        const u32x2 w0 = {vw[i][0], vw[i][1]}, w1 = {vw[i][2], vw[i][3]};
        if constexpr (TV == FT_Q8_0) {
          const int at = operand_slot(vg_, vr & 15);
          L.v[buf][vr >> 4][0][at] = __builtin_bit_cast(u32x4, codes8_q8(w0));
          L.v[buf][vr >> 4][1][at] = __builtin_bit_cast(u32x4, codes8_q8(w1));
        } else {
          const int at = operand_slot(vg_, vr & 15), b = vr >> 4;
          L.v[buf][2 * b][0][at] = __builtin_bit_cast(u32x4, codes8_q4_bytes<0>(w0));
          L.v[buf][2 * b][1][at] = __builtin_bit_cast(u32x4, codes8_q4_bytes<0>(w1));
          L.v[buf][2 * b + 1][0][at] = __builtin_bit_cast(u32x4, codes8_q4_bytes<1>(w0));
          L.v[buf][2 * b + 1][1][at] = __builtin_bit_cast(u32x4, codes8_q4_bytes<1>(w1));
        }
      }
    }
    if (wave == 0) {
      const int kk = key0 + 8 * (lane & 7), b = lane >> 3;
      uint32_t top = 0;
      const bool all_seen = key0 >= part_lo && key0 > any.above && key0 + ATTN_STEP <= any.below;   // by some row
      if (__builtin_expect(!all_seen, 0)) only_seen(sc, any, part_lo, kk);
      if (lane < NB * 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, max(sc[k] & 0x7FFFu, (sc[k] >> 16) & 0x7FFFu));
      }
      top = wave_umax(top);
      if (lane == 0) L.vmax[buf] = top;
      if constexpr (PREC == PREC_BF16)   // as multiples of a power of two: the largest is in [1, 2)
        sc = __builtin_bit_cast(u32x4, times(__builtin_bit_cast(h16x8, sc), pow2_pair(15 - min((int)(top >> 10), 30))));
      if (lane < NB * 8) *(u32x4*)&L.vd[buf][b][8 * (lane & 7)] = sc;
    } else if (PREC != PREC_BF16 && wave == 1) {
      if (lane < NB * 8) *(u32x4*)&L.kd[buf][lane >> 3][8 * (lane & 7)] = sc;
    }
  };

  // A step's keys are fetched during the step before it and laid out at its end, between two
  // barriers.  Where one workgroup fills a CU (ALONE) half of its waves, which share the
  // SIMDs with the other half, lay out a step earlier, before their products in place of
  // after them, so that one half's matrix instructions run beside the other's vector
  // instructions (4096 bf16 rows over 16384 keys: 1379 us against 1445, fp32 causal prompts
  // 732 against 767).  Two workgroups are out of step already (fp16 the same to 2 % slower).
  constexpr bool ALONE = CT == 2 || NB == 8 || (NB == 4 && PREC == PREC_F32);
  const bool late = ALONE && wave >= NW / 2;
  const auto get = [&](int i) {
    if (i >= s_end) return;
    fetch(steps.block(i) * ATTN_STEP);
    if constexpr (AHEAD) fetch_ids(steps.block(min(i + 1, s_end - 1)) * ATTN_STEP);
  };
  const auto lay_out = [&](int i) {
    if (i < s_end) commit((i - s0) & 1, steps.block(i) * ATTN_STEP);
  };
  if constexpr (AHEAD) {
    if (s0 < s_end) fetch_ids(steps.block(s0) * ATTN_STEP);
  }
  get(s0);
  lay_out(s0);
  if constexpr (ALONE) {
    get(s0 + 1);
    lds_barrier();
    if (late) {
      lay_out(s0 + 1);
      get(s0 + 2);
    }
  }
  for (int i = s0; i < s_end; ++i) {
    const int buf = (i - s0) & 1;
    const int key0 = steps.block(i) * ATTN_STEP;
    if constexpr (!ALONE) {
      lds_barrier();
      get(i + 1);
    }
    // the products first where waves compete (fp32 chunk: 351 us against 360)
    if constexpr (LO) __builtin_amdgcn_s_setprio(1);
    const int last = key0 + ATTN_STEP - 1;
    {
      const bool all = key0 >= part_lo && last < min(min_len, part_hi) &&
                       (((!A.causal || last <= min_pos) && (!A.window || key0 > max_pos - (int)A.window)) || last < min_pfx);
      const int kg = key0 + 16 * g;
      f32x4 s[CT][4];
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int t = 0; t < 4; ++t) s[c][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      // ALONE, which leaves registers for it: a block's operands are read from LDS while the
      // one before is multiplied, V's first ones ahead of the softmax (fp32 chunk 332 us
      // against 365; head size 256 825, 1026 and 1334 us against 836, 1072 and 1370; 4096 bf16
      // rows 1318 against 1344; elsewhere it spills or gains nothing)
      u32x4 ka[ALONE ? 2 : 1][4], kd[ALONE ? 2 : 1][2];
      const auto read_k = [&](int b) {
        const int to = ALONE ? b & 1 : 0;
        if constexpr (ALONE) {
#pragma unroll
          for (int t = 0; t < 4; ++t) ka[to][t] = L.k[buf][t][b][slot];
        }
        if constexpr (PREC != PREC_BF16) {
          kd[to][0] = *(const u32x4*)&L.kd[buf][b][16 * g];
          kd[to][1] = *(const u32x4*)&L.kd[buf][b][16 * g + 8];
        }
      };
      if constexpr (ALONE) read_k(0);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (!ALONE) read_k(b);
        else if (b + 1 < NB) read_k(b + 1);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const h16x8 a = __builtin_bit_cast(h16x8, ALONE ? ka[b & 1][t] : L.k[buf][t][b][slot]);
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            if constexpr (PREC == PREC_BF16) {
              s[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, qh[c][b], s[c][t], 0, 0, 0);
            } else {
              f32x4 x = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, qh[c][b], f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
              if constexpr (LO) x = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ql[c][b], x, 0, 0, 0);
              const u32x4 d = kd[ALONE ? b & 1 : 0][t >> 1];
              const h16x2 d0 = halves(d[2 * (t & 1)]), d1 = halves(d[2 * (t & 1) + 1]);
              s[c][t][0] = fmaf((float)d0[0], x[0], s[c][t][0]);
              s[c][t][1] = fmaf((float)d0[1], x[1], s[c][t][1]);
              s[c][t][2] = fmaf((float)d1[0], x[2], s[c][t][2]);
              s[c][t][3] = fmaf((float)d1[1], x[3], s[c][t][3]);
            }
          }
        }
        if constexpr (PREC != PREC_BF16) __builtin_amdgcn_sched_barrier(0);
      }
      u32x4 va[2][2][2], vd[2][2];
      const auto read_v = [&](int b) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          vd[b & 1][h] = *(const u32x4*)&L.vd[buf][b][16 * g + 8 * h];
#pragma unroll
          for (int d2 = 0; d2 < 2; ++d2) va[b & 1][h][d2] = L.v[buf][2 * b + d2][h][slot];
        }
      };
      if constexpr (ALONE) read_v(0);
      if constexpr (LO) __builtin_amdgcn_s_setprio(0);
      const int ev = min((int)(L.vmax[buf] >> 10), 30);
      const float lift = (float)(29 - ev);
      if constexpr (PREC == PREC_BF16) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const f32x4 kf = *(const f32x4*)&L.kf[buf][16 * g + 4 * t];
#pragma unroll
          for (int c = 0; c < CT; ++c) s[c][t] *= kf;
        }
      }
      h16x8 ph[PREC == PREC_BF16 ? CT : 1][2];
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        float top = -INFINITY;
        const bool plain = !capped && !A.slopes;   // the factor can wait for the exponent
        if (!plain) {
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[c][t][e] *= c0[c];
          if (capped) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[c][t][e] = capped_score<LO>(s[c][t][e], cap);
          }
          if (A.slopes) {
            const float far = (float)(pos[c] - kg), slope = s_slope[wave][c][col];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[c][t][e] -= slope * fabsf(far - (float)(4 * t + e));
          }
        }
        if (!all) {
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[c][t][e] = sees(seen[c], part_lo, kg + 4 * t + e) ? s[c][t][e] : -INFINITY;
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, s[c][t][e]);
        const float k0 = plain ? c0[c] : 1.0f;
        top = groups_max(top) * k0;
        const float mn = fmaxf(m[c], top - lift);
        if (__ballot(mn != m[c])) {
          const float al = __builtin_amdgcn_exp2f(m[c] - mn);
          l[c] *= al;
#pragma unroll
          for (int i2 = 0; i2 < 2 * NB; ++i2) o[c][i2] *= al;
          m[c] = mn;
        }
        // bf16 rows: p in units that the scales below 2 leave under 2^15
        const float shift = PREC == PREC_BF16 ? (float)(ev - 15) - m[c] : -m[c];
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[c][t][e] = __builtin_amdgcn_exp2f(fmaf(s[c][t][e], k0, shift));
            sum += s[c][t][e];
          }
        if constexpr (PREC == PREC_BF16) {
          l[c] = fmaf(sum, __uint_as_float((uint32_t)(15 - ev + 127) << 23), l[c]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 8; ++k) ph[c][h][k] = (_Float16)s[c][2 * h + (k >> 2)][k & 3];
        } else {
          l[c] += sum;
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (ALONE && b + 1 < NB) read_v(b + 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4 dw = ALONE ? vd[b & 1][h] : *(const u32x4*)&L.vd[buf][b][16 * g + 8 * h];
          h16x8 hi[CT], lo[LO ? CT : 1];
          if constexpr (PREC == PREC_BF16) {
            const h16x8 d = __builtin_bit_cast(h16x8, dw);
#pragma unroll
            for (int c = 0; c < CT; ++c) hi[c] = ph[c][h] * d;
          } else {
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              float p[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const h16x2 d = halves(dw[k >> 1]);
                p[k] = s[c][2 * h + (k >> 2)][k & 3] * (float)d[k & 1];
              }
              split8<LO>(p, hi[c], lo[LO ? c : 0]);
            }
          }
#pragma unroll
          for (int d2 = 0; d2 < 2; ++d2) {
            const h16x8 a = __builtin_bit_cast(h16x8, ALONE ? va[b & 1][h][d2] : L.v[buf][2 * b + d2][h][slot]);
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              o[c][2 * b + d2] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, hi[c], o[c][2 * b + d2], 0, 0, 0);
              if constexpr (LO) o[c][2 * b + d2] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, lo[c], o[c][2 * b + d2], 0, 0, 0);
            }
          }
        }
        if constexpr (PREC != PREC_BF16) __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (ALONE) {
      if (late) lds_barrier();
      lay_out(i + 1 + (late ? 1 : 0));
      get(i + 2 + (late ? 1 : 0));
      if (!late) lds_barrier();
    } else {
      lay_out(i + 1);
    }
  }

  wave_lds_sync();   // s_tok and s_head, also of a workgroup that has no step and so no barrier
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const float L_ = groups_sum(l[c]);
    const int tok = s_tok[wave][c][col], oh = s_head[wave][c][col];
    if (tok < 0) continue;
    if (A.part_o) {
      const int64_t ps = (A.split0 + split) * A.part_rows + (int64_t)tok * A.n_head + oh;
      if (g == 0) *(f32x2*)(A.part_ml + 2 * ps) = f32x2{L_ != 0.0f ? m[c] : NO_MAX, L_};
      if (L_ == 0.0f) continue;
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i) *(f32x4*)(A.part_o + ps * D + 16 * i + 4 * g) = o[c][i];
    } else {
      const float inv = L_ != 0.0f ? 1.0f / L_ : 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i) {
        const float y[4] = {o[c][i][0] * inv, o[c][i][1] * inv, o[c][i][2] * inv, o[c][i][3] * inv};
        kv_store_n<4>(A.ftype, A.out, tok * A.out_token + oh * A.out_head + 16 * i + 4 * g, A.out_vec, y);
      }
    }
  }
}

// the tile kernel: rows of a workgroup with one 16-row operand per wave, or with two (wide)
constexpr int TILE_WAVES = 8, TILE_ROWS = 16 * TILE_WAVES;
// where two fit the registers
constexpr bool tile_has_wide(int prec, int nb) { return prec == PREC_BF16 && nb == 4; }

template <int TK, int TV, int NB, int PREC>
static hipError_t tile_launch(const AttnArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.tiles * a.n_kv_head), a.n_split);
  if constexpr (tile_has_wide(PREC, NB)) {
    if (a.tile_wide) {
      attn_tile_kernel<TK, TV, NB, TILE_WAVES, 2, PREC><<<grid, 64 * TILE_WAVES, 0, st>>>(a);
      return hipGetLastError();
    }
  }
  attn_tile_kernel<TK, TV, NB, TILE_WAVES, 1, PREC><<<grid, 64 * TILE_WAVES, 0, st>>>(a);
  return hipGetLastError();
}

template <int TK, int TV, int NB>
static hipError_t attn_launch(const AttnArgs& a, hipStream_t st) {
  const int prec = attn_prec(a);
  if (a.tile_kernel) {
    if (prec == PREC_F32) return tile_launch<TK, TV, NB, PREC_F32>(a, st);
    if (prec == PREC_F16) return tile_launch<TK, TV, NB, PREC_F16>(a, st);
    return tile_launch<TK, TV, NB, PREC_BF16>(a, st);
  }
  const dim3 grid((unsigned)(a.tiles * a.n_kv_head), a.n_split);
  if (NB <= 4 && a.eight) {   // eight waves for a few blocks of keys: one launch, nothing to join
    constexpr int B = NB <= 4 ? NB : 4;
    if (prec == PREC_F32) attn_step_kernel<TK, TV, B, 8, true><<<grid, 512, 0, st>>>(a);
    else attn_step_kernel<TK, TV, B, 8, false><<<grid, 512, 0, st>>>(a);
    return hipGetLastError();
  }
  if (prec == PREC_F32) attn_step_kernel<TK, TV, NB, 4, true><<<grid, 256, 0, st>>>(a);
  else attn_step_kernel<TK, TV, NB, 4, false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

template <int NB>
static hipError_t attn_pick(const AttnArgs& a, hipStream_t st) {
  if (a.k_type == FT_Q8_0)
    return a.v_type == FT_Q8_0 ? attn_launch<FT_Q8_0, FT_Q8_0, NB>(a, st) : attn_launch<FT_Q8_0, FT_Q4_0, NB>(a, st);
  return a.v_type == FT_Q8_0 ? attn_launch<FT_Q4_0, FT_Q8_0, NB>(a, st) : attn_launch<FT_Q4_0, FT_Q4_0, NB>(a, st);
}

}  // namespace ftk
