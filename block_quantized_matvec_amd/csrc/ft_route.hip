// ft_route.hip -- router with softmax or sigmoid scores over all experts, a bias for
// balance, groups and renormalised weights (ft_moe_route_ex).
//
//   score_e = softmax(x)_e or 1 / (1 + exp(-x_e)),  choice_e = score_e + bias_e;
//   group_g = the sum of its group_top largest choices; the topk_group best groups stay;
//   ids = the topk largest choices among them, ties to the lower index;
//   w = the scores of ids, over their sum where renorm says so, times scale.
//
// The result is that of 64-bit scores and choices: the order of two experts may hang on
// the last bits of an exponential, and in fp64 it depends on the formula alone (fp32
// would reorder neighbours by its own rounding).  Almost always fp32 is enough to know
// that order: route_fast_kernel works in fp32 with a bound of its error, and where two
// neighbours in the order lie closer than the bound (ties among them, groups that are equal
// in fp32) the wave decides that token again in fp64 (route_exact).
//
// Bound by instruction issue and the length of a token's chain, not by HBM: 16384 tokens
// x 256 experts, sigmoid, bias, 8 groups, top 8 (16.8 MB in) take 17 to 18.5 us (10.2 us
// without bias and groups), of which 4 us are the tail of the few tokens that fp64 decides
// (bf16 logits without a bias, where one token in a hundred has three equal ones at the last
// slot: 16.4 us); with every exponential in fp64 and a wave per token 33 us.  3 tokens x 128
// experts: 4.7 us.  More than 14 slots go to the kernels with more lanes per token (top 16
// of 1024, 16384 tokens: 45 us; every token in fp64: 126).
#include "ft_device.h"
#include "ft_internal.h"
#include "ft_kv.h"

namespace ftk {

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}
// order-preserving 64-bit key (-0 folded into +0)
__device__ __forceinline__ uint64_t choice_key(double c) {
  const uint64_t u = (uint64_t)__double_as_longlong(c + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// logit e of a token; a NaN counts as -inf (it is never preferred)
__device__ __forceinline__ float logit_at(const RouteArgs& A, int64_t tok, int e) {
  const int64_t at = tok * A.ld + e;
  float x;
  if (A.ftype == FT_F32) x = ((const float*)A.logits)[at];
  else if (A.ftype == FT_BF16) x = bf16_value(((const uint16_t*)A.logits)[at]);
  else x = h2f(((const uint16_t*)A.logits)[at]);
  return x == x ? x : -INFINITY;
}

// logits e .. e+3 of rows whose quads are aligned
__device__ __forceinline__ f32x4 quad_at(const RouteArgs& A, int64_t tok, int e) {
  if (A.ftype == FT_F32) return *(const f32x4*)((const float*)A.logits + tok * A.ld + e);
  const u32x2 w = *(const u32x2*)((const uint16_t*)A.logits + tok * A.ld + e);
  f32x4 v;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t h = (w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu;
    v[k] = A.ftype == FT_BF16 ? bf16_value(h) : h2f(h);
  }
  return v;
}

// One token by a whole wave in fp64: lane l holds experts l*M .. l*M + M-1, so lane
// order is expert order.  LDS of the wave's own: choices (groups only), w and id.
template <int MAXE>
__device__ __forceinline__ void route_exact(const RouteArgs& A, int64_t tok, double* s_choice, double* s_w, int* s_id) {
  const int lane = threadIdx.x & 63;
  const int E = A.n_expert, M = (E + 63) / 64;
  float x[MAXE];
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < MAXE; ++j) {
    const int e = lane * M + j;
    x[j] = j < M && e < E ? logit_at(A, tok, e) : -INFINITY;
    top = fmaxf(top, x[j]);
  }
  double score[MAXE], choice[MAXE];
  if (A.sigmoid) {
#pragma unroll
    for (int j = 0; j < MAXE; ++j) score[j] = 1.0 / (1.0 + exp(-(double)x[j]));
  } else {
    top = route_val(wave_umax(route_key(top)));
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < MAXE; ++j) {
      score[j] = top > -INFINITY ? exp((double)x[j] - (double)top) : 0.0;
      sum += score[j];
    }
    sum = wave_sum(sum);
    const double r = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
    for (int j = 0; j < MAXE; ++j) score[j] *= r;
  }
#pragma unroll
  for (int j = 0; j < MAXE; ++j) {
    const int e = lane * M + j;
    choice[j] = score[j];
    if (A.bias && j < M && e < E) choice[j] += (double)A.bias[e];
    if (!(choice[j] == choice[j])) choice[j] = -INFINITY;
  }

  uint64_t kept = ~0ull;
  const int S = E / A.n_group;
  if (A.n_group > 1) {
#pragma unroll
    for (int j = 0; j < MAXE; ++j)
      if (j < M) s_choice[lane * M + j] = choice[j];
    wave_lds_sync();
    double a = -INFINITY, b = -INFINITY;   // the group's two largest
    if (lane < A.n_group) {
#pragma unroll 8
      for (int i = 0; i < S; ++i) {
        const double c = s_choice[lane * S + i];
        b = fmax(b, fmin(a, c));
        a = fmax(a, c);
      }
      if (A.group_top == 2 && S > 1) a += b;
    }
    int rank = 0;
    for (int k = 0; k < A.n_group; ++k) {
      const double o = __shfl(a, k, 64);
      rank += o > a || (o == a && k < lane);
    }
    kept = __ballot(lane < A.n_group && rank < A.topk_group);
  }

  uint64_t key[MAXE];
#pragma unroll
  for (int j = 0; j < MAXE; ++j) {
    const int e = lane * M + j;
    const bool in = j < M && e < E && (A.n_group == 1 || ((kept >> (e / S)) & 1));
    key[j] = in ? choice_key(choice[j]) : 0;
  }
  for (int r = 0; r < A.topk; ++r) {
    uint64_t best = 0;
#pragma unroll
    for (int j = 0; j < MAXE; ++j) best = key[j] > best ? key[j] : best;
    const uint32_t hi = wave_umax((uint32_t)(best >> 32));
    const uint32_t lo = wave_umax((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
    const uint64_t most = ((uint64_t)hi << 32) | lo;
    const uint64_t who = __ballot(best == most);
    if (lane == __builtin_ctzll(who)) {
      bool taken = false;
#pragma unroll
      for (int j = 0; j < MAXE; ++j) {
        if (!taken && key[j] == most) {
          taken = true;
          key[j] = 0;
          s_w[r] = score[j];
          s_id[r] = lane * M + j;
        }
      }
    }
  }
  wave_lds_sync();
  double f = A.scale;
  if (A.renorm) {
    double sum = 0.0;
    for (int r = 0; r < A.topk; ++r) sum += s_w[r];
    f = sum > 0.0 ? f / sum : 0.0;
  }
  if (lane < A.topk) {
    A.ids[tok * A.topk + lane] = min(s_id[lane], E - 1);
    A.w[tok * A.topk + lane] = (float)(s_w[lane] * f);
  }
  wave_lds_sync();   // the LDS may be used again
}

// ---------------------------------------------------------------------------
// fp32 with a bound: LANES lanes per token, lane l holds experts 4 (i LANES + l) ..+3,
// i < Q (16-byte loads, a token's lanes side by side).  topk + 2 <= LANES.
//
// With s the largest score and c the largest choice, expert e's key is its distance
// from c in units of s 2^-20 above its index (24 bits and 8 for up to 256 experts, else
// 22 and 10): keys differ, a smaller key is a better choice, or an equal one of a lower
// index, and a round is one minimum over the token's lanes.
//
// A distance is off by at most: the exponent's argument is rounded (|x| 2^-24 relative in
// the exponential, which its own size or 1 - score take back to under 2^-21 s, unless
// every sigmoid's x is under -8: then up to 2^-17 s); exp2 and rcp are within 2^-23 each,
// the softmax's sum within 2^-21; together under 2^-19 s = 2 units (2^-16 s = 16 in the
// exception).  Adding the bias and taking the distance round by 2^-24 of |c| + 16 s, one
// unit and |c| / 16 s; the unit itself half of one.  Two keys that lie `room` = 10 (50) +
// |c| / 4 s units apart are in the right order; where that is over 10^6, a part of the
// range that keys have, the token goes through route_exact.
//
// The rounds go two past topk.  Where neighbours among them are closer than `room`, the
// slots' own 64-bit choices settle their order; only if the one after next to the last
// slot is that close too, or a group kept is that close to one left out, does the whole
// token go through route_exact.
// ---------------------------------------------------------------------------
// value of the lane at distance S (as xchg), as an operand the compiler can fold
template <int S> __device__ __forceinline__ uint32_t near_lane(uint32_t v, uint32_t identity) {
  constexpr int ctrl = S == 1 ? 0xB1 : S == 2 ? 0x4E : S == 4 ? 0x141 : 0x140;
  return (uint32_t)__builtin_amdgcn_update_dpp((int)identity, (int)v, ctrl, 0xF, 0xF, false);
}
template <int LANES> __device__ __forceinline__ uint32_t lanes_umin(uint32_t v) {
  v = min(v, near_lane<1>(v, ~0u));
  v = min(v, near_lane<2>(v, ~0u));
  v = min(v, near_lane<4>(v, ~0u));
  v = min(v, near_lane<8>(v, ~0u));
  if constexpr (LANES >= 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = min((uint32_t)a[0], (uint32_t)a[1]);
  }
  if constexpr (LANES == 64) {
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = min((uint32_t)b[0], (uint32_t)b[1]);
  }
  return v;
}
template <int LANES> __device__ __forceinline__ float lanes_max(float v) {
  return route_val(~lanes_umin<LANES>(~route_key(v)));
}
template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
  v += xchg<1>(v);
  v += xchg<2>(v);
  v += xchg<4>(v);
  v += xchg<8>(v);
#pragma unroll
  for (int d = 16; d < LANES; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}
template <int S> __device__ __forceinline__ double near_lane(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint64_t lo = near_lane<S>((uint32_t)u, 0u), hi = near_lane<S>((uint32_t)(u >> 32), 0u);
  return __longlong_as_double((long long)(lo | (hi << 32)));
}
template <int LANES> __device__ __forceinline__ double lanes_sum(double v) {
  v += near_lane<1>(v);
  v += near_lane<2>(v);
  v += near_lane<4>(v);
  v += near_lane<8>(v);
#pragma unroll
  for (int d = 16; d < LANES; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}
// (a, b): the two largest of this lane's and the partner's
template <int S> __device__ __forceinline__ void top2_with(float& a, float& b) {
  const float oa = xchg<S>(a), ob = xchg<S>(b);
  b = fmaxf(fminf(a, oa), fmaxf(b, ob));
  a = fmaxf(a, oa);
}

// ascending; a lane's four smallest keys
__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {
  const uint32_t lo = min(a, b);
  b = max(a, b);
  a = lo;
}
__device__ __forceinline__ void sort4(uint32_t (&v)[4]) {
  order2(v[0], v[1]);
  order2(v[2], v[3]);
  order2(v[0], v[2]);
  order2(v[1], v[3]);
  order2(v[1], v[2]);
}
// the four smallest of two sorted fours, sorted
__device__ __forceinline__ void merge4(uint32_t (&v)[4], const uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = min(v[i], o[3 - i]);
  order2(v[0], v[2]);
  order2(v[1], v[3]);
  order2(v[0], v[1]);
  order2(v[2], v[3]);
}
// the four smallest of N keys that are past `last`
template <int N>
__device__ __forceinline__ void smallest4(const uint32_t (&key)[N], bool all, uint32_t last, uint32_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    uint32_t q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = all || key[i + k] > last ? key[i + k] : ~0u;
    sort4(q);
    if (i == 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = q[k];
    } else {
      merge4(v, q);
    }
  }
}

template <int LANES, int Q, int MAXE>
__global__ void __launch_bounds__(256)
route_fast_kernel(RouteArgs A) {
  constexpr int TPW = 64 / LANES;   // tokens per wave
  constexpr int N = 4 * Q;
  constexpr int EMAX = LANES * N;
  constexpr int IB = EMAX <= 256 ? 8 : 10;              // bits of the index in a key
  constexpr uint32_t FAR = (1u << (32 - IB)) - 1;       // the largest distance
  // per wave: its tokens' logits; their choices (a word of padding per 32), or what
  // route_exact needs, after all else is done; group values
  constexpr int CW = EMAX + EMAX / 32, XB = 64 * MAXE * 8 + 32 * 8 + 32 * 4, CB = TPW * CW * 4;
  __shared__ __align__(16) float s_x[4 * TPW][EMAX];
  __shared__ __align__(16) uint8_t s_c[4][(CB > XB ? CB : XB) + 15 & ~15];
  __shared__ float s_g[4 * TPW][64];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int l = lane & (LANES - 1), sub = lane / LANES;
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * TPW;
  if (t0 >= A.t) return;
  const int64_t tok = min(t0 + sub, A.t - 1);   // past the end: the last token again, not written
  const bool real = t0 + sub < A.t;
  const int E = A.n_expert;

  // every load goes out before anything is computed
  float x[N], c[N], bias[N];
  if (A.vec) {   // E is a multiple of 4: quads are whole
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int e = 4 * (i * LANES + l), at = e < E ? e : 0;
      const f32x4 v = quad_at(A, tok, at);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[4 * i + k] = v[k];
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = logit_at(A, tok, min(4 * ((j >> 2) * LANES + l) + (j & 3), E - 1));
  }
  if (A.bias) {
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int e = 4 * (i * LANES + l);
      f32x4 v;
      if (A.vec_bias) {
        v = *(const f32x4*)(A.bias + (e < E ? e : 0));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = A.bias[min(e + k, E - 1)];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) bias[4 * i + k] = v[k];
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) bias[j] = 0.0f;
  }
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = 4 * ((j >> 2) * LANES + l) + (j & 3);
    x[j] = EMAX == E || e < E ? fmaxf(x[j], -INFINITY) : -INFINITY;   // a NaN counts as -inf
    top = fmaxf(top, x[j]);
  }
  float* sx = s_x[wave * TPW + sub];
#pragma unroll
  for (int i = 0; i < Q; ++i) *(f32x4*)(sx + 4 * (i * LANES + l)) = f32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
  top = lanes_max<LANES>(top);
  float s, units;   // the largest score; its error in units of s 2^-20, see above
  if (A.sigmoid) {
#pragma unroll
    for (int j = 0; j < N; ++j) c[j] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[j] * -1.44269504f));
    s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(top * -1.44269504f));
    units = top < -8.0f ? 50.0f : 10.0f;
  } else {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      c[j] = __builtin_amdgcn_exp2f((x[j] - top) * 1.44269504f);
      sum += c[j];
    }
    s = __builtin_amdgcn_rcpf(lanes_sum<LANES>(sum));
#pragma unroll
    for (int j = 0; j < N; ++j) c[j] *= s;
    units = 10.0f;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) c[j] += bias[j];
  if (E < EMAX) {
#pragma unroll
    for (int j = 0; j < N; ++j) c[j] = 4 * ((j >> 2) * LANES + l) + (j & 3) < E ? c[j] : -INFINITY;
  }

  bool close = false;   // fp32 cannot settle this token
  if (A.n_group > 1) {
    float* sc = (float*)s_c[wave] + sub * CW;
    float* sg = s_g[wave * TPW + sub];
    const int S = E / A.n_group;
    float big = -INFINITY;
    if ((S & (S - 1)) == 0 && S >= 4 && S <= 64) {   // whole quads of 1, 2 .. 16 neighbouring lanes
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        float a = fmaxf(c[4 * i], c[4 * i + 1]), b = fminf(c[4 * i], c[4 * i + 1]);
        const float a2 = fmaxf(c[4 * i + 2], c[4 * i + 3]), b2 = fminf(c[4 * i + 2], c[4 * i + 3]);
        b = fmaxf(fminf(a, a2), fmaxf(b, b2));
        a = fmaxf(a, a2);
        if (S > 4) top2_with<1>(a, b);
        if (S > 8) top2_with<2>(a, b);
        if (S > 16) top2_with<4>(a, b);
        if (S > 32) top2_with<8>(a, b);
        const int e = 4 * (i * LANES + l);
        if (e < E && (e & (S - 1)) == 0) sg[e / S] = A.group_top == 2 ? a + b : a;
      }
    } else {
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int e = 4 * (i * LANES + l);   // four stay on one side of a multiple of 32
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[e + (e >> 5) + k] = c[4 * i + k];
      }
      wave_lds_sync();
      for (int g = l; g < A.n_group; g += LANES) {
        float a = -INFINITY, b = -INFINITY;
        for (int i = 0; i < S; ++i) {
          const int e = g * S + i;
          const float v = sc[e + (e >> 5)];
          b = fmaxf(b, fminf(a, v));
          a = fmaxf(a, v);
        }
        sg[g] = A.group_top == 2 && S > 1 ? a + b : a;
      }
    }
    wave_lds_sync();
    uint64_t kept = 0;
    const float err = units * (s * 0x1p-19f);   // twice a choice's own
    uint64_t alike = 0;   // groups within both errors of this lane's (or no difference to speak of: infinities)
    for (int g0 = 0; g0 < A.n_group; g0 += LANES) {
      const int g = g0 + l;
      int rank = 0;
      uint64_t with = 0;
      if (g < A.n_group) {
        const float a = sg[g];
#pragma unroll 8
        for (int k = 0; k < A.n_group; ++k) {
          const float o = sg[k];
          rank += o > a;
          with |= (uint64_t)!(fabsf(o - a) > err + (fabsf(o) + fabsf(a)) * 0x1p-22f) << k;
        }
      }
      const uint64_t in = __ballot(g < A.n_group && rank < A.topk_group) >> (sub * LANES);
      kept |= (LANES == 64 ? in : in & ((1ull << (LANES & 63)) - 1)) << g0;
      // with more groups than lanes: any likeness counts
      if (A.n_group <= LANES) alike = with;
      else close |= (with & ~(1ull << (g & 63))) != 0;
    }
    if (l < A.n_group) close |= (alike & (((kept >> (l & 63)) & 1) ? ~kept : kept)) != 0;
    // groups equal in fp32 have one rank: at the border all of them were kept
    close |= __popcll(kept) != A.topk_group;
    if ((S & (S - 1)) == 0 && S >= 4) {   // quads are of one group
      const int shift = 31 - __builtin_clz(S);
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const bool in = (kept >> ((4 * (i * LANES + l)) >> shift & 63)) & 1;
#pragma unroll
        for (int k = 0; k < 4; ++k) c[4 * i + k] = in ? c[4 * i + k] : -INFINITY;
      }
    } else {
      const float rS = 1.0f / (float)S;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = 4 * ((j >> 2) * LANES + l) + (j & 3);
        const int g = (int)(((float)e + 0.5f) * rS);   // exact below 1024
        c[j] = (kept >> (g & 63)) & 1 ? c[j] : -INFINITY;
      }
    }
  }

  float most = -INFINITY;
#pragma unroll
  for (int j = 0; j < N; ++j) most = fmaxf(most, c[j]);
  most = lanes_max<LANES>(most);
  const float inv = __builtin_amdgcn_rcpf(s) * 0x1p20f;
  // no distances without a finite choice and a scale (every logit closed, or infinite)
  close |= !(fabsf(most) < INFINITY && inv < INFINITY && fabsf(top) < INFINITY);
  const float apart = units + fabsf(most) * inv * 0x1p-22f;
  close |= !(apart <= 1e6f);   // scores far below the choice's last bits: no distance tells them apart
  const uint32_t room = (uint32_t)fminf(apart, 1e6f);
  uint32_t key[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = 4 * ((j >> 2) * LANES + l) + (j & 3);
    const float d = fminf(fmaf(c[j], -inv, most * inv), (float)FAR);   // closed: as far as can be
    key[j] = ((uint32_t)d << IB) | (uint32_t)e;
  }
  // Rounds of the smallest; lane r keeps slot r.  A lane has its four smallest in order
  // and gives them up one by one; a lane that runs out (one round in a few tokens) has
  // every lane look for its next four.
  uint32_t mine4[4];
  smallest4<N>(key, true, 0u, mine4);
  uint32_t my_key = ~0u, last = 0;
  int left = 4;
  bool gave = false;
  for (int r = 0; r < A.topk + 2; ++r) {
    const uint32_t best = lanes_umin<LANES>(mine4[0]);
    my_key = l == r ? best : my_key;
    const bool won = mine4[0] == best;
    last = won ? best : last;
    left -= won;
    gave |= won;
#pragma unroll
    for (int k = 0; k < 3; ++k) mine4[k] = won ? mine4[k + 1] : mine4[k];
    mine4[3] = won ? ~0u : mine4[3];
    if (N > 4 && __ballot(left == 0)) {
      // a lane that gave none up yet starts over; for the others keys up to `last` are gone
      smallest4<N>(key, !gave, last, mine4);
      left = 4;
    }
  }

  // the slots' scores in fp64, a slot per lane; softmax: over exp of the largest logit
  wave_lds_sync();
  const uint32_t far = my_key >> IB;
  const bool have = far < FAR;
  const int my_id = min((int)(my_key & ((1u << IB) - 1)), E - 1);
  const float xv = have ? sx[my_id] : 0.0f;
  const double v = (double)xv;
  // The order of the slots, and of the last with the first left out, is open between
  // neighbours that close; but equal logits (16-bit ones often are) without a bias are equal
  // in 64 bits too, and their keys are in the order of the index ...
  const uint32_t before = __shfl_up(far, 1, 64), two_before = __shfl_up(far, 2, 64);
  const bool same = !A.bias && __shfl_up(xv, 1, 64) == xv;
  const bool near = (l > 0) & (l <= A.topk) & (far - before < room) & !same;
  // ... and cannot be settled among the slots: too far to tell, or a third that close
  close |= (far >= FAR) & ((l < A.topk) | ((l == A.topk) & (FAR - before < room)));
  close |= (l == A.topk + 1) & (far - two_before < room);
  double w = A.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - (double)top);
  const bool settle = __ballot(near) != 0;
  if (!A.sigmoid && (!A.renorm || (settle && A.bias))) {
    double sum = 0.0;
#pragma unroll 1
    for (int e = l; e < E; e += LANES) sum += exp((double)sx[e] - (double)top);
    w /= lanes_sum<LANES>(sum);
  }
  int rank = l;
  if (settle) {
    const double mine = A.bias ? w + (double)A.bias[my_id] : w;
    rank = 0;
    for (int k = 0; k < A.topk + 2; ++k) {
      const int from = sub * LANES + k;
      const double o = __shfl(mine, from, 64);
      const int oid = __shfl(have ? my_id : E, from, 64);
      rank += oid < E && (o > mine || (o == mine && oid < my_id));
    }
  }
  const bool slot = have && rank < A.topk && l < A.topk + 2;
  double f = A.scale;
  if (A.renorm) {
    const double sum = lanes_sum<LANES>(slot ? w : 0.0);
    f = sum > 0.0 ? f / sum : 0.0;
  }
  if (slot && real) {
    A.ids[tok * A.topk + rank] = my_id;
    A.w[tok * A.topk + rank] = (float)(w * f);
  }
  const uint64_t again = __ballot(close && real);
  if (again == 0) return;
  wave_lds_sync();
  for (int q = 0; q < TPW; ++q) {
    const uint64_t mask = LANES == 64 ? ~0ull : ((1ull << (LANES & 63)) - 1) << (q * LANES);
    double* sd = (double*)s_c[wave];
    if (again & mask) route_exact<MAXE>(A, t0 + q, sd, sd + 64 * MAXE, (int*)(sd + 64 * MAXE + 32));
  }
}

}  // namespace ftk

hipError_t ftk_launch_route_ex(const RouteArgs& a0, hipStream_t st) {
  using namespace ftk;
  RouteArgs a = a0;
  const int64_t step = a.ftype == FT_F32 ? 4 : 8;   // elements in 16 bytes
  a.vec = ((uintptr_t)a.logits & 15) == 0 && a.ld % step == 0 && a.n_expert % 4 == 0;
  a.vec_bias = ((uintptr_t)a.bias & 15) == 0 && a.n_expert % 4 == 0;
  const int E = a.n_expert;
  const auto grid = [&](int per) { return (unsigned)((a.t + per - 1) / per); };
  if (E <= 256 && (a.t <= 2048 || a.topk > 14)) {   // a wave per token: fewer steps after one another
    route_fast_kernel<64, 1, 4><<<grid(4), 256, 0, st>>>(a);
  } else if (E <= 64) {
    route_fast_kernel<16, 1, 1><<<grid(16), 256, 0, st>>>(a);
  } else if (E <= 128) {
    route_fast_kernel<16, 2, 2><<<grid(16), 256, 0, st>>>(a);
  } else if (E <= 256) {
    route_fast_kernel<16, 4, 4><<<grid(16), 256, 0, st>>>(a);
  } else if (E <= 512 && a.topk <= 30) {
    route_fast_kernel<32, 4, 8><<<grid(8), 256, 0, st>>>(a);
  } else {
    route_fast_kernel<64, 4, 16><<<grid(4), 256, 0, st>>>(a);
  }
  return hipGetLastError();
}
