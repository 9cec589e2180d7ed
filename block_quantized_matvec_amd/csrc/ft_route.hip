// ft_route.hip -- router with softmax or sigmoid scores over all experts, a bias for
// balance, groups and renormalised weights (ft_moe_route_ex).
//
//   score_e = softmax(x)_e or 1 / (1 + exp(-x_e)),  choice_e = score_e + bias_e;
//   group_g = the sum of its group_top largest choices; the topk_group best groups stay;
//   ids = the topk largest choices among them, ties to the lower index;
//   w = the scores of ids, over their sum where renorm says so, times scale.
//
// Scores and choices are held in 64 bits: the order of two experts may hang on the
// last bits of an exponential, and in fp64 it depends on the formula alone (fp32
// would reorder neighbours by its own rounding).  One wave per token; lane l holds
// experts l*M .. l*M + M-1, so lane order is expert order.
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

// what this wave's lanes wrote to LDS is there for all of them (LDS serves a wave in
// order; the fence keeps the compiler from moving accesses across)
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int MAXE>
__global__ void __launch_bounds__(256)
route_ex_kernel(RouteArgs A) {
  __shared__ double s_choice[4][64 * MAXE];
  __shared__ double s_w[4][32];
  __shared__ int s_id[4][32];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int64_t tok = (int64_t)blockIdx.x * 4 + wave;
  if (tok >= A.t) return;   // no barrier below: a wave meets only itself
  const int E = A.n_expert, M = (E + 63) / 64;

  float x[MAXE];
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < MAXE; ++j) {
    const int e = lane * M + j;
    x[j] = -INFINITY;
    if (j < M && e < E) {
      const int64_t at = tok * A.ld + e;
      if (A.ftype == FT_F32) x[j] = ((const float*)A.logits)[at];
      else if (A.ftype == FT_BF16) x[j] = bf16_value(((const uint16_t*)A.logits)[at]);
      else x[j] = h2f(((const uint16_t*)A.logits)[at]);
      if (!(x[j] == x[j])) x[j] = -INFINITY;   // a NaN is never preferred
    }
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
      if (j < M) s_choice[wave][lane * M + j] = choice[j];
    wave_lds_sync();
    double a = -INFINITY, b = -INFINITY;   // the group's two largest
    if (lane < A.n_group) {
      for (int i = 0; i < S; ++i) {
        const double c = s_choice[wave][lane * S + i];
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
          s_w[wave][r] = score[j];
          s_id[wave][r] = lane * M + j;
        }
      }
    }
  }
  wave_lds_sync();
  double f = A.scale;
  if (A.renorm) {
    double sum = 0.0;
    for (int r = 0; r < A.topk; ++r) sum += s_w[wave][r];
    f = sum > 0.0 ? f / sum : 0.0;
  }
  if (lane < A.topk) {
    A.ids[tok * A.topk + lane] = min(s_id[wave][lane], E - 1);
    A.w[tok * A.topk + lane] = (float)(s_w[wave][lane] * f);
  }
}

}  // namespace ftk

hipError_t ftk_launch_route_ex(const RouteArgs& a, hipStream_t st) {
  using namespace ftk;
  const unsigned grid = (unsigned)((a.t + 3) / 4);
  if (a.n_expert <= 64) route_ex_kernel<1><<<grid, 256, 0, st>>>(a);
  else if (a.n_expert <= 128) route_ex_kernel<2><<<grid, 256, 0, st>>>(a);
  else if (a.n_expert <= 256) route_ex_kernel<4><<<grid, 256, 0, st>>>(a);
  else if (a.n_expert <= 512) route_ex_kernel<8><<<grid, 256, 0, st>>>(a);
  else route_ex_kernel<16><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}
