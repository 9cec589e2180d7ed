// ft_attn.hip -- attention over the cache: how the keys are split, and the join of
// the parts.
#include <algorithm>

#include "ft_attn_kernels.h"

namespace ftk {

// One row's parts into its output: with M = max m, o = sum exp2(m - M) o_part / sum
// exp2(m - M) l, the parts in order, so the result does not depend on which part was
// done first.  D / 4 threads per row, four elements each.
template <int D>
__global__ void __launch_bounds__(256)
attn_join_kernel(AttnArgs A, int parts) {
  constexpr int TPR = D / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = id / TPR;
  const int64_t rows = (int64_t)A.n_tok * A.n_head;
  if (row >= rows) return;
  const int tok = (int)(row / A.n_head), head = (int)(row % A.n_head);
  if (tok < A.q_start[0] || tok >= A.q_start[A.n_seq]) return;   // no sequence's token
  const int e = (int)(id - row * TPR) * 4;
  const f32x2* ml = (const f32x2*)A.part_ml;
  float M = NO_MAX;
  for (int p = 0; p < parts; ++p) M = fmaxf(M, ml[p * rows + row][0]);
  float L = 0.0f;
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const f32x2 v = ml[p * rows + row];
    if (v[1] > 0.0f) {   // a part without keys wrote no row
      const float f = __builtin_amdgcn_exp2f(v[0] - M);
      L += f * v[1];
      x += f * *(const f32x4*)(A.part_o + (p * rows + row) * D + e);
    }
  }
  const float inv = L > 0.0f ? 1.0f / L : 0.0f;
  const float y[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
  kv_store_n<4>(A.ftype, A.out, tok * A.out_token + head * A.out_head + e, A.out_vec, y);
}

template <int D>
static hipError_t join(const AttnArgs& a, int parts, hipStream_t st) {
  const int64_t threads = (int64_t)a.n_tok * a.n_head * (D / 4);
  attn_join_kernel<D><<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(a, parts);
  return hipGetLastError();
}

static hipError_t attn_dim(const AttnArgs& a, hipStream_t st) {
  switch (a.dim) {
    case 64: return ftk_attn_d64(a, st);
    case 96: return ftk_attn_d96(a, st);
    case 128: return ftk_attn_d128(a, st);
    case 256: return ftk_attn_d256(a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace ftk

// Splits: enough workgroups for two on every CU, but four steps (one per wave) at
// least in each.  Depends on the host's bounds alone (max_kv, not the lengths on the
// device), so a captured call can be replayed with other lengths.
static void split_keys(int64_t wgs, int64_t steps, int* n_split, int* split_steps) {
  const int64_t want = 2 * 256;
  int64_t n = std::max<int64_t>(1, std::min<int64_t>((want + wgs - 1) / std::max<int64_t>(wgs, 1), (steps + 3) / 4));
  int64_t per = (steps + n - 1) / n;
  per = std::max<int64_t>(4, (per + 3) / 4 * 4);
  *split_steps = (int)per;
  *n_split = (int)std::max<int64_t>(1, (steps + per - 1) / per);
}

AttnPlan ftk_attn_plan(const AttnArgs& a) {
  AttnPlan p = {};
  p.tiles = (int64_t)a.n_tok * a.group / 16 + a.n_seq;
  int64_t span = a.max_kv - a.n_shared;
  // under a causal window a tile sees the window of its rows (at most 16 tokens) only
  if (a.window > 0 && a.causal && !a.prefix_len) span = std::min<int64_t>(span, a.window + 16 / a.group + 2);
  const int64_t steps = (span + 63) / 64 + 1;   // the first block may start before the span
  split_keys(p.tiles * a.n_kv_head, steps, &p.n_split, &p.split_steps);
  if (a.n_shared > 0) {
    p.shared_tiles = ((int64_t)a.n_tok * a.group + 15) / 16;
    split_keys(p.shared_tiles * a.n_kv_head, (a.n_shared + 63) / 64, &p.shared_splits, &p.shared_steps);
  }
  const int64_t parts = p.n_split + p.shared_splits;
  if (parts > 1) p.scratch = (size_t)parts * a.n_tok * a.n_head * (a.dim + 2) * sizeof(float);
  return p;
}

hipError_t ftk_launch_attn(AttnArgs a, const AttnPlan& p, void* scratch, hipStream_t st) {
  using namespace ftk;
  const int parts = p.n_split + p.shared_splits;
  const int64_t rows = (int64_t)a.n_tok * a.n_head;
  a.part_o = parts > 1 ? (float*)scratch : nullptr;
  a.part_ml = parts > 1 ? (float*)scratch + parts * rows * a.dim : nullptr;
  hipError_t e = hipSuccess;
  if (a.n_shared > 0) {
    a.shared_part = 1;
    a.tiles = p.shared_tiles;
    a.n_split = p.shared_splits;
    a.split_steps = p.shared_steps;
    a.split0 = 0;
    e = attn_dim(a, st);
  }
  a.shared_part = 0;
  a.tiles = p.tiles;
  a.n_split = p.n_split;
  a.split_steps = p.split_steps;
  a.split0 = p.shared_splits;
  if (e == hipSuccess) e = attn_dim(a, st);
  if (e != hipSuccess || parts == 1) return e;
  switch (a.dim) {
    case 64: return join<64>(a, parts, st);
    case 96: return join<96>(a, parts, st);
    case 128: return join<128>(a, parts, st);
    default: return join<256>(a, parts, st);
  }
}
