// ft_attn.hip -- attention over the cache: which kernel takes which rows, how the keys
// are split, and the join of the parts.
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
  if (row >= A.part_rows) return;
  int tok, head;
  if (A.step_rows && !A.tile_kernel) {   // the step kernel's rows: [seq][step_rows][n_kv_head]
    const int64_t i = row / A.n_kv_head;
    const int seq = (int)(i / A.step_rows), r = (int)(i % A.step_rows);
    const int n = seq_rows(A, seq);
    if (n > A.step_rows || r >= n) return;
    tok = min(max(A.q_start[seq], 0), A.n_tok) + r / A.group;
    head = (int)(row % A.n_kv_head) * A.group + r % A.group;
  } else {
    tok = (int)(row / A.n_head);
    head = (int)(row % A.n_head);
    if (tok < A.q_start[0] || tok >= A.q_start[A.n_seq]) return;   // no sequence's token
    if (A.step_rows && seq_rows(A, seq_of_token(A, tok)) <= A.step_rows) return;
  }
  const int e = (int)(id - row * TPR) * 4;
  const f32x2* ml = (const f32x2*)A.part_ml;
  float M = NO_MAX;
  for (int p = 0; p < parts; ++p) M = fmaxf(M, ml[p * A.part_rows + row][0]);
  float L = 0.0f;
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const f32x2 v = ml[p * A.part_rows + row];
    if (v[1] > 0.0f) {   // a part without keys wrote no row
      const float f = __builtin_amdgcn_exp2f(v[0] - M);
      L += f * v[1];
      x += f * *(const f32x4*)(A.part_o + (p * A.part_rows + row) * D + e);
    }
  }
  const float inv = L > 0.0f ? 1.0f / L : 0.0f;
  const float y[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
  kv_store_n<4>(A.ftype, A.out, tok * A.out_token + head * A.out_head + e, A.out_vec, y);
}

static hipError_t join(const AttnArgs& a, int parts, hipStream_t st) {
  const unsigned grid = (unsigned)((a.part_rows * (a.dim / 4) + 255) / 256);
  switch (a.dim) {
    case 64: attn_join_kernel<64><<<grid, 256, 0, st>>>(a, parts); break;
    case 96: attn_join_kernel<96><<<grid, 256, 0, st>>>(a, parts); break;
    case 128: attn_join_kernel<128><<<grid, 256, 0, st>>>(a, parts); break;
    default: attn_join_kernel<256><<<grid, 256, 0, st>>>(a, parts); break;
  }
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

// Splits: `want` workgroups, but `least` steps in each.  Depends on the host's bounds
// alone (max_kv, not the lengths on the device), so a captured call can be replayed
// with other lengths.
static AttnSplit split_keys(const AttnArgs& a, int64_t tiles, int64_t steps, int64_t want, int64_t least) {
  const int64_t wgs = std::max<int64_t>(tiles * a.n_kv_head, 1);
  const int64_t n = std::max<int64_t>(1, std::min<int64_t>((want + wgs - 1) / wgs, steps / least));
  int64_t per = (steps + n - 1) / n;
  per = std::max<int64_t>(least, (per + 3) / 4 * 4);
  return {tiles, (int)std::max<int64_t>(1, (steps + per - 1) / per), (int)per};
}

AttnPlan ftk_attn_plan(const AttnArgs& a) {
  using namespace ftk;
  AttnPlan p = {};
  constexpr int kStepRows = 32;
  const int64_t rows = (int64_t)a.n_tok * a.group;
  constexpr int tile_rows = TILE_ROWS;
  // under a causal window a tile sees the window of its tokens only
  const auto steps = [&](int64_t tile) {
    int64_t span = a.max_kv - a.n_shared;
    if (a.window > 0 && a.causal && !a.prefix_len) span = std::min<int64_t>(span, a.window + tile / a.group + 2);
    return (span + 63) / 64 + 1;   // the first block may start before the span
  };
  const bool many = rows > (int64_t)kStepRows * a.n_seq;   // more rows per sequence than the step kernel is for
  const int64_t part = (a.dim + 2) * sizeof(float);
  if (many) p.tile = split_keys(a, rows / tile_rows + a.n_seq, steps(tile_rows), 512, 8);
  if (many && a.n_seq > 1 && !a.n_shared) p.step_rows = kStepRows;
  if (p.step_rows) p.step = split_keys(a, (int64_t)a.n_seq * (kStepRows / 16), steps(16), 512, 4);
  else if (!many) p.step = split_keys(a, rows / 16 + a.n_seq, steps(16), 512, 4);
  if (a.n_shared > 0) {
    p.shared_tile = rows > kStepRows;
    const int64_t n = a.n_shared / 64 + 1;
    p.shared = p.shared_tile ? split_keys(a, (rows + tile_rows - 1) / tile_rows, n, 512, 8)
                             : split_keys(a, (rows + 15) / 16, n, 512, 4);
  }
  const int64_t all = (int64_t)a.n_tok * a.n_head;
  const int64_t parts = p.shared.n_split + (p.step_rows ? p.tile.n_split : p.tile.n_split + p.step.n_split);
  if (parts > 1) p.scratch = (size_t)(parts * all * part);
  p.step_at = (p.scratch + 255) & ~(size_t)255;
  if (p.step_rows && p.step.n_split > 1)
    p.scratch = p.step_at + (size_t)((int64_t)p.step.n_split * a.n_seq * kStepRows * a.n_kv_head * part);
  return p;
}

hipError_t ftk_launch_attn(AttnArgs a, const AttnPlan& p, void* scratch, hipStream_t st) {
  using namespace ftk;
  const int parts = p.shared.n_split + p.tile.n_split + (p.step_rows ? 0 : p.step.n_split);
  const auto with_parts = [&](int n, int64_t rows, size_t at) {
    a.part_rows = rows;
    a.part_o = n > 1 ? (float*)((uint8_t*)scratch + at) : nullptr;
    a.part_ml = n > 1 ? a.part_o + (int64_t)n * rows * a.dim : nullptr;
  };
  const auto run = [&](const AttnSplit& s, int split0) {
    a.tiles = s.tiles;
    a.n_split = s.n_split;
    a.split_steps = s.split_steps;
    a.split0 = split0;
    return attn_dim(a, st);
  };
  with_parts(parts, (int64_t)a.n_tok * a.n_head, 0);
  hipError_t e = hipSuccess;
  if (p.shared.tiles) {
    a.shared_part = 1;
    a.tile_kernel = p.shared_tile;
    e = run(p.shared, 0);
    a.shared_part = 0;
  }
  a.step_rows = p.step_rows;
  if (e == hipSuccess && p.tile.tiles) {
    a.tile_kernel = 1;
    e = run(p.tile, p.shared.n_split);
  }
  if (e == hipSuccess && parts > 1 && p.step_rows) e = join(a, parts, st);
  if (p.step_rows) with_parts(p.step.n_split, (int64_t)a.n_seq * p.step_rows * a.n_kv_head, p.step_at);
  if (e == hipSuccess && p.step.tiles) {
    a.tile_kernel = 0;
    e = run(p.step, p.step_rows ? 0 : p.shared.n_split);
  }
  const int last = p.step_rows ? p.step.n_split : parts;
  if (e == hipSuccess && last > 1) e = join(a, last, st);
  return e;
}
