// ft_attn.hip -- attention over the cache: which kernel takes which rows, how the keys
// are split, and the join of the parts.
#include <algorithm>
#include <cmath>

#include "ft_attn_kernels.h"

namespace ftk {

// One row's parts into its output: with M = max m, o = sum exp2(m - M) o_part / sum
// exp2(m - M) l; a part whose l is NaN makes the row NaN.  A wave per row: a lane per part for m and l, then D / 4 lanes per part
// and 64 / (D / 4) parts at a time for o, added up in an order of their own, so the
// result does not depend on which part was done first.  Bound by the latency of the
// loads: all of a row's (m, l) go out at once, then four rounds of parts (31 parts of 80
// rows: 22 us with a thread walking the parts, 6 us so).
template <int D>
__global__ void __launch_bounds__(256)
attn_join_kernel(AttnArgs A, int parts) {
  constexpr int TPR = D / 4, PG = 64 / TPR;
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + wave_id();
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
  const f32x2* ml = (const f32x2*)A.part_ml;
  float M = NO_MAX, L = 0.0f;
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
  const int sub = lane / TPR, e = (lane - sub * TPR) * 4;
  for (int p0 = 0; p0 < parts; p0 += 64) {
    const int p = p0 + lane;
    const f32x2 v = p < parts ? ml[p * A.part_rows + row] : f32x2{NO_MAX, 0.0f};
    const float m = v[1] != 0.0f ? v[0] : NO_MAX;   // a part without keys wrote no row
    const float Mn = fmaxf(M, route_val(wave_umax(route_key(m))));
    const float back = __builtin_amdgcn_exp2f(M - Mn), f = v[1] != 0.0f ? __builtin_amdgcn_exp2f(m - Mn) : 0.0f;
    M = Mn;
    L = L * back + f * v[1];
    x *= back;
    const int n = min(64, parts - p0);
    for (int q0 = 0; q0 < n; q0 += 4 * PG) {
      float w[4];
      f32x4 y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int at = q0 + u * PG + sub;
        w[u] = __shfl(f, min(at, 63), 64);
        y[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (at < n && sub < PG && w[u] != 0.0f) y[u] = *(const f32x4*)(A.part_o + ((p0 + at) * A.part_rows + row) * D + e);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) x += w[u] * y[u];
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) L += __shfl_xor(L, d, 64);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float y = x[k];
#pragma unroll
    for (int s = 1; s < PG; ++s) y += __shfl(x[k], (lane + s * TPR) & 63, 64);   // lanes of the first part group
    x[k] = y;
  }
  if (sub != 0) return;
  const float inv = L != 0.0f ? 1.0f / L : 0.0f;
  const float y[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
  kv_store_n<4>(A.ftype, A.out, tok * A.out_token + head * A.out_head + e, A.out_vec, y);
}

static hipError_t join(const AttnArgs& a, int parts, hipStream_t st) {
  const unsigned grid = (unsigned)((a.part_rows + 3) / 4);
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

// Splits: `want` workgroups, of `least` steps or a few more each (whole rounds of `waves`
// steps where a workgroup's waves take them in turn).  Depends on the host's bounds alone
// (max_kv, not the lengths on the device), so a captured call can be replayed with other
// lengths.
static AttnSplit split_keys(const AttnArgs& a, int64_t tiles, int64_t steps, int64_t want, int64_t least, int64_t waves) {
  const int64_t wgs = std::max<int64_t>(tiles * a.n_kv_head, 1);
  // the join walks the parts 64 at a time (one KV head, 100000 keys: 391 parts 43 us, 128 31,
  // 64 33; 30000 keys: 118 parts 24.5 us, 64 18.9)
  const int64_t most = std::max<int64_t>(64, steps / 12);
  const int64_t n = std::max<int64_t>(1, std::min<int64_t>({(want + wgs - 1) / wgs, (steps + least - 1) / least, most}));
  int64_t per = (steps + n - 1) / n;
  per = std::max<int64_t>(least, (per + waves - 1) / waves * waves);
  // n grows with the steps; the splits it comes to do not always
  return {tiles, (int)std::max<int64_t>(1, (steps + per - 1) / per), (int)per, 0, (int)n};
}

// Time of the tile kernel with n splits of `per` steps, in steps of one CU (256 rows, 64
// keys; 3 to 4 us at head size 128), as measured over 130 to 4000 rows and 130 to 6000
// keys of each type.  A CU holds one workgroup, or two where the registers allow; a step
// of two costs 1 (bf16 rows 1.12 of a wide step), one alone 0.7 of that.  A workgroup's
// start and end take two steps, the join 1.4 and one per 20000 rows of each part.  Under
// the causal mask the workgroups' shares of the keys run from 1 down to 2 seen - 1; whole
// ones start longest first and fill the CUs, the first of several splits are all full.
static double tile_cost(const AttnArgs& a, int prec, int wide, int64_t wgs, int64_t n, int64_t per, double seen) {
  const bool two = !wide && a.dim <= (prec == ftk::PREC_F32 ? 96 : 128);
  const double pair = prec == ftk::PREC_BF16 ? 1.12 : 1.0;
  const double c = wgs * (double)n / 256, rounds = std::ceil(c), least = 2 * seen - 1;
  const double load = n == 1 ? std::max(c * seen, rounds * (1 - (1 - least) * rounds / (2 * c)))
                             : std::min(rounds, c * seen + least);
  const double rate = two ? pair * (0.5 + (std::fmod(rounds, 2) != 0 ? 0.2 * least / rounds : 0.0)) : 1.0;
  const double join = n > 1 ? 1.4 + n * (double)a.n_tok * a.n_head / 20000 : 0.0;
  return ((double)per + 2) * std::max(load * rate, two ? 0.7 * pair : 1.0) + join;
}

AttnPlan ftk_attn_plan(const AttnArgs& a, int most_tile) {
  using namespace ftk;
  AttnPlan p = {};
  constexpr int kStepRows = 32;
  const int64_t rows = (int64_t)a.n_tok * a.group;
  const int prec = attn_prec(a);
  // under a causal window a tile sees the window of its tokens only
  const auto steps = [&](int64_t tile) {
    int64_t span = a.max_kv - a.n_shared;
    if (a.window > 0 && a.causal && !a.prefix_len) span = std::min<int64_t>(span, a.window + tile / a.group + 2);
    return (span + 63) / 64 + 1;   // the first block may start before the span
  };
  const bool many = rows > (int64_t)kStepRows * a.n_seq;   // more rows per sequence than the step kernel is for
  const int64_t part = (a.dim + 2) * sizeof(float);
  const auto tiles = [&](int64_t n_rows, int64_t seqs, bool shared) {
    AttnSplit best = {};
    double best_cost = 0.0;
    for (int wide = 0; wide <= (tile_has_wide(prec, a.dim / 32) ? 1 : 0); ++wide) {
      const int64_t tile = wide ? 2 * TILE_ROWS : TILE_ROWS;
      const int64_t n_tiles = shared ? (n_rows + tile - 1) / tile : n_rows / tile + seqs;
      const int64_t filled = seqs == 1 ? (n_rows + tile - 1) / tile : n_rows / tile + seqs / 2;   // about
      const int64_t n_steps = shared ? (int64_t)a.n_shared / 64 + 1 : steps(tile);
      // under the causal mask a row sees half of its sequence's new tokens on average
      double seen = 1.0;
      if (!shared && a.causal && !a.prefix_len)
        seen -= 0.5 * std::min(n_rows / (64.0 * a.group * seqs), (double)n_steps) / n_steps;
      for (int64_t n = 1, per; n <= n_steps && (shared || n <= most_tile); n = (n_steps + per - 2) / (per - 1)) {
        per = (n_steps + n - 1) / n;
        const double cost = tile_cost(a, prec, wide, filled * a.n_kv_head, n, per, seen);
        if (best.tiles == 0 || cost < best_cost) {
          best = {n_tiles, (int)n, (int)per, wide};
          best_cost = cost;
        }
        if (per <= 4 || n * filled * a.n_kv_head > 2048) break;   // eight rounds of the chip
      }
    }
    return best;
  };
  if (many) p.tile = tiles(rows, a.n_seq, false);
  if (many && a.n_seq > 1 && !a.n_shared) p.step_rows = kStepRows;
  // Two workgroups per CU; twice as many, of eight steps at least, where there are some
  // sequences already but not that many workgroups (32 ragged sequences of 8 heads: 80 us
  // against 86; 8 of them: 28 against 33; two of 100000 keys: 90 against 101 the other way,
  // as each workgroup takes 5 us to start and end)
  const auto step_split = [&](int64_t tiles) {
    const int64_t wgs = tiles * a.n_kv_head;
    return wgs >= 64 && wgs < 512 ? split_keys(a, tiles, steps(16), 1024, 8, 4) : split_keys(a, tiles, steps(16), 512, 4, 4);
  };
  if (p.step_rows) p.step = step_split((int64_t)a.n_seq * (kStepRows / 16));
  else if (!many) p.step = step_split(rows / 16 + a.n_seq);
  // few workgroups with a block for each of eight waves: no split, no join (one user, 250
  // keys: 9.2 us against 11.7; with two rounds, 777 keys, 13.8 against 11.2)
  const AttnSplit whole = {rows / 16 + a.n_seq, 1, (int)steps(16), 0, p.step.most};
  if (!many && !a.n_shared && a.dim <= 128 && p.step.n_split > 1 && whole.tiles * a.n_kv_head <= 256 && whole.split_steps <= 9) {
    p.step = whole;
    p.eight = 1;
  }
  // beside the tile kernel there may be no such sequence at all, and a join would still be
  // launched (three prompts of 130 to 200 tokens: 23.3 us against 25.0; with 64 steps and a
  // short sequence among eight, 79 against 65 the other way)
  if (p.step_rows && a.dim <= 128 && p.step.n_split > 1 && steps(16) <= 16) {
    p.step = {p.step.tiles, 1, (int)steps(16), 0, p.step.most};
    p.eight = 1;
  }
  if (a.n_shared > 0) {
    p.shared_tile = rows > kStepRows;
    p.shared = p.shared_tile ? tiles(rows, 1, true) : split_keys(a, (rows + 15) / 16, a.n_shared / 64 + 1, 512, 4, 4);
  }
  const int64_t all = (int64_t)a.n_tok * a.n_head;
  const auto scratch = [&](int step_split) {
    const int64_t parts = p.shared.n_split + p.tile.n_split + (p.step_rows ? 0 : step_split);
    size_t n = parts > 1 ? (size_t)(parts * all * part) : 0;
    p.step_at = (n + 255) & ~(size_t)255;
    if (p.step_rows && step_split > 1) n = p.step_at + (size_t)((int64_t)step_split * a.n_seq * kStepRows * a.n_kv_head * part);
    return n;
  };
  p.scratch_most = scratch(p.step.most);
  p.scratch = scratch(p.step.n_split);   // and step_at
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
    a.tile_wide = s.wide;
    a.split0 = split0;
    return attn_dim(a, st);
  };
  with_parts(parts, (int64_t)a.n_tok * a.n_head, 0);
  hipError_t e = hipSuccess;
  if (p.shared.tiles && !p.shared_tile && p.step.tiles) {   // both on the step kernel: one launch
    a.shared_splits = p.shared.n_split;
    a.shared_steps = p.shared.split_steps;
    a.shared_tiles = (int)p.shared.tiles;
    AttnSplit s = p.step;
    s.tiles = std::max(p.step.tiles, p.shared.tiles);
    s.n_split += p.shared.n_split;
    e = run(s, 0);
    return e == hipSuccess ? join(a, parts, st) : e;
  }
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
    a.eight = p.eight;
    e = run(p.step, p.step_rows ? 0 : p.shared.n_split);
  }
  const int last = p.step_rows ? p.step.n_split : parts;
  if (e == hipSuccess && last > 1) e = join(a, last, st);
  return e;
}
