// ft_rope.hip -- rotary positions: rows of queries or keys turned by their position
// (ft_rope), the same on the way into the paged cache (ft_kv_store_rope), and the table of
// angles (ft_rope_table).
//
// Pair j of a row at position p is the vector (a, b), turned by the angle p * f_j:
//   a' = a cos - b sin,  b' = b cos + a sin,
// every product and sum one fp32 operation (no fused multiply-add: this file is compiled
// without contraction), so that a key's code in the cache does not hang on how a compiler
// pairs them.  cos and sin come from a table with a row per position, rounded once from
// 64-bit angles: at position 131072 an fp32 product p * f is off by 2^-8 of a radian, and in
// 64 bits a sine costs more than all else that a row needs, while its row of the table is
// shared by every head (512 bytes beside the 8 KB of 32 heads of 128 in bf16).
//
// A wave holds 64 / L rows, L lanes of eight elements each (L the power of two from
// dim / 8 on): the rows of that many consecutive tokens of one head, so that keys of
// consecutive slots leave as whole pieces of a page.  The lane keeps its cosines and sines
// for several heads.  A pair's other half comes over LDS (half layout) or lies in the lane
// (neighbours).
//
// Bound by memory: 6000 bf16 tokens of 20 heads of 256 (126 MB) 25 us, 5.0 TB/s, a large copy's rate.
// 8192 tokens of 32 query and 8 key/value heads of 128 in bf16, K to Q8_0 and V to Q4_0 (182 MB): 44 us in one
// launch (14 for the plain store, 27 for as many queries alone); with the values' workgroups
// spread between the others 48.  6000 bf16 tokens of 20 heads of 128, normed (64 MB): 18 us, the norm's 64-bit sums on top of
// the loads.  A table of 131072 positions by 64 pairs (67 MB): 27 us, its sines and cosines in 64 bits.  At a decode step (24 tokens, norms of every head) 3.9 us, the launch and
// three memory latencies: positions and slots, the table's row beside the values, the stores.
#include "ft_kv_store.h"
#include "ft_rowstat.h"

namespace ftk {

constexpr int ROPE_MANY = 4;   // heads per wave, where there are waves enough

struct RopeRows {
  const void* x;
  int64_t x_token, x_head;   // strides in elements
  int heads, chunks;         // chunks: groups of heads that a wave takes together
  int vec;                   // rows stay 16-byte aligned
  const float* weight;       // nullable: the rows are normed first
  int vec_w;
};
struct RopeOut {
  void* x;
  int64_t x_token, x_head;
  int vec;
};
struct RopeTurn {
  const int32_t* pos;
  const float* table;        // [n_pos][rot]: cosines, then sines
  int64_t n_pos, t;
  int dim, rot, log_lanes, interleaved, ftype;
  int vec_t;                 // a lane's cosines are aligned quads of one region
  double eps, inv_dim;
};

// The rows of heads h0 .. h0+HC-1 of token group g: loaded, normed, turned and handed to
// put(head, token, first element, values) by the lanes that hold a row.  s_x: this wave's
// 64 * 8 floats of LDS.
template <int HC, class Put>
__device__ __forceinline__ void rope_rows(const RopeTurn& c, const RopeRows& rows, uint32_t g, int h0, float* s_x, Put&& put) {
  const int lane = threadIdx.x & 63, ls = c.log_lanes;
  const int l = lane & ((1 << ls) - 1), e0 = 8 * l, rot = c.rot, half = rot >> 1;
  const int64_t tok = (int64_t)g * (64 >> ls) + (lane >> ls);
  const bool live = tok < c.t && e0 < c.dim;
  const int64_t tk = min(tok, c.t - 1);   // lanes without a row read one that is there
  const int el = e0 < c.dim ? e0 : 0;
  int64_t p = c.pos[tk];
  const bool whole = (c.dim & 7) == 0;
  u32x4 raw[HC][2];
  if (whole) {
    int64_t at[HC];
#pragma unroll
    for (int n = 0; n < HC; ++n) at[n] = tk * rows.x_token + min(h0 + n, rows.heads - 1) * rows.x_head + el;
    kv_load_raw<HC>(c.ftype, rows.x, at, rows.vec, raw);
  } else {   // the row's last lane holds fewer than eight
#pragma unroll
    for (int n = 0; n < HC; ++n) {
      const int64_t at = tk * rows.x_token + min(h0 + n, rows.heads - 1) * rows.x_head + el;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = 0.0f;
        if (el + i < c.dim) {
          if (c.ftype == FT_F32) v = ((const float*)rows.x)[at + i];
          else if (c.ftype == FT_BF16) v = bf16_value(((const uint16_t*)rows.x)[at + i]);
          else v = h2f(((const uint16_t*)rows.x)[at + i]);
        }
        raw[n][i >> 2][i & 3] = __float_as_uint(v);
      }
    }
  }
  p = p < 0 ? 0 : p >= c.n_pos ? c.n_pos - 1 : p;
  const float* row = c.table + p * rot;
  float w[8];
  if (rows.weight) {
    if (rows.vec_w) kv_load8(FT_F32, rows.weight, el, true, w);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = el + i < c.dim ? rows.weight[el + i] : 0.0f;
  }
  // the lane's cosines, and its sines with the sign of their term
  float cs[8], sn[8];
  if (c.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = 1.0f, sn[i] = 0.0f;
    if (c.vec_t) {
      if (e0 < rot) {
        const f32x4 a = *(const f32x4*)(row + (e0 >> 1)), b = *(const f32x4*)(row + half + (e0 >> 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = a[i], sn[i] = b[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + 2 * i < rot) cs[i] = row[(e0 >> 1) + i], sn[i] = row[half + (e0 >> 1) + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = 1.0f, sn[i] = 0.0f;
    if (c.vec_t) {   // half is a multiple of eight: the lane lies in one half
      if (e0 < rot) {
        const int j = e0 < half ? e0 : e0 - half;
        kv_load8(FT_F32, row, j, true, cs);
        kv_load8(FT_F32, row, half + j, true, sn);
      }
      if (e0 < half)
#pragma unroll
        for (int i = 0; i < 8; ++i) sn[i] = -sn[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        if (e < rot) {
          const int j = e < half ? e : e - half;
          cs[i] = row[j];
          sn[i] = e < half ? -row[half + j] : row[half + j];
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < HC; ++n) {
    if (h0 + n >= rows.heads) break;
    float v[8];
    kv_raw_values(whole ? c.ftype : FT_F32, raw[n], v);
    if (rows.weight) {
      const float r = rstd_of(fma(lanes_sum(e0 < c.dim ? sum_squares(v) : 0.0, ls), c.inv_dim, c.eps));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (v[i] * r) * w[i];
    }
    if (c.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1], x = a * cs[i] - b * sn[i], y = b * cs[i] + a * sn[i];
        if (e0 + 2 * i < rot) v[2 * i] = x, v[2 * i + 1] = y;
      }
    } else {
      float* mine = s_x + 8 * lane;
      *(f32x4*)mine = f32x4{v[0], v[1], v[2], v[3]};
      *(f32x4*)(mine + 4) = f32x4{v[4], v[5], v[6], v[7]};
      wave_lds_sync();
      float o[8];
      const float* base = s_x + 8 * (lane - l);
      if (c.vec_t) {
        const float* other = base + (e0 < half ? e0 + half : e0 < rot ? e0 - half : e0);
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const f32x4 q = *(const f32x4*)(other + i);
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i + k] = q[k];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = e0 + i;
          o[i] = base[e < half ? e + half : e < rot ? e - half : e];
        }
      }
      wave_lds_sync();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = v[i] * cs[i] + o[i] * sn[i];
        if (e0 + i < rot) v[i] = x;
      }
    }
    if (live) put(h0 + n, tok, e0, v);
  }
}

__device__ __forceinline__ void rope_put(const RopeTurn& c, const RopeOut& out, int head, int64_t tok, int e0, const float (&v)[8]) {
  const int64_t at = tok * out.x_token + head * out.x_head + e0;
  if (e0 + 8 <= c.dim) {
    kv_store_n<8>(c.ftype, out.x, at, out.vec, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (e0 + i >= c.dim) break;
    if (c.ftype == FT_F32) ((float*)out.x)[at + i] = v[i];
    else ((uint16_t*)out.x)[at + i] = (uint16_t)float_bits16x2(c.ftype, v[i], v[i]);
  }
}

// the workgroup's number, in a grid of two dimensions (each holds fewer than 2^24 of 256 threads)
__device__ __forceinline__ uint32_t rope_group() { return blockIdx.y * gridDim.x + blockIdx.x; }

template <int HC>
__global__ void __launch_bounds__(256)
rope_kernel(RopeTurn c, RopeRows rows, RopeOut out, uint32_t tasks) {
  __shared__ __align__(16) float s_x[4][512];
  const uint32_t task = rope_group() * 4 + wave_id();
  if (task >= tasks) return;
  const uint32_t g = task / rows.chunks;
  rope_rows<HC>(c, rows, g, (int)(task - g * rows.chunks) * HC, s_x[wave_id()],
                [&](int head, int64_t tok, int e0, const float (&v)[8]) { rope_put(c, out, head, tok, e0, v); });
}

// the first workgroups take the values (as kv_store_kernel's), a wave of the others rows of keys, then of queries
template <int TK, int TV, int NB, int HC>
__global__ void __launch_bounds__(256)
kv_store_rope_kernel(RopeTurn c, RopeRows k, RopeRows q, RopeOut out, KvIo kio, KvIo vio, const int64_t* __restrict__ slots,
                     int span, uint32_t v_groups, uint32_t k_tasks, uint32_t tasks) {
  __shared__ KvTokens s_tok;
  __shared__ __align__(16) uint8_t s_tile[NB * 32 * KV_PITCH > 8192 ? NB * 32 * KV_PITCH : 8192];
  const uint32_t wg = rope_group();
  if (wg < v_groups) {
    const uint32_t tile = wg / vio.heads;
    const int t0 = (int)tile * span;
    kv_store_side<TV, NB, true>(vio, c.ftype, slots, min((int)c.t, t0 + span), t0, (int)(wg - tile * vio.heads), s_tok, s_tile);
    return;
  }
  uint32_t task = (wg - v_groups) * 4 + wave_id();
  if (task >= tasks) return;
  float* s_x = (float*)s_tile + 512 * wave_id();
  if (task >= k_tasks) {
    task -= k_tasks;
    const uint32_t g = task / q.chunks;
    rope_rows<HC>(c, q, g, (int)(task - g * q.chunks) * HC, s_x,
                  [&](int head, int64_t tok, int e0, const float (&v)[8]) { rope_put(c, out, head, tok, e0, v); });
    return;
  }
  constexpr int D = NB * 32;
  const uint32_t g = task / k.chunks;
  const int lane = threadIdx.x & 63;
  const int64_t tok = (int64_t)g * (64 >> c.log_lanes) + (lane >> c.log_lanes);
  int64_t s = tok < c.t ? slots[tok] : -1;
  if (s >= kio.n_slot) s = -1;
  const int hb = kv_head_bytes(TK, D, kio.page), cb = kv_code_bytes(TK, D, kio.page);
  const int j = (int)(s & (kio.page - 1));
  uint8_t* page = kio.pages + (s < 0 ? 0 : s >> kio.page_shift) * ((int64_t)kio.heads * hb);
  rope_rows<HC>(c, k, g, (int)(task - g * k.chunks) * HC, s_x, [&](int head, int64_t, int e0, const float (&v)[8]) {
    uint32_t u[8];
    const int b = e0 >> 5, l4 = (e0 >> 3) & 3;
    const uint32_t dh = kv_quantize<TK>(v, l4, u);
    if (s < 0) return;
    uint8_t* ph = page + (int64_t)head * hb;
    if (l4 == 0) *(uint16_t*)(ph + cb + 2 * (b * kio.page + j)) = (uint16_t)dh;
    uint8_t* o = ph + kv_k_at<TK, NB>(kio.page, j, b, l4);
    if constexpr (TK == FT_Q8_0) *(u32x2*)o = kv_bytes(u);
    else *(uint32_t*)o = kv_nibbles(u);
  });
}

// Row p of the table: cos and sin of p * f_j in 64 bits, times m, rounded once.
__global__ void __launch_bounds__(256)
rope_table_kernel(const double* __restrict__ freqs, uint32_t half, int64_t n, double m, float* __restrict__ table) {
  const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  const int64_t p = i / half;
  const uint32_t j = (uint32_t)(i - p * half);
  double s, c;
  sincos((double)p * freqs[j], &s, &c);
  float* o = table + p * (2 * (int64_t)half) + j;
  o[0] = (float)(c * m);
  o[half] = (float)(s * m);
}

static dim3 rope_grid(int64_t groups) {
  const int64_t x = groups < (1 << 20) ? groups : 1 << 20;
  return dim3((unsigned)x, (unsigned)((groups + x - 1) / x));
}

static RopeTurn rope_turn(const RopeArgs& a) {
  RopeTurn c;
  c.pos = a.pos;
  c.table = a.table;
  c.n_pos = a.n_pos;
  c.t = a.t;
  c.dim = a.dim;
  c.rot = a.rot;
  c.log_lanes = 0;
  while (8 << c.log_lanes < a.dim) ++c.log_lanes;
  c.interleaved = a.interleaved;
  c.ftype = a.ftype;
  // half layout: a lane's eight elements in one half, at aligned quads; neighbours: its four pairs
  c.vec_t = a.rot % (a.interleaved ? 8 : 16) == 0 && ((uintptr_t)a.table & 15) == 0;
  c.eps = a.eps;
  c.inv_dim = 1.0 / a.dim;
  return c;
}
static bool rope_vec(const void* x, int64_t token, int64_t head, int dim, int ftype) {
  const int64_t step = ftype == FT_F32 ? 4 : 8;   // elements in 16 bytes
  return ((uintptr_t)x & 15) == 0 && token % step == 0 && head % step == 0 && dim % 8 == 0;
}
static RopeRows rope_rows_of(const void* x, int64_t token, int64_t head, int heads, const float* weight, const RopeArgs& a, int hc) {
  RopeRows r;
  r.x = x;
  r.x_token = token;
  r.x_head = head;
  r.heads = heads;
  r.chunks = (heads + hc - 1) / hc;
  r.vec = rope_vec(x, token, head, a.dim, a.ftype);
  r.weight = weight;
  r.vec_w = ((uintptr_t)weight & 15) == 0 && a.dim % 8 == 0;
  return r;
}

}  // namespace ftk

hipError_t ftk_launch_rope_table(const double* freqs, int64_t half, int64_t n_pos, double scale, float* table, hipStream_t st) {
  const int64_t n = half * n_pos;
  ftk::rope_table_kernel<<<ftk::rope_grid((n + 255) / 256), 256, 0, st>>>(freqs, (uint32_t)half, n, scale, table);
  return hipGetLastError();
}

namespace ftk {

template <int HC>
static hipError_t rope_launch(const RopeArgs& a, hipStream_t st) {
  const RopeTurn c = rope_turn(a);
  const RopeRows q = rope_rows_of(a.q, a.q_token, a.q_head, a.n_head, a.q_weight, a, HC);
  const RopeOut out = {a.out, a.out_token, a.out_head, rope_vec(a.out, a.out_token, a.out_head, a.dim, a.ftype)};
  const int64_t per = 64 >> c.log_lanes, tasks = (a.t + per - 1) / per * q.chunks;
  rope_kernel<HC><<<rope_grid((tasks + 3) / 4), 256, 0, st>>>(c, q, out, (uint32_t)tasks);
  return hipGetLastError();
}

template <int TK, int TV, int NB, int HC>
static hipError_t store_launch(const RopeArgs& a, hipStream_t st) {
  const RopeTurn c = rope_turn(a);
  const RopeRows q = rope_rows_of(a.q, a.q_token, a.q_head, a.n_head, a.q_weight, a, HC);
  const RopeRows k = rope_rows_of(a.kv.k, a.kv.k_token, a.kv.k_head, a.kv.heads, a.k_weight, a, HC);
  const RopeOut out = {a.out, a.out_token, a.out_head, rope_vec(a.out, a.out_token, a.out_head, a.dim, a.ftype)};
  const int64_t per = 64 >> c.log_lanes, groups = (a.t + per - 1) / per;
  const int span = kv_span(a.t, a.kv.heads);
  const int64_t v_groups = (a.t + span - 1) / span * a.kv.heads, k_tasks = groups * k.chunks, tasks = k_tasks + groups * q.chunks;
  kv_store_rope_kernel<TK, TV, NB, HC><<<rope_grid(v_groups + (tasks + 3) / 4), 256, 0, st>>>(
      c, k, q, out, kv_io(a.kv, false), kv_io(a.kv, true), a.kv.slots, span, (uint32_t)v_groups, (uint32_t)k_tasks, (uint32_t)tasks);
  return hipGetLastError();
}

// Several heads per wave share its table row and have their loads in flight together, once 16 waves
// per CU remain.
static bool rope_many(const RopeArgs& a, int heads) {
  int per = 64;
  while (per > 1 && (64 / per) * 8 < a.dim) per >>= 1;
  return (a.t + per - 1) / per * ((heads + ROPE_MANY - 1) / ROPE_MANY) >= 16 * (int64_t)ftk_num_cus();
}

template <int TK, int TV, int NB>
static hipError_t store_many(const RopeArgs& a, hipStream_t st) {
  return rope_many(a, a.n_head + a.kv.heads) ? store_launch<TK, TV, NB, ROPE_MANY>(a, st) : store_launch<TK, TV, NB, 1>(a, st);
}
template <int TK, int TV>
static hipError_t store_pick(const RopeArgs& a, hipStream_t st) {
  switch (a.dim) {
    case 64: return store_many<TK, TV, 2>(a, st);
    case 96: return store_many<TK, TV, 3>(a, st);
    case 128: return store_many<TK, TV, 4>(a, st);
    case 256: return store_many<TK, TV, 8>(a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace ftk

hipError_t ftk_launch_rope(const RopeArgs& a, hipStream_t st) {
  using namespace ftk;
  return rope_many(a, a.n_head) ? rope_launch<ROPE_MANY>(a, st) : rope_launch<1>(a, st);
}

hipError_t ftk_launch_kv_store_rope(const RopeArgs& a, hipStream_t st) {
  using namespace ftk;
  if (a.kv.k_type == FT_Q8_0)
    return a.kv.v_type == FT_Q8_0 ? store_pick<FT_Q8_0, FT_Q8_0>(a, st) : store_pick<FT_Q8_0, FT_Q4_0>(a, st);
  return a.kv.v_type == FT_Q8_0 ? store_pick<FT_Q4_0, FT_Q8_0>(a, st) : store_pick<FT_Q4_0, FT_Q4_0>(a, st);
}
