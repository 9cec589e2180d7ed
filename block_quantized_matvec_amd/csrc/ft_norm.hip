// ft_norm.hip -- the norm around a block (ft_norm): a block's output normed, gated, scaled
// and added to the residual stream, and the stream's norm for the next block, as rows or as
// the quantized blocks that the next product reads.
//
//   b = x;  b = norm(b) w_post + b_post;  b = b gate;  b = scale b;  r = residual + b;
//   n = norm(r) w + bias;   norm(v) = (v - mean) / sqrt(var + eps), or v / sqrt(mean v^2 + eps)
//
// (each step where it is asked for.)  Sums are 64-bit, everything per element is one fp32
// operation after the other (this file is compiled without contraction), so a code next to
// a half-integer does not hang on the order of the sum.
//
// A row is read once: it stays in the registers of one workgroup, eight consecutive
// elements a chunk, between its two norms, and every load of a row (x, residual, gate) is
// issued before the first is used.  The quantizers' blocks lie in neighbouring lanes (four
// for 32 elements, 32 for 256), so their maxima meet in lane exchanges.
#include "ft_kv.h"
#include "ft_rowstat.h"
#include "ft_internal.h"

namespace ftk {

struct NormSide {
  const void* x;
  int64_t ld;
  int vec;   // rows stay 16-byte aligned
};
struct NormIo {
  NormSide x, residual, gate, r, out;   // x.x null: not there
  const float *post_weight, *post_bias, *weight, *bias;
  int vec_w, post, layer, ftype, act, scaled, width;
  float scale;
  double eps, inv_width;
  uint8_t* xq;
  int64_t xq_row;
  int64_t rows;
};

// eight elements of a row from e on (those past the width: 0), as 32-bit words
__device__ __forceinline__ void norm_load(int type, const NormSide& s, int64_t row, int e, int width, u32x4 (&raw)[2]) {
  const int64_t at[1] = {row * s.ld + e};
  if (e + 8 <= width) {
    u32x4 r[1][2];
    kv_load_raw<1>(type, s.x, at, s.vec, r);
    raw[0] = r[0][0];
    if (type == FT_F32) raw[1] = r[0][1];
    return;
  }
  raw[0] = raw[1] = u32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (e + i >= width) break;
    if (type == FT_F32) raw[i >> 2][i & 3] = ((const uint32_t*)s.x)[at[0] + i];
    else raw[0][i >> 1] |= (uint32_t)((const uint16_t*)s.x)[at[0] + i] << (16 * (i & 1));
  }
}
__device__ __forceinline__ void norm_store(int type, const NormSide& s, int64_t row, int e, int width, const float (&v)[8]) {
  const int64_t at = row * s.ld + e;
  void* base = const_cast<void*>(s.x);
  if (e + 8 <= width) {
    kv_store_n<8>(type, base, at, s.vec, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (e + i >= width) break;
    if (type == FT_F32) ((float*)base)[at + i] = v[i];
    else ((uint16_t*)base)[at + i] = (uint16_t)float_bits16x2(type, v[i], v[i]);
  }
}
__device__ __forceinline__ void norm_weights(const float* p, bool vec, int e, int width, float (&w)[8]) {
  if (vec && e + 8 <= width) {
    kv_load8(FT_F32, p, e, true, w);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = e + i < width ? p[e + i] : 0.0f;
}

// Q8_0's 34-byte block: as q8_1_part without the sum
__device__ __forceinline__ void norm_q8_0(const float (&v)[8], int l4, uint8_t* ob) {
  float a = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(v[j]));
  a = fmaxf(a, xchg<1>(a));
  a = fmaxf(a, xchg<2>(a));
  const uint32_t dh = f2h_bits(a / 127.0f);
  const float d = h2f(dh);
  int q[8];
  q8_codes<8>(v, d, q);
  uint16_t* o = (uint16_t*)(ob + 2 + 8 * l4);
#pragma unroll
  for (int j = 0; j < 8; j += 2) o[j >> 1] = (uint16_t)((q[j] & 255) | ((q[j + 1] & 255) << 8));
  if (l4 == 0) *(uint16_t*)ob = (uint16_t)(d == 0.0f ? 0u : dh);
}
// Q8_K's 292-byte block in 32 lanes: as q8_k_part, two lanes to a 16-element sum
__device__ __forceinline__ void norm_q8_k(const float (&v)[8], int l32, uint8_t* ob) {
  float a = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(v[j]));
  a = fmaxf(a, xchg<1>(a));
  a = fmaxf(a, xchg<2>(a));
  a = fmaxf(a, xchg<4>(a));
  a = fmaxf(a, xchg<8>(a));
  a = fmaxf(a, xchg<16>(a));
  const float d = a / 127.0f;
  int q[8], s = 0;
  q8_codes<8>(v, d, q);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s += q[j];
    w[j >> 2] |= (uint32_t)(q[j] & 255) << (8 * (j & 3));
  }
  s += __float_as_int(xchg<1>(__int_as_float(s)));
  uint32_t* o = (uint32_t*)(ob + 4 + 8 * l32);
  o[0] = w[0];
  o[1] = w[1];
  if (!(l32 & 1)) *(int16_t*)(ob + 260 + l32) = (int16_t)s;
  if (l32 == 0) *(float*)ob = d;
}

// sum over the lanes that share a row: a wave, or the workgroup (s_sum: a slot per wave and use)
template <int THREADS>
__device__ __forceinline__ double norm_sum(double s, double* s_sum) {
  s = lanes_sum(s, 6);
  if constexpr (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) s += s_sum[i];
  }
  return s;
}

// THREADS threads share a row, C chunks of eight elements each.  With 64 a workgroup holds four rows.
template <int THREADS, int C>
__global__ void __launch_bounds__(THREADS < 256 ? 256 : THREADS)
norm_kernel(NormIo io) {
  constexpr int WAVES = THREADS / 64;
  __shared__ double s_sum[4][WAVES];
  const int tid = threadIdx.x & (THREADS - 1);
  const int64_t wg = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t row = THREADS == 64 ? wg * 4 + wave_id() : wg;
  if (row >= io.rows) return;   // a whole workgroup, or waves that no barrier waits for
  const int width = io.width;
  u32x4 rx[C][2], rr[C][2], rg[C][2];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = 8 * (tid + THREADS * c);
    if (e < width) norm_load(io.ftype, io.x, row, e, width, rx[c]);
    else rx[c][0] = rx[c][1] = u32x4{0, 0, 0, 0};
  }
  if (io.residual.x)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 8 * (tid + THREADS * c);
      if (e < width) norm_load(io.ftype, io.residual, row, e, width, rr[c]);
    }
  if (io.gate.x)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 8 * (tid + THREADS * c);
      if (e < width) norm_load(io.ftype, io.gate, row, e, width, rg[c]);
    }
  float v[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) kv_raw_values(io.ftype, rx[c], v[c]);

  // v <- norm(v) w + b, elements past the width left at 0
  auto norm = [&](const float* weight, const float* bias, double* sums) {
    double s = 0.0, mean = 0.0;
    if (io.layer) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += (double)v[c][i];
      mean = norm_sum<THREADS>(s, sums) * io.inv_width;
      s = 0.0;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double d = (double)v[c][i] - mean;
          if (8 * (tid + THREADS * c) + i < width) s = fma(d, d, s);
          v[c][i] = (float)d;
        }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) s += sum_squares(v[c]);
    }
    const float r = rstd_of(fma(norm_sum<THREADS>(s, sums + WAVES), io.inv_width, io.eps));
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 8 * (tid + THREADS * c);
      if (e >= width) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * r;
      float w[8];
      if (weight) {
        norm_weights(weight, io.vec_w, e, width, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * w[i];
      }
      if (bias) {
        norm_weights(bias, io.vec_w, e, width, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] + w[i];
      }
    }
  };

  if (io.post) norm(io.post_weight, io.post_bias, s_sum[0]);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = 8 * (tid + THREADS * c);
    if (e >= width) {   // a layer's norm leaves -mean there
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = 0.0f;
      continue;
    }
    float o[8];
    if (io.gate.x) {
      kv_raw_values(io.ftype, rg[c], o);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * o[i];
    }
    if (io.scaled)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * io.scale;
    if (io.residual.x) {
      kv_raw_values(io.ftype, rr[c], o);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = o[i] + v[c][i];
    }
    if (e + 8 > width)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i >= width) v[c][i] = 0.0f;
    if (io.r.x) norm_store(io.ftype, io.r, row, e, width, v[c]);
  }
  if (!io.out.x && !io.xq) return;
  norm(io.weight, io.bias, s_sum[2]);
  uint8_t* xq = io.xq + row * io.xq_row;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int g = tid + THREADS * c, e = 8 * g;
    if (e >= width) continue;
    if (io.out.x) norm_store(io.ftype, io.out, row, e, width, v[c]);
    if (io.xq) {   // whole blocks: a block's lanes are all here
      if (io.act == FT_Q8_1) q8_1_part(v[c], g & 3, xq + (g >> 2) * 36);
      else if (io.act == FT_Q8_0) norm_q8_0(v[c], g & 3, xq + (g >> 2) * 34);
      else norm_q8_k(v[c], g & 31, xq + (g >> 5) * 292);
    }
  }
}

template <int THREADS, int C>
static hipError_t norm_launch(const NormIo& io, hipStream_t st) {
  const int64_t groups = THREADS == 64 ? (io.rows + 3) / 4 : io.rows;
  const int64_t x = groups < (1 << 20) ? groups : 1 << 20;   // fewer than 2^32 threads along a dimension
  norm_kernel<THREADS, C><<<dim3((unsigned)x, (unsigned)((groups + x - 1) / x)), THREADS < 256 ? 256 : THREADS, 0, st>>>(io);
  return hipGetLastError();
}

static NormSide norm_side(const void* x, int64_t ld, int ftype) {
  return {x, ld, ((uintptr_t)x & 15) == 0 && ld % (ftype == FT_F32 ? 4 : 8) == 0};
}

}  // namespace ftk

hipError_t ftk_launch_norm(const NormArgs& a, hipStream_t st) {
  using namespace ftk;
  NormIo io;
  io.x = norm_side(a.x, a.ldx, a.ftype);
  io.residual = norm_side(a.residual, a.ld_residual, a.ftype);
  io.gate = norm_side(a.gate, a.ld_gate, a.ftype);
  io.r = norm_side(a.r, a.ld_r, a.ftype);
  io.out = norm_side(a.out, a.ld_out, a.ftype);
  io.post_weight = a.post_weight;
  io.post_bias = a.post_bias;
  io.weight = a.weight;
  io.bias = a.bias;
  io.vec_w = (((uintptr_t)a.post_weight | (uintptr_t)a.post_bias | (uintptr_t)a.weight | (uintptr_t)a.bias) & 15) == 0;
  io.post = a.post;
  io.layer = a.layer;
  io.ftype = a.ftype;
  io.act = a.act;
  io.scaled = a.scale != 1.0f;
  io.width = (int)a.width;
  io.scale = a.scale;
  io.eps = a.eps;
  io.inv_width = 1.0 / a.width;
  io.xq = (uint8_t*)a.xq;
  io.xq_row = a.xq_row;
  io.rows = a.rows;
  // the fewest threads whose lanes hold a row in four chunks, but a chunk each while rows are few
  const int64_t w = a.width;
  if (w <= 512) return norm_launch<64, 1>(io, st);
  if (w <= 2048) return norm_launch<256, 1>(io, st);
  if (w <= 4096) return norm_launch<256, 2>(io, st);
  if (w <= 8192) return norm_launch<256, 4>(io, st);
  if (w <= 16384) return norm_launch<512, 4>(io, st);
  return norm_launch<1024, 4>(io, st);
}
