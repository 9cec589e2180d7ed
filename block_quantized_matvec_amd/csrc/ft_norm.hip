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
// elements a thread, between its two norms, and every load of a row (x, residual, gate, the
// coming norm's weights) is issued before the first is used.  The quantizers' blocks lie in
// neighbouring lanes (four for 32 elements, 32 for 256), so their maxima meet in lane
// exchanges.
//
// Bound by memory once there are rows for the chip (a 2 GiB copy moves 5.0 TB/s here): 8192 rows of 4096,
// bf16, both norms and the residual 46-52 us (5.2-5.8 TB/s; 91 with two chunks per thread and loads that
// waited for each other); fp32 to Q8_K blocks 82 us (5.4); 8192 rows of 2048 fp32 41 us (64 with the registers
// held to eight waves per SIMD, which spilled).  1500 layer-normed rows of 5002 fp16 with a gate 21 us, 3.5 TB/s: two
// sums one after the other, each with a barrier, and 8 us of vector issue, which the three workgroups that a CU holds do
// not hide.  One row of 4096: 2.8 us, the launch and two memory latencies.  Wide bf16 rows with a residual, 134 MB each: 2048 of 8200
// 29 us (two chunks a thread, half of them empty), 1024 of 16384 27, 512 of 32768 36 and 1024 of 16390 65 (four chunks, whose
// registers spill to memory: 17 to 29 of a thread, 25 to 121 where the width is no multiple of eight).
#include "ft_kv.h"
#include "ft_rowstat.h"
#include "ft_internal.h"

namespace ftk {

struct NormSide {
  const void* x;
  int64_t ld;
};
struct NormIo {
  NormSide x, residual, gate, r, out;   // x.x null: not there
  const float *post_weight, *post_bias, *weight, *bias;
  int post, layer, act, scaled, width;
  float scale;
  double eps, inv_width;
  uint8_t* xq;
  int64_t xq_row;
  int64_t rows;
};

// Rows need no alignment past their elements': the vector loads and stores below are whole
// whatever their address (a row of 5002 fp16 starts at any fourth byte).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
template <int TYPE> constexpr int NORM_WORDS = TYPE == FT_F32 ? 2 : 1;   // of 16 bytes for eight elements

// eight elements of a row from e on; TAIL: those past the width are 0
template <int TYPE, bool TAIL>
__device__ __forceinline__ void norm_load(const NormSide& s, int64_t row, int e, int width, u32x4 (&raw)[NORM_WORDS<TYPE>]) {
  const int64_t at = row * s.ld + e;
  if (!TAIL || e + 8 <= width) {
    const u32x4_any* p = (const u32x4_any*)((const uint8_t*)s.x + at * (TYPE == FT_F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < NORM_WORDS<TYPE>; ++i) raw[i] = p[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t u = 0;
    if (e + i < width) u = TYPE == FT_F32 ? ((const uint32_t*)s.x)[at + i] : ((const uint16_t*)s.x)[at + i];
    if constexpr (TYPE == FT_F32) raw[i >> 2][i & 3] = u;
    else raw[0][i >> 1] = i & 1 ? raw[0][i >> 1] | (u << 16) : u;
  }
}
template <int TYPE>
__device__ __forceinline__ void norm_values(const u32x4 (&raw)[NORM_WORDS<TYPE>], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (TYPE == FT_F32) v[i] = __uint_as_float(raw[i >> 2][i & 3]);
    else if constexpr (TYPE == FT_BF16) v[i] = __uint_as_float(i & 1 ? raw[0][i >> 1] & 0xFFFF0000u : raw[0][i >> 1] << 16);
    else v[i] = h2f((raw[0][i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
  }
}
template <int TYPE, bool TAIL>
__device__ __forceinline__ void norm_store(const NormSide& s, int64_t row, int e, int width, const float (&v)[8]) {
  const int64_t at = row * s.ld + e;
  uint8_t* base = (uint8_t*)const_cast<void*>(s.x) + at * (TYPE == FT_F32 ? 4 : 2);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (TYPE == FT_F32) w[i] = __float_as_uint(v[i]);
    else if (!(i & 1)) w[i >> 1] = float_bits16x2(TYPE, v[i], v[i + 1]);
  }
  if (!TAIL || e + 8 <= width) {
#pragma unroll
    for (int i = 0; i < NORM_WORDS<TYPE>; ++i) ((u32x4_any*)base)[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (e + i < width) {
      if constexpr (TYPE == FT_F32) ((uint32_t*)base)[i] = w[i];
      else ((uint16_t*)base)[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
  }
}
template <bool TAIL>
__device__ __forceinline__ void norm_weights(const float* p, int e, int width, float (&w)[8]) {
  if (!TAIL || e + 8 <= width) {
    const f32x4 a = ((const f32x4_any*)(p + e))[0], b = ((const f32x4_any*)(p + e))[1];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < 4 ? a[i & 3] : b[i & 3];
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

// sum over the lanes that share a row: a wave, or the workgroup (s_sum: a slot per wave, another array for
// every use)
template <bool WAVE>
__device__ __forceinline__ double norm_sum(double s, double* s_sum) {
  s = lanes_sum(s, 6);
  if constexpr (!WAVE) {
    const int lane = threadIdx.x & 63;
    if (lane == 0) s_sum[wave_id()] = s;
    __syncthreads();
    s = lanes_sum((lane & 15) < (int)(blockDim.x >> 6) ? s_sum[lane & 15] : 0.0, 4);
  }
  return s;
}

// A workgroup of up to 1024 threads has a row, C chunks of eight elements per thread; with WAVE it
// has four, one a wave.  TAIL: the width is no multiple of eight.
template <int TYPE, int C, bool WAVE, bool TAIL>
__global__ void __launch_bounds__(WAVE ? 256 : 1024)
norm_kernel(NormIo io) {
  constexpr int W = NORM_WORDS<TYPE>;
  __shared__ double s_sum[4][16];
  const int tid = WAVE ? threadIdx.x & 63 : threadIdx.x, threads = C == 1 ? 0 : 1024;
  const int64_t wg = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t row = WAVE ? wg * 4 + wave_id() : wg;
  if (row >= io.rows) return;   // a whole workgroup, or waves that no barrier waits for
  const int width = io.width;
  const auto at = [&](int c) { return 8 * (tid + threads * c); };
  u32x4 rx[C][W], rr[C][W], rg[C][W];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int i = 0; i < W; ++i) rx[c][i] = rr[c][i] = rg[c][i] = u32x4{0, 0, 0, 0};
    if (at(c) < width) norm_load<TYPE, TAIL>(io.x, row, at(c), width, rx[c]);
  }
  constexpr bool AHEAD = C <= 2;   // room for every load that is still to come
  if (AHEAD && io.residual.x)
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (at(c) < width) norm_load<TYPE, TAIL>(io.residual, row, at(c), width, rr[c]);
  if (AHEAD && io.gate.x)
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (at(c) < width) norm_load<TYPE, TAIL>(io.gate, row, at(c), width, rg[c]);
  float v[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) norm_values<TYPE>(rx[c], v[c]);

  // v <- norm(v) weight + bias; elements past the width are 0 before it, and anything after
  auto norm = [&](const float* weight, const float* bias, double* sums) {
    float w[C][8];
    if (AHEAD && weight)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (at(c) < width) norm_weights<TAIL>(weight, at(c), width, w[c]);
    double s = 0.0;
    if (io.layer) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += (double)v[c][i];
      const double mean = norm_sum<WAVE>(s, sums) * io.inv_width;
      s = 0.0;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double d = (double)v[c][i] - mean;
          if (at(c) + i < width) s = fma(d, d, s);
          v[c][i] = (float)d;
        }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) s += sum_squares(v[c]);
    }
    const float r = rstd_of(fma(norm_sum<WAVE>(s, sums + 16), io.inv_width, io.eps));
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (at(c) >= width) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * r;
      if (weight) {
        if (!AHEAD) norm_weights<TAIL>(weight, at(c), width, w[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * w[c][i];
      }
      if (bias) {
        float b[8];
        norm_weights<TAIL>(bias, at(c), width, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] + b[i];
      }
    }
  };

  if (io.post) norm(io.post_weight, io.post_bias, s_sum[0]);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = at(c);
    float o[8];
    if (io.gate.x) {
      if (!AHEAD && e < width) norm_load<TYPE, TAIL>(io.gate, row, e, width, rg[c]);
      norm_values<TYPE>(rg[c], o);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * o[i];
    }
    if (io.scaled)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * io.scale;
    if (io.residual.x) {
      if (!AHEAD && e < width) norm_load<TYPE, TAIL>(io.residual, row, e, width, rr[c]);
      norm_values<TYPE>(rr[c], o);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = o[i] + v[c][i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)   // a norm leaves -mean or a bias past the width
      if (TAIL ? e + i >= width : e >= width) v[c][i] = 0.0f;
    if (io.r.x && e < width) norm_store<TYPE, TAIL>(io.r, row, e, width, v[c]);
  }
  if (!io.out.x && !io.xq) return;
  norm(io.weight, io.bias, s_sum[2]);
  uint8_t* xq = io.xq + row * io.xq_row;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int g = tid + threads * c;
    if (at(c) >= width) continue;
    if (io.out.x) norm_store<TYPE, TAIL>(io.out, row, at(c), width, v[c]);
    if (!TAIL && io.xq) {   // whole blocks: a block's lanes are all here
      if (io.act == FT_Q8_1) q8_1_part(v[c], g & 3, xq + (g >> 2) * 36);
      else if (io.act == FT_Q8_0) norm_q8_0(v[c], g & 3, xq + (g >> 2) * 34);
      else norm_q8_k(v[c], g & 31, xq + (g >> 5) * 292);
    }
  }
}

template <int TYPE, int C, bool WAVE>
static hipError_t norm_launch(const NormIo& io, hipStream_t st) {
  const int64_t groups = WAVE ? (io.rows + 3) / 4 : io.rows;
  const int64_t x = groups < (1 << 20) ? groups : 1 << 20;   // fewer than 2^32 threads along a dimension
  const dim3 grid((unsigned)x, (unsigned)((groups + x - 1) / x));
  const int block = WAVE ? 256 : C > 1 ? 1024 : (io.width + 511) / 512 * 64;
  if (io.width % 8) norm_kernel<TYPE, C, WAVE, true><<<grid, block, 0, st>>>(io);
  else norm_kernel<TYPE, C, WAVE, false><<<grid, block, 0, st>>>(io);
  return hipGetLastError();
}

// a chunk per thread while a workgroup's threads last; rows of at most 512 go to single waves
template <int TYPE>
static hipError_t norm_pick(const NormIo& io, hipStream_t st) {
  if (io.width <= 512) return norm_launch<TYPE, 1, true>(io, st);
  if (io.width <= 8192) return norm_launch<TYPE, 1, false>(io, st);
  if (io.width <= 16384) return norm_launch<TYPE, 2, false>(io, st);
  return norm_launch<TYPE, 4, false>(io, st);
}

}  // namespace ftk

hipError_t ftk_launch_norm(const NormArgs& a, hipStream_t st) {
  using namespace ftk;
  NormIo io;
  io.x = {a.x, a.ldx};
  io.residual = {a.residual, a.ld_residual};
  io.gate = {a.gate, a.ld_gate};
  io.r = {a.r, a.ld_r};
  io.out = {a.out, a.ld_out};
  io.post_weight = a.post_weight;
  io.post_bias = a.post_bias;
  io.weight = a.weight;
  io.bias = a.bias;
  io.post = a.post;
  io.layer = a.layer;
  io.act = a.act;
  io.scaled = a.scale != 1.0f;
  io.width = (int)a.width;
  io.scale = a.scale;
  io.eps = a.eps;
  io.inv_width = 1.0 / a.width;
  io.xq = (uint8_t*)a.xq;
  io.xq_row = a.xq_row;
  io.rows = a.rows;
  if (a.ftype == FT_F32) return norm_pick<FT_F32>(io, st);
  return a.ftype == FT_F16 ? norm_pick<FT_F16>(io, st) : norm_pick<FT_BF16>(io, st);
}
