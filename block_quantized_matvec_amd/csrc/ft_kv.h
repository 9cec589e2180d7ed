// ft_kv.h -- the paged key/value cache's page layout (include/ft.h defines it) and
// the element types of the tensors around it, shared by the store, load and
// attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ft.h"

namespace ftk {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 h16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));

// what this wave's lanes wrote to LDS is there for all of them (LDS serves a wave in
// order; the fence keeps the compiler from moving accesses across)
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// One page head: the codes of `page` keys (D elements each), then the fp16 scales
// [D/32][page].
__host__ __device__ constexpr int kv_code_bytes(int type, int dim, int page) {
  return type == FT_Q8_0 ? dim * page : dim * page / 2;
}
__host__ __device__ constexpr int kv_head_bytes(int type, int dim, int page) {
  return kv_code_bytes(type, dim, page) + dim / 32 * page * 2;
}

// K codes: the blocks of a key are taken in groups (two of Q8_0, four of Q4_0, the
// last group may hold fewer); a group's keys lie one after the other, and within a
// key its four 8-element eighths-of-a-pair lie one after the other with the group's
// blocks side by side.  Lane group g of a matrix operand (k = 8g .. 8g+7 of a
// 32-element block) so finds its codes of the whole group in one load.
template <int T> struct KvCodes;
template <> struct KvCodes<FT_Q8_0> { static constexpr int GROUP = 2, CB = 8; };   // blocks per group, bytes per 8 codes
template <> struct KvCodes<FT_Q4_0> { static constexpr int GROUP = 4, CB = 4; };
// byte of the first of codes 8g .. 8g+7 of block b of key j
template <int T, int NB>
__host__ __device__ inline int kv_k_at(int page, int j, int b, int g) {
  constexpr int G = KvCodes<T>::GROUP, CB = KvCodes<T>::CB;
  const int p = b / G, left = NB - p * G, m = left < G ? left : G;
  return page * 64 * p + j * 4 * m * CB + g * m * CB + (b - p * G) * CB;
}

// Eight codes (each plus 128, or plus 8, in the low byte of a word) as the cache holds
// them: Q8_0, and Q4_0 where a byte each is wanted, in element order; Q4_0 with element e
// in nibble e/2 + 4*(e%2), so that (w >> 4i) & 0x000F000F is the pair of elements 2i, 2i+1
// in the two halves of a register.
__device__ __forceinline__ uint32_t kv_bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u), 0x05040100u);
}
__device__ __forceinline__ u32x2 kv_bytes(const uint32_t (&u)[8]) {
  return u32x2{kv_bytes4(u[0], u[1], u[2], u[3]), kv_bytes4(u[4], u[5], u[6], u[7])};
}
__device__ __forceinline__ uint32_t kv_nibbles(const uint32_t (&u)[8]) {
  return kv_bytes4(u[0], u[4], u[1], u[5]) | (kv_bytes4(u[2], u[6], u[3], u[7]) << 4);
}

// eight consecutive elements of a float tensor; vec: 16-byte aligned
__device__ __forceinline__ float bf16_value(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ void kv_load8(int type, const void* base, int64_t at, bool vec, float (&v)[8]) {
  if (type == FT_F32) {
    const float* p = (const float*)base + at;
    if (vec) {
      const f32x4 a = ((const f32x4*)p)[0], b = ((const f32x4*)p)[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[i];
    }
    return;
  }
  const uint16_t* p = (const uint16_t*)base + at;
  uint32_t h[8];
  if (vec) {
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    const u4 a = *(const u4*)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (a[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = p[i];
  }
  if (type == FT_BF16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = bf16_value(h[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)h[i]);
  }
}

// The same N times as loaded (two words of 16 bytes for fp32, one else), all loads in
// flight together; and the values of one.
template <int N>
__device__ __forceinline__ void kv_load_raw(int type, const void* base, const int64_t (&at)[N], bool vec,
                                            uint32_t __attribute__((ext_vector_type(4))) (&r)[N][2]) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  if (type == FT_F32) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t* p = (const uint32_t*)base + at[n];
      if (vec) {
        r[n][0] = ((const u4*)p)[0];
        r[n][1] = ((const u4*)p)[1];
      } else {
        r[n][0] = u4{p[0], p[1], p[2], p[3]};
        r[n][1] = u4{p[4], p[5], p[6], p[7]};
      }
    }
    return;
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint16_t* p = (const uint16_t*)base + at[n];
    if (vec) r[n][0] = *(const u4*)p;
    else
#pragma unroll
      for (int i = 0; i < 4; ++i) r[n][0][i] = p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
  }
}
__device__ __forceinline__ void kv_raw_values(int type, const uint32_t __attribute__((ext_vector_type(4))) (&r)[2], float (&v)[8]) {
  if (type == FT_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i >> 2][i & 3]);
  } else if (type == FT_BF16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? r[0][i >> 1] & 0xFFFF0000u : r[0][i >> 1] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = r[0][i >> 1];
      v[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(i & 1 ? w >> 16 : w));
    }
  }
}

// Of N blocks, 32 elements apart: every load goes out before the first value
// is converted.
template <int N>
__device__ __forceinline__ void kv_load_row(int type, const void* base, int64_t at, bool vec, float (&v)[N][8]) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  if (!vec) {
#pragma unroll
    for (int b = 0; b < N; ++b) kv_load8(type, base, at + 32 * b, false, v[b]);
    return;
  }
  if (type == FT_F32) {
    const f32x4* p = (const f32x4*)((const float*)base + at);
    f32x4 r[N][2];
#pragma unroll
    for (int b = 0; b < N; ++b) {
      r[b][0] = p[8 * b];
      r[b][1] = p[8 * b + 1];
    }
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[b][i] = r[b][i >> 2][i & 3];
    return;
  }
  const u4* p = (const u4*)((const uint16_t*)base + at);
  u4 r[N];
#pragma unroll
  for (int b = 0; b < N; ++b) r[b] = p[4 * b];
  if (type == FT_BF16) {
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[b][i] = __uint_as_float(i & 1 ? r[b][i >> 1] & 0xFFFF0000u : r[b][i >> 1] << 16);
  } else {
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w = r[b][i >> 1];
        v[b][i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(i & 1 ? w >> 16 : w));
      }
  }
}

// two values as bf16 or fp16, to nearest even
__device__ __forceinline__ uint32_t float_bits16x2(int type, float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  if (type == FT_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, h16x2));
}
template <int N>   // N consecutive elements (4 or 8)
__device__ __forceinline__ void kv_store_n(int type, void* base, int64_t at, bool vec, const float (&v)[N]) {
  if (type == FT_F32) {
    float* p = (float*)base + at;
    if (vec) {
#pragma unroll
      for (int i = 0; i < N; i += 4) *(f32x4*)(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = v[i];
    }
    return;
  }
  uint16_t* p = (uint16_t*)base + at;
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w[i] = float_bits16x2(type, v[2 * i], v[2 * i + 1]);
  if (vec) {
#pragma unroll
    for (int i = 0; i < N / 2; i += 2) *(u32x2*)(p + 2 * i) = u32x2{w[i], w[i + 1]};
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}

}  // namespace ftk
