// ft_rowstat.h -- statistics of rows in 64 bits, for the norms (ft_norm.hip, ft_rope.hip).
//
// A row's sums are doubles and 1 / sqrt is rounded to fp32 once, so that the result does
// not depend on the order of the sum: an element is then one fp32 operation after the
// other on that factor, and its quantized code is the same on any lane split.  At four
// cycles per wave (a conversion and a multiply-add per element) the doubles stay far
// below the time of the row's loads.
#pragma once

#include "ft_device.h"

namespace ftk {

template <int S>
__device__ __forceinline__ double xchg_d(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __float_as_uint(xchg<S>(__uint_as_float((uint32_t)u)));
  const uint32_t hi = __float_as_uint(xchg<S>(__uint_as_float((uint32_t)(u >> 32))));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// s plus the other half's (or the other 16 lanes' of a half): both registers of the exchange hold one side
__device__ __forceinline__ double halves_sum(double v, bool wide) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)u, hi = (uint32_t)(u >> 32);
  const auto a = wide ? __builtin_amdgcn_permlane32_swap(lo, lo, false, false) : __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
  const auto b = wide ? __builtin_amdgcn_permlane32_swap(hi, hi, false, false) : __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
  return __builtin_bit_cast(double, ((uint64_t)b[0] << 32) | a[0]) + __builtin_bit_cast(double, ((uint64_t)b[1] << 32) | a[1]);
}
// sum over 1 << log_lanes aligned lanes (uniform over the wave), in all of them
__device__ __forceinline__ double lanes_sum(double s, int log_lanes) {
  if (log_lanes > 0) s += xchg_d<1>(s);
  if (log_lanes > 1) s += xchg_d<2>(s);
  if (log_lanes > 2) s += xchg_d<4>(s);
  if (log_lanes > 3) s += xchg_d<8>(s);
  if (log_lanes > 4) s = halves_sum(s, false);
  if (log_lanes > 5) s = halves_sum(s, true);
  return s;
}
template <int N>
__device__ __forceinline__ double sum_squares(const float (&v)[N]) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) s = fma((double)v[i], (double)v[i], s);
  return s;
}
// 1 / sqrt(m), rounded to fp32.  The instruction is good for about half of the bits; one
// step of third order leaves an error near 2^-53.  0, infinities and NaN as they come.
__device__ __forceinline__ float rstd_of(double m) {
  double r = __builtin_amdgcn_rsq(m);
  const double e = fma(-(m * r), r, 1.0);
  const double f = fma(r * e, fma(0.375, e, 0.5), r);
  if (m > 0.0 && m < __builtin_huge_val()) r = f;
  return (float)r;
}

}  // namespace ftk
