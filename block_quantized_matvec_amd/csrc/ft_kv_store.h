// ft_kv_store.h -- the paged cache's quantizer and the device side of a store: shared by the plain
// store and load (ft_kv.hip) and the store that turns its rows first (ft_rope.hip).
#pragma once

#include "ft_device.h"
#include "ft_internal.h"
#include "ft_kv.h"

namespace ftk {

constexpr int KV_TILE = 64;    // tokens per workgroup
constexpr int KV_PITCH = 68;   // bytes between the rows of the transposed tile in LDS (a bank further per row)

// The codes of eight values of one block, each plus HIGH + 1, in the low bytes of u.  top:
// the block's largest magnitude; d is an fp16 number.  The sum of v * rcp(d) and 3 * 2^22 +
// HIGH + 1 leaves the rounded quotient in its last bits; v * rcp(d) is within 1.5 * 2^-16 of
// v / d while that is below 128, so the rounding is the code's unless it lies within 2^-14
// of a half-integer (bf16 values often lie on one).  There a code n is held against
// (|n| -+ 1/2) |d|, which are exact.  Past the range of codes (a scale that fp16 holds
// with few bits or not at all) the lane divides.
template <int LOW, int HIGH>
__device__ __forceinline__ void kv_codes(const float (&v)[8], float d, float top, uint32_t (&u)[8]) {
  constexpr float MAGIC = 12582912.0f + HIGH + 1;
  const float r = __builtin_amdgcn_rcpf(d);
  float off = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // Q4_0: the last code stands for everything above it
    const float t = LOW == -8 ? fminf(v[j] * r, (float)HIGH) : v[j];
    const float c = LOW == -8 ? t + MAGIC : fmaf(t, r, MAGIC);
    const float e = LOW == -8 ? t - (c - MAGIC) : fmaf(t, r, MAGIC - c);
    off = fmaxf(off, fabsf(e));
    u[j] = __float_as_uint(c);
  }
  if (!(top * fabsf(r) < 0.4f - LOW)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = roundf(v[j] / (d == 0.0f ? 1.0f : d));
      u[j] = (uint32_t)((d == 0.0f ? 0 : (int)fminf(fmaxf(t, (float)LOW), (float)HIGH)) + HIGH + 1);
    }
  } else if (off >= 0.5f - 0x1p-14f) {
    const float ad = fabsf(d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float n = fabsf(__uint_as_float(u[j]) - MAGIC);
      const float x = fabsf(v[j]), up = fmaf(n, ad, 0.5f * ad), down = fmaf(n, ad, -0.5f * ad);
      n += x >= up ? 1.0f : x < down ? -1.0f : 0.0f;
      n = __uint_as_float(__float_as_uint(n) | ((__float_as_uint(v[j]) ^ __float_as_uint(d)) & 0x80000000u));
      u[j] = __float_as_uint(fminf(n, (float)HIGH) + MAGIC);
    }
  }
}

// One block's scale (fp16 bits) and this lane's eight codes as kv_codes leaves them; its four lanes call it
// together, lane l4 with elements 8*l4 .. 8*l4+7.
template <int T>
__device__ __forceinline__ uint32_t kv_quantize(const float (&v)[8], int l4, uint32_t (&u)[8]) {
  float d;
  uint32_t dh;
  if constexpr (T == FT_Q8_0) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(v[j]));
    a = fmaxf(a, xchg<1>(a));
    a = fmaxf(a, xchg<2>(a));
    // a / 127, correctly rounded: a product with the rounded reciprocal, and its remainder
    const float q = a * (1.0f / 127.0f), q1 = fmaf(fmaf(-127.0f, q, a), 1.0f / 127.0f, q);
    dh = f2h_bits(fminf(q1, 65504.0f));
    d = h2f(dh);
    kv_codes<-127, 127>(v, d, a, u);
  } else {
    float m = v[0] == v[0] ? v[0] : 0.0f;   // a NaN has no magnitude; behind the first it is never the larger
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fabsf(v[j]) > fabsf(m) ? v[j] : m;
    // of two of equal magnitude the lower lane's stands first
    const float o1 = xchg<1>(m);
    m = (l4 & 1) ? (fabsf(o1) >= fabsf(m) ? o1 : m) : (fabsf(o1) > fabsf(m) ? o1 : m);
    const float o2 = xchg<2>(m);
    m = (l4 & 2) ? (fabsf(o2) >= fabsf(m) ? o2 : m) : (fabsf(o2) > fabsf(m) ? o2 : m);
    dh = f2h_bits(fminf(fmaxf(m * -0.125f, -65504.0f), 65504.0f));
    d = h2f(dh);
    kv_codes<-8, 7>(v, d, fabsf(m), u);
  }
  return d == 0.0f ? 0u : dh;
}

// this lane's token's slot
__device__ __forceinline__ int64_t kv_slot(const int64_t* slots, int t0, int t) {
  const int lane = threadIdx.x & 63;
  return t0 + lane < t ? slots[t0 + lane] : -1;
}
struct KvTokens {
  int64_t at[KV_TILE];   // byte of the page head in the pool
  int key[KV_TILE];      // the key in its page; -1: not in the cache (padding, or out of range)
  uint8_t rest[KV_TILE]; // the tokens of the cache that no run covers, in order
};
__device__ __forceinline__ uint64_t cover16(uint64_t m) {   // bits j .. j+15 of every bit j
  m |= m << 1;
  m |= m << 2;
  m |= m << 4;
  return m | (m << 8);
}
// The tile's slots, and which of its tokens start a run that fills 16 slots from a
// multiple of 16 on.  Every wave computes the same masks.  LIST: the tokens that no run covers are listed, where there are any
// (unconditionally, and for keys too, it took 3 % of an aligned prompt's store).
template <bool LIST, class IO>
__device__ __forceinline__ uint64_t kv_runs(const IO& io, int64_t s, int head_bytes, int head, KvTokens& tk, uint64_t& valid) {
  const int lane = threadIdx.x & 63;
  if (s >= io.n_slot) s = -1;
  if (threadIdx.x < 64) {
    tk.at[lane] = (s >> io.page_shift) * ((int64_t)io.heads * head_bytes) + (int64_t)head * head_bytes;
    tk.key[lane] = s < 0 ? -1 : (int)(s & (io.page - 1));
  }
  const int64_t before = __shfl_up(s, 1, 64);
  valid = __ballot(s >= 0);
  const uint64_t next = __ballot(lane > 0 && s >= 0 && s == before + 1);   // continues the token before it
  uint64_t run = next >> 1;   // bit j: tokens j+1 .. continue j
  run &= run >> 1;            // two
  run &= run >> 2;            // four
  run &= run >> 4;            // eight
  run &= (next >> 9) & (next >> 10) & (next >> 11) & (next >> 12);   // ... fifteen
  run &= (next >> 13) & (next >> 14) & (next >> 15);
  run &= __ballot(s >= 0 && (s & 15) == 0 && lane <= 48);
  const uint64_t rest = valid & ~cover16(run);
  if (LIST && rest != 0 && threadIdx.x < 64 && ((rest >> lane) & 1)) tk.rest[__popcll(rest & ((1ull << lane) - 1))] = (uint8_t)lane;
  return run;
}

// n-th set bit of m (m has more than n)
__device__ __forceinline__ int nth_bit(uint64_t m, int n) {
  for (int i = 0; i < n; ++i) m &= m - 1;
  return __builtin_ctzll(m);
}
// A unit is one block of four tokens, in 16 lanes: lane 16r + 4u + l4 of a wave holds
// elements 8 l4 .. 8 l4 + 7 of its token r, u one of the wave's four units.  A workgroup
// takes 16 units at a time, NB times; unit n is block n % NB of tokens 4 (n / NB) ..
struct KvUnit {
  int tok, b, l4;
};
template <int NB>
__device__ __forceinline__ KvUnit kv_unit(int it) {
  const int lane = threadIdx.x & 63, n = it * 16 + (threadIdx.x >> 6) * 4 + ((lane >> 2) & 3);
  const int quad = n / NB;
  return {4 * quad + (lane >> 4), n - quad * NB, lane & 3};
}
template <int NB>   // the first token of the wave's first unit
__device__ __forceinline__ int kv_unit_first(int it) {
  return 4 * ((it * 16 + wave_id() * 4) / NB);
}

// Eight bytes of a token per lane (a: 0..3, b: 4..7) <-> two bytes of four tokens: lane
// 16r + .. gets bytes 2r and 2r + 1 of tokens 0, 1, 2, 3.
__device__ __forceinline__ u32x2 kv_to_rows(u32x2 w) {
  const auto h = __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false);   // of tokens r & 1 and (r & 1) + 2
  const uint32_t lo = __builtin_amdgcn_perm(h[1], h[0], 0x05010400u), hi = __builtin_amdgcn_perm(h[1], h[0], 0x07030602u);
  const auto q = __builtin_amdgcn_permlane16_swap(lo, hi, false, false);
  return u32x2{__builtin_amdgcn_perm(q[1], q[0], 0x05010400u), __builtin_amdgcn_perm(q[1], q[0], 0x07030602u)};
}
__device__ __forceinline__ u32x2 kv_from_rows(u32x2 w) {
  const uint32_t lo = __builtin_amdgcn_perm(w[1], w[0], 0x06040200u), hi = __builtin_amdgcn_perm(w[1], w[0], 0x07050301u);
  const auto q = __builtin_amdgcn_permlane16_swap(lo, hi, false, false);
  const uint32_t a = __builtin_amdgcn_perm(q[1], q[0], 0x06040200u), b = __builtin_amdgcn_perm(q[1], q[0], 0x07050301u);
  const auto h = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return u32x2{h[0], h[1]};
}

// Rounds of units whose loads go out together (four at head size 128: 1.5 us slower, for
// the registers).
template <int NB> constexpr int KV_AHEAD = NB % 2 ? 1 : 2;

struct KvIo {
  uint8_t* pages;
  int64_t n_slot;              // n_pages * page
  int page, page_shift, heads;
  void* x;
  int64_t x_token, x_head;     // strides in elements
  int vec;                     // rows stay 16-byte aligned
};

template <int T, int NB, bool V>
__device__ __forceinline__ void kv_store_side(const KvIo& io, int ftype, const int64_t* slots, int t, int t0,
                                              int head, KvTokens& tk, uint8_t* s_tile) {
  constexpr int D = NB * 32;
  constexpr int ROWS = T == FT_Q8_0 ? D : D / 2;   // rows of the transposed tile
  constexpr int N = KV_AHEAD<NB>;
  const int tid = threadIdx.x;
  const int nt = min(KV_TILE, t - t0);
  const int hb = kv_head_bytes(T, D, io.page), cb = kv_code_bytes(T, D, io.page);
  const int64_t my_slot = kv_slot(slots, t0, t);
  uint64_t valid, runs = 0;
  for (int it0 = 0; it0 < NB; it0 += N) {
    // the rows' loads wait for nothing (those behind the last token: its own once more)
    u32x4 raw[N][2];
    int64_t at[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const KvUnit u = kv_unit<NB>(it0 + n);
      at[n] = (int64_t)min(t0 + u.tok, t - 1) * io.x_token + head * io.x_head + 32 * u.b + 8 * u.l4;
    }
    kv_load_raw<N>(ftype, io.x, at, io.vec, raw);
    if (it0 == 0) {
      runs = kv_runs<V>(io, my_slot, hb, head, tk, valid);
      __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (kv_unit_first<NB>(it0 + n) >= nt) break;   // the wave's units are all behind the last token
      const KvUnit u = kv_unit<NB>(it0 + n);
      float v[8];
      kv_raw_values(ftype, raw[n], v);
      uint32_t q[8];
      const uint32_t dh = kv_quantize<T>(v, u.l4, q);
      const int j = tk.key[u.tok];
      uint8_t* ph = io.pages + tk.at[u.tok];   // not followed where j < 0
      if (j >= 0 && u.l4 == 0) *(uint16_t*)(ph + cb + 2 * (u.b * io.page + j)) = (uint16_t)dh;
      if constexpr (!V) {
        if (j >= 0) {
          uint8_t* o = ph + kv_k_at<T, NB>(io.page, j, u.b, u.l4);
          if constexpr (T == FT_Q8_0) *(u32x2*)o = kv_bytes(q);
          else *(uint32_t*)o = kv_nibbles(q);
        }
      } else {
        u32x2 w = kv_bytes(q);
        int row = 32 * u.b + 8 * u.l4;
        if constexpr (T == FT_Q4_0) {   // elements 0..15, in lanes 0, 1, share their bytes with 16..31, in lanes 2, 3
#pragma unroll
          for (int i = 0; i < 2; ++i) w[i] |= __float_as_uint(xchg<2>(__uint_as_float(w[i]))) << 4;
          row = 16 * u.b + 8 * (u.l4 & 1);
        }
        w = kv_to_rows(w);
        const int r = row + 2 * (u.tok & 3);
        if (T == FT_Q8_0 || u.l4 < 2) {
          *(uint32_t*)(s_tile + r * KV_PITCH + (u.tok & ~3)) = w[0];
          *(uint32_t*)(s_tile + (r + 1) * KV_PITCH + (u.tok & ~3)) = w[1];
        }
      }
    }
  }
  if constexpr (V) {
    __syncthreads();
    const int n_run = __popcll(runs);
    for (int i = tid; i < n_run * ROWS; i += 256) {   // a row's runs side by side: often one piece of a page
      const int r = i / n_run, c = i - r * n_run;
      const int tok = nth_bit(runs, c);
      uint8_t* ph = io.pages + tk.at[tok];
      u32x4 w;
      const uint8_t* src = s_tile + r * KV_PITCH + tok;
      if ((tok & 3) == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = ((const uint32_t*)src)[k];
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = src[4 * k] | (src[4 * k + 1] << 8) | (src[4 * k + 2] << 16) | ((uint32_t)src[4 * k + 3] << 24);
      }
      *(u32x4*)(ph + r * io.page + tk.key[tok]) = w;
    }
    const int n_rest = __popcll(valid & ~cover16(runs));
    for (int i = tid; i < n_rest * ROWS; i += 256) {
      const int c = i / ROWS, r = i - c * ROWS;
      const int tok = tk.rest[c];
      uint8_t* ph = io.pages + tk.at[tok];
      ph[r * io.page + tk.key[tok]] = s_tile[r * KV_PITCH + tok];
    }
  }
}

// Tokens that a workgroup takes.  Values of tokens that lie far apart are single bytes, and what a workgroup of 64 does
// with them one after the other takes longer than all else: while there are CUs to spare it takes 16 or 4, at the
// price of runs of 16 that two workgroups share (stored and read back, with queries turned: 44 tokens of one head of
// 256 92 -> 9.7 us, 137 tokens of 4 heads of 256 56 -> 10.4, 24 of 4 heads of 128 20 -> 7.1).  16 tokens up to
// halves / 2 workgroups a CU: two, but one and a half where Q8_0 values are stored alone, whose single bytes cost the
// most (first slots 0 and 5; 2000 tokens of 4 heads of 128: by 16 tokens 5.0 and 9.2 us, by 64 5.4 and 6.9; 760 of 8
// heads: 4.6 and 7.9, 5.5 and 6.8).
inline int kv_span(int64_t t, int heads, int halves = 4) {
  if ((t + 3) / 4 * heads <= ftk_num_cus()) return 4;
  return (t + 15) / 16 * heads * 2 <= (int64_t)halves * ftk_num_cus() ? 16 : KV_TILE;
}

inline KvIo kv_io(const KvArgs& a, bool v) {
  KvIo io;
  io.pages = (uint8_t*)(v ? a.v_pages : a.k_pages);
  io.n_slot = a.n_pages * a.page;
  io.page = a.page;
  io.page_shift = __builtin_ctz(a.page);
  io.heads = a.heads;
  io.x = v ? a.v : a.k;
  io.x_token = v ? a.v_token : a.k_token;
  io.x_head = v ? a.v_head : a.k_head;
  const int64_t step = a.ftype == FT_F32 ? 4 : 8;   // elements in 16 bytes
  io.vec = ((uintptr_t)io.x & 15) == 0 && io.x_token % step == 0 && io.x_head % step == 0;
  return io;
}

}  // namespace ftk
