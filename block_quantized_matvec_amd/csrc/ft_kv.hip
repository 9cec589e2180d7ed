// ft_kv.hip -- the paged key/value cache: rows quantized as they are written
// (ft_kv_store) and read back (ft_kv_load).
//
// Blocks of 32 elements as the library's weight formats hold them, d in fp16 and the
// codes decided against the stored d with the exact quotient:
//   Q8_0  d = fp16(amax / 127),  q = clamp(round_half_away(x / d), -127, 127)
//   Q4_0  d = fp16(m / -8), m the first element of largest magnitude,
//         q = clamp(round_half_away(x / d), -8, 7)
// (d limited to the largest finite fp16; a zero d gives zero codes.)
//
// Both are bound by HBM at thousands of tokens and by latency at a decode step.  A
// workgroup takes 64 consecutive tokens of one head and of K or V; four lanes hold a
// block, eight elements each, so amax (or m) meets in two DPP steps.  K codes go
// straight to the page, eight at a time.  V is held transposed (a row per element,
// the page's keys side by side: the operand order of the attention's second
// product), so its codes meet in LDS and leave as 16-byte rows wherever 16
// consecutive tokens fill 16 consecutive slots from a multiple of 16 on; other
// tokens' codes are single bytes.
#include "ft_device.h"
#include "ft_internal.h"
#include "ft_kv.h"

namespace ftk {

constexpr int KV_TILE = 64;    // tokens per workgroup
constexpr int KV_PITCH = 68;   // bytes between the rows of the transposed tile in LDS (a bank further per row)

// The codes of N values of one block.  t = v * rcp(d) is within 1.5 * 2^-16 of v / d
// while |v / d| < 128, so it rounds to the code unless it lies within 2^-14 of a
// half-integer; there, and for a scale outside 2^+-100, the lane divides.
template <int LOW, int HIGH, int N>
__device__ __forceinline__ void kv_codes(const float (&v)[N], float d, int (&q)[N]) {
  const float r = __builtin_amdgcn_rcpf(d), ad = fabsf(d);
  bool slow = !(ad >= 0x1p-100f && ad <= 0x1p100f);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float t = v[j] * r;
    slow |= fabsf(__builtin_amdgcn_fractf(t) - 0.5f) <= 0x1p-14f;
    q[j] = (int)__builtin_rintf(fminf(fmaxf(t, (float)LOW), (float)HIGH));
  }
  if (slow) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float t = roundf(v[j] / (d == 0.0f ? 1.0f : d));
      q[j] = d == 0.0f ? 0 : (int)fminf(fmaxf(t, (float)LOW), (float)HIGH);
    }
  }
}

// One block's scale (fp16 bits) and this lane's eight codes; its four lanes call it
// together, lane l4 with elements 8*l4 .. 8*l4+7.
template <int T>
__device__ __forceinline__ uint32_t kv_quantize(const float (&v)[8], int l4, int (&q)[8]) {
  float d;
  uint32_t dh;
  if constexpr (T == FT_Q8_0) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(v[j]));
    a = fmaxf(a, xchg<1>(a));
    a = fmaxf(a, xchg<2>(a));
    dh = f2h_bits(fminf(a / 127.0f, 65504.0f));
    d = h2f(dh);
    kv_codes<-127, 127, 8>(v, d, q);
  } else {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fabsf(v[j]) > fabsf(m) ? v[j] : m;
    // of two of equal magnitude the lower lane's stands first
    const float o1 = xchg<1>(m);
    m = (l4 & 1) ? (fabsf(o1) >= fabsf(m) ? o1 : m) : (fabsf(o1) > fabsf(m) ? o1 : m);
    const float o2 = xchg<2>(m);
    m = (l4 & 2) ? (fabsf(o2) >= fabsf(m) ? o2 : m) : (fabsf(o2) > fabsf(m) ? o2 : m);
    dh = f2h_bits(fminf(fmaxf(m * -0.125f, -65504.0f), 65504.0f));
    d = h2f(dh);
    kv_codes<-8, 7, 8>(v, d, q);
  }
  return d == 0.0f ? 0u : dh;
}

// The tile's slots, and which of its tokens start a run that fills 16 slots from a
// multiple of 16 on.  Every wave computes the same masks; s_slot[j] < 0: token j is
// not in the cache (padding, or out of range).
__device__ __forceinline__ uint64_t kv_runs(const int64_t* slots, int64_t t0, int64_t t, int64_t n_slot, int64_t* s_slot,
                                            uint64_t& valid) {
  const int lane = threadIdx.x & 63;
  int64_t s = -1;
  if (t0 + lane < t) s = slots[t0 + lane];
  if (s >= n_slot) s = -1;
  if (threadIdx.x < 64) s_slot[lane] = s;
  const int64_t before = __shfl_up(s, 1, 64);
  valid = __ballot(s >= 0);
  const uint64_t next = __ballot(lane > 0 && s >= 0 && s == before + 1);   // continues the token before it
  uint64_t run = next >> 1;   // bit j: tokens j+1 .. continue j
  run &= run >> 1;            // two
  run &= run >> 2;            // four
  run &= run >> 4;            // eight
  run &= (next >> 9) & (next >> 10) & (next >> 11) & (next >> 12);   // ... fifteen
  run &= (next >> 13) & (next >> 14) & (next >> 15);
  return run & __ballot(s >= 0 && (s & 15) == 0 && lane <= 48);
}

// n-th set bit of m (m has more than n)
__device__ __forceinline__ int nth_bit(uint64_t m, int n) {
  for (int i = 0; i < n; ++i) m &= m - 1;
  return __builtin_ctzll(m);
}
__device__ __forceinline__ uint64_t cover16(uint64_t m) {   // bits j .. j+15 of every bit j
  m |= m << 1;
  m |= m << 2;
  m |= m << 4;
  return m | (m << 8);
}

struct KvIo {
  uint8_t* pages;
  int64_t n_slot;              // n_pages * page
  int page, page_shift, heads;
  void* x;
  int64_t x_token, x_head;     // strides in elements
  int vec;                     // rows stay 16-byte aligned
};

template <int T, int NB, bool V>
__device__ __forceinline__ void kv_store_side(const KvIo& io, int ftype, const int64_t* slots, int64_t t, int64_t t0,
                                              int head, int64_t* s_slot, uint8_t* s_tile) {
  constexpr int D = NB * 32;
  constexpr int ROWS = T == FT_Q8_0 ? D : D / 2;   // rows of the transposed tile
  const int tid = threadIdx.x, l4 = tid & 3;
  uint64_t valid;
  const uint64_t runs = kv_runs(slots, t0, t, io.n_slot, s_slot, valid);
  __syncthreads();
  const int nt = (int)min((int64_t)KV_TILE, t - t0);
  const int hb = kv_head_bytes(T, D, io.page), cb = kv_code_bytes(T, D, io.page);
  const int64_t page_bytes = (int64_t)io.heads * hb;
  for (int i = tid >> 2; i < nt * NB; i += 64) {
    const int tok = i / NB, b = i - tok * NB;
    const int64_t slot = s_slot[tok];
    if (slot < 0) continue;   // the block's four lanes together
    float v[8];
    kv_load8(ftype, io.x, (t0 + tok) * io.x_token + head * io.x_head + 32 * b + 8 * l4, io.vec, v);
    int q[8];
    const uint32_t dh = kv_quantize<T>(v, l4, q);
    const int j = (int)(slot & (io.page - 1));
    uint8_t* ph = io.pages + (slot >> io.page_shift) * page_bytes + (int64_t)head * hb;
    if (l4 == 0) *(uint16_t*)(ph + cb + 2 * (b * io.page + j)) = (uint16_t)dh;
    if constexpr (!V) {
      uint8_t* o = ph + kv_k_at<T, NB>(io.page, j, b, l4);
      if constexpr (T == FT_Q8_0) *(u32x2*)o = kv_pack8(q);
      else *(uint32_t*)o = kv_pack4(q);
    } else if constexpr (T == FT_Q8_0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s_tile[(32 * b + 8 * l4 + e) * KV_PITCH + tok] = (uint8_t)(q[e] + 128);
    } else {   // lanes 0, 1 hold elements 0..15, whose partners in lanes 2, 3 share their bytes
      int hi[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) hi[e] = __float_as_int(xchg<2>(__int_as_float(q[e] + 8)));
      if (l4 < 2) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          s_tile[(16 * b + 8 * l4 + e) * KV_PITCH + tok] = (uint8_t)((q[e] + 8) | (hi[e] << 4));
      }
    }
  }
  if constexpr (V) {
    __syncthreads();
    const int n_run = __popcll(runs);
    for (int i = tid; i < n_run * ROWS; i += 256) {
      const int c = i / ROWS, r = i - c * ROWS;
      const int tok = nth_bit(runs, c);
      const int64_t slot = s_slot[tok];
      uint8_t* ph = io.pages + (slot >> io.page_shift) * page_bytes + (int64_t)head * hb;
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
      *(u32x4*)(ph + r * io.page + (int)(slot & (io.page - 1))) = w;
    }
    const uint64_t rest = valid & ~cover16(runs);
    const int n_rest = __popcll(rest);
    for (int i = tid; i < n_rest * ROWS; i += 256) {
      const int c = i / ROWS, r = i - c * ROWS;
      const int tok = nth_bit(rest, c);
      const int64_t slot = s_slot[tok];
      uint8_t* ph = io.pages + (slot >> io.page_shift) * page_bytes + (int64_t)head * hb;
      ph[r * io.page + (int)(slot & (io.page - 1))] = s_tile[r * KV_PITCH + tok];
    }
  }
}

// grid: (token tiles, heads, 2): z = 0 the keys, 1 the values
template <int TK, int TV, int NB>
__global__ void __launch_bounds__(256)
kv_store_kernel(KvIo k, KvIo v, int ftype, const int64_t* __restrict__ slots, int64_t t) {
  __shared__ int64_t s_slot[KV_TILE];
  __shared__ __align__(16) uint8_t s_tile[NB * 32 * KV_PITCH];
  const int64_t t0 = (int64_t)blockIdx.x * KV_TILE;
  if (blockIdx.z == 0) kv_store_side<TK, NB, false>(k, ftype, slots, t, t0, blockIdx.y, s_slot, s_tile);
  else kv_store_side<TV, NB, true>(v, ftype, slots, t, t0, blockIdx.y, s_slot, s_tile);
}

template <int T, int NB, bool V>
__device__ __forceinline__ void kv_load_side(const KvIo& io, int ftype, const int64_t* slots, int64_t t, int64_t t0,
                                             int head, int64_t* s_slot, uint8_t* s_tile) {
  constexpr int D = NB * 32;
  constexpr int ROWS = T == FT_Q8_0 ? D : D / 2;
  const int tid = threadIdx.x, l4 = tid & 3;
  uint64_t valid;
  const uint64_t runs = kv_runs(slots, t0, t, io.n_slot, s_slot, valid);
  __syncthreads();
  const int nt = (int)min((int64_t)KV_TILE, t - t0);
  const int hb = kv_head_bytes(T, D, io.page), cb = kv_code_bytes(T, D, io.page);
  const int64_t page_bytes = (int64_t)io.heads * hb;
  if constexpr (V) {   // the codes into the transposed tile first
    const int n_run = __popcll(runs);
    for (int i = tid; i < n_run * ROWS; i += 256) {
      const int c = i / ROWS, r = i - c * ROWS;
      const int tok = nth_bit(runs, c);
      const int64_t slot = s_slot[tok];
      const uint8_t* ph = io.pages + (slot >> io.page_shift) * page_bytes + (int64_t)head * hb;
      const u32x4 w = *(const u32x4*)(ph + r * io.page + (int)(slot & (io.page - 1)));
      uint8_t* dst = s_tile + r * KV_PITCH + tok;
      if ((tok & 3) == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) ((uint32_t*)dst)[k] = w[k];
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) dst[k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
      }
    }
    const uint64_t rest = valid & ~cover16(runs);
    const int n_rest = __popcll(rest);
    for (int i = tid; i < n_rest * ROWS; i += 256) {
      const int c = i / ROWS, r = i - c * ROWS;
      const int tok = nth_bit(rest, c);
      const int64_t slot = s_slot[tok];
      const uint8_t* ph = io.pages + (slot >> io.page_shift) * page_bytes + (int64_t)head * hb;
      s_tile[r * KV_PITCH + tok] = ph[r * io.page + (int)(slot & (io.page - 1))];
    }
    __syncthreads();
  }
  for (int i = tid >> 2; i < nt * NB; i += 64) {
    const int tok = i / NB, b = i - tok * NB;
    const int64_t slot = s_slot[tok];
    float x[8];
    if (slot < 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    } else {
      const int j = (int)(slot & (io.page - 1));
      const uint8_t* ph = io.pages + (slot >> io.page_shift) * page_bytes + (int64_t)head * hb;
      const float d = h2f(*(const uint16_t*)(ph + cb + 2 * (b * io.page + j)));
      int q[8];
      if constexpr (V) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if constexpr (T == FT_Q8_0) q[e] = (int)s_tile[(32 * b + 8 * l4 + e) * KV_PITCH + tok] - 128;
          else q[e] = (int)((s_tile[(16 * b + 8 * (l4 & 1) + e) * KV_PITCH + tok] >> (l4 & 2 ? 4 : 0)) & 15u) - 8;
        }
      } else if constexpr (T == FT_Q8_0) {
        const u32x2 w = *(const u32x2*)(ph + kv_k_at<T, NB>(io.page, j, b, l4));
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = (int)((w[e >> 2] >> (8 * (e & 3))) & 255u) - 128;
      } else {
        const uint32_t w = *(const uint32_t*)(ph + kv_k_at<T, NB>(io.page, j, b, l4));
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = (int)((w >> (4 * ((e >> 1) + 4 * (e & 1)))) & 15u) - 8;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = d * (float)q[e];   // exact in fp32
    }
    kv_store_n<8>(ftype, io.x, (t0 + tok) * io.x_token + head * io.x_head + 32 * b + 8 * l4, io.vec, x);
  }
}

template <int TK, int TV, int NB>
__global__ void __launch_bounds__(256)
kv_load_kernel(KvIo k, KvIo v, int ftype, const int64_t* __restrict__ slots, int64_t t, int first) {
  __shared__ int64_t s_slot[KV_TILE];
  __shared__ __align__(16) uint8_t s_tile[NB * 32 * KV_PITCH];
  const int64_t t0 = (int64_t)blockIdx.x * KV_TILE;
  if (blockIdx.z + first == 0) kv_load_side<TK, NB, false>(k, ftype, slots, t, t0, blockIdx.y, s_slot, s_tile);
  else kv_load_side<TV, NB, true>(v, ftype, slots, t, t0, blockIdx.y, s_slot, s_tile);
}

static KvIo kv_io(const KvArgs& a, bool v) {
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

template <int TK, int TV, int NB>
static hipError_t kv_launch(const KvArgs& a, bool load, hipStream_t st) {
  const KvIo k = kv_io(a, false), v = kv_io(a, true);
  const unsigned tiles = (unsigned)((a.t + KV_TILE - 1) / KV_TILE);
  if (!load) {
    kv_store_kernel<TK, TV, NB><<<dim3(tiles, a.heads, 2), 256, 0, st>>>(k, v, a.ftype, a.slots, a.t);
  } else {
    const int first = a.k ? 0 : 1;
    kv_load_kernel<TK, TV, NB><<<dim3(tiles, a.heads, (a.k ? 1 : 0) + (a.v ? 1 : 0)), 256, 0, st>>>(k, v, a.ftype, a.slots,
                                                                                                  a.t, first);
  }
  return hipGetLastError();
}

template <int TK, int TV>
static hipError_t kv_pick(const KvArgs& a, bool load, hipStream_t st) {
  switch (a.dim) {
    case 64: return kv_launch<TK, TV, 2>(a, load, st);
    case 96: return kv_launch<TK, TV, 3>(a, load, st);
    case 128: return kv_launch<TK, TV, 4>(a, load, st);
    case 256: return kv_launch<TK, TV, 8>(a, load, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace ftk

hipError_t ftk_launch_kv(const KvArgs& a, bool load, hipStream_t st) {
  using namespace ftk;
  if (a.k_type == FT_Q8_0)
    return a.v_type == FT_Q8_0 ? kv_pick<FT_Q8_0, FT_Q8_0>(a, load, st) : kv_pick<FT_Q8_0, FT_Q4_0>(a, load, st);
  return a.v_type == FT_Q8_0 ? kv_pick<FT_Q4_0, FT_Q8_0>(a, load, st) : kv_pick<FT_Q4_0, FT_Q4_0>(a, load, st);
}
