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
// A workgroup takes 64, 16 or 4 consecutive tokens (kv_span) of one head and of K or V; four lanes hold a
// block, eight elements each, so amax (or m) meets in two DPP steps, and a wave takes four
// tokens of each of its blocks.  K codes go straight to the page, eight at a time.  V is
// held transposed (a row per element, the page's keys side by side: the operand order of
// the attention's second product): the codes of four tokens change places between lanes,
// so that words of four keys meet in LDS, and leave as 16-byte rows wherever 16
// consecutive tokens fill 16 consecutive slots from a multiple of 16 on; other tokens'
// codes are single bytes.
//
// At a decode step both are launch and latency (3.5 us each).  8192 bf16 tokens of 8 heads
// of 128, K in Q8_0 and V in Q4_0 (33 MB of rows, 14 MB of cache), first slot a multiple of 16: reading
// back 9.5 us, at the rate of a copy; writing 13.7 us, of which vector instructions issue for 9, 170 per
// eight elements and wave, while the waves wait for half of their time (208 instructions, and
// 18 us, while every value near a half-integer divided; byte writes to LDS in place of the
// exchange between lanes: 17.6 and 12.6 us).  From slot 5 on, where a quarter of V leaves and
// returns as single bytes, 15.9 and 12.0.  fp32 rows, twice the bytes, K in Q4_0 and V in Q8_0: 16 and 18.
#include "ft_kv_store.h"

namespace ftk {

// grid: (token tiles, heads, 2): z = 0 the keys, 1 the values
template <int TK, int TV, int NB>
__global__ void __launch_bounds__(256)
kv_store_kernel(KvIo k, KvIo v, int ftype, const int64_t* __restrict__ slots, int t, int span) {
  __shared__ KvTokens s_tok;
  __shared__ __align__(16) uint8_t s_tile[NB * 32 * KV_PITCH];
  const int t0 = blockIdx.x * span;
  t = min(t, t0 + span);
  if (blockIdx.z == 0) kv_store_side<TK, NB, false>(k, ftype, slots, t, t0, blockIdx.y, s_tok, s_tile);
  else kv_store_side<TV, NB, true>(v, ftype, slots, t, t0, blockIdx.y, s_tok, s_tile);
}

template <int T, int NB, bool V>
__device__ __forceinline__ void kv_load_side(const KvIo& io, int ftype, const int64_t* slots, int t, int t0,
                                             int head, KvTokens& tk, uint8_t* s_tile) {
  constexpr int D = NB * 32;
  constexpr int ROWS = T == FT_Q8_0 ? D : D / 2;
  constexpr int N = KV_AHEAD<NB>;
  const int tid = threadIdx.x;
  uint64_t valid;
  const int hb = kv_head_bytes(T, D, io.page), cb = kv_code_bytes(T, D, io.page);
  const uint64_t runs = kv_runs<V>(io, kv_slot(slots, t0, t), hb, head, tk, valid);
  __syncthreads();
  const int nt = min(KV_TILE, t - t0);
  if constexpr (V) {   // the codes into the transposed tile first
    const int n_run = __popcll(runs), n_rest = __popcll(valid & ~cover16(runs));
    for (int i = tid; i < n_run * ROWS; i += 256) {   // a row's runs side by side: often one piece of a page
      const int r = i / n_run, c = i - r * n_run;
      const int tok = nth_bit(runs, c);
      const u32x4 w = *(const u32x4*)(io.pages + tk.at[tok] + r * io.page + tk.key[tok]);
      uint8_t* dst = s_tile + r * KV_PITCH + tok;
      if ((tok & 3) == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) ((uint32_t*)dst)[k] = w[k];
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) dst[k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
      }
    }
    // four loads per thread in flight before the first is put down
    for (int i0 = tid; i0 < n_rest * ROWS; i0 += 1024) {
      uint8_t b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + 256 * q, c = i / ROWS;
        if (i >= n_rest * ROWS) continue;
        const int tok = tk.rest[c];
        b[q] = (io.pages + tk.at[tok])[(i - c * ROWS) * io.page + tk.key[tok]];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + 256 * q, c = i / ROWS;
        if (i < n_rest * ROWS) s_tile[(i - c * ROWS) * KV_PITCH + tk.rest[c]] = b[q];
      }
    }
    __syncthreads();
  }
  for (int it0 = 0; it0 < NB; it0 += N) {
    uint32_t d[N];
    u32x2 w[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const KvUnit u = kv_unit<NB>(it0 + n);
      const int j = tk.key[u.tok];
      d[n] = 0;
      w[n] = u32x2{0u, 0u};
      if (j >= 0) {
        const uint8_t* ph = io.pages + tk.at[u.tok];
        d[n] = *(const uint16_t*)(ph + cb + 2 * (u.b * io.page + j));
        if constexpr (!V) {
          if constexpr (T == FT_Q8_0) w[n] = *(const u32x2*)(ph + kv_k_at<T, NB>(io.page, j, u.b, u.l4));
          else w[n][0] = *(const uint32_t*)(ph + kv_k_at<T, NB>(io.page, j, u.b, u.l4));
        }
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (kv_unit_first<NB>(it0 + n) >= nt) break;
      const KvUnit u = kv_unit<NB>(it0 + n);
      if constexpr (V) {
        const int r = (T == FT_Q8_0 ? 32 * u.b + 8 * u.l4 : 16 * u.b + 8 * (u.l4 & 1)) + 2 * (u.tok & 3);
        w[n] = kv_from_rows(u32x2{*(const uint32_t*)(s_tile + r * KV_PITCH + (u.tok & ~3)),
                                  *(const uint32_t*)(s_tile + (r + 1) * KV_PITCH + (u.tok & ~3))});
      }
      if constexpr (T == FT_Q4_0) {   // a byte per code
        if constexpr (V) {
          w[n] = (w[n] >> (u.l4 & 2 ? 4 : 0)) & 0x0F0F0F0Fu;
        } else {
          const uint32_t even = w[n][0] & 0x0F0F0F0Fu, odd = (w[n][0] >> 4) & 0x0F0F0F0Fu;   // elements 0 4 1 5, 2 6 3 7
          w[n] = u32x2{__builtin_amdgcn_perm(odd, even, 0x06040200u), __builtin_amdgcn_perm(odd, even, 0x07050301u)};
        }
      }
      // d * (code - 128), exact in fp32; a token that is not there has d = 0
      const float df = h2f(d[n]), less = df * (T == FT_Q8_0 ? -128.0f : -8.0f);
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(df, (float)((w[n][e >> 2] >> (8 * (e & 3))) & 255u), less);
      if (u.tok < nt)
        kv_store_n<8>(ftype, io.x, (int64_t)(t0 + u.tok) * io.x_token + head * io.x_head + 32 * u.b + 8 * u.l4, io.vec, x);
    }
  }
}

template <int TK, int TV, int NB>
__global__ void __launch_bounds__(256)
kv_load_kernel(KvIo k, KvIo v, int ftype, const int64_t* __restrict__ slots, int t, int span, int first) {
  __shared__ KvTokens s_tok;
  __shared__ __align__(16) uint8_t s_tile[NB * 32 * KV_PITCH];
  const int t0 = blockIdx.x * span;
  t = min(t, t0 + span);
  if (blockIdx.z + first == 0) kv_load_side<TK, NB, false>(k, ftype, slots, t, t0, blockIdx.y, s_tok, s_tile);
  else kv_load_side<TV, NB, true>(v, ftype, slots, t, t0, blockIdx.y, s_tok, s_tile);
}

template <int TK, int TV, int NB>
static hipError_t kv_launch(const KvArgs& a, bool load, hipStream_t st) {
  const KvIo k = kv_io(a, false), v = kv_io(a, true);
  const int span = kv_span(a.t, a.heads, !load && TV == FT_Q8_0 ? 3 : 4);
  const unsigned tiles = (unsigned)((a.t + span - 1) / span);
  if (!load) {
    kv_store_kernel<TK, TV, NB><<<dim3(tiles, a.heads, 2), 256, 0, st>>>(k, v, a.ftype, a.slots, (int)a.t, span);
  } else {
    const int first = a.k ? 0 : 1;
    kv_load_kernel<TK, TV, NB><<<dim3(tiles, a.heads, (a.k ? 1 : 0) + (a.v ? 1 : 0)), 256, 0, st>>>(k, v, a.ftype, a.slots, (int)a.t, span,
                                                                                                  first);
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
