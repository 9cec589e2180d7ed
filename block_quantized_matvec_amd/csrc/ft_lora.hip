// ft_lora.hip -- low-rank adapters of many requests beside a shared projection (ft_lora):
//   out_i = y_i + s_a B_a (A_a x_i),  a the adapter of token i.
//
// Tokens of one adapter are taken together, up to 64 a tile: up to 64 tokens in all, every
// workgroup finds its tile from the ids by ballots; beyond, one workgroup sorts the tokens
// first (lora_plan_kernel).  Then two launches: h = A x (lora_shrink_kernel), the long axis split
// over waves and over workgroups whose partial sums the second adds up, and out = y + B h
// (lora_expand_kernel).  A tile of 16 or fewer tokens gives its workgroup's four waves four
// shares of the axis (or of the columns), one of 64 gives each 16 tokens.
//
// Both products run on v_mfma_f32_16x16x32 with the weights' rows as rows of the result and
// the tokens as columns.  Accuracy is fp32's: an fp32 operand is taken as three bf16 pieces
// (8 bits each, cut off, so their sum is exact), an fp16 one as two, and the products of pieces
// down to 2^-16 of the first are summed (those left out are below 2^-24 of it).  fp16 rows with
// fp16 weights, and bf16 with bf16, are one product.  h stays in fp32 between the launches.
#include <algorithm>

#include "ft_internal.h"
#include "ft_kv.h"
#include "ft_device.h"

namespace ftk {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int LORA_TILE = 64;    // tokens per tile
constexpr int LORA_RANKS = 64;   // ranks per workgroup of the first product

struct LoraIo {
  const void* x;
  int64_t ldx;
  const float* y;      // nullable
  int64_t ldy;
  float* out;
  int64_t ldo;
  const void *a, *b;   // [adapters][rank][k], [adapters][n][rank]
  const int32_t *ids, *ranks;
  const float* scales;
  int64_t k, n;
  int t, rank, adapters, rank_pad;   // rank_pad: rank, rounded up to 16
  int vec_x, vec_a, vec_b, vec_y, copies;   // copies: out is not y, rows without an adapter are copied
  int parts, part_k;                 // shares of the long axis
  float* h;            // [parts][t][rank_pad]
  const int32_t* order;              // null: tiles from the ids
  const int4* tiles;                 // adapter, first place in order, tokens
  const int32_t* n_tiles;
};

// eight elements of a row from e on, those from `end` on as zeros; vec: 16-byte aligned and no end within
template <int T>
__device__ __forceinline__ void lora_load(const void* base, int64_t at, int e, int end, bool vec, u32x4 (&r)[T == FT_F32 ? 2 : 1]) {
  if (vec && e + 8 <= end) {
    if constexpr (T == FT_F32) {
      const u32x4* p = (const u32x4*)((const float*)base + at);
      r[0] = p[0];
      r[1] = p[1];
    } else {
      r[0] = *(const u32x4*)((const uint16_t*)base + at);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < (T == FT_F32 ? 2 : 1); ++i) r[i] = u32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (e + i >= end) break;
    if constexpr (T == FT_F32) r[i >> 2][i & 3] = ((const uint32_t*)base)[at + i];
    else r[0][i >> 1] |= (uint32_t)((const uint16_t*)base)[at + i] << (16 * (i & 1));
  }
}

// The pieces of eight values.  Cut off, not rounded: what is left is exact in fp32, and
// the last piece of an fp32 (or fp16) value holds all that is left.
template <int P>
__device__ __forceinline__ void lora_pieces(const float (&v)[8], bf16x8 (&o)[P]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __builtin_amdgcn_perm(__float_as_uint(r[2 * i + 1]), __float_as_uint(r[2 * i]), 0x07060302u);
    o[p] = __builtin_bit_cast(bf16x8, w);
    if (p + 1 < P)
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] -= __uint_as_float(__float_as_uint(r[i]) & 0xFFFF0000u);
  }
}
// of eight loaded elements; WITH: the other operand's type (two fp16 operands stay as they are)
template <int T, int WITH> constexpr int LORA_PIECES = T == FT_F32 ? 3 : T == FT_F16 && WITH != FT_F16 ? 2 : 1;
template <int T, int P>
__device__ __forceinline__ void lora_operand(const u32x4 (&r)[T == FT_F32 ? 2 : 1], bf16x8 (&o)[P]) {
  if constexpr (P == 1) {
    o[0] = __builtin_bit_cast(bf16x8, r[0]);
  } else {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (T == FT_F32) v[i] = __uint_as_float(r[i >> 2][i & 3]);
      else v[i] = h2f((r[0][i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
    }
    lora_pieces<P>(v, o);
  }
}
template <bool F16, int PA, int PB>
__device__ __forceinline__ f32x4 lora_mfma(const bf16x8 (&a)[PA], const bf16x8 (&b)[PB], f32x4 c) {
  if constexpr (F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h16x8, a[0]), __builtin_bit_cast(h16x8, b[0]), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int s = 2; s >= 0; --s)   // the smallest products first
#pragma unroll
      for (int i = 0; i < PA; ++i) {
        const int j = s - i;
        if (j >= 0 && j < PB) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], c, 0, 0, 0);
      }
    return c;
  }
}

// A tile: its adapter (or -1), how many tokens, and which.
struct LoraTile {
  int adapter, count, rank;
  int groups, ways;   // groups of 16 tokens (1, 2 or 4), waves per group
  int token;          // the lane's, in lane l of all waves the tile's token l
};
__device__ __forceinline__ bool lora_tile(const LoraIo& io, int index, LoraTile& t) {
  const int lane = threadIdx.x & 63;
  if (io.order) {
    if (index >= *io.n_tiles) return false;
    const int4 e = io.tiles[index];
    t.adapter = e.x;
    t.count = e.z;
    t.token = io.order[e.y + min(lane, e.z - 1)];
  } else {   // the tokens of token `index`'s adapter, if it is the first of them
    int a = lane < io.t ? io.ids[lane] : -2;
    if (lane < io.t && (a < 0 || a >= io.adapters)) a = -1;
    t.adapter = __builtin_amdgcn_readlane(a, index);
    const uint64_t m = __ballot(a == t.adapter);
    if (__builtin_ctzll(m) != index) return false;
    t.count = __builtin_popcountll(m);
    // lane l finds the l-th set bit: every lane tells its token to the lane of its rank
    const int place = __builtin_popcountll(m & ((1ull << lane) - 1));
    const bool in = (m >> lane) & 1;
    int src = 0;
    src = __builtin_amdgcn_ds_permute(4 * (in ? place : 63), in ? lane : 0);
    if (t.count < 64 && lane >= t.count) src = index;
    t.token = src;
  }
  t.adapter = __builtin_amdgcn_readfirstlane(t.adapter);
  t.count = __builtin_amdgcn_readfirstlane(t.count);
  t.rank = 0;
  if (t.adapter >= 0) t.rank = io.ranks ? __builtin_amdgcn_readfirstlane(max(0, min(io.ranks[t.adapter], io.rank))) : io.rank;
  t.groups = t.count <= 16 ? 1 : t.count <= 32 ? 2 : 4;
  t.ways = 4 / t.groups;
  return true;
}

// h[part][token][rank] of a tile, for 64 ranks and one share of the long axis
template <int TX, int TW>
__global__ void __launch_bounds__(256)
lora_shrink_kernel(LoraIo io) {
  constexpr bool F16 = TX == FT_F16 && TW == FT_F16;
  constexpr int PX = LORA_PIECES<TX, TW>, PW = LORA_PIECES<TW, TX>, RX = TX == FT_F32 ? 2 : 1, RW = TW == FT_F32 ? 2 : 1;
  __shared__ __align__(16) float s_h[3][64][4][4];   // the other waves' sums
  LoraTile tile;
  if (!lora_tile(io, blockIdx.x, tile)) return;
  const int r0 = blockIdx.z * LORA_RANKS;
  if (r0 >= tile.rank) return;
  const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, quad = lane >> 4;
  const int group = wave & (tile.groups - 1), way = wave / tile.groups;
  const int k = (int)io.k;
  // the workgroup's share of the axis, in steps of 32, dealt to its ways
  const int first = blockIdx.y * io.part_k, last = min(k, first + io.part_k);
  const int n_rt = min(4, (tile.rank - r0 + 15) >> 4);   // tiles of 16 ranks
  const int tok = __shfl(tile.token, min(16 * group + l16, tile.count - 1), 64);
  const int64_t xrow = (int64_t)tok * io.ldx;
  int64_t arow[4];
  bool there[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 16 * i + l16;
    there[i] = r < tile.rank;
    arow[i] = ((int64_t)tile.adapter * io.rank + (there[i] ? r : 0)) * k;
  }
  f32x4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = f32x4{0, 0, 0, 0};
  const bool used = 16 * group < tile.count;   // three groups: the fourth wave has none
  if (used) {
    for (int k0 = first + 32 * way; k0 < last; k0 += 32 * tile.ways) {
      const int e = k0 + 8 * quad;
      u32x4 rx[RX], rw[4][RW];
      lora_load<TX>(io.x, xrow + e, e, last, io.vec_x, rx);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n_rt) lora_load<TW>(io.a, arow[i] + e, e, there[i] ? last : 0, io.vec_a, rw[i]);
      bf16x8 px[PX];
      lora_operand<TX, PX>(rx, px);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n_rt) {
          bf16x8 pw[PW];
          lora_operand<TW, PW>(rw[i], pw);
          acc[i] = lora_mfma<F16>(pw, px, acc[i]);
        }
    }
  }
  if (tile.ways > 1) {
    if (way > 0)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n_rt) *(f32x4*)s_h[wave - tile.groups][lane][i] = acc[i];
    __syncthreads();
    if (way > 0) return;
    for (int j = 1; j < tile.ways; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n_rt) acc[i] += *(const f32x4*)s_h[(j - 1) * tile.groups + group][lane][i];
  }
  if (!used || 16 * group + l16 >= tile.count) return;
  float* o = io.h + ((int64_t)blockIdx.y * io.t + tok) * io.rank_pad + r0 + 4 * quad;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n_rt) *(f32x4*)(o + 16 * i) = acc[i];
}

constexpr int LORA_COLS = 256;   // columns per workgroup of the second product

// out = y + B h for a tile and 256 columns.  S: steps of 32 ranks
template <int TW, int S>
__global__ void __launch_bounds__(256)
lora_expand_kernel(LoraIo io) {
  constexpr int PW = LORA_PIECES<TW, FT_F32>, RW = TW == FT_F32 ? 2 : 1;
  LoraTile tile;
  if (!lora_tile(io, blockIdx.y, tile)) return;
  if (tile.rank == 0 && !io.copies) return;
  const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, quad = lane >> 4;
  const int group = wave & (tile.groups - 1), way = wave / tile.groups;
  if (16 * group >= tile.count) return;
  const bool live = 16 * group + l16 < tile.count;
  const int tok = __shfl(tile.token, min(16 * group + l16, tile.count - 1), 64);
  bf16x8 ph[S][3];
  const float scale = tile.rank && io.scales ? io.scales[tile.adapter] : 1.0f;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int r = 32 * s + 8 * quad;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (r < tile.rank) {
      const float* p = io.h + (int64_t)tok * io.rank_pad + r;
      const int64_t step = (int64_t)io.t * io.rank_pad;
      f32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
      for (int j = 0; j < io.parts; ++j, p += step) {
        a += *(const f32x4*)p;
        b += *(const f32x4*)(p + 4);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = r + i < tile.rank ? (i < 4 ? a[i & 3] : b[i & 3]) * scale : 0.0f;
    }
    lora_pieces<3>(v, ph[s]);
  }
  const int64_t yrow = (int64_t)tok * io.ldy, orow = (int64_t)tok * io.ldo;
  const int64_t n1 = min(io.n, (int64_t)(blockIdx.x + 1) * LORA_COLS);
  for (int64_t n0 = (int64_t)blockIdx.x * LORA_COLS + 16 * way; n0 < n1; n0 += 16 * tile.ways) {
    const int64_t c = n0 + 4 * quad;   // the lane's columns of the result
    f32x4 acc = {0, 0, 0, 0};
    const int64_t bn = min(n0 + l16, io.n - 1);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (32 * s >= tile.rank) break;
      const int r = 32 * s + 8 * quad;
      u32x4 rw[RW];
      lora_load<TW>(io.b, ((int64_t)tile.adapter * io.n + bn) * io.rank + r, r, tile.rank, io.vec_b, rw);
      bf16x8 pw[PW];
      lora_operand<TW, PW>(rw, pw);
      acc = lora_mfma<false>(pw, ph[s], acc);
    }
    if (!live) continue;
    if (io.vec_y && c + 4 <= io.n) {
      if (io.y) acc += *(const f32x4*)(io.y + yrow + c);
      *(f32x4*)(io.out + orow + c) = acc;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < io.n) io.out[orow + c + i] = acc[i] + (io.y ? io.y[yrow + c + i] : 0.0f);
    }
  }
}

// The tokens sorted by adapter (those of none last) and cut into tiles, by one workgroup.
// Within an adapter the order is free: a token's result does not depend on its place.
__global__ void __launch_bounds__(1024)
lora_plan_kernel(const int32_t* __restrict__ ids, int t, int adapters, int32_t* __restrict__ order, int4* __restrict__ tiles,
                 int32_t* __restrict__ n_tiles) {
  extern __shared__ int s_count[];   // [adapters + 1], then places
  __shared__ int s_wave[2][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), many = adapters + 1;
  for (int a = tid; a < many; a += 1024) s_count[a] = 0;
  __syncthreads();
  for (int i0 = 0; i0 < t; i0 += 1024) {
    const int i = i0 + tid;
    int a = i < t ? ids[i] : -2;
    if (i < t && (a < 0 || a >= adapters)) a = adapters;
    const int a0 = __builtin_amdgcn_readfirstlane(a);
    if (a0 >= 0 && __ballot(a == a0) == ~0ull) {
      if (lane == 0) atomicAdd(&s_count[a0], 64);
    } else if (a >= 0) {
      atomicAdd(&s_count[a], 1);
    }
  }
  __syncthreads();
  // places and tiles before each adapter's: a run of adapters per thread, then over the threads
  const int per = (many + 1023) / 1024, b0 = min(many, tid * per), b1 = min(many, b0 + per);
  int n = 0, m = 0;
  for (int a = b0; a < b1; ++a) {
    n += s_count[a];
    m += (s_count[a] + LORA_TILE - 1) / LORA_TILE;
  }
  int before_n = n, before_m = m;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int un = __shfl_up(before_n, s, 64), um = __shfl_up(before_m, s, 64);
    if (lane >= s) before_n += un, before_m += um;
  }
  if (lane == 63) s_wave[0][wave] = before_n, s_wave[1][wave] = before_m;
  __syncthreads();
  before_n -= n;
  before_m -= m;
  for (int w = 0; w < wave; ++w) before_n += s_wave[0][w], before_m += s_wave[1][w];
  if (tid == 1023) *n_tiles = before_m + m;
  for (int a = b0; a < b1; ++a) {
    const int c = s_count[a];
    s_count[a] = before_n;
    for (int j = 0; j < c; j += LORA_TILE) tiles[before_m++] = int4{a == adapters ? -1 : a, before_n + j, min(LORA_TILE, c - j), 0};
    before_n += c;
  }
  __syncthreads();
  for (int i0 = 0; i0 < t; i0 += 1024) {
    const int i = i0 + tid;
    int a = i < t ? ids[i] : -2;
    if (i < t && (a < 0 || a >= adapters)) a = adapters;
    const int a0 = __builtin_amdgcn_readfirstlane(a);
    int at = 0;
    if (a0 >= 0 && __ballot(a == a0) == ~0ull) {
      if (lane == 0) at = atomicAdd(&s_count[a0], 64);
      at = __builtin_amdgcn_readfirstlane(at) + lane;
    } else if (a >= 0) {
      at = atomicAdd(&s_count[a], 1);
    }
    if (i < t) order[at] = i;
  }
}

// Partial sums: enough workgroups for two per CU, a share of at least 128 elements.  Adapters
// that no token names cannot be told from here; each is counted as a tile.
struct LoraPlan {
  int parts, part_k, tiles;
  size_t h, order, list, total;
};
static LoraPlan lora_plan(int64_t t, int64_t k, int rank, int64_t adapters) {
  LoraPlan p;
  const int64_t some = std::min<int64_t>(t, adapters + 1);
  const int64_t likely = std::max<int64_t>((t + LORA_TILE - 1) / LORA_TILE, std::min<int64_t>(t, adapters));
  int64_t parts = std::min<int64_t>(16, (2 * ftk_num_cus() + likely - 1) / likely);
  parts = std::max<int64_t>(1, std::min(parts, (k + 127) / 128));
  p.part_k = (int)(((k + parts - 1) / parts + 127) / 128 * 128);
  p.parts = (int)((k + p.part_k - 1) / p.part_k);
  p.tiles = (int)(t <= 64 ? t : t / LORA_TILE + some);
  const size_t rank_pad = (size_t)(rank + 15) / 16 * 16;
  // parts * t grows with t up to here whatever the parts: a bound for every smaller t too
  p.h = (size_t)std::min<int64_t>(16 * t, 128 * ftk_num_cus() + t) * rank_pad * 4;
  p.order = (p.h + 255) & ~(size_t)255;
  p.list = (p.order + (size_t)t * 4 + 255) & ~(size_t)255;
  p.total = p.list + 16 + (size_t)(t / LORA_TILE + some) * 16;
  return p;
}

template <int TX, int TW>
static hipError_t lora_shrink(const LoraIo& io, dim3 grid, hipStream_t st) {
  lora_shrink_kernel<TX, TW><<<grid, 256, 0, st>>>(io);
  return hipGetLastError();
}
template <int TW>
static hipError_t lora_shrink_x(int tx, const LoraIo& io, dim3 grid, hipStream_t st) {
  if (tx == FT_F32) return lora_shrink<FT_F32, TW>(io, grid, st);
  return tx == FT_F16 ? lora_shrink<FT_F16, TW>(io, grid, st) : lora_shrink<FT_BF16, TW>(io, grid, st);
}
template <int TW>
static hipError_t lora_expand(const LoraIo& io, dim3 grid, hipStream_t st) {
  if (io.rank <= 32) lora_expand_kernel<TW, 1><<<grid, 256, 0, st>>>(io);
  else if (io.rank <= 64) lora_expand_kernel<TW, 2><<<grid, 256, 0, st>>>(io);
  else if (io.rank <= 128) lora_expand_kernel<TW, 4><<<grid, 256, 0, st>>>(io);
  else lora_expand_kernel<TW, 8><<<grid, 256, 0, st>>>(io);
  return hipGetLastError();
}

}  // namespace ftk

size_t ftk_lora_scratch(int64_t t, int64_t k, int rank, int64_t adapters) { return ftk::lora_plan(t, k, rank, adapters).total; }

hipError_t ftk_launch_lora(const LoraArgs& a, void* scratch, hipStream_t st) {
  using namespace ftk;
  const LoraPlan p = lora_plan(a.t, a.k, a.rank, a.adapters);
  uint8_t* s = (uint8_t*)scratch;
  LoraIo io;
  io.x = a.x;
  io.ldx = a.ldx;
  io.y = a.y;
  io.ldy = a.ldy;
  io.out = a.out;
  io.ldo = a.ldo;
  io.a = a.a;
  io.b = a.b;
  io.ids = a.ids;
  io.ranks = a.ranks;
  io.scales = a.scales;
  io.k = a.k;
  io.n = a.n;
  io.t = (int)a.t;
  io.rank = a.rank;
  io.adapters = (int)a.adapters;
  io.rank_pad = (a.rank + 15) / 16 * 16;
  const int64_t wx = a.xtype == FT_F32 ? 4 : 8, ww = a.wtype == FT_F32 ? 4 : 8;
  io.vec_x = ((uintptr_t)a.x & 15) == 0 && a.ldx % wx == 0;
  io.vec_a = ((uintptr_t)a.a & 15) == 0 && a.k % ww == 0;
  io.vec_b = ((uintptr_t)a.b & 15) == 0 && a.rank % ww == 0;
  io.vec_y = (((uintptr_t)a.y | (uintptr_t)a.out) & 15) == 0 && (a.ldy % 4 == 0 || !a.y) && a.ldo % 4 == 0;
  io.copies = a.out != a.y;
  io.parts = p.parts;
  io.part_k = p.part_k;
  io.h = (float*)s;
  io.order = nullptr;
  io.tiles = nullptr;
  io.n_tiles = nullptr;
  hipError_t e = hipSuccess;
  if (a.t > 64) {
    io.order = (int32_t*)(s + p.order);
    io.n_tiles = (int32_t*)(s + p.list);
    io.tiles = (int4*)(s + p.list + 16);
    lora_plan_kernel<<<1, 1024, (size_t)(a.adapters + 1) * 4, st>>>(a.ids, io.t, io.adapters, (int32_t*)io.order, (int4*)io.tiles,
                                                                     (int32_t*)io.n_tiles);
    e = hipGetLastError();
  }
  const dim3 shrink((unsigned)p.tiles, (unsigned)p.parts, (unsigned)((a.rank + LORA_RANKS - 1) / LORA_RANKS));
  const dim3 expand((unsigned)((a.n + LORA_COLS - 1) / LORA_COLS), (unsigned)p.tiles);   // tiles < 2^15: t is at most 2^20
  if (e == hipSuccess)
    e = a.wtype == FT_F32   ? lora_shrink_x<FT_F32>(a.xtype, io, shrink, st)
        : a.wtype == FT_F16 ? lora_shrink_x<FT_F16>(a.xtype, io, shrink, st)
                            : lora_shrink_x<FT_BF16>(a.xtype, io, shrink, st);
  if (e == hipSuccess)
    e = a.wtype == FT_F32   ? lora_expand<FT_F32>(io, expand, st)
        : a.wtype == FT_F16 ? lora_expand<FT_F16>(io, expand, st)
                            : lora_expand<FT_BF16>(io, expand, st);
  return e;
}
