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
constexpr int LORA_FEW = 1024;   // adapters up to which a workgroup finds its tile by itself

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
  int copies;                        // out is not y: rows without an adapter are copied
  int parts, part_k;                 // shares of the long axis
  float* h;            // [parts][t][rank_pad]
  const int32_t* order;              // null: tiles from the ids
  const int4* tiles;                 // adapter, first place in order, tokens
  const int32_t* n_tiles;
  int words;                         // bytes of LDS for finding tiles
};

// Loads and stores below are whole whatever their address: rows need only their elements' alignment.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
template <int T> constexpr int LORA_WORDS = T == FT_F32 ? 2 : 1;   // of 16 bytes for eight elements

// eight elements, and the same of which those from `end` on count as zeros (e: the first's number in its row)
template <int T>
__device__ __forceinline__ void lora_load(const void* base, int64_t at, u32x4 (&r)[LORA_WORDS<T>]) {
  const u32x4_any* p = (const u32x4_any*)((const uint8_t*)base + at * (T == FT_F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < LORA_WORDS<T>; ++i) r[i] = p[i];
}
template <int T>
__device__ __forceinline__ void lora_load_end(const void* base, int64_t at, int e, int end, u32x4 (&r)[LORA_WORDS<T>]) {
  if (e + 8 <= end) {
    lora_load<T>(base, at, r);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t u = 0;
    if (e + i < end) u = T == FT_F32 ? ((const uint32_t*)base)[at + i] : ((const uint16_t*)base)[at + i];
    if constexpr (T == FT_F32) r[i >> 2][i & 3] = u;
    else r[0][i >> 1] = i & 1 ? r[0][i >> 1] | (u << 16) : u;
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
__device__ __forceinline__ void lora_operand(const u32x4 (&r)[LORA_WORDS<T>], bf16x8 (&o)[P]) {
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

// A tile: its adapter (or -1), that adapter's rank, how many tokens, and which.
struct LoraTile {
  int adapter, rank, count;
  int first;          // the first token of the 16 that are asked for
  int token;          // lane l of every wave: the tile's token l
};
// Tile `index` of the plan's, or of those that up to 64 ids make; with SIXTEENS the index counts
// groups of 16 tokens, tile by tile.  False: there are fewer.  Without a plan s_word has a word per adapter.
template <bool SIXTEENS>
__device__ __forceinline__ bool lora_tile(const LoraIo& io, int index, int* s_word, LoraTile& t) {
  const int lane = threadIdx.x & 63;
  t.first = 0;
  if (io.order) {
    if (SIXTEENS) {
      t.first = index & 3;
      index >>= 2;
      t.first *= 16;
    }
    const int n = *io.n_tiles;
    const int4 e = io.tiles[index];   // one beyond the last: whatever is there
    if (index >= n || t.first >= e.z) return false;
    t.adapter = e.x;
    t.count = e.z;
    t.rank = e.w;
    t.token = io.order[e.y + min(lane, e.z - 1)];
  } else {
    // each adapter's word: its first token, and from bit 8 on its tokens
    int a = lane < io.t ? io.ids[lane] : -2, rank = 0;
    const bool here = lane < io.t;
    if (here && (a < 0 || a >= io.adapters)) a = -1;
    if (a >= 0) rank = io.ranks ? max(0, min(io.ranks[a], io.rank)) : io.rank;
    int* word = s_word + (here ? a + 1 : 0);
    const bool counts = threadIdx.x < 64 && here;
    if (counts) *word = 64;
    __syncthreads();
    if (counts) atomicMin(word, lane);
    __syncthreads();
    if (counts) atomicAdd(word, 256);
    __syncthreads();
    const int w = here ? *word : 0;
    const bool leads = here && (w & 255) == lane;
    const int groups = SIXTEENS ? ((w >> 8) + 15) >> 4 : 1;
    const uint64_t below = (1ull << lane) - 1;
    int before = 0;
#pragma unroll
    for (int k = 1; k <= (SIXTEENS ? 4 : 1); ++k) before += __builtin_popcountll(__ballot(leads && groups >= k) & below);
    const uint64_t mine = __ballot(leads && before <= index && index < before + groups);
    if (!mine) return false;
    const int leader = __builtin_ctzll(mine);
    t.first = 16 * (index - __builtin_amdgcn_readlane(before, leader));
    t.adapter = __builtin_amdgcn_readlane(a, leader);
    t.rank = __builtin_amdgcn_readlane(rank, leader);
    const uint64_t m = __ballot(a == t.adapter);
    t.count = __builtin_popcountll(m);
    // every token of the tile goes to the lane of its rank among them; lanes behind the last take any
    const bool in = (m >> lane) & 1;
    const int src = __builtin_amdgcn_ds_permute(4 * (in ? __builtin_popcountll(m & below) : 63), in ? lane : leader);
    t.token = lane < t.count ? src : leader;
  }
  t.adapter = __builtin_amdgcn_readfirstlane(t.adapter);
  t.count = __builtin_amdgcn_readfirstlane(t.count);
  t.rank = __builtin_amdgcn_readfirstlane(t.rank);
  t.first = __builtin_amdgcn_readfirstlane(t.first);
  return true;
}

// h[part][token][rank] of 16 of a tile's tokens, for 16 * R ranks and one share of the long axis, which
// the four waves take in turn, U steps of 32 elements at a time with all of their loads in flight.
template <int TX, int TW, int R>
__global__ void __launch_bounds__(256)
lora_shrink_kernel(LoraIo io) {
  constexpr bool F16 = TX == FT_F16 && TW == FT_F16;
  constexpr int PX = LORA_PIECES<TX, TW>, PW = LORA_PIECES<TW, TX>, RX = LORA_WORDS<TX>, RW = LORA_WORDS<TW>;
  constexpr int U = RX + R * RW <= 3 ? 8 : RX + R * RW <= 6 ? 4 : 2;
  __shared__ __align__(16) float s_h[3][R][64][4];   // the other waves' sums
  extern __shared__ int s_word[];
  LoraTile tile;
  if (!lora_tile<true>(io, blockIdx.x, s_word, tile)) return;
  const int t0 = tile.first;
  const int r0 = blockIdx.z * (16 * R);
  if (r0 >= tile.rank) return;
  const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, quad = lane >> 4;
  const int k = (int)io.k, n_rt = (tile.rank - r0 + 15) >> 4;   // tiles of 16 ranks
  const int first = blockIdx.y * io.part_k, last = min(k, first + io.part_k);
  const int tok = __shfl(tile.token, min(t0 + l16, tile.count - 1), 64);
  const int64_t xrow = (int64_t)tok * io.ldx + 8 * quad;
  int64_t arow[R];
#pragma unroll
  for (int i = 0; i < R; ++i)   // rows past the adapter's rank: sums that nobody reads
    arow[i] = ((int64_t)tile.adapter * io.rank + min(r0 + 16 * i + l16, tile.rank - 1)) * k + 8 * quad;
  f32x4 acc[R];
#pragma unroll
  for (int i = 0; i < R; ++i) acc[i] = f32x4{0, 0, 0, 0};
  const auto sum = [&](const u32x4 (&rx)[RX], const u32x4 (&rw)[R][RW]) {
    bf16x8 px[PX];
    lora_operand<TX, PX>(rx, px);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i < n_rt) {
        bf16x8 pw[PW];
        lora_operand<TW, PW>(rw[i], pw);
        acc[i] = lora_mfma<F16>(pw, px, acc[i]);
      }
  };
  for (int k0 = first + 32 * U * wave; k0 < last; k0 += 32 * U * 4) {
    if (k0 + 32 * U <= last) {
      u32x4 rx[U][RX], rw[U][R][RW];
#pragma unroll
      for (int u = 0; u < U; ++u) lora_load<TX>(io.x, xrow + k0 + 32 * u, rx[u]);
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n_rt)
#pragma unroll
          for (int u = 0; u < U; ++u) lora_load<TW>(io.a, arow[i] + k0 + 32 * u, rw[u][i]);
#pragma unroll
      for (int u = 0; u < U; ++u) sum(rx[u], rw[u]);
    } else {
      for (int e = k0; e < last; e += 32) {
        u32x4 rx[RX], rw[R][RW];
        lora_load_end<TX>(io.x, xrow + e, e + 8 * quad, last, rx);
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (i < n_rt) lora_load_end<TW>(io.a, arow[i] + e, e + 8 * quad, last, rw[i]);
        sum(rx, rw);
      }
    }
  }
  // one wave for each tile of ranks adds the four up
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int to = R == 1 ? 0 : i & 3;
    if (wave != to) *(f32x4*)s_h[wave - (wave > to)][i][lane] = acc[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (wave != i || i >= n_rt || t0 + l16 >= tile.count) continue;
#pragma unroll
    for (int j = 0; j < 3; ++j) acc[i] += *(const f32x4*)s_h[j][i][lane];
    *(f32x4*)(io.h + ((int64_t)blockIdx.y * io.t + tok) * io.rank_pad + r0 + 16 * i + 4 * quad) = acc[i];
  }
}

// out = y + B h for a tile and 64 * C columns, 16 * C a wave: the wave's rows of B stay in its registers while it
// goes over the tile's tokens, 16 at a time, the next ones' y and h on their way.  With C = 4 the sums change
// places over LDS, so that y and out are read and written 256 bytes of a row at a time.  S: steps of 32 ranks; ONE: most
// tiles hold 16 tokens or fewer, nothing is kept ready for more
template <int TW, int S, int C, bool ONE>
__global__ void __launch_bounds__(256)
lora_expand_kernel(LoraIo io) {
  constexpr int PW = LORA_PIECES<TW, FT_F32>, RW = LORA_WORDS<TW>, PITCH = 16 * C + 4;
  constexpr int L = 4 * C, ROWS = 64 / L;   // lanes that share a row of y, rows they take at once
  __shared__ __align__(16) float s_out[C == 1 ? 1 : 4][C == 1 ? 1 : 16 * PITCH];
  extern __shared__ int s_word[];
  LoraTile tile;
  if (!lora_tile<false>(io, blockIdx.y, s_word, tile)) return;
  if (tile.rank == 0 && !io.copies) return;
  const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, quad = lane >> 4;
  const int n = (int)io.n, n0 = ((int)blockIdx.x * 4 + wave) * 16 * C;
  if (n0 >= n) return;
  // the lane's place in y: columns at .. at + 3 of row i * ROWS + line of 16
  const int line = C == 1 ? l16 : lane / L, at = n0 + 4 * (C == 1 ? quad : lane % L);
  constexpr int B = ONE ? 1 : 2;
  f32x4 y[B][C];
  f32x4 h[B][S][2];
  int tok[B][C];
  const auto load = [&](int t0, f32x4 (&y)[C], f32x4 (&h)[S][2], int (&tok)[C]) {
    const float* p = io.h + (int64_t)__shfl(tile.token, min(t0 + l16, tile.count - 1), 64) * io.rank_pad + 8 * quad;
    const int64_t step = (int64_t)io.t * io.rank_pad;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int row = t0 + i * ROWS + line;
      tok[i] = row < tile.count ? __shfl(tile.token, row, 64) : -1;
      y[i] = f32x4{0, 0, 0, 0};
      if (io.y && tok[i] >= 0) {
        const float* q = io.y + tok[i] * io.ldy + at;
        if (at + 4 <= n) y[i] = *(const f32x4_any*)q;
        else
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (at + e < n) y[i][e] = q[e];
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      h[s][0] = h[s][1] = f32x4{0, 0, 0, 0};
      if (32 * s + 8 * quad >= tile.rank) continue;
#pragma unroll 4
      for (int j = 0; j < io.parts; ++j) {
        h[s][0] += *(const f32x4*)(p + j * step + 32 * s);
        h[s][1] += *(const f32x4*)(p + j * step + 32 * s + 4);
      }
    }
  };
  u32x4 rw[S][C][RW];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int r = 32 * s + 8 * quad, bn = min(n0 + 16 * c + l16, n - 1);
#pragma unroll
      for (int i = 0; i < RW; ++i) rw[s][c][i] = u32x4{0, 0, 0, 0};
      if (r < tile.rank) lora_load_end<TW>(io.b, ((int64_t)tile.adapter * io.n + bn) * io.rank + r, r, tile.rank, rw[s][c]);
    }
  load(0, y[0], h[0], tok[0]);
  const float scale = tile.rank && io.scales ? io.scales[tile.adapter] : 1.0f;
  bf16x8 pw[S][C][PW];
  const auto operands = [&] {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int c = 0; c < C; ++c) lora_operand<TW, PW>(rw[s][c], pw[s][c]);
  };
  if (!ONE) operands();
#pragma unroll(ONE ? 1 : 4)
  for (int g = 0; g < 4; ++g) {
    const int b = ONE ? 0 : g & 1;
    if (16 * g >= tile.count) break;
    if (ONE && g) load(16 * g, y[0], h[0], tok[0]);
    if (ONE) operands();
    if (!ONE && 16 * (g + 1) < tile.count) load(16 * (g + 1), y[B - 1 - b], h[B - 1 - b], tok[B - 1 - b]);
    f32x4 acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (32 * s >= tile.rank) break;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 32 * s + 8 * quad + i < tile.rank ? h[b][s][i >> 2][i & 3] * scale : 0.0f;
      bf16x8 ph[3];
      lora_pieces<3>(v, ph);
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = lora_mfma<false>(pw[s][c], ph, acc[c]);
    }
    if constexpr (C > 1) {
      float* mine = s_out[wave];
#pragma unroll
      for (int c = 0; c < C; ++c) *(f32x4*)(mine + l16 * PITCH + 16 * c + 4 * quad) = acc[c];
      wave_lds_sync();
#pragma unroll
      for (int i = 0; i < C; ++i) acc[i] = *(const f32x4*)(mine + (i * ROWS + line) * PITCH + 4 * (lane % L));
      wave_lds_sync();
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (tok[b][i] < 0) continue;
      float* q = io.out + tok[b][i] * io.ldo + at;
      const f32x4 o = y[b][i] + acc[i];
      if (at + 4 <= n) *(f32x4_any*)q = o;
      else
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at + e < n) q[e] = o[e];
    }
  }
}

// the adapters of tokens i, i + 1024, .. (adapters: none; -2: no such token)
__device__ __forceinline__ void lora_ids(const int32_t* ids, int t, int adapters, int i, int (&a)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) a[j] = i + 1024 * j < t ? ids[i + 1024 * j] : -2;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + 1024 * j < t && (a[j] < 0 || a[j] >= adapters)) a[j] = adapters;
}

// The tokens sorted by adapter (those of none last) and cut into tiles, by one workgroup.
// Within an adapter the order is free: a token's result does not depend on its place.
__global__ void __launch_bounds__(1024)
lora_plan_kernel(const int32_t* __restrict__ ids, const int32_t* __restrict__ ranks, int most, int t, int adapters, int32_t* __restrict__ order,
                 int4* __restrict__ tiles, int32_t* __restrict__ n_tiles) {
  extern __shared__ int s_count[];   // [adapters + 1], then places
  __shared__ int s_wave[2][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), many = adapters + 1;
  for (int a = tid; a < many; a += 1024) s_count[a] = 0;
  __syncthreads();
  for (int i0 = 0; i0 < t; i0 += 4096) {
    int a[4];
    lora_ids(ids, t, adapters, i0 + tid, a);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int a0 = __builtin_amdgcn_readfirstlane(a[j]);
      if (a0 >= 0 && __ballot(a[j] == a0) == ~0ull) {
        if (lane == 0) atomicAdd(&s_count[a0], 64);
      } else if (a[j] >= 0) {
        atomicAdd(&s_count[a[j]], 1);
      }
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
    const int rank = a == adapters || c == 0 ? 0 : ranks ? max(0, min(ranks[a], most)) : most;
    for (int j = 0; j < c; j += LORA_TILE) tiles[before_m++] = int4{a == adapters ? -1 : a, before_n + j, min(LORA_TILE, c - j), rank};
    before_n += c;
  }
  __syncthreads();
  for (int i0 = 0; i0 < t; i0 += 4096) {
    int a[4];
    lora_ids(ids, t, adapters, i0 + tid, a);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 1024 * j + tid, a0 = __builtin_amdgcn_readfirstlane(a[j]);
      int at = 0;
      if (a0 >= 0 && __ballot(a[j] == a0) == ~0ull) {
        if (lane == 0) at = atomicAdd(&s_count[a0], 64);
        at = __builtin_amdgcn_readfirstlane(at) + lane;
      } else if (a[j] >= 0) {
        at = atomicAdd(&s_count[a[j]], 1);
      }
      if (i < t) order[at] = i;
    }
  }
}

// Shares of the long axis: enough workgroups for two per CU, at least 128 elements each.  Adapters that no
// token names cannot be told from here; each is counted as a tile.
struct LoraPlan {
  int parts, part_k, tiles, sixteens;   // tiles, and groups of 16 tokens, that there can be
  bool sorts;          // tiles from a plan, not from the ids
  int64_t likely;      // tiles that probably hold tokens
  size_t h, order, list, total;
};
static LoraPlan lora_plan(int64_t t, int64_t k, int rank, int64_t adapters) {
  LoraPlan p;
  const int64_t some = std::min<int64_t>(t, adapters + 1), cus = ftk_num_cus();
  p.likely = std::max<int64_t>((t + LORA_TILE - 1) / LORA_TILE, std::min<int64_t>(t, adapters));
  const int64_t sixteens = std::max<int64_t>((t + 15) / 16, std::min<int64_t>(t, adapters));
  int64_t parts = std::min<int64_t>(16, (2 * cus + sixteens - 1) / sixteens);
  parts = std::max<int64_t>(1, std::min(parts, (k + 127) / 128));
  p.part_k = (int)(((k + parts - 1) / parts + 127) / 128 * 128);
  p.parts = (int)((k + p.part_k - 1) / p.part_k);
  p.sorts = t > 64 || adapters > LORA_FEW;
  p.tiles = (int)(t <= 64 ? some : t / LORA_TILE + some);
  p.sixteens = (int)(p.sorts ? 4 * p.tiles : some + (t - 1) / 16);
  const size_t rank_pad = (size_t)(rank + 15) / 16 * 16;
  // no fewer than parts * t, here and for every smaller t
  p.h = (size_t)std::min<int64_t>(16 * t, 32 * cus + t) * rank_pad * 4;
  p.order = (p.h + 255) & ~(size_t)255;
  p.list = (p.order + (size_t)t * 4 + 255) & ~(size_t)255;
  p.total = p.list + 16 + (size_t)(t / LORA_TILE + some) * 16;
  return p;
}

template <int TX, int TW>
static hipError_t lora_shrink(const LoraIo& io, dim3 grid, hipStream_t st) {
  if (io.rank <= 16) lora_shrink_kernel<TX, TW, 1><<<grid, 256, io.words, st>>>(io);
  else if (io.rank <= 32) lora_shrink_kernel<TX, TW, 2><<<grid, 256, io.words, st>>>(io);
  else lora_shrink_kernel<TX, TW, 4><<<grid, 256, io.words, st>>>(io);
  return hipGetLastError();
}
template <int TW>
static hipError_t lora_shrink_x(int tx, const LoraIo& io, dim3 grid, hipStream_t st) {
  if (tx == FT_F32) return lora_shrink<FT_F32, TW>(io, grid, st);
  return tx == FT_F16 ? lora_shrink<FT_F16, TW>(io, grid, st) : lora_shrink<FT_BF16, TW>(io, grid, st);
}
// columns of a workgroup; ranks past 128 fill the registers with fewer
static int lora_cols(bool wide, int rank) { return 64 * (!wide || rank > 128 ? 1 : rank > 64 ? 2 : 4); }
template <int TW, int C, bool ONE>
static hipError_t lora_expand(const LoraIo& io, dim3 grid, hipStream_t st) {
  if (io.rank <= 32) lora_expand_kernel<TW, 1, C, ONE><<<grid, 256, io.words, st>>>(io);
  else if (io.rank <= 64) lora_expand_kernel<TW, 2, C, ONE><<<grid, 256, io.words, st>>>(io);
  else if (io.rank <= 128) lora_expand_kernel<TW, 4, C == 1 ? 1 : 2, ONE><<<grid, 256, io.words, st>>>(io);
  else lora_expand_kernel<TW, 8, 1, true><<<grid, 256, io.words, st>>>(io);
  return hipGetLastError();
}
template <int TW>
static hipError_t lora_expand_c(bool wide, bool one, const LoraIo& io, dim3 grid, hipStream_t st) {
  if (one) return wide ? lora_expand<TW, 4, true>(io, grid, st) : lora_expand<TW, 1, true>(io, grid, st);
  return wide ? lora_expand<TW, 4, false>(io, grid, st) : lora_expand<TW, 1, false>(io, grid, st);
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
  io.copies = a.out != a.y;
  io.parts = p.parts;
  io.part_k = p.part_k;
  io.h = (float*)s;
  io.order = nullptr;
  io.tiles = nullptr;
  io.n_tiles = nullptr;
  io.words = p.sorts ? 0 : (int)(a.adapters + 1) * 4;
  hipError_t e = hipSuccess;
  if (p.sorts) {
    io.order = (int32_t*)(s + p.order);
    io.n_tiles = (int32_t*)(s + p.list);
    io.tiles = (int4*)(s + p.list + 16);
    lora_plan_kernel<<<1, 1024, (size_t)(a.adapters + 1) * 4, st>>>(a.ids, a.ranks, a.rank, io.t, io.adapters, (int32_t*)io.order, (int4*)io.tiles,
                                                                     (int32_t*)io.n_tiles);
    e = hipGetLastError();
  }
  const dim3 shrink((unsigned)p.sixteens, (unsigned)p.parts, (unsigned)((a.rank + LORA_RANKS - 1) / LORA_RANKS));
  // 64 columns a wave where that still gives every CU a workgroup
  const bool wide = p.likely * a.n >= 256 * (int64_t)ftk_num_cus();
  const bool one = p.likely * 16 >= a.t;
  const int cols = lora_cols(wide, a.rank);
  const dim3 expand((unsigned)((a.n + cols - 1) / cols), (unsigned)p.tiles);   // tiles < 2^15: t is at most 2^20
  if (e == hipSuccess)
    e = a.wtype == FT_F32   ? lora_shrink_x<FT_F32>(a.xtype, io, shrink, st)
        : a.wtype == FT_F16 ? lora_shrink_x<FT_F16>(a.xtype, io, shrink, st)
                            : lora_shrink_x<FT_BF16>(a.xtype, io, shrink, st);
  if (e == hipSuccess)
    e = a.wtype == FT_F32   ? lora_expand_c<FT_F32>(wide, one, io, expand, st)
        : a.wtype == FT_F16 ? lora_expand_c<FT_F16>(wide, one, io, expand, st)
                            : lora_expand_c<FT_BF16>(wide, one, io, expand, st);
  return e;
}
