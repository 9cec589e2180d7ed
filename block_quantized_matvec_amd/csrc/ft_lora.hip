// ft_lora.hip -- low-rank adapters of many requests beside a shared projection (ft_lora):
//   out_i = y_i + s_a B_a (A_a x_i),  a the adapter of token i.
//
// Tokens of one adapter are taken together, up to 64 a tile: up to 64 tokens in all, every
// workgroup of the first product finds its tile from the ids by itself and leaves it for the
// second; beyond, one workgroup sorts the tokens first (lora_plan_kernel, 5 us).  Two launches:
// h = A x (lora_shrink_kernel), the long axis split over a workgroup's waves and over workgroups,
// and out = y + B h (lora_expand_kernel), whose workgroups first add up the shares of h.
//
// Both products run on v_mfma_f32_16x16x32 with the weights' rows as rows of the result and
// the tokens as columns, so that a token's values come from its own row alone.  Accuracy is about fp32's:
// an fp32 operand is taken as three bf16 pieces (8 bits each, cut off, so their sum is exact), an
// fp16 one as two, and six (or five) products of pieces are summed.  Left out are the second piece times
// the third, both ways: as pieces are cut off these are below 2^-7 and 2^-15 of a value and have its sign, so
// a product comes out short by up to 2^-21 of itself (2^-24.5 on average).  fp16 rows with fp16 weights, and bf16
// with bf16, are one product and exact.  h stays in fp32 between the launches.
//
// Bound by memory: x, y, out and the rows of A and B that the tokens name.  4096 fp32 tokens,
// 4096 -> 14336, rank 64, bf16 weights (540 MB): 116 us (4.7 TB/s; a 2 GiB copy 5.0), of which 97 the
// second product, 19 the first.  1500 bf16 tokens of 16 adapters in any order, 14336 -> 4096, ranks
// 8 to 64 (110 MB): 41 us, a third of it two chains of dependent loads (tile, tokens, rows) and the sort.
// 48 tokens of 32 adapters, ranks 8 to 64, fp16 weights, 4096 -> 14336: 25 us; B's rows of 8 to 32 ranks lie
// 128 bytes apart, and whole lines come (59 MB for 27).  One token, 4096 -> 6144, rank 16: 7.2 us, two launches; in
// one launch, every workgroup reading all of A again, 9.5 to 11.
#include <algorithm>

#include "ft_internal.h"
#include "ft_kv.h"
#include "ft_device.h"

namespace ftk {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int LORA_TILE = 64;    // tokens per tile
constexpr int LORA_RANKS = 64;   // ranks per workgroup of the first product
constexpr int LORA_WGS = 2;      // workgroups per CU that the first product's split of the long axis aims at
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
  int blocks;                        // blocks of columns per workgroup of the second product
  float* h;            // [parts][t][rank_pad]
  int32_t* order;      // [tiles][64] tokens
  int4* tiles;         // adapter, rank, tokens
  int32_t* n_tiles;
  int sorted;          // the plan has run: they are there for the first product too
};

// Loads and stores below are whole whatever their address: rows need only their elements' alignment.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
template <int T> constexpr int LORA_WORDS = T == FT_F32 ? 2 : 1;   // of 16 bytes for eight elements

// eight elements, and the same of which those from `end` on count as zeros (e: the first's number in its row,
// which has one at least before the end, or reads the last one that is)
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
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {   // past the end the row's last again: no branches
    const int64_t j = at + min(i, end - 1 - e);
    u[i] = T == FT_F32 ? ((const uint32_t*)base)[j] : ((const uint16_t*)base)[j];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (e + i >= end) u[i] = 0;
    if constexpr (T == FT_F32) r[i >> 2][i & 3] = u[i];
    else if (i & 1) r[0][i >> 1] = u[i - 1] | (u[i] << 16);
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
__device__ __forceinline__ bool lora_tile(const LoraIo& io, int index, LoraTile& t) {
  const int lane = threadIdx.x & 63;
  const int n = *io.n_tiles;
  const int4 e = io.tiles[index];   // one beyond the last: whatever is there, as behind a tile's last token
  const int token = io.order[64 * index + lane];
  if (index >= n || t.first >= e.z) return false;
  t.adapter = __builtin_amdgcn_readfirstlane(e.x);
  t.rank = __builtin_amdgcn_readfirstlane(e.y);
  t.count = __builtin_amdgcn_readfirstlane(e.z);
  t.token = lane < t.count ? token : __builtin_amdgcn_readfirstlane(token);
  return true;
}
// The same from up to 64 ids, the index counting groups of 16 tokens, tile by tile; `leave`: the workgroup
// of a tile's first group writes it down.  s_word: a word per adapter and one for none.
__device__ __forceinline__ bool lora_find(const LoraIo& io, int index, int* s_word, bool leave, LoraTile& t) {
  const int lane = threadIdx.x & 63;
  int a = lane < io.t ? io.ids[lane] : -2, rank = 0;
  const bool here = lane < io.t;
  if (here && (a < 0 || a >= io.adapters)) a = -1;
  if (a >= 0) rank = io.ranks ? max(0, min(io.ranks[a], io.rank)) : io.rank;
  // an adapter's word: its first token, and from bit 8 on how many it has
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
  const int groups = ((w >> 8) + 15) >> 4;
  const uint64_t below = (1ull << lane) - 1, leaders = __ballot(leads);
  int before = 0;
#pragma unroll
  for (int k = 1; k <= 4; ++k) before += __builtin_popcountll(__ballot(leads && groups >= k) & below);
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
  if (leave && t.first == 0 && threadIdx.x < 64) {
    const int tile = __builtin_popcountll(leaders & ((1ull << leader) - 1));
    io.order[64 * tile + lane] = t.token;
    if (lane == 0) {
      io.tiles[tile] = int4{t.adapter, t.rank, t.count, 0};
      if (tile == 0) *io.n_tiles = __builtin_popcountll(leaders);
    }
  }
  return true;
}

// h[part][token][rank] of 16 * G of a tile's tokens, for 16 * R ranks and one share of the long axis, which
// the W waves take in turn, U steps of 32 elements at a time, a run's loads ahead of the one before.  G is 4
// where tiles are likely to be full: a row of A is then read once for 64 tokens (it comes from an L2 that all
// of them share, at half of the time of the whole kernel with G = 1).  The share is the fastest of
// the grid's indices: with eight of them, or four, each of the chip's eight L2s holds its own part of A.
template <int TX, int TW, int R, int G, int W>
__global__ void __launch_bounds__(64 * W)
lora_shrink_kernel(LoraIo io) {
  constexpr bool F16 = TX == FT_F16 && TW == FT_F16;
  constexpr int PX = LORA_PIECES<TX, TW>, PW = LORA_PIECES<TW, TX>, RX = LORA_WORDS<TX>, RW = LORA_WORDS<TW>;
  constexpr int U = G * RX + R * RW <= 8 && (G * R < 16 || PW == 1) ? 2 : 1;   // the last: for the registers
  __shared__ __align__(16) float s_h[W - 1][G * R][64][4];   // the other waves' sums
  extern __shared__ int s_word[];
  LoraTile tile;
  if (io.sorted) {
    tile.first = G == 1 ? 16 * (blockIdx.y & 3) : 0;
    if (!lora_tile(io, G == 1 ? blockIdx.y >> 2 : blockIdx.y, tile)) return;
  } else if (!lora_find(io, blockIdx.y, s_word, blockIdx.x == 0 && blockIdx.z == 0, tile)) {
    return;
  }
  const int r0 = blockIdx.z * (16 * R);
  if (r0 >= tile.rank) return;
  const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, quad = lane >> 4;
  const int k = (int)io.k, n_rt = (tile.rank - r0 + 15) >> 4;   // tiles of 16 ranks
  const int n_g = min(G, (tile.count - tile.first + 15) >> 4);  // groups of 16 tokens
  const int first = blockIdx.x * io.part_k, last = min(k, first + io.part_k);
  int tok[G];
  int64_t xrow[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    tok[g] = __shfl(tile.token, min(tile.first + 16 * g + l16, tile.count - 1), 64);
    xrow[g] = (int64_t)tok[g] * io.ldx + 8 * quad;
  }
  // the adapter's rows from one base: offsets of 32 bits (256 ranks of 2^20 fp32).  Rows past the adapter's
  // rank: sums that nobody reads
  const uint8_t* a = (const uint8_t*)io.a + (int64_t)tile.adapter * io.rank * k * (TW == FT_F32 ? 4 : 2);
  uint32_t arow[R];
#pragma unroll
  for (int i = 0; i < R; ++i) arow[i] = (uint32_t)min(r0 + 16 * i + l16, tile.rank - 1) * (uint32_t)k + 8 * quad;
  f32x4 acc[G][R];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int i = 0; i < R; ++i) acc[g][i] = f32x4{0, 0, 0, 0};
  u32x4 rx[2][U][G][RX], rw[2][U][R][RW];
  const auto load = [&](int k0, u32x4 (&rx)[U][G][RX], u32x4 (&rw)[U][R][RW]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (g < n_g) lora_load<TX>(io.x, xrow[g] + k0 + 32 * u, rx[u][g]);
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n_rt) {
          const u32x4_any* p = (const u32x4_any*)(a + (size_t)((arow[i] + k0 + 32 * u) * (TW == FT_F32 ? 4u : 2u)));
#pragma unroll
          for (int w = 0; w < RW; ++w) rw[u][i][w] = p[w];
        }
    }
  };
  const auto sum = [&](const u32x4 (&rx)[G][RX], const u32x4 (&rw)[R][RW]) {
    bf16x8 pw[R][PW];
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i < n_rt) lora_operand<TW, PW>(rw[i], pw[i]);
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (g < n_g) {
        bf16x8 px[PX];
        lora_operand<TX, PX>(rx[g], px);
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (i < n_rt) acc[g][i] = lora_mfma<F16>(pw[i], px, acc[g][i]);
      }
  };
  // whole runs of U steps, the next one's loads ahead of each; then what is left of the share, by the last wave
  const int run = 32 * U, runs = (last - first) / run, mine = runs > wave ? (runs - wave + W - 1) / W : 0, k0 = first + run * wave;
  if (mine > 0) load(k0, rx[0], rw[0]);
  for (int j = 0; j < mine; j += 2) {
    if (j + 1 < mine) load(k0 + (j + 1) * W * run, rx[1], rw[1]);
#pragma unroll
    for (int u = 0; u < U; ++u) sum(rx[0][u], rw[0][u]);
    if (j + 1 >= mine) break;
    if (j + 2 < mine) load(k0 + (j + 2) * W * run, rx[0], rw[0]);
#pragma unroll
    for (int u = 0; u < U; ++u) sum(rx[1][u], rw[1][u]);
  }
  if (wave == W - 1)
    for (int e = first + runs * run; e < last; e += 32) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (g < n_g) lora_load_end<TX>(io.x, xrow[g] + e, e + 8 * quad, last, rx[0][0][g]);
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n_rt) lora_load_end<TW>(a, arow[i] + e, e + 8 * quad, last, rw[0][0][i]);
      sum(rx[0][0], rw[0][0]);
    }
  // the waves' sums meet: wave (g R + i) % W adds up group g's ranks 16 i ..
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int to = (g * R + i) & (W - 1);
      if (wave != to && g < n_g && i < n_rt) *(f32x4*)s_h[wave - (wave > to)][g * R + i][lane] = acc[g][i];
    }
  __syncthreads();
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int to = (g * R + i) & (W - 1);
      if (wave != to || i >= n_rt || tile.first + 16 * g + l16 >= tile.count) continue;
      f32x4 s = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < W; ++j)   // in the waves' order, whichever group the token is in
        s += j == to ? acc[g][i] : *(const f32x4*)s_h[j - (j > to)][g * R + i][lane];
      *(f32x4*)(io.h + ((int64_t)blockIdx.x * io.t + tok[g]) * io.rank_pad + r0 + 16 * i + 4 * quad) = s;
    }
}

// LDS of a tile's h in the second product: [token][piece][LORA_PITCH], the pieces of a token's ranks one after the other
template <int S> constexpr int LORA_PITCH = 32 * S + 8;   // 16 bytes more: rows start on other banks

// out = y + B h for a tile and io.blocks * 64 * C columns, 16 * C a wave and block.  The workgroup adds up the parts of
// the tile's h once and leaves their pieces in LDS.  A wave's rows of B stay in its registers while it goes over the
// tile's tokens, 16 at a time.  What comes next is on its way meanwhile: the next tokens' y or, with ONE (most tiles
// hold 16 tokens or fewer, and B is what takes the time), the next block's B and y.  With C > 1 the sums
// change places over LDS, so that y and out are read and written 64 * C bytes of a row at a time.  S: steps of 32 ranks
template <int TW, int S, int C, bool ONE>
__global__ void __launch_bounds__(256, 2)
lora_expand_kernel(LoraIo io) {
  constexpr int PW = LORA_PIECES<TW, FT_F32>, RW = LORA_WORDS<TW>, PITCH = 16 * C + 4, HP = LORA_PITCH<S>;
  constexpr int L = 4 * C, ROWS = 64 / L;   // lanes that share a row of y, rows they take at once
  // with four tiles of columns y and out are larger than the L2s together: they pass them by (4096 rows of 14336:
  // 133 -> 120 us for the whole call)
  constexpr bool STREAM = C == 4;
  __shared__ __align__(16) float s_out[C == 1 ? 1 : 4][C == 1 ? 1 : 16 * PITCH];
  extern __shared__ __align__(16) uint8_t s_dyn[];
  __bf16* s_h = (__bf16*)s_dyn;
  LoraTile tile;
  tile.first = 0;
  if (!lora_tile(io, blockIdx.y, tile)) return;
  if (tile.rank == 0 && !io.copies) return;
  const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, quad = lane >> 4;
  const int n = (int)io.n, b0 = blockIdx.x * io.blocks, blocks = min(io.blocks, (n + 64 * C - 1) / (64 * C) - b0);
  // the lane's place in y: columns at .. at + 3 of row i * ROWS + line of 16
  const int line = C == 1 ? l16 : lane / L, column = 16 * C * wave + 4 * (C == 1 ? quad : lane % L);
  const auto load_y = [&](int at, int t0, f32x4 (&y)[C], int (&tok)[C]) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int row = t0 + i * ROWS + line, token = __shfl(tile.token, row, 64);   // of a lane that takes part
      tok[i] = row < tile.count && at < n ? token : -1;
      y[i] = f32x4{0, 0, 0, 0};
      if (io.y && tok[i] >= 0) {
        const float* q = io.y + tok[i] * io.ldy + at;
        if (at + 4 <= n) y[i] = STREAM ? __builtin_nontemporal_load((const f32x4_any*)q) : *(const f32x4_any*)q;
        else
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (at + e < n) y[i][e] = q[e];
      }
    }
  };
  const auto load_b = [&](int block, u32x4 (&rw)[S][C][RW]) {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int r = 32 * s + 8 * quad, bn = min(64 * C * block + 16 * (C * wave + c) + l16, n - 1);
#pragma unroll
        for (int i = 0; i < RW; ++i) rw[s][c][i] = u32x4{0, 0, 0, 0};
        if (r < tile.rank) lora_load_end<TW>(io.b, ((int64_t)tile.adapter * io.n + bn) * io.rank + r, r, tile.rank, rw[s][c]);
      }
  };
  const auto store = [&](int at, const f32x4 (&y)[C], const int (&tok)[C], int t0, const bf16x8 (&pw)[S][C][PW]) {
    f32x4 acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = f32x4{0, 0, 0, 0};
    const __bf16* h = s_h + min(t0 + l16, tile.count - 1) * (3 * HP) + 8 * quad;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (32 * s >= tile.rank) break;
      bf16x8 ph[3];
#pragma unroll
      for (int q = 0; q < 3; ++q) ph[q] = *(const bf16x8*)(h + q * HP + 32 * s);
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
      if (tok[i] < 0) continue;
      float* q = io.out + tok[i] * io.ldo + at;
      const f32x4 o = tile.rank ? y[i] + acc[i] : y[i];   // without ranks y's own bits: -0 + 0 is +0
      if (at + 4 <= n) {
        if constexpr (STREAM) __builtin_nontemporal_store(o, (f32x4_any*)q);
        else *(f32x4_any*)q = o;
      }
      if (at + 4 > n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at + e < n) q[e] = o[e];
    }
  };
  const auto operands = [&](const u32x4 (&rw)[S][C][RW], bf16x8 (&pw)[S][C][PW]) {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int c = 0; c < C; ++c) lora_operand<TW, PW>(rw[s][c], pw[s][c]);
  };
  u32x4 rw[ONE ? 2 : 1][S][C][RW];
  f32x4 y[ONE ? 2 : 1][C];
  int tok[ONE ? 2 : 1][C];
  load_b(b0, rw[0]);
  load_y(64 * C * b0 + column, 0, y[0], tok[0]);
  const float scale = tile.rank && io.scales ? io.scales[tile.adapter] : 1.0f;
  // eight ranks of a token per thread; those past the adapter's are zeros
  for (int i0 = 64 * wave; i0 < tile.count * 4 * S && tile.rank; i0 += 256) {
    const int i = i0 + lane, row = i / (4 * S), r = 8 * (i - row * (4 * S));
    const int token = __shfl(tile.token, min(row, tile.count - 1), 64);
    if (row >= tile.count) continue;
    f32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
    if (r < tile.rank) {
      const float* p = io.h + (int64_t)token * io.rank_pad + r;
      const int64_t step = (int64_t)io.t * io.rank_pad;
#pragma unroll 8
      for (int j = 0; j < io.parts; ++j) {
        a += *(const f32x4*)(p + j * step);
        b += *(const f32x4*)(p + j * step + 4);
      }
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = r + e < tile.rank ? (e < 4 ? a[e & 3] : b[e & 3]) * scale : 0.0f;
    bf16x8 o[3];
    lora_pieces<3>(v, o);
#pragma unroll
    for (int q = 0; q < 3; ++q) *(bf16x8*)(s_h + (row * 3 + q) * HP + r) = o[q];
  }
  __syncthreads();
  bf16x8 pw[S][C][PW];
  if constexpr (ONE) {
    const auto block = [&](int j, const u32x4 (&rw)[S][C][RW], f32x4 (&y)[C], int (&tok)[C]) {
      const int at = 64 * C * (b0 + j) + column;
      operands(rw, pw);
      store(at, y, tok, 0, pw);
      for (int t0 = 16; t0 < tile.count; t0 += 16) {
        load_y(at, t0, y, tok);
        store(at, y, tok, t0, pw);
      }
    };
    for (int j = 0; j < blocks; j += 2) {
      if (j + 1 < blocks) {
        load_b(b0 + j + 1, rw[1]);
        load_y(64 * C * (b0 + j + 1) + column, 0, y[1], tok[1]);
      }
      block(j, rw[0], y[0], tok[0]);
      if (j + 1 >= blocks) break;
      if (j + 2 < blocks) {
        load_b(b0 + j + 2, rw[0]);
        load_y(64 * C * (b0 + j + 2) + column, 0, y[0], tok[0]);
      }
      block(j + 1, rw[1], y[1], tok[1]);
    }
  } else {
    const int at = 64 * C * b0 + column;
    operands(rw[0], pw);
    // all of the tile's y before the first row is written: a load behind a store waits for it
    f32x4 more[3][C];
    int rows[3][C];
#pragma unroll
    for (int g = 1; g < 4; ++g)
      if (16 * g < tile.count) load_y(at, 16 * g, more[g - 1], rows[g - 1]);
    store(at, y[0], tok[0], 0, pw);
#pragma unroll
    for (int g = 1; g < 4; ++g)
      if (16 * g < tile.count) store(at, more[g - 1], rows[g - 1], 16 * g, pw);
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
  __shared__ int s_wave[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), many = adapters + 1;
  for (int a = tid; a < many; a += 1024) s_count[a] = 0;
  int kept[4];   // the first tokens' adapters, for both passes; the rank of this thread's first adapter, for the list
  lora_ids(ids, t, adapters, tid, kept);
  const int per = (many + 1023) / 1024, b0 = min(many, tid * per), b1 = min(many, b0 + per);
  int rank0 = most;
  if (ranks && b0 < adapters) rank0 = max(0, min(ranks[b0], most));
  __syncthreads();
  for (int i0 = 0; i0 < t; i0 += 4096) {
    int a[4] = {kept[0], kept[1], kept[2], kept[3]};
    if (i0) lora_ids(ids, t, adapters, i0 + tid, a);
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
  // the tiles before each adapter's: a run of adapters per thread, then over the threads
  int m = 0;
  for (int a = b0; a < b1; ++a) m += (s_count[a] + LORA_TILE - 1) / LORA_TILE;
  int before_m = m;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int um = __shfl_up(before_m, s, 64);
    if (lane >= s) before_m += um;
  }
  if (lane == 63) s_wave[wave] = before_m;
  __syncthreads();
  before_m -= m;
  for (int w = 0; w < wave; ++w) before_m += s_wave[w];
  if (tid == 1023) *n_tiles = before_m + m;
  for (int a = b0; a < b1; ++a) {
    const int c = s_count[a];
    s_count[a] = LORA_TILE * before_m;
    const int rank = a == adapters || c == 0 ? 0 : a == b0 || !ranks ? rank0 : max(0, min(ranks[a], most));
    for (int j = 0; j < c; j += LORA_TILE) tiles[before_m++] = int4{a == adapters ? -1 : a, rank, min(LORA_TILE, c - j), 0};
  }
  __syncthreads();
  for (int i0 = 0; i0 < t; i0 += 4096) {
    int a[4] = {kept[0], kept[1], kept[2], kept[3]};
    if (i0) lora_ids(ids, t, adapters, i0 + tid, a);
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

// Shares of the long axis, at least 128 elements each: so many that LORA_WGS workgroups of 16 tokens, or one of
// 64, come to a CU.  Adapters that no token names cannot be told from here; each is counted as a tile.
struct LoraPlan {
  int parts, part_k, tiles, sixteens;   // tiles, and groups of 16 tokens, that there can be
  bool sorts;          // tiles from a plan, not from the ids
  bool full;           // tiles hold more than 16 tokens on average, if every adapter is named
  int64_t likely;      // tiles that probably hold tokens
  size_t h, order, list, total;
};
static LoraPlan lora_plan(int64_t t, int64_t k, int rank, int64_t adapters) {
  LoraPlan p;
  const int64_t some = std::min<int64_t>(t, adapters + 1), cus = ftk_num_cus();
  p.likely = std::max<int64_t>((t + LORA_TILE - 1) / LORA_TILE, std::min<int64_t>(t, adapters));
  p.sorts = t > 64 || adapters > LORA_FEW;
  p.full = p.sorts && p.likely * 16 < t;
  const int64_t sixteens = std::max<int64_t>((t + 15) / 16, std::min<int64_t>(t, adapters));
  int64_t parts = p.full ? (cus + p.likely - 1) / p.likely : (LORA_WGS * cus + sixteens - 1) / sixteens;
  if (p.full)
    for (; parts & (parts - 1); parts &= parts - 1) {}   // a power of two
  parts = std::max<int64_t>(1, std::min(std::min<int64_t>(16, parts), (k + 127) / 128));
  p.part_k = (int)(((k + parts - 1) / parts + 127) / 128 * 128);
  p.parts = (int)((k + p.part_k - 1) / p.part_k);
  p.tiles = (int)(t <= 64 ? some : t / LORA_TILE + some);
  p.sixteens = (int)(p.sorts ? 4 * p.tiles : some + (t - 1) / 16);
  const size_t rank_pad = (size_t)(rank + 15) / 16 * 16;
  // no fewer than parts * t, here and for every smaller t: parts < cus * most / t + 1
  const int64_t most = std::max(16 * LORA_WGS, 64);
  p.h = (size_t)std::min<int64_t>(16 * t, most * cus + t) * rank_pad * 4;
  p.order = (p.h + 255) & ~(size_t)255;
  const size_t most_tiles = (size_t)(t / LORA_TILE + some);
  p.list = p.order + most_tiles * LORA_TILE * 4;
  p.total = p.list + 16 + most_tiles * 16;
  return p;
}

template <int TX, int TW, int R, int G>
static hipError_t lora_shrink_r(const LoraIo& io, bool eight, dim3 grid, hipStream_t st) {
  const int words = io.sorted ? 0 : (io.adapters + 1) * 4;   // for finding tiles
  // 64 ranks with many pieces: no registers for eight waves
  if constexpr (G == 4 && (R < 4 || LORA_PIECES<TX, TW> + LORA_PIECES<TW, TX> <= 4))
    if (eight) {
      lora_shrink_kernel<TX, TW, R, G, 8><<<grid, 512, words, st>>>(io);
      return hipGetLastError();
    }
  lora_shrink_kernel<TX, TW, R, G, 4><<<grid, 256, words, st>>>(io);
  return hipGetLastError();
}
template <int TX, int TW, int G>
static hipError_t lora_shrink(const LoraIo& io, bool eight, dim3 grid, hipStream_t st) {
  if (io.rank <= 16) return lora_shrink_r<TX, TW, 1, G>(io, eight, grid, st);
  if (io.rank <= 32) return lora_shrink_r<TX, TW, 2, G>(io, eight, grid, st);
  return lora_shrink_r<TX, TW, 4, G>(io, eight, grid, st);
}
template <int TW>
static hipError_t lora_shrink_x(int tx, bool full, bool eight, const LoraIo& io, dim3 grid, hipStream_t st) {
  if (full) {
    if (tx == FT_F32) return lora_shrink<FT_F32, TW, 4>(io, eight, grid, st);
    return tx == FT_F16 ? lora_shrink<FT_F16, TW, 4>(io, eight, grid, st) : lora_shrink<FT_BF16, TW, 4>(io, eight, grid, st);
  }
  if (tx == FT_F32) return lora_shrink<FT_F32, TW, 1>(io, eight, grid, st);
  return tx == FT_F16 ? lora_shrink<FT_F16, TW, 1>(io, eight, grid, st) : lora_shrink<FT_BF16, TW, 1>(io, eight, grid, st);
}
// tiles of 16 columns that a wave takes at a time; ranks past 64 fill the registers with fewer
static int lora_wide(bool wide, bool one, int rank) { return !wide || rank > 128 ? 1 : one || rank > 64 ? 2 : 4; }
template <int TW, int S, int C, bool ONE>
static hipError_t lora_expand_s(const LoraIo& io, dim3 grid, hipStream_t st) {
  const int h = std::min(io.t, LORA_TILE) * 3 * LORA_PITCH<S> * 2;   // at most 101 KB
  lora_expand_kernel<TW, S, C, ONE><<<grid, 256, h, st>>>(io);
  return hipGetLastError();
}
template <int TW, int C, bool ONE>
static hipError_t lora_expand(const LoraIo& io, dim3 grid, hipStream_t st) {
  if (io.rank <= 32) return lora_expand_s<TW, 1, C, ONE>(io, grid, st);
  if (io.rank <= 64) return lora_expand_s<TW, 2, C, ONE>(io, grid, st);
  if (io.rank <= 128) return lora_expand_s<TW, 4, C == 1 ? 1 : 2, ONE>(io, grid, st);
  return lora_expand_s<TW, 8, 1, true>(io, grid, st);
}
template <int TW>
static hipError_t lora_expand_c(bool wide, bool one, const LoraIo& io, dim3 grid, hipStream_t st) {
  if (one) return wide ? lora_expand<TW, 2, true>(io, grid, st) : lora_expand<TW, 1, true>(io, grid, st);
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
  io.order = (int32_t*)(s + p.order);
  io.n_tiles = (int32_t*)(s + p.list);
  io.tiles = (int4*)(s + p.list + 16);
  io.sorted = p.sorts;
  hipError_t e = hipSuccess;
  if (p.sorts) {
    lora_plan_kernel<<<1, 1024, (size_t)(a.adapters + 1) * 4, st>>>(a.ids, a.ranks, a.rank, io.t, io.adapters, io.order, io.tiles, io.n_tiles);
    e = hipGetLastError();
  }
  const int64_t cus = ftk_num_cus();
  const dim3 shrink((unsigned)p.parts, (unsigned)(p.full ? p.tiles : p.sixteens), (unsigned)((a.rank + LORA_RANKS - 1) / LORA_RANKS));
  // many columns a wave where that still gives every CU a workgroup; full tiles take a block of them, others so
  // many that three workgroups come to a CU
  const bool wide = p.likely * a.n >= 256 * cus, one = !p.full;
  const int64_t cols = 64 * lora_wide(wide, one, a.rank), across = (a.n + cols - 1) / cols;
  io.blocks = one || a.rank > 128 ? (int)std::max<int64_t>(1, std::min(across, p.likely * across / (3 * cus))) : 1;
  const dim3 expand((unsigned)((across + io.blocks - 1) / io.blocks), (unsigned)p.tiles);   // tiles < 2^15: t is at most 2^20
  // A workgroup that has a CU to itself keeps more loads on their way with eight waves (4096 fp32 tokens of one
  // adapter: first product 21.3 -> 19.0 us); where several share a CU four are faster (20000 bf16 tokens of 40, rank 64: 74 -> 69)
  const bool eight = p.likely * shrink.x * shrink.z <= cus;
  if (e == hipSuccess)
    e = a.wtype == FT_F32   ? lora_shrink_x<FT_F32>(a.xtype, p.full, eight, io, shrink, st)
        : a.wtype == FT_F16 ? lora_shrink_x<FT_F16>(a.xtype, p.full, eight, io, shrink, st)
                            : lora_shrink_x<FT_BF16>(a.xtype, p.full, eight, io, shrink, st);
  if (e == hipSuccess)
    e = a.wtype == FT_F32   ? lora_expand_c<FT_F32>(wide, one, io, expand, st)
        : a.wtype == FT_F16 ? lora_expand_c<FT_F16>(wide, one, io, expand, st)
                            : lora_expand_c<FT_BF16>(wide, one, io, expand, st);
  return e;
}
