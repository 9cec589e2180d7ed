// ft_api.cpp -- the C ABI of libft.so: argument validation, the per-format
// capability table, the per-stream grow-only scratch pool and dispatch.
//
// Refusal happens on the host before anything is enqueued, and the capability
// table is the one the dispatcher uses (vllm.cpp PR #523, review and rework:
// per-dtype availability instead of a boolean; refuse before the first
// forward).  Scratch comes from a per-stream pool that only grows and retires
// buffers instead of freeing them while work may be in flight (same PR: a
// grow-only per-stream pool, no per-call malloc/free/synchronize).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

#include "ft.h"
#include "ft_internal.h"

namespace {

constexpr int kTypes = 13;
constexpr int kElems[kTypes] = {32, 32, 256, 256, 256, 32, 32, 256, 256, 256, 32, 32, 32};
constexpr int kBytes[kTypes] = {18, 34, 144, 176, 210, 17, 36, 292, 84, 110, 20, 22, 24};

bool is_weight(int t) { return (t >= FT_Q4_0 && t <= FT_MXFP4) || (t >= FT_Q2_K && t <= FT_Q5_1); }
// Q8_0 is a weight format and, with the same block layout, an activation format
bool is_act(int t) { return t == FT_Q8_1 || t == FT_Q8_K || t == FT_Q8_0; }
bool is_kv_type(int t) { return t == FT_Q8_0 || t == FT_Q4_0; }
bool is_float(int t) { return t == FT_F32 || t == FT_F16 || t == FT_BF16; }
bool float_aligned(const void* p, int t) { return ((uintptr_t)p & (t == FT_F32 ? 3 : 1)) == 0; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
int64_t row_bytes_of(int type, int64_t k) { return k / kElems[type] * kBytes[type]; }

hipStream_t hs(ft_stream_t s) { return (hipStream_t)s; }

ft_status hip_status(hipError_t e) { return e == hipSuccess ? FT_OK : FT_ERR_HIP; }

// --------------------------------------------------------------------------
// scratch pool
// --------------------------------------------------------------------------
struct Pool {
  std::mutex use;   // held from a call's look-up until its last launch is enqueued
  void* ptr = nullptr;
  size_t size = 0;
  std::vector<void*> retired;
};
// A stream orders what is enqueued on it, but two host threads that call on one stream may
// enqueue their launches in turn, and one would read what the other's wrote to the pool.  So a
// call that uses the pool holds it until it has enqueued everything.
using PoolUse = std::unique_lock<std::mutex>;
std::mutex g_pool_mu;
// by device too: every device has the null stream
std::map<std::pair<int, hipStream_t>, Pool> g_pools;

Pool* pool_hold(hipStream_t st, PoolUse& use) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return nullptr;
  Pool* p;
  {
    std::lock_guard<std::mutex> lk(g_pool_mu);
    p = &g_pools[{dev, st}];   // entries stay where they are
  }
  use = PoolUse(p->use);
  return p;
}

ft_status pool_get(hipStream_t st, size_t bytes, void** out, PoolUse& use, size_t* held = nullptr) {
  Pool* pool = pool_hold(st, use);
  if (!pool) return FT_ERR_HIP;
  Pool& p = *pool;
  *out = p.ptr;
  if (held) *held = p.size;
  if (p.size >= bytes) return FT_OK;
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(st, &cs) != hipSuccess) return FT_ERR_HIP;
  if (cs != hipStreamCaptureStatusNone) return FT_ERR_NO_SCRATCH;
  size_t want = std::max(bytes, 2 * p.size);
  want = (want + ((size_t)1 << 20) - 1) & ~(((size_t)1 << 20) - 1);
  void* np = nullptr;
  if (hipMalloc(&np, want) != hipSuccess) {
    (void)hipGetLastError();   // told by the status; the next launch's check would find it again
    return FT_ERR_HIP;
  }
  if (p.ptr) p.retired.push_back(p.ptr);  // work already enqueued may still use it
  p.ptr = np;
  p.size = want;
  *out = np;
  if (held) *held = want;
  return FT_OK;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// scratch layout of ft_moe_q_vec
struct MoeScratch {
  size_t xq, h, hq, d, ids, w, tab, total;
};
MoeScratch moe_layout(int w, int act, int64_t hidden, int64_t inter, int64_t t, int topk) {
  (void)w;
  MoeScratch s;
  size_t off = 0;
  s.xq = off;
  off += align256((size_t)t * row_bytes_of(act, hidden));
  s.h = off;
  off += align256((size_t)t * topk * inter * sizeof(float));
  s.hq = off;
  off += align256((size_t)t * topk * row_bytes_of(act, inter));
  s.d = off;
  off += align256((size_t)t * topk * hidden * sizeof(float));
  s.ids = off;   // the routing when the layer routes from logits
  off += align256((size_t)t * topk * 4);
  s.w = off;
  off += align256((size_t)t * topk * 4);
  s.tab = off;   // the fused Q4_K layer's routing table (its first launch -> its second)
  off += align256(ftk_moe_fused_table_bytes());
  s.total = off;
  return s;
}

// scratch layout of the grouped GEMM: the sort, then (MXFP4) the FP8 halves of
// the activation rows (512 bytes per row and superblock)
struct SortScratch {
  size_t counts, offsets, pairs, xf8, total;
};
SortScratch sort_layout(int64_t n_expert, int64_t t, int topk, size_t xf8_bytes = 0) {
  SortScratch s;
  size_t off = 0;
  s.counts = off;
  off += align256((size_t)n_expert * 4);
  s.offsets = off;
  off += align256((size_t)(n_expert + 1) * 4);
  s.pairs = off;
  off += align256((size_t)t * topk * 4);
  s.xf8 = off;
  off += align256(xf8_bytes);
  s.total = off;
  return s;
}
size_t xf8_bytes_of(int w, int64_t rows, int64_t k) { return w == FT_MXFP4 ? (size_t)rows * (k / 256) * 512 : 0; }

// every weight format x Q8_1 or Q8_0; the grouped-GEMM formats x Q8_K
bool mmvq_pair(int w, int a) {
  return ((a == FT_Q8_1 || a == FT_Q8_0) && is_weight(w)) ||
         (a == FT_Q8_K && (w == FT_Q4_K || w == FT_Q5_K || w == FT_Q6_K || w == FT_MXFP4));
}
// the direct route: Q4_K x Q8_1 on dot4, MXFP4 x Q8_K on the FP4 MFMA; the sorted
// tiles: every grouped-GEMM format x Q8_K
bool moe_direct_pair(int w, int a) { return (w == FT_Q4_K && a == FT_Q8_1) || (w == FT_MXFP4 && a == FT_Q8_K); }
bool moe_tile_pair(int w, int a) {
  return a == FT_Q8_K && (w == FT_Q4_K || w == FT_Q5_K || w == FT_Q6_K || w == FT_MXFP4);
}
bool moe_pair(int w, int a) { return moe_direct_pair(w, a) || moe_tile_pair(w, a); }
// the tile route splits x, then h, into FP8 halves in one buffer
size_t moe_xf8_bytes(int w, int64_t hidden, int64_t inter, int64_t t, int topk) {
  const size_t a = xf8_bytes_of(w, t, hidden), b = xf8_bytes_of(w, t * topk, inter);
  return a > b ? a : b;
}
bool grouped_pair(int w, int a) {
  return a == FT_Q8_K && (w == FT_Q4_K || w == FT_Q5_K || w == FT_Q6_K || w == FT_MXFP4);
}

bool kv_sizes(int64_t page, int64_t heads, int64_t dim) {
  return (page == 16 || page == 32 || page == 64 || page == 128 || page == 256) && heads >= 1 && heads <= 1024 &&
         (dim == 64 || dim == 96 || dim == 128 || dim == 256);
}
// the cache itself: types, sizes, pools
ft_status kv_check(const ft_kv_cache* c) {
  if (!c) return FT_ERR_INVALID_ARG;
  if (!is_kv_type(c->k_type) || !is_kv_type(c->v_type)) return FT_ERR_UNSUPPORTED;
  if (!kv_sizes(c->page_size, c->n_kv_head, c->head_dim)) return FT_ERR_SHAPE;
  if (c->n_pages < 1 || c->n_pages > INT32_MAX) return FT_ERR_SHAPE;
  if (!c->k_pages || !c->v_pages) return FT_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return FT_ERR_ALIGNMENT;
  return FT_OK;
}
// strides of a [rows][heads][dim] tensor whose rows may not run into each other
bool strides_ok(int64_t rows, int64_t heads, int64_t dim, int64_t token, int64_t head) {
  if ((rows > 1 && token < dim) || (heads > 1 && head < dim) || token < 0 || head < 0) return false;
  const int64_t lim = (int64_t)1 << 40;   // offsets stay far from 63 bits
  return token <= lim && head <= lim;
}

KvArgs kv_args(const ft_kv_cache* c, ft_float type, void* k, int64_t k_token, int64_t k_head, void* v,
               int64_t v_token, int64_t v_head, const int64_t* slots, int64_t t) {
  KvArgs a = {};
  a.k_type = c->k_type;
  a.v_type = c->v_type;
  a.k_pages = c->k_pages;
  a.v_pages = c->v_pages;
  a.n_pages = c->n_pages;
  a.page = (int)c->page_size;
  a.heads = (int)c->n_kv_head;
  a.dim = (int)c->head_dim;
  a.ftype = type;
  a.k = k;
  a.k_token = k_token;
  a.k_head = k_head;
  a.v = v;
  a.v_token = v_token;
  a.v_head = v_head;
  a.slots = slots;
  a.t = t;
  return a;
}

// Sizes and options of ft_attn_kv into the arguments that the planner needs.
ft_status attn_sizes(const ft_kv_cache* c, int64_t n_tok, int64_t n_head, int64_t n_seq, int64_t max_kv,
                     const ft_attn_opts& o, AttnArgs* a) {
  if (!kv_sizes(c->page_size, c->n_kv_head, c->head_dim)) return FT_ERR_SHAPE;
  if (n_tok < 0 || n_seq < 0 || max_kv < 0 || o.window < 0 || o.n_shared < 0) return FT_ERR_INVALID_ARG;
  if (!(o.softcap >= 0.0f) || std::isinf(o.softcap) || !std::isfinite(o.scale)) return FT_ERR_INVALID_ARG;
  if (o.bidirectional != 0 && o.bidirectional != 1) return FT_ERR_INVALID_ARG;
  if (n_head < 1 || n_head > 1024 || n_head % c->n_kv_head) return FT_ERR_SHAPE;
  if (n_tok > (1 << 24) || n_seq > (1 << 20) || max_kv > (1 << 30)) return FT_ERR_SHAPE;
  if (o.n_shared % c->page_size || o.n_shared > max_kv) return FT_ERR_SHAPE;
  a->page = (int)c->page_size;
  a->page_shift = __builtin_ctz((unsigned)a->page);
  a->n_kv_head = (int)c->n_kv_head;
  a->dim = (int)c->head_dim;
  a->n_head = (int)n_head;
  a->group = (int)(n_head / c->n_kv_head);
  a->group_mul = ((1ull << 40) + (unsigned)a->group - 1) / (unsigned)a->group;
  if (n_tok * a->group >= (1 << 30)) return FT_ERR_SHAPE;
  a->n_tok = (int)n_tok;
  a->n_seq = (int)n_seq;
  a->max_kv = (int)max_kv;
  a->scale = o.scale != 0.0f ? o.scale : 1.0f / std::sqrt((float)c->head_dim);
  a->softcap = std::min(o.softcap, 1e30f);   // in powers of two it stays finite; no score comes near it
  a->causal = !o.bidirectional;
  a->window = std::min<int64_t>(o.window, 1 << 30);
  a->slopes = o.slopes;
  a->prefix_len = o.prefix_len;
  a->n_shared = (int)o.n_shared;
  return FT_OK;
}

}  // namespace

extern "C" {

int ft_block_elems(ft_type t) { return ((int)t >= 0 && (int)t < kTypes) ? kElems[t] : 0; }
size_t ft_block_bytes(ft_type t) { return ((int)t >= 0 && (int)t < kTypes) ? (size_t)kBytes[t] : 0; }

const char* ft_version(void) { return "ft 0.1 (gfx950)"; }

int ft_supported(ft_op op, ft_type w, ft_type act) {
  switch (op) {
    case FT_OP_QUANTIZE: return is_act(act);
    case FT_OP_DEQUANT: return is_weight(w);
    case FT_OP_MMVQ: return mmvq_pair(w, act);
    case FT_OP_MOE_VEC: return moe_pair(w, act);
    case FT_OP_GROUPED: return grouped_pair(w, act);
    case FT_OP_BLOCK_DOTS: return is_weight(w) && is_act(act);
    case FT_OP_KV_CACHE: return is_kv_type(w) && is_kv_type(act);
  }
  return 0;
}

const char* ft_status_str(ft_status s) {
  switch (s) {
    case FT_OK: return "ok";
    case FT_ERR_INVALID_ARG: return "invalid argument";
    case FT_ERR_UNSUPPORTED: return "unsupported format combination";
    case FT_ERR_SHAPE: return "shape not supported (block multiple, topk or size limit)";
    case FT_ERR_ALIGNMENT: return "pointer not 16-byte aligned";
    case FT_ERR_NO_SCRATCH: return "scratch too small (pool while capturing, or the given workspace)";
    case FT_ERR_HIP: return "HIP runtime error";
  }
  return "unknown status";
}

ft_status ft_quantize_act(ft_type act, const float* x, int64_t rows, int64_t k, int64_t ldx, void* xq,
                          ft_stream_t stream) {
  if (!is_act(act)) return FT_ERR_UNSUPPORTED;
  if (rows < 0 || k < 0 || ldx < k) return FT_ERR_INVALID_ARG;
  if (k % kElems[act]) return FT_ERR_SHAPE;
  if (rows == 0 || k == 0) return FT_OK;
  if (!x || !xq) return FT_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(xq)) return FT_ERR_ALIGNMENT;
  return hip_status(ftk_launch_quantize(act, x, rows, k, ldx, xq, hs(stream)));
}

ft_status ft_dequant(ft_type w, const void* blocks, int64_t rows, int64_t k, float* out, ft_stream_t stream) {
  if (!is_weight(w)) return FT_ERR_UNSUPPORTED;
  if (rows < 0 || k < 0) return FT_ERR_INVALID_ARG;
  if (k % kElems[w]) return FT_ERR_SHAPE;
  if (rows == 0 || k == 0) return FT_OK;
  if (!blocks || !out) return FT_ERR_INVALID_ARG;
  if (!aligned16(blocks) || !aligned16(out)) return FT_ERR_ALIGNMENT;
  return hip_status(ftk_launch_dequant(w, blocks, rows, k, out, hs(stream)));
}

ft_status ft_mul_mat_vec_q(ft_type w, const void* W, int64_t n, int64_t k, ft_type act, const void* xq, int64_t t,
                           float* y, int64_t ldy, ft_stream_t stream) {
  if (!is_weight(w) || !is_act(act) || !mmvq_pair(w, act)) return FT_ERR_UNSUPPORTED;
  if (n < 0 || k < 0 || t < 0 || ldy < n) return FT_ERR_INVALID_ARG;
  if (k % kElems[w] || k % kElems[act]) return FT_ERR_SHAPE;
  if (k > 32768 || n > ((int64_t)1 << 31) / 2) return FT_ERR_SHAPE;
  if (n == 0 || t == 0) return FT_OK;
  if (!W || !xq || !y) return FT_ERR_INVALID_ARG;
  if (k == 0) return FT_ERR_SHAPE;
  if (!aligned16(W) || !aligned16(xq) || !aligned16(y)) return FT_ERR_ALIGNMENT;
  PoolUse use;
  if (act == FT_Q8_0) {   // the Q8_1 layout of the same blocks, in the stream's pool
    void* rp = nullptr;
    const int64_t nblk = t * (k / 32);
    const ft_status ps = pool_get(hs(stream), align256((size_t)nblk * 36), &rp, use);
    if (ps != FT_OK) return ps;
    const hipError_t e = ftk_launch_repack_q8_0(xq, nblk, rp, hs(stream));
    if (e != hipSuccess) return FT_ERR_HIP;
    xq = rp;
    act = FT_Q8_1;
  }
  MmvqArgs a;
  a.w = w;
  a.act = act;
  a.W = W;
  a.n = n;
  a.row_bytes = (int)row_bytes_of(w, k);
  a.units_per_row = 0;
  a.xrow_bytes = (int)row_bytes_of(act, k);
  a.ldy = ldy;
  for (int64_t t0 = 0; t0 < t; t0 += 8) {
    a.t = (int)std::min<int64_t>(8, t - t0);
    a.xq = (const uint8_t*)xq + t0 * a.xrow_bytes;
    a.y = y + t0 * ldy;
    const hipError_t e = ftk_launch_mmvq(a, k, hs(stream));
    if (e != hipSuccess) return FT_ERR_HIP;
  }
  return FT_OK;
}

ft_status ft_moe_route(const float* logits, int64_t t, int64_t n_expert, int topk, int32_t* ids, float* w,
                       ft_stream_t stream) {
  if (t < 0 || n_expert < 1 || n_expert > 1024) return FT_ERR_SHAPE;
  if (topk < 1 || topk > 8 || topk > n_expert) return FT_ERR_SHAPE;
  if (t == 0) return FT_OK;
  if (!logits || !ids || !w) return FT_ERR_INVALID_ARG;
  return hip_status(ftk_launch_route(logits, t, n_expert, topk, ids, w, hs(stream)));
}

ft_status ft_moe_route_ex(const void* logits, ft_float type, int64_t t, int64_t n_expert, int64_t ld, int topk,
                          const ft_route_opts* opts, int32_t* ids, float* w, ft_stream_t stream) {
  ft_route_opts o = {};
  if (opts) o = *opts;
  if (!is_float(type)) return FT_ERR_UNSUPPORTED;
  if (t < 0 || n_expert < 1 || n_expert > 1024 || t > (1 << 25)) return FT_ERR_SHAPE;
  if ((o.sigmoid != 0 && o.sigmoid != 1) || (o.no_renorm != 0 && o.no_renorm != 1) || !std::isfinite(o.scale) ||
      o.group_top < 0 || o.group_top > 2 || (ld < n_expert && t > 1) || ld < 0 || ld > ((int64_t)1 << 30))
    return FT_ERR_INVALID_ARG;
  const int64_t groups = o.n_group ? o.n_group : 1;
  const int64_t keep = o.topk_group ? o.topk_group : groups;
  if (groups < 1 || groups > 64 || n_expert % groups || keep < 1 || keep > groups) return FT_ERR_SHAPE;
  if (topk < 1 || topk > 32 || topk > keep * (n_expert / groups)) return FT_ERR_SHAPE;
  if (t == 0) return FT_OK;
  if (!logits || !ids || !w) return FT_ERR_INVALID_ARG;
  if (!float_aligned(logits, type)) return FT_ERR_ALIGNMENT;
  RouteArgs a = {};
  a.logits = logits;
  a.ftype = type;
  a.ld = ld;
  a.t = t;
  a.n_expert = (int)n_expert;
  a.topk = topk;
  a.sigmoid = o.sigmoid;
  a.bias = o.bias;
  a.n_group = (int)groups;
  a.topk_group = (int)keep;
  a.group_top = o.group_top ? o.group_top : 1;
  a.renorm = !o.no_renorm;
  a.scale = o.scale != 0.0 ? o.scale : 1.0;
  a.ids = ids;
  a.w = w;
  return hip_status(ftk_launch_route_ex(a, hs(stream)));
}

size_t ft_kv_page_bytes(ft_type type, int64_t page_size, int64_t n_kv_head, int64_t head_dim) {
  if (!is_kv_type(type) || !kv_sizes(page_size, n_kv_head, head_dim)) return 0;
  return (size_t)(page_size * n_kv_head * row_bytes_of(type, head_dim));
}

ft_status ft_kv_store(const ft_kv_cache* cache, ft_float type, const void* k, int64_t k_token, int64_t k_head,
                      const void* v, int64_t v_token, int64_t v_head, const int64_t* slots, int64_t t,
                      ft_stream_t stream) {
  const ft_status s = kv_check(cache);
  if (s != FT_OK) return s;
  if (!is_float(type)) return FT_ERR_UNSUPPORTED;
  const int64_t H = cache->n_kv_head, D = cache->head_dim;
  if (t < 0 || !strides_ok(t, H, D, k_token, k_head) || !strides_ok(t, H, D, v_token, v_head))
    return FT_ERR_INVALID_ARG;
  if (t > ((int64_t)1 << 24)) return FT_ERR_SHAPE;
  if (t == 0) return FT_OK;
  if (!k || !v || !slots) return FT_ERR_INVALID_ARG;
  if (!float_aligned(k, type) || !float_aligned(v, type) || ((uintptr_t)slots & 7)) return FT_ERR_ALIGNMENT;
  const KvArgs a = kv_args(cache, type, (void*)k, k_token, k_head, (void*)v, v_token, v_head, slots, t);
  return hip_status(ftk_launch_kv(a, false, hs(stream)));
}

ft_status ft_kv_load(const ft_kv_cache* cache, const int64_t* slots, int64_t t, ft_float type, void* k,
                     int64_t k_token, int64_t k_head, void* v, int64_t v_token, int64_t v_head, ft_stream_t stream) {
  const ft_status s = kv_check(cache);
  if (s != FT_OK) return s;
  if (!is_float(type)) return FT_ERR_UNSUPPORTED;
  const int64_t H = cache->n_kv_head, D = cache->head_dim;
  if (t < 0 || (k && !strides_ok(t, H, D, k_token, k_head)) || (v && !strides_ok(t, H, D, v_token, v_head)))
    return FT_ERR_INVALID_ARG;
  if (t > ((int64_t)1 << 24)) return FT_ERR_SHAPE;
  if (t == 0 || (!k && !v)) return FT_OK;
  if (!slots) return FT_ERR_INVALID_ARG;
  if (!float_aligned(k, type) || !float_aligned(v, type) || ((uintptr_t)slots & 7)) return FT_ERR_ALIGNMENT;
  const KvArgs a = kv_args(cache, type, k, k_token, k_head, v, v_token, v_head, slots, t);
  return hip_status(ftk_launch_kv(a, true, hs(stream)));
}

size_t ft_attn_kv_scratch_bytes(const ft_kv_cache* cache, int64_t n_tok, int64_t n_head, int64_t n_seq, int64_t max_kv,
                                const ft_attn_opts* opts) {
  ft_attn_opts o = {};
  if (opts) o = *opts;
  AttnArgs a = {};
  if (!cache || attn_sizes(cache, n_tok, n_head, n_seq, max_kv, o, &a) != FT_OK || n_tok == 0 || n_seq == 0) return 0;
  size_t most = 0;
  for (const int type : {FT_F32, FT_F16, FT_BF16}) {   // the split depends on the type
    a.ftype = type;
    most = std::max(most, ftk_attn_plan(a).scratch_most);
  }
  return align256(most);
}

ft_status ft_attn_kv(const ft_kv_cache* cache, ft_float type, const void* q, int64_t q_token, int64_t q_head,
                     int64_t n_tok, int64_t n_head, const int32_t* q_start, const int32_t* kv_len,
                     const int32_t* table, int64_t table_ld, int64_t n_col, int64_t n_seq, int64_t max_kv, void* out,
                     int64_t out_token, int64_t out_head, const ft_attn_opts* opts, ft_stream_t stream) {
  ft_attn_opts o = {};
  if (opts) o = *opts;
  ft_status s = kv_check(cache);
  if (s != FT_OK) return s;
  if (!is_float(type)) return FT_ERR_UNSUPPORTED;
  if (n_col < 1 || n_col > INT32_MAX || (n_seq > 1 && table_ld < n_col) || table_ld < 0) return FT_ERR_INVALID_ARG;
  AttnArgs a = {};
  // no key lies past the table
  const int64_t room = std::min<int64_t>(n_col * cache->page_size, 1 << 30);
  s = attn_sizes(cache, n_tok, n_head, n_seq, std::min(max_kv, room), o, &a);
  if (s != FT_OK) return s;
  const int64_t D = cache->head_dim;
  if (!strides_ok(n_tok, n_head, D, q_token, q_head) || !strides_ok(n_tok, n_head, D, out_token, out_head))
    return FT_ERR_INVALID_ARG;
  if (n_tok == 0 || n_seq == 0) return FT_OK;
  if (!q || !q_start || !kv_len || !table || !out) return FT_ERR_INVALID_ARG;
  if (!float_aligned(q, type) || !float_aligned(out, type) || (((uintptr_t)q_start | (uintptr_t)kv_len |
      (uintptr_t)table | (uintptr_t)o.slopes | (uintptr_t)o.prefix_len) & 3) || !aligned16(o.workspace))
    return FT_ERR_ALIGNMENT;
  a.k_type = cache->k_type;
  a.v_type = cache->v_type;
  a.k_pages = (const uint8_t*)cache->k_pages;
  a.v_pages = (const uint8_t*)cache->v_pages;
  a.n_pages = (int)cache->n_pages;
  a.ftype = type;
  const int64_t step = type == FT_F32 ? 4 : 8;   // elements in 16 bytes
  a.q = q;
  a.q_token = q_token;
  a.q_head = q_head;
  a.q_vec = aligned16(q) && q_token % step == 0 && q_head % step == 0;
  a.out = out;
  a.out_token = out_token;
  a.out_head = out_head;
  a.out_vec = aligned16(out) && out_token % step == 0 && out_head % step == 0;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.table = table;
  a.table_ld = table_ld;
  a.cols = (int)n_col;
  AttnPlan p = ftk_attn_plan(a);
  // launches of under 2^32 threads (512 a tile, 64 a row of a join)
  const auto too_large = [&] {
    for (const AttnSplit& x : {p.shared, p.tile, p.step})
      if (x.tiles * a.n_kv_head >= (1 << 23) || x.n_split > 65535) return true;
    return p.scratch && std::max(n_tok * n_head, p.step_rows * n_seq * cache->n_kv_head) >= (1 << 26);
  };
  if (too_large()) return FT_ERR_SHAPE;
  void* base = o.workspace;
  size_t room_bytes = o.workspace_bytes;
  PoolUse use;
  if (p.scratch && !base) {
    s = pool_get(hs(stream), align256(p.scratch), &base, use, &room_bytes);
    if (s != FT_OK && s != FT_ERR_NO_SCRATCH) return s;
  }
  // many rows do with fewer splits, down to none: so the size for a larger max_kv is enough
  while (p.scratch > room_bytes && p.tile.n_split > 1) p = ftk_attn_plan(a, p.tile.n_split - 1);
  if (p.scratch > room_bytes) return FT_ERR_NO_SCRATCH;
  if (too_large()) return FT_ERR_SHAPE;
  return hip_status(ftk_launch_attn(a, p, base, hs(stream)));
}

ft_status ft_moe_sort(const int32_t* ids, int64_t t, int topk, int64_t n_expert, int32_t* counts, int32_t* offsets,
                      int32_t* pairs, ft_stream_t stream) {
  if (t < 0 || n_expert < 1 || n_expert > 8192 || topk < 1 || topk > 8) return FT_ERR_SHAPE;
  if (!counts || !offsets || (t > 0 && (!ids || !pairs))) return FT_ERR_INVALID_ARG;
  return hip_status(ftk_launch_sort(ids, t, topk, n_expert, counts, offsets, pairs, hs(stream)));
}

size_t ft_moe_scratch_bytes(ft_type w, ft_type act, int64_t n_expert, int64_t hidden, int64_t inter, int64_t t,
                            int topk) {
  if (!is_act(act) || t < 0 || topk < 0 || n_expert < 1) return 0;
  // the sorted-tile route also needs the sort's buffers
  return moe_layout(w, act, hidden, inter, t, topk).total +
         (moe_tile_pair(w, act) ? sort_layout(n_expert, t, topk, moe_xf8_bytes(w, hidden, inter, t, topk)).total : 0);
}

size_t ft_grouped_scratch_bytes(ft_type w, int64_t n_expert, int64_t k, int64_t t, int topk, int x_per_pair) {
  if (n_expert < 1 || k < 0 || t < 0 || topk < 1) return 0;
  return sort_layout(n_expert, t, topk, xf8_bytes_of(w, x_per_pair ? t * topk : t, k)).total;
}

}  // extern "C"

namespace {

// Host-side checks of ft_moe_q_vec; on FT_OK, *tiles says which route runs and
// *need the scratch bytes it takes.
ft_status moe_check(ft_type w, const void* w_gate, const void* w_up, const void* w_down, int64_t n_expert,
                    int64_t hidden, int64_t inter, ft_type act, const float* x, int64_t t,
                    const int32_t* expert_ids, const float* expert_w, int topk, float* y, const ft_moe_opts& o,
                    bool* tiles, size_t* need) {
  if (!is_weight(w) || !is_act(act) || !moe_pair(w, act)) return FT_ERR_UNSUPPORTED;
  if (n_expert < 1 || hidden < 0 || inter < 0 || t < 0) return FT_ERR_INVALID_ARG;
  if (topk < 1 || topk > 8 || topk > n_expert) return FT_ERR_SHAPE;
  if (hidden % kElems[w] || hidden % kElems[act] || inter % kElems[w] || inter % kElems[act]) return FT_ERR_SHAPE;
  if (hidden == 0 || inter == 0 || hidden > 16384 || inter > 16384) return FT_ERR_SHAPE;
  if (o.route < 0 || o.route > 2 || o.direct_max_t < 0) return FT_ERR_INVALID_ARG;
  const bool tile_ok = moe_tile_pair(w, act), direct_ok = moe_direct_pair(w, act);
  if ((o.route == 2 && !tile_ok) || (o.route == 1 && !direct_ok)) return FT_ERR_UNSUPPORTED;
  // default threshold: up to 8 tokens (one launch chunk of the direct MXFP4 kernels)
  // the direct route wins on MI355X (measured per layer: t = 8: 284 vs 290 us; t = 9:
  // 317 vs 298 us for the sorted tiles); pairs with no direct kernels take the tiles
  const int64_t dmax = o.direct_max_t > 0 ? o.direct_max_t : 8;
  *tiles = o.route == 2 || (o.route == 0 && (!direct_ok || (tile_ok && t > dmax)));
  // the sort behind the tiles holds one counter per expert in LDS
  if (*tiles && n_expert > 8192) return FT_ERR_SHAPE;
  if (o.logits && n_expert > 1024) return FT_ERR_SHAPE;   // the router's limit
  if (t == 0) return FT_OK;
  if (!w_gate || !w_up || !w_down || !x || !y) return FT_ERR_INVALID_ARG;
  if (!o.logits && (!expert_ids || !expert_w)) return FT_ERR_INVALID_ARG;
  if (!aligned16(w_gate) || !aligned16(w_up) || !aligned16(w_down) || !aligned16(x) || !aligned16(y))
    return FT_ERR_ALIGNMENT;
  if ((o.tap_g && !aligned16(o.tap_g)) || (o.tap_u && !aligned16(o.tap_u)) || (o.tap_h && !aligned16(o.tap_h)) ||
      (o.tap_hq && !aligned16(o.tap_hq)) || (o.tap_down && !aligned16(o.tap_down)) ||
      (o.in_hq && !aligned16(o.in_hq)))
    return FT_ERR_ALIGNMENT;
  *need = moe_layout(w, act, hidden, inter, t, topk).total +
          (*tiles ? sort_layout(n_expert, t, topk, moe_xf8_bytes(w, hidden, inter, t, topk)).total : 0);
  return FT_OK;
}

// The layer on checked arguments, its scratch at b (moe_check's `need` bytes).
ft_status moe_run(ft_type w, const void* w_gate, const void* w_up, const void* w_down, int64_t n_expert,
                  int64_t hidden, int64_t inter, ft_type act, const float* x, int64_t t,
                  const int32_t* expert_ids, const float* expert_w, int topk, float* y, const ft_moe_opts& o,
                  bool tiles, uint8_t* b, hipStream_t st) {
  const MoeScratch L = moe_layout(w, act, hidden, inter, t, topk);
  const SortScratch S = sort_layout(n_expert, t, topk, moe_xf8_bytes(w, hidden, inter, t, topk));
  MoeArgs a = {};
  a.w = w;
  a.act = act;
  a.w_gate = w_gate;
  a.w_up = w_up;
  a.w_down = w_down;
  a.n_expert = n_expert;
  a.hidden = hidden;
  a.inter = inter;
  a.t = t;
  a.topk = topk;
  a.ids = expert_ids;
  a.ew = expert_w;
  a.x = x;
  a.xq = b + L.xq;
  a.h = o.tap_h ? o.tap_h : (float*)(b + L.h);
  a.g_tap = o.tap_g;
  a.u_tap = o.tap_u;
  a.hq = o.in_hq ? const_cast<void*>(o.in_hq) : (o.tap_hq ? o.tap_hq : (void*)(b + L.hq));
  a.hq_tap = o.tap_hq;
  a.in_hq = o.in_hq;
  a.dpair = o.tap_down ? o.tap_down : (float*)(b + L.d);
  a.d_tap = o.tap_down;
  a.h_tap = o.tap_h;
  a.y = y;

  hipError_t e = hipSuccess;
  a.logits = nullptr;
  a.ids_out = o.ids_out;
  a.w_out = o.w_out;
  const bool fused = !tiles && ftk_moe_fused_ok(w, act, hidden, inter, topk);
  if (o.logits && fused && ftk_moe_fused_routes(n_expert)) {
    a.logits = o.logits;   // the fused layer routes itself
    a.ids = nullptr;
    a.ew = nullptr;
  } else if (o.logits && !tiles && w == FT_MXFP4 && act == FT_Q8_K && n_expert <= 256 && t <= 2) {
    // the MXFP4 direct gate/up launch routes the tokens itself (the router's
    // selection and weights) and leaves the routing here for the later stages
    // (1-2 tokens: 1.2-1.5 us less per layer; from 4 tokens on, every workgroup
    // routing its chunk costs more than the router's launch)
    a.logits = o.logits;
    a.ids = o.ids_out ? o.ids_out : (int32_t*)(b + L.ids);
    a.ew = o.w_out ? o.w_out : (float*)(b + L.w);
    expert_ids = a.ids;
  } else if (o.logits) {   // route first, into the caller's outputs or scratch
    int32_t* ri = o.ids_out ? o.ids_out : (int32_t*)(b + L.ids);
    float* rw = o.w_out ? o.w_out : (float*)(b + L.w);
    e = ftk_launch_route(o.logits, t, n_expert, topk, ri, rw, st);
    if (e != hipSuccess) return FT_ERR_HIP;
    a.ids = ri;
    a.ew = rw;
    expert_ids = ri;
  }
  if (tiles) {
    e = ftk_launch_quantize(act, x, t, hidden, hidden, (void*)a.xq, st);
    uint8_t* sb = b + L.total;
    int32_t* counts = (int32_t*)(sb + S.counts);
    int32_t* offsets = (int32_t*)(sb + S.offsets);
    int32_t* pairs = (int32_t*)(sb + S.pairs);
    void* xf8 = sb + S.xf8;
    if (e == hipSuccess) e = ftk_launch_sort(expert_ids, t, topk, n_expert, counts, offsets, pairs, st);
    if (e == hipSuccess && w == FT_MXFP4) e = ftk_launch_fp8_split(a.xq, t, hidden, xf8, st);
    GroupedArgs gu = {};
    gu.w = w;
    gu.act = act;
    gu.W = w_gate;
    gu.W2 = w_up;
    gu.g_tap = o.tap_g;
    gu.u_tap = o.tap_u;
    gu.n_expert = n_expert;
    gu.n = inter;
    gu.k = hidden;
    gu.xq = a.xq;
    gu.xf8 = w == FT_MXFP4 ? xf8 : nullptr;
    gu.x_per_pair = 0;
    gu.t = t;
    gu.topk = topk;
    gu.counts = counts;
    gu.offsets = offsets;
    gu.pairs = pairs;
    gu.y = a.h;
    if (e == hipSuccess) e = ftk_launch_grouped(gu, st);
    if (e == hipSuccess && !o.in_hq) e = ftk_launch_quantize(act, a.h, t * topk, inter, inter, a.hq, st);
    if (e == hipSuccess && o.in_hq && o.tap_hq)
      e = hipMemcpyAsync(o.tap_hq, o.in_hq, (size_t)t * topk * row_bytes_of(act, inter), hipMemcpyDeviceToDevice,
                         st);
    if (e == hipSuccess && w == FT_MXFP4) e = ftk_launch_fp8_split(a.hq, t * topk, inter, xf8, st);
    GroupedArgs dn = gu;
    dn.W = w_down;
    dn.W2 = nullptr;
    dn.g_tap = dn.u_tap = nullptr;
    dn.n = hidden;
    dn.k = inter;
    dn.xq = a.hq;
    dn.xf8 = w == FT_MXFP4 ? xf8 : nullptr;
    dn.x_per_pair = 1;
    dn.y = a.dpair;
    if (e == hipSuccess) e = ftk_launch_grouped(dn, st);
    if (e == hipSuccess) e = ftk_launch_moe_combine(a, st);
    return hip_status(e);
  }
  // direct route, Q4_K x Q8_1 shapes that fit: the whole layer in two launches per 4-token chunk
  if (fused) return hip_status(ftk_launch_moe_fused(a, b + L.tab, st));
  // otherwise gate/up (quantizes x itself), down (quantizes each expert's h rows
  // itself, or reads in_hq), slot-order combine
  e = ftk_launch_moe_gate_up(a, st);
  if (e == hipSuccess && w == FT_MXFP4 && ftk_moe_fp4_down_combine_ok(a))
    return hip_status(ftk_launch_moe_fp4_down_combine(a, st));   // 1-2 tokens: down + combine
  if (e == hipSuccess) e = ftk_launch_moe_down(a, st);
  if (e == hipSuccess) e = ftk_launch_moe_combine(a, st);
  return hip_status(e);
}

// --------------------------------------------------------------------------
// fixed scratch of ft_moe_q_vec_noalloc: a device array of every GPU the library
// runs on, held until the process ends.  Host code never passes the array's name
// to a kernel (on the host it is a stand-in, not a device address): the address
// comes from hipGetSymbolAddress once per device and is kept here.
// --------------------------------------------------------------------------
static __device__ __align__(256) uint8_t scratch[FT_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_static_use[kMaxDevices];   // held as a pool's is
void* g_static_ptr[kMaxDevices] = {};

ft_status static_scratch(void** out, PoolUse& use) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return FT_ERR_HIP;
  use = PoolUse(g_static_use[dev]);
  if (!g_static_ptr[dev]) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return FT_ERR_HIP;
    g_static_ptr[dev] = p;
  }
  *out = g_static_ptr[dev];
  return FT_OK;
}

}  // namespace

extern "C" {

ft_status ft_moe_q_vec(ft_type w, const void* w_gate, const void* w_up, const void* w_down, int64_t n_expert,
                       int64_t hidden, int64_t inter, ft_type act, const float* x, int64_t t,
                       const int32_t* expert_ids, const float* expert_w, int topk, float* y, const ft_moe_opts* opts,
                       ft_stream_t stream) {
  ft_moe_opts o = {};
  if (opts) o = *opts;
  bool tiles = false;
  size_t need = 0;
  ft_status s = moe_check(w, w_gate, w_up, w_down, n_expert, hidden, inter, act, x, t, expert_ids, expert_w, topk,
                          y, o, &tiles, &need);
  if (s != FT_OK || t == 0) return s;
  hipStream_t st = hs(stream);
  void* base = nullptr;
  PoolUse use;
  s = pool_get(st, need, &base, use);
  if (s != FT_OK) return s;
  return moe_run(w, w_gate, w_up, w_down, n_expert, hidden, inter, act, x, t, expert_ids, expert_w, topk, y, o,
                 tiles, (uint8_t*)base, st);
}

ft_status ft_moe_q_vec_noalloc(ft_type w, const void* w_gate, const void* w_up, const void* w_down,
                               int64_t n_expert, int64_t hidden, int64_t inter, ft_type act, const float* x,
                               int64_t t, const int32_t* expert_ids, const float* expert_w, int topk, float* y,
                               const ft_moe_opts* opts, ft_stream_t stream) {
  ft_moe_opts o = {};
  if (opts) o = *opts;
  bool tiles = false;
  size_t need = 0;
  ft_status s = moe_check(w, w_gate, w_up, w_down, n_expert, hidden, inter, act, x, t, expert_ids, expert_w, topk,
                          y, o, &tiles, &need);
  if (s != FT_OK || t == 0) return s;
  if (need > (size_t)FT_NOALLOC_SCRATCH_BYTES) return FT_ERR_SHAPE;
  void* base = nullptr;
  PoolUse use;
  s = static_scratch(&base, use);
  if (s != FT_OK) return s;
  return moe_run(w, w_gate, w_up, w_down, n_expert, hidden, inter, act, x, t, expert_ids, expert_w, topk, y, o,
                 tiles, (uint8_t*)base, hs(stream));
}

ft_status ft_grouped_gemm_q(ft_type w, const void* W, int64_t n_expert, int64_t n, int64_t k, ft_type act,
                            const void* xq, int x_per_pair, const int32_t* expert_ids, int64_t t, int topk, float* y,
                            ft_stream_t stream) {
  if (!is_weight(w) || !is_act(act) || !grouped_pair(w, act)) return FT_ERR_UNSUPPORTED;
  if (n_expert < 1 || n < 0 || k < 0 || t < 0) return FT_ERR_INVALID_ARG;
  if (topk < 1 || topk > 8 || topk > n_expert || n_expert > 8192) return FT_ERR_SHAPE;
  if (k % kElems[w] || k % kElems[act] || k == 0 || k > 16384) return FT_ERR_SHAPE;
  if (n == 0 || t == 0) return FT_OK;
  if (!W || !xq || !expert_ids || !y) return FT_ERR_INVALID_ARG;
  if (!aligned16(W) || !aligned16(xq) || !aligned16(y)) return FT_ERR_ALIGNMENT;
  hipStream_t st = hs(stream);
  const SortScratch L = sort_layout(n_expert, t, topk, xf8_bytes_of(w, x_per_pair ? t * topk : t, k));
  void* base = nullptr;
  PoolUse use;
  ft_status s = pool_get(st, L.total, &base, use);
  if (s != FT_OK) return s;
  uint8_t* b = (uint8_t*)base;
  GroupedArgs a = {};
  a.w = w;
  a.act = act;
  a.W = W;
  a.n_expert = n_expert;
  a.n = n;
  a.k = k;
  a.xq = xq;
  a.x_per_pair = x_per_pair ? 1 : 0;
  a.t = t;
  a.topk = topk;
  a.counts = (const int32_t*)(b + L.counts);
  a.offsets = (const int32_t*)(b + L.offsets);
  a.pairs = (const int32_t*)(b + L.pairs);
  a.y = y;
  a.xf8 = w == FT_MXFP4 ? (const void*)(b + L.xf8) : nullptr;
  hipError_t e = ftk_launch_sort(expert_ids, t, topk, n_expert, (int32_t*)(b + L.counts), (int32_t*)(b + L.offsets),
                                 (int32_t*)(b + L.pairs), st);
  if (e == hipSuccess && w == FT_MXFP4) e = ftk_launch_fp8_split(xq, x_per_pair ? t * topk : t, k, b + L.xf8, st);
  if (e == hipSuccess) e = ftk_launch_grouped(a, st);
  return hip_status(e);
}

ft_status ft_debug_block_dots(ft_type w, const void* W, int64_t n, int64_t k, ft_type act, const void* xq, int64_t t,
                              int32_t* partials, ft_stream_t stream) {
  if (!is_weight(w) || !is_act(act)) return FT_ERR_UNSUPPORTED;
  if (n < 0 || k < 0 || t < 0) return FT_ERR_INVALID_ARG;
  if (k % kElems[w] || k % kElems[act]) return FT_ERR_SHAPE;
  if (n == 0 || t == 0 || k == 0) return FT_OK;
  if (!W || !xq || !partials) return FT_ERR_INVALID_ARG;
  if (!aligned16(W) || !aligned16(xq)) return FT_ERR_ALIGNMENT;
  PoolUse use;
  if (act == FT_Q8_0) {   // as the matvec: the Q8_1 layout of the same blocks
    void* rp = nullptr;
    const int64_t nblk = t * (k / 32);
    const ft_status ps = pool_get(hs(stream), align256((size_t)nblk * 36), &rp, use);
    if (ps != FT_OK) return ps;
    const hipError_t e = ftk_launch_repack_q8_0(xq, nblk, rp, hs(stream));
    if (e != hipSuccess) return FT_ERR_HIP;
    xq = rp;
    act = FT_Q8_1;
  }
  return hip_status(ftk_launch_block_dots(w, W, n, k, act, xq, t, partials, hs(stream)));
}

ft_status ft_debug_ceiling(int which, const void* buf, int64_t bytes, int64_t iters, void* out,
                           ft_stream_t stream) {
  if (which < 0 || which > 3 || !out || iters < 0) return FT_ERR_INVALID_ARG;
  if (which == 0) {
    if (!buf || bytes < 0 || bytes % 16) return FT_ERR_INVALID_ARG;
    if (!aligned16(buf)) return FT_ERR_ALIGNMENT;
    if (bytes == 0) return FT_OK;
  }
  return hip_status(ftk_launch_probe(which, buf, bytes, iters, (uint32_t*)out, hs(stream)));
}

ft_status ft_scratch_reserve(ft_stream_t stream, size_t bytes) {
  void* p = nullptr;
  PoolUse use;
  return pool_get(hs(stream), bytes, &p, use);
}

void ft_shutdown(void) {
  std::lock_guard<std::mutex> lk(g_pool_mu);
  for (auto& kv : g_pools) {
    if (kv.second.ptr) (void)hipFree(kv.second.ptr);
    for (void* r : kv.second.retired) (void)hipFree(r);
  }
  g_pools.clear();
}

}  // extern "C"
