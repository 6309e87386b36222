// Host side of the calls around a drafted block: the paged cache, the shared-prefix
// attention over it and the verification.  Validation and launch order only.
#include <float.h>
#include <limits.h>

#include <algorithm>
#include <new>
#include <numeric>

#include "xp_internal.h"

namespace {

inline size_t align_up(size_t x) { return (x + 255) / 256 * 256; }
inline xp_status cuda_status(cudaError_t e) { return e == cudaSuccess ? XP_OK : XP_ECUDA; }

// a b c < 2^31, whatever they are (none negative)
bool fits(int a, int b, int c) {
  return (int64_t)a * b <= INT_MAX && (int64_t)a * b * c <= INT_MAX;
}

// heads outside the tokens of a page, tokens outside the heads, or neither (-1)
int page_order(const xp_cache_desc* d) {
  const int64_t D = d->head_dim, H = d->kv_heads, ps = d->page_size;
  if ((d->stride_token == H * D || ps == 1) && (d->stride_head == D || H == 1)) return 0;
  if ((d->stride_head == ps * D || H == 1) && (d->stride_token == D || ps == 1)) return 1;
  return -1;
}

bool valid_desc(const xp_cache_desc* d) {
  if (!d || d->pages <= 0 || d->page_size <= 0 || d->layers <= 0 || d->kv_heads <= 0 ||
      d->head_dim <= 0 || d->head_dim > 256 || d->max_seqs <= 0)
    return false;
  if (d->dtype != XP_BF16 && d->dtype != XP_F32) return false;
  if (!fits(d->page_size, d->kv_heads, d->head_dim) || page_order(d) < 0) return false;
  const int64_t block = (int64_t)d->page_size * d->kv_heads * d->head_dim;
  return d->stride_page >= block && d->stride_layer >= 0;
}

struct CachePrep {
  size_t err, src, dst, cnt, n_moves, map, row_a, row_b, row_c, row_d, total;
};
CachePrep cache_prep(const xp_cache_desc* d) {
  CachePrep L;
  size_t o = 0;
  auto take = [&](size_t words) { size_t at = o; o = align_up(o + words * 4); return at; };
  L.err = take(64);
  L.n_moves = take(64);
  L.src = take(d->pages);
  L.dst = take(d->pages);
  L.cnt = take(d->pages);
  L.map = take(d->pages);
  L.row_a = take(d->max_seqs);
  L.row_b = take(d->max_seqs);
  L.row_c = take(d->max_seqs);
  L.row_d = take(d->max_seqs);
  L.total = o;
  return L;
}

bool on_device(const xp_cache* c) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == c->device;
}

// `rows` rows of `width` columns: what the table calls share
xp_status check_table(const xp_cache* c, const int32_t* table, int64_t ld, const int32_t* lens,
                      int rows, int width) {
  if (!c) return XP_ENOTPREPARED;
  if (rows < 0 || (rows > 0 && (!table || !lens)) || width <= 0 || ld < width || !on_device(c) ||
      (int64_t)width * c->d.page_size > INT_MAX)
    return XP_EINVAL;
  return rows > c->d.max_seqs ? XP_ECAPACITY : XP_OK;
}

bool valid_attn(const xp_cache* c, const xp_attn* a) {
  return a && a->layer >= 0 && a->layer < c->d.layers && a->N >= 0 && a->T > 0 && a->heads > 0 &&
         a->head_dim == c->d.head_dim && a->dtype == c->d.dtype &&
         a->scale > 0.0f && a->scale <= FLT_MAX && a->heads % c->d.kv_heads == 0 && a->prefix_len >= 0 && a->max_len >= 0 &&
         fits(a->N, a->T, a->heads) &&
         (int64_t)a->prefix_len + a->max_len <= INT_MAX - 1024;
}

xp_attn_plan attn_plan(const xp_cache* c, const xp_attn* a) {
  if (c->attn_tc) {
    const xp_attn_plan tc = xp_attn_tc_plan(c, a);
    if (tc.total) return tc;   // 0: more work than its line can count
  }
  xp_attn_plan p = xp_attn_simt_plan(c, a);
  const size_t rows = (size_t)a->N * a->T * a->heads;
  p.stat_off = 0;
  p.acc_off = align_up(rows * p.parts * 8);
  p.total = p.acc_off + align_up(rows * p.parts * c->d.head_dim * 4);
  return p;
}

// Whether rows of two tables (a: na rows lda apart, b likewise) share entries: 0 no, 1 the same
// columns of the same rows only, -1 an entry of another column too (or strides too unlike to tell).
int table_overlap(const int32_t* a, int64_t lda, int na, const int32_t* b, int64_t ldb, int nb,
                  int width) {
  if (na == 0 || nb == 0) return 0;
  if (na == 1) lda = nb == 1 ? 2 * (int64_t)width : ldb;   // one row has no stride of its own
  if (nb == 1) ldb = lda;
  const intptr_t a0 = (intptr_t)a, b0 = (intptr_t)b, es = sizeof(int32_t);
  if (a0 + ((na - 1) * lda + width) * es <= b0 || b0 + ((nb - 1) * ldb + width) * es <= a0) return 0;
  // all rows of both begin at multiples of `unit` from a, or d behind one (told apart only where a
  // unit holds a row)
  const int64_t unit = std::gcd(lda, ldb), d = (((b0 - a0) / es) % unit + unit) % unit;
  if (d == 0 && unit >= width) return 1;
  return d >= width && d + width <= unit ? 0 : -1;
}

xp_status append(const xp_cache* c, int layer, const void* k, const void* v, int64_t stride_n,
                 int64_t stride_t, int64_t stride_h, int heads, int head_dim, xp_dtype dtype,
                 const int32_t* table, int64_t ld_table, int64_t width, const int32_t* lens, int N,
                 int T, cudaStream_t stream) {
  if (!c) return XP_ENOTPREPARED;
  if (heads != c->d.kv_heads || head_dim != c->d.head_dim || dtype != c->d.dtype || layer < 0 ||
      layer >= c->d.layers || N < 0 || T <= 0 || width <= 0 || ld_table < width ||
      !fits(N, T, c->d.kv_heads) || !on_device(c))
    return XP_EINVAL;
  if (N == 0) return XP_OK;   // an empty batch needs no pointers, here and in the calls below
  if (!k || !v || !table || !lens) return XP_EINVAL;
  return cuda_status(xp_launch_append(c, layer, k, v, stride_n, stride_t, stride_h, table, ld_table,
                                      width, lens, N, T, stream));
}

}  // namespace

extern "C" {

size_t xp_cache_prep_bytes(const xp_cache_desc* d) { return valid_desc(d) ? cache_prep(d).total : 0; }

xp_status xp_cache_create(const xp_cache_desc* d, void* prep_dev, size_t prep_bytes,
                          cudaStream_t stream, xp_cache** out) {
  if (!out) return XP_EINVAL;
  *out = nullptr;
  if (!valid_desc(d) || !d->k || !d->v || !prep_dev || (uintptr_t)prep_dev % 256) return XP_EINVAL;
  const size_t es = xp_elem(d->dtype);
  if ((uintptr_t)d->k % es || (uintptr_t)d->v % es) return XP_EINVAL;
  const CachePrep L = cache_prep(d);
  if (prep_bytes < L.total) return XP_ECAPACITY;
  xp_cache* c = new (std::nothrow) xp_cache();
  if (!c) return XP_ECAPACITY;
  c->d = *d;
  c->heads_outside = page_order(d) == 1;
  // What one head, token, page or layer has for a stride is never used: set to the dense one, so that
  // an odd value does not keep the pools from 16-byte accesses and TMA.
  if (d->kv_heads == 1) c->d.stride_head = d->head_dim;
  if (d->page_size == 1) c->d.stride_token = (int64_t)d->kv_heads * d->head_dim;
  if (d->pages == 1) c->d.stride_page = (int64_t)d->page_size * d->kv_heads * d->head_dim;
  if (d->layers == 1) c->d.stride_layer = c->d.stride_page * d->pages;
  if (cudaGetDevice(&c->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, c->device) !=
          cudaSuccess) {
    delete c;
    return XP_ECUDA;
  }
  char* p = (char*)prep_dev;
  c->err = (uint32_t*)(p + L.err);
  c->n_moves = (int32_t*)(p + L.n_moves);
  c->src = (int32_t*)(p + L.src);
  c->dst = (int32_t*)(p + L.dst);
  c->cnt = (int32_t*)(p + L.cnt);
  c->map = (int32_t*)(p + L.map);
  c->row_a = (int32_t*)(p + L.row_a);
  c->row_b = (int32_t*)(p + L.row_b);
  c->row_c = (int32_t*)(p + L.row_c);
  c->row_d = (int32_t*)(p + L.row_d);
  c->attn_tc = xp_attn_tc_maps(c);
  if (cudaMemsetAsync(prep_dev, 0, L.total, stream) != cudaSuccess) {
    delete c;
    return XP_ECUDA;
  }
  *out = c;
  return XP_OK;
}

void xp_cache_destroy(xp_cache* c) { delete c; }

xp_status xp_cache_get_error(const xp_cache* c, cudaStream_t stream) {
  if (!c) return XP_ENOTPREPARED;
  if (!on_device(c)) return XP_EINVAL;
  uint32_t word = 0;
  if (xp_take_error(c->err, stream, &word) != cudaSuccess) return XP_ECUDA;
  if (word & XP_ERR_TIMEOUT) return XP_ETIMEOUT;
  if (word & XP_ERR_LENGTH) return XP_ELENGTH;
  if (word & XP_ERR_SHARED) return XP_ESHARED;
  if (word & XP_ERR_NOPAGES) return XP_ENOPAGES;
  if (word & XP_ERR_BADPAGE) return XP_EBADPAGE;
  return XP_OK;
}

xp_status xp_cache_append(const xp_cache* c, int layer, const void* k, const void* v,
                          int64_t stride_n, int64_t stride_t, int64_t stride_h,
                          int heads, int head_dim, xp_dtype dtype, const int32_t* table,
                          int64_t ld_table, const int32_t* lens, int N, int T,
                          cudaStream_t stream) {
  return append(c, layer, k, v, stride_n, stride_t, stride_h, heads, head_dim, dtype, table,
                ld_table, ld_table, lens, N, T, stream);
}

xp_status xp_cache_append_columns(const xp_cache* c, int layer, const void* k, const void* v,
                                  int64_t stride_n, int64_t stride_t, int64_t stride_h,
                                  int heads, int head_dim, xp_dtype dtype, const int32_t* table,
                                  int64_t ld_table, int width, const int32_t* lens, int N, int T,
                                  cudaStream_t stream) {
  return append(c, layer, k, v, stride_n, stride_t, stride_h, heads, head_dim, dtype, table,
                ld_table, width, lens, N, T, stream);
}

xp_status xp_cache_copy(const xp_cache* c, const int32_t* src, const int32_t* dst, int count,
                        cudaStream_t stream) {
  if (!c) return XP_ENOTPREPARED;
  if (count < 0 || (count > 0 && (!src || !dst)) || !on_device(c)) return XP_EINVAL;
  if (count == 0) return XP_OK;
  return cuda_status(xp_launch_copy_pages(c, src, dst, nullptr, count, nullptr, stream));
}

xp_status xp_cache_resize(const xp_cache* c, const int32_t* table, int64_t ld_table,
                          const int32_t* lens, const int32_t* new_lens, const int32_t* refs,
                          int pages, int N, int width, int32_t* table_out, int64_t ld_out, int32_t* lens_out,
                          int32_t* refs_out, cudaStream_t stream) {
  const xp_status st = check_table(c, table, ld_table, lens, N, width);
  if (st != XP_OK) return st;
  if (!refs || pages != c->d.pages || !refs_out || ld_out < width || !fits(N, width, 1) ||
      (N > 0 && (!new_lens || !table_out || !lens_out)))
    return XP_EINVAL;
  return cuda_status(xp_launch_resize(c, table, ld_table, lens, new_lens, refs, N, width, table_out,
                                      ld_out, lens_out, refs_out, stream));
}

xp_status xp_cache_fork(const xp_cache* c, const int32_t* table, int64_t ld_table,
                        const int32_t* lens, int rows, const int32_t* parent, const int32_t* cut,
                        int M, int width, const int32_t* refs, int pages, int32_t* child_table,
                        int64_t ld_child, int32_t* child_lens, int32_t* refs_out,
                        cudaStream_t stream) {
  const xp_status st = check_table(c, table, ld_table, lens, rows, width);
  if (st != XP_OK) return st;
  if (!refs || pages != c->d.pages || !refs_out || ld_child < width || M < 0 ||
      (M > 0 && (!parent || !child_table || !child_lens)))
    return XP_EINVAL;
  const int shared = table_overlap(table, ld_table, rows, child_table, ld_child, M, width);
  if (shared < 0) return XP_EINVAL;
  if (M > c->d.max_seqs) return XP_ECAPACITY;
  return cuda_status(xp_launch_fork(c, table, ld_table, lens, rows, parent, cut, M, width, refs,
                                    shared != 0, child_table, ld_child, child_lens, refs_out, stream));
}

xp_status xp_cache_compact(const xp_cache* c, const int32_t* table, int64_t ld_table,
                           const int32_t* lens, int N, int width, const int32_t* refs, int pages,
                           int32_t* table_out, int64_t ld_out, int32_t* refs_out, int32_t* map,
                           int32_t* live, cudaStream_t stream) {
  const xp_status st = check_table(c, table, ld_table, lens, N, width);
  if (st != XP_OK) return st;
  if (!refs || pages != c->d.pages || (N > 0 && !table_out) || !refs_out || ld_out < width)
    return XP_EINVAL;
  return cuda_status(xp_launch_compact(c, table, ld_table, lens, N, width, refs, table_out, ld_out,
                                       refs_out, map, live, stream));
}

size_t xp_attention_workspace_bytes(const xp_cache* c, const xp_attn* a) {
  return c && valid_attn(c, a) ? std::max<size_t>(256, attn_plan(c, a).total) : 0;
}

xp_status xp_prefix_attention(const xp_cache* c, const xp_attn* a, const void* q,
                              const int32_t* prefix_table, int prefix_pages, const int32_t* table,
                              int64_t ld_table, int width, const int32_t* lens, void* out, float* lse,
                              void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!c) return XP_ENOTPREPARED;
  if (!valid_attn(c, a) || !on_device(c)) return XP_EINVAL;
  if (a->N == 0) return XP_OK;
  if (!q || !out || !ws || (uintptr_t)ws % 256) return XP_EINVAL;
  const int ps = c->d.page_size;
  if (a->prefix_len > 0 && (!prefix_table || prefix_pages < (a->prefix_len - 1) / ps + 1))
    return XP_EINVAL;
  if (a->max_len > 0 &&
      (!table || !lens || width < (a->max_len - 1) / ps + 1 || (a->N > 1 && ld_table < width)))
    return XP_EINVAL;
  const xp_attn_plan plan = attn_plan(c, a);
  if (ws_bytes < plan.total) return XP_ECAPACITY;
  const size_t es = xp_elem(c->d.dtype);
  xp_attn_args g;
  g.a = *a;
  g.kv_heads = c->d.kv_heads;
  g.group = a->heads / c->d.kv_heads;
  g.dim = c->d.head_dim;
  g.page_size = c->d.page_size;
  g.pages = c->d.pages;
  g.q = q;
  g.k = (const char*)c->d.k + a->layer * c->d.stride_layer * es;
  g.v = (const char*)c->d.v + a->layer * c->d.stride_layer * es;
  g.kv_page = c->d.stride_page;
  g.kv_token = c->d.stride_token;
  g.kv_head = c->d.stride_head;
  g.prefix_table = prefix_table;
  g.table = table;
  g.lens = lens;
  g.ld_table = ld_table;
  g.out = out;
  g.lse = lse;
  g.stat = (float*)((char*)ws + plan.stat_off);
  g.acc = (float*)((char*)ws + plan.acc_off);
  g.line = (int*)((char*)ws + plan.line_off);
  g.err = c->err;
  g.plan = plan;
  if (plan.tc) return cuda_status(xp_launch_attn_tc(c, g, stream));
  cudaError_t e = xp_launch_attn_simt(c, g, stream);
  if (e == cudaSuccess) e = xp_launch_attn_combine(c, g, stream);
  return cuda_status(e);
}

size_t xp_verify_workspace_bytes(const xp_head* h, int N) {
  return h && N >= 0 && N <= h->max_N ? xp_verify_layout(h, N).total : 0;
}

xp_status xp_verify_drafts(const xp_head* h, const void* target, int64_t stride_n,
                           int64_t stride_b, const float* draft, int64_t ld_draft,
                           const int64_t* blk, const int32_t* n_draft, int N, int B, int V,
                           xp_dtype dtype, const float* temperature, const float* u, const float* noise,
                           int64_t ld_noise, int64_t* tokens, int32_t* counts, float* prob,
                           void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!h) return XP_ENOTPREPARED;
  if (N < 0 || B != h->B || V != h->V || dtype != h->dtype || !xp_on_head_device(h))
    return XP_EINVAL;
  if (N == 0) return XP_OK;
  if (!target || !blk || !u || !noise || !tokens || !counts || !ws || (uintptr_t)ws % 256 ||
      stride_n < 0 || stride_b < 0 || (draft && ld_draft < h->V) || ld_noise < h->V)
    return XP_EINVAL;
  if (N > h->max_N || N > 65535) return XP_ECAPACITY;
  const xp_verify_ws L = xp_verify_layout(h, N);
  if (ws_bytes < L.total) return XP_ECAPACITY;
  char* w = (char*)ws;
  xp_verify_args a;
  a.target = target;
  a.sn = stride_n;
  a.sb = stride_b;
  a.draft = draft;
  a.ld_draft = ld_draft;
  a.blk = blk;
  a.n_draft = n_draft;
  a.temperature = temperature;
  a.u = u;
  a.noise = noise;
  a.ld_noise = ld_noise;
  a.tokens = tokens;
  a.counts = counts;
  a.prob = prob;
  a.N = N;
  a.B = h->B;
  a.V = h->V;
  a.err = h->err;
  a.marks = (unsigned*)(w + L.marks);
  a.tickets = (unsigned*)(w + L.tickets);
  a.packed = (unsigned long long*)(w + L.packed);
  a.draw_ticket = (unsigned*)(w + L.draw_ticket);
  a.next = (unsigned*)(w + L.next);
  a.part = (float*)(w + L.part);
  a.row = (float*)(w + L.row);
  return cuda_status(xp_launch_verify(h, a, stream));
}

}  // extern "C"
