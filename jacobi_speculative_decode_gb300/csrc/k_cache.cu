// The paged cache: appending tokens, copying pages, and the table calls (resize, fork,
// compact).  A table call is one cluster of 8 CTAs: its phases (release, rank the free
// pages, hand them out) each need the whole of the one before, and a cluster's barrier and
// shared memory order them within one launch.  Their bound is latency: four or five cluster barriers and the
// loads between them, about 10 us on the GPU (12 a call) for 256 rows and 16,384 pages, whose bytes
// would take less than one.  (One CTA would order the phases more cheaply, but read 16,384 counts
// in 16 rounds; a grid-wide barrier costs more than a cluster's.)
#include <cooperative_groups.h>

#include <algorithm>

#include "quant.cuh"
#include "sm100_ptx.cuh"
#include "xp_device.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kCtas = 8;
constexpr int kThreads = 1024;
constexpr int kForkHeld = 8;   // entries that a thread holds of children made in their parents' places

struct Scan {
  int warp[32];
  int total[3][kCtas];   // every CTA's sums, one row a use of cluster_base
};

__device__ __forceinline__ void flag(uint32_t* err, uint32_t bit) { atomicOr(err, bit); }

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// Exclusive prefix of v over the CTA's threads; *sum gets the CTA's total.  Two barriers.
__device__ __forceinline__ int block_scan(int v, Scan& s, int* sum) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) s.warp[w] = inc;
  __syncthreads();
  int ws = s.warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, ws, o);
    if (lane >= o) ws += t;
  }
  const int before = __shfl_sync(0xFFFFFFFFu, ws, w == 0 ? 0 : w - 1);
  *sum = __shfl_sync(0xFFFFFFFFu, ws, 31);
  __syncthreads();
  return (w == 0 ? 0 : before) + inc - v;
}

// Every CTA says at its start that it runs, and waits for the others' word just before the first
// store into their shared memory (which may not be reached before): the reads between hide it.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Sum of v over the CTA's threads, then the CTA's exclusive prefix among the cluster's (use:
// the sum's own row; 0 comes first).  Orders the cluster: whatever any CTA wrote before is visible
// behind it.
__device__ __forceinline__ int cluster_base(cg::cluster_group& cl, int use, int v, Scan& s,
                                            int* total) {
  int sum;
  block_scan(v, s, &sum);
  const int rank = (int)cl.block_rank();
  if (use == 0) cluster_wait();
  if (threadIdx.x < kCtas) *cl.map_shared_rank(&s.total[use][rank], threadIdx.x) = sum;
  cl.sync();
  int base = 0, all = 0;
  for (int r = 0; r < kCtas; ++r) {
    const int t = s.total[use][r];
    base += r < rank ? t : 0;
    all += t;
  }
  *total = all;
  return base;
}

__device__ __forceinline__ int checked_len(int len, int most, uint32_t* err) {
  if (len < 0 || len > most) {
    flag(err, XP_ERR_LENGTH);
    len = len < 0 ? 0 : most;
  }
  return len;
}

// The pages of [lo, hi) that are free (refs <= 0), in ascending order, to free_list: ranks
// below `want` only; each is taken (refs = 1).  Returns the number of free pages of all CTAs.
__device__ int take_free(cg::cluster_group& cl, int32_t* refs, int lo, int hi, int want,
                         int32_t* free_list, Scan& s, uint32_t* err) {
  int mine = 0;
  for (int p = lo + (int)threadIdx.x; p < hi; p += kThreads) {
    const int r = refs[p];
    if (r < 0) {   // let go more often than it was held
      refs[p] = 0;
      flag(err, XP_ERR_BADPAGE);
    }
    mine += r <= 0;
  }
  int total;
  int base = cluster_base(cl, 1, mine, s, &total);
  for (int p0 = lo; p0 < hi && base < want; p0 += kThreads) {
    const int p = p0 + (int)threadIdx.x;
    const int is_free = p < hi && refs[p] <= 0;
    int sum;
    const int rank = base + block_scan(is_free, s, &sum);
    if (is_free && rank < want) {
      free_list[rank] = p;
      refs[p] = 1;
    }
    base += sum;
  }
  cl.sync();
  return total;
}

struct ResizeArgs {
  const int32_t* table;
  int64_t ld;
  const int32_t *lens, *new_lens, *refs;
  int N, width, pages, ps;
  int32_t* table_out;
  int64_t ld_out;
  int32_t *lens_out, *refs_out;
  int32_t *row_old, *row_new, *row_off, *free_list;
  uint32_t* err;
};

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    resize_kernel(const ResizeArgs a) {
  __shared__ Scan s;
  cluster_arrive();
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), tid = (int)threadIdx.x;
  const int r0 = (int)((int64_t)a.N * rank / kCtas), r1 = (int)((int64_t)a.N * (rank + 1) / kCtas);
  const int p0 = (int)((int64_t)a.pages * rank / kCtas);
  const int p1 = (int)((int64_t)a.pages * (rank + 1) / kCtas);

  // each row's lengths, on the counts as they were
  if (a.refs_out != a.refs)
    for (int p = p0 + tid; p < p1; p += kThreads) a.refs_out[p] = a.refs[p];
  int need = 0;
  for (int n = r0 + tid; n < r1; n += kThreads) {
    const int len = checked_len(a.lens[n], a.width * a.ps, a.err);
    int now = checked_len(a.new_lens[n], a.width * a.ps, a.err);
    const int low = min(len, now);
    if (now != len && low % a.ps != 0) {
      const int p = a.table[n * a.ld + low / a.ps];
      if (p >= 0 && p < a.pages && a.refs[p] > 1) {
        flag(a.err, XP_ERR_SHARED);
        now = len;
      }
    }
    a.row_old[n] = len;
    a.row_new[n] = now;
    need += max(0, ceil_div(now, a.ps) - ceil_div(len, a.ps));
  }
  int all_need;
  int base = cluster_base(cl, 0, need, s, &all_need);   // from here on refs_out may change
  for (int n0 = r0; n0 < r1; n0 += kThreads) {
    const int n = n0 + tid;
    const int v = n < r1 ? max(0, ceil_div(a.row_new[n], a.ps) - ceil_div(a.row_old[n], a.ps)) : 0;
    int sum;
    const int off = base + block_scan(v, s, &sum);
    if (n < r1) a.row_off[n] = off;
    base += sum;
  }

  // kept entries, and the pages let go
  const int lane = tid & 31;
  for (int n = r0 + (tid >> 5); n < r1; n += kThreads / 32) {
    const int have = ceil_div(a.row_old[n], a.ps), want = ceil_div(a.row_new[n], a.ps);
    for (int j = lane; j < a.width; j += 32) {
      int out = -1;
      if (j < have) {
        const int p = a.table[n * a.ld + j];
        const bool ok = p >= 0 && p < a.pages;
        if (!ok) flag(a.err, XP_ERR_BADPAGE);
        if (j < want) out = p;
        else if (ok) atomicSub(&a.refs_out[p], 1);
      }
      if (j < have || j >= want) a.table_out[n * a.ld_out + j] = out;
    }
  }
  cl.sync();

  const int n_free = take_free(cl, a.refs_out, p0, p1, all_need, a.free_list, s, a.err);

  // the free pages go to the rows in order
  for (int n = r0 + (tid >> 5); n < r1; n += kThreads / 32) {
    const int old_len = a.row_old[n], now = a.row_new[n], off = a.row_off[n];
    const int have = ceil_div(old_len, a.ps), want = ceil_div(now, a.ps);
    for (int j = have + lane; j < want; j += 32) {
      const int r = off + j - have;
      a.table_out[n * a.ld_out + j] = r < n_free ? a.free_list[r] : -1;
    }
    if (lane == 0) {
      int len = now;
      if (want > have) {
        const int got = min(want - have, max(0, n_free - off));
        if (got < want - have) flag(a.err, XP_ERR_NOPAGES);
        len = min(len, (have + got) * a.ps);
      }
      a.lens_out[n] = len;
    }
  }
}

struct ForkArgs {
  const int32_t* table;
  int64_t ld;
  const int32_t* lens;
  int rows;
  const int32_t *parent, *cut, *refs;
  int M, width, pages, ps;
  bool in_place;   // children are rows of the parents' table: all are read before any is written
  int32_t* child;
  int64_t ld_child;
  int32_t *child_lens, *refs_out;
  int32_t *row_parent, *row_len, *row_off, *row_entry;
  int32_t *src, *dst, *cnt, *n_moves;
  uint32_t* err;
};

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    fork_kernel(const ForkArgs a) {
  __shared__ Scan s;
  cluster_arrive();
  ptx::pdl_trigger();   // the next kernel's CTAs come up as this one's leave, and wait there
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), tid = (int)threadIdx.x;
  const int r0 = (int)((int64_t)a.M * rank / kCtas), r1 = (int)((int64_t)a.M * (rank + 1) / kCtas);
  const int p0 = (int)((int64_t)a.pages * rank / kCtas);
  const int p1 = (int)((int64_t)a.pages * (rank + 1) / kCtas);

  if (a.refs_out != a.refs)
    for (int p = p0 + tid; p < p1; p += kThreads) a.refs_out[p] = a.refs[p];
  int need = 0;
  for (int i = r0 + tid; i < r1; i += kThreads) {
    int p = a.parent[i], len = 0;
    if (p < 0 || p >= a.rows) {
      flag(a.err, XP_ERR_LENGTH);
      p = 0;
    } else {
      len = checked_len(a.lens[p], a.width * a.ps, a.err);
      if (a.cut) len = min(len, max(0, a.cut[i]));
      // a last page that is none cannot be copied: the child ends before it
      if (len % a.ps) {
        const int last = a.table[p * a.ld + len / a.ps];
        if (last < 0 || last >= a.pages) {
          flag(a.err, XP_ERR_BADPAGE);
          len -= len % a.ps;
        }
      }
    }
    a.row_parent[i] = p;
    a.row_len[i] = len;
    need += len % a.ps != 0;
  }
  int all_need;
  int base = cluster_base(cl, 0, need, s, &all_need);   // from here on refs_out may change
  for (int i0 = r0; i0 < r1; i0 += kThreads) {
    const int i = i0 + tid;
    int sum;
    const int part = i < r1 ? a.row_len[i] % a.ps : 0;
    const int off = base + block_scan(part != 0, s, &sum);
    if (i < r1) a.row_off[i] = off;
    if (part && off < a.pages) {   // there are no more moves than pages
      a.src[off] = a.table[a.row_parent[i] * a.ld + a.row_len[i] / a.ps];
      a.cnt[off] = part;
    }
    base += sum;
  }

  // full pages are shared
  auto shared_page = [&](const int32_t* row, int full, int j) {
    int out = -1;
    if (j < full) {
      out = row[j];
      if (out >= 0 && out < a.pages) atomicAdd(&a.refs_out[out], 1);
      else flag(a.err, XP_ERR_BADPAGE);
    }
    return out;
  };
  if (!a.in_place) {
    for (int i = r0 + (tid >> 5); i < r1; i += kThreads / 32) {
      const int full = a.row_len[i] / a.ps;
      const int32_t* row = a.table + a.row_parent[i] * a.ld;
      for (int j = tid & 31; j < a.width; j += 32)
        a.child[i * a.ld_child + j] = shared_page(row, full, j);
    }
  } else {
    // some columns of all rows at a time: a child's column is made from its parent's alone
    const int rows = (a.M + kCtas - 1) / kCtas, cols = kThreads * kForkHeld / rows;
    for (int j = 0; cols == 0 && j < a.width; ++j) {   // more rows than entries held: from memory
      for (int i = r0 + tid; i < r1; i += kThreads)
        a.row_entry[i] = shared_page(a.table + a.row_parent[i] * a.ld, a.row_len[i] / a.ps, j);
      cl.sync();
      for (int i = r0 + tid; i < r1; i += kThreads) a.child[i * a.ld_child + j] = a.row_entry[i];
    }
    for (int c0 = 0; cols > 0 && c0 < a.width; c0 += cols) {
      const int cw = min(cols, a.width - c0), entries = (r1 - r0) * cw;
      int out[kForkHeld];
#pragma unroll
      for (int k = 0; k < kForkHeld; ++k) {
        const int e = tid + k * kThreads;
        const int i = r0 + e / cw;
        if (e < entries)
          out[k] = shared_page(a.table + a.row_parent[i] * a.ld, a.row_len[i] / a.ps, c0 + e % cw);
      }
      cl.sync();
#pragma unroll
      for (int k = 0; k < kForkHeld; ++k) {
        const int e = tid + k * kThreads;
        if (e < entries) a.child[(r0 + e / cw) * a.ld_child + c0 + e % cw] = out[k];
      }
    }
  }
  cl.sync();

  const int n_free = take_free(cl, a.refs_out, p0, p1, all_need, a.dst, s, a.err);

  // the partly filled last pages are copied
  for (int i = r0 + tid; i < r1; i += kThreads) {
    int len = a.row_len[i];
    const int part = len % a.ps, full = len / a.ps, off = a.row_off[i];
    if (part) {
      if (off < n_free) {
        a.child[i * a.ld_child + full] = a.dst[off];
      } else {
        flag(a.err, XP_ERR_NOPAGES);
        len -= part;
      }
    }
    a.child_lens[i] = len;
  }
  if (rank == 0 && tid == 0) *a.n_moves = min(all_need, n_free);
}

struct CompactArgs {
  const int32_t* table;
  int64_t ld;
  const int32_t *lens, *refs;
  int N, width, pages, ps;
  int32_t* table_out;
  int64_t ld_out;
  int32_t *refs_out, *map, *live;
  int32_t *src, *dst, *n_moves;
  uint32_t* err;
};

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    compact_kernel(const CompactArgs a) {
  __shared__ Scan s;
  cluster_arrive();
  ptx::pdl_trigger();   // the next kernel's CTAs come up as this one's leave, and wait there
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), tid = (int)threadIdx.x;
  const int r0 = (int)((int64_t)a.N * rank / kCtas), r1 = (int)((int64_t)a.N * (rank + 1) / kCtas);
  const int p0 = (int)((int64_t)a.pages * rank / kCtas);
  const int p1 = (int)((int64_t)a.pages * (rank + 1) / kCtas);

  int used = 0;
  for (int p = p0 + tid; p < p1; p += kThreads) used += a.refs[p] > 0;
  int live;
  cluster_base(cl, 0, used, s, &live);

  // pages in use behind the line, and holes before it: equally many
  int high = 0, holes = 0;
  for (int p = p0 + tid; p < p1; p += kThreads) {
    const bool u = a.refs[p] > 0;
    high += u && p >= live;
    holes += !u && p < live;
  }
  int moves, same;
  int base_h = cluster_base(cl, 1, high, s, &moves);
  int base_o = cluster_base(cl, 2, holes, s, &same);
  for (int q0 = p0; q0 < p1; q0 += kThreads) {
    const int p = q0 + tid;
    const bool u = p < p1 && a.refs[p] > 0;
    const int is_high = u && p >= live, is_hole = p < p1 && !u && p < live;
    int sum_h, sum_o;
    const int rh = base_h + block_scan(is_high, s, &sum_h);
    const int ro = base_o + block_scan(is_hole, s, &sum_o);
    if (is_high) a.src[rh] = p;
    if (is_hole) a.dst[ro] = p;
    if (p < p1 && !is_high) a.map[p] = u ? p : -1;
    base_h += sum_h;
    base_o += sum_o;
  }
  cl.sync();
  const int m0 = (int)((int64_t)moves * rank / kCtas), m1 = (int)((int64_t)moves * (rank + 1) / kCtas);
  // counts first stay or clear, then follow the moves (refs_out may be refs)
  for (int i = m0 + tid; i < m1; i += kThreads) {
    a.map[a.src[i]] = a.dst[i];
    a.refs_out[a.dst[i]] = a.refs[a.src[i]];
  }
  if (a.refs_out != a.refs)
    for (int p = p0 + tid; p < p1; p += kThreads) {
      const int r = a.refs[p];
      if (p < live ? r > 0 : true) a.refs_out[p] = p < live ? r : 0;
    }
  cl.sync();
  if (a.refs_out == a.refs)
    for (int p = max(p0, live) + tid; p < p1; p += kThreads) a.refs_out[p] = 0;
  for (int n = r0 + (tid >> 5); n < r1; n += kThreads / 32) {
    const int held = ceil_div(checked_len(a.lens[n], a.width * a.ps, a.err), a.ps);
    for (int j = tid & 31; j < a.width; j += 32) {
      int out = -1;
      if (j < held) {
        const int p = a.table[n * a.ld + j];
        if (p >= 0 && p < a.pages) out = a.map[p];
        else flag(a.err, XP_ERR_BADPAGE);
      }
      a.table_out[n * a.ld_out + j] = out;
    }
  }
  if (rank == 0 && tid == 0) {
    *a.n_moves = moves;
    if (a.live) *a.live = live;
  }
}

// ---------------------------------------------------------------------------
// Page copies: (move, plane, chunk) items, a plane being K or V of one layer.  Bound by HBM: the
// call that moves 491 pages of 2 MB in 8 layers takes 321 us, 6.4 TB/s read and written together
// (95% of measured); 256 partial pages, 520 MB, take 71 us of their call's 83.  32 KB a CTA are in
// flight, all loads before the first store; 68 registers a thread leave three CTAs an SM, so that
// the grid of eight an SM comes in turns.
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kPerThread = 8;   // vectors of a thread in flight: 32 KB a CTA

struct CopyArgs {
  char *k, *v;
  int64_t layer_bytes, page_bytes;   // strides
  int layers, pages;
  int64_t block_bytes;               // one page of K or V
  int64_t seg_bytes, token_bytes;    // a page is segments of tokens: one, or one a head
  const int32_t *src, *dst, *tokens;
  int n;
  const int32_t* n_dev;
  uint32_t* err;
};

template <typename U>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const CopyArgs a) {
  ptx::pdl_wait();
  constexpr int kChunk = kCopyThreads * kPerThread * (int)sizeof(U);
  const int n = a.n_dev ? *a.n_dev : a.n;
  const int chunks = (int)((a.block_bytes + kChunk - 1) / kChunk);
  const int64_t items = (int64_t)n * a.layers * 2 * chunks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int c = (int)(it % chunks);
    const int64_t mp = it / chunks;
    const int plane = (int)(mp % (2 * a.layers)), i = (int)(mp / (2 * a.layers));
    const int sp = a.src[i], dp = a.dst[i];
    if (sp < 0 || dp < 0 || sp >= a.pages || dp >= a.pages) {
      if ((sp >= a.pages || dp >= a.pages) && threadIdx.x == 0 && c == 0 && plane == 0)
        flag(a.err, XP_ERR_BADPAGE);
      continue;
    }
    const int64_t keep = a.tokens ? a.tokens[i] * a.token_bytes : a.seg_bytes;
    // a page of one segment has nothing to copy behind its tokens
    if (a.seg_bytes == a.block_bytes && (int64_t)c * kChunk >= keep) continue;
    // which bytes move: no division where a page is one segment, or moves whole
    const bool plain = a.seg_bytes == a.block_bytes || keep == a.seg_bytes;
    const int64_t end = keep == a.seg_bytes ? a.block_bytes : plain ? keep : a.block_bytes;
    auto moves = [&](int64_t o) { return o < end && (plain || o % a.seg_bytes < keep); };
    char* pool = plane & 1 ? a.v : a.k;
    pool += (plane >> 1) * a.layer_bytes;
    const char* from = pool + sp * a.page_bytes;
    char* to = pool + dp * a.page_bytes;
    U val[kPerThread];
    const int64_t at = (int64_t)c * kChunk + threadIdx.x * sizeof(U);
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      const int64_t o = at + (int64_t)k * kCopyThreads * sizeof(U);
      if (moves(o)) val[k] = *(const U*)(from + o);
    }
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      const int64_t o = at + (int64_t)k * kCopyThreads * sizeof(U);
      if (moves(o)) *(U*)(to + o) = val[k];
    }
  }
}

// ---------------------------------------------------------------------------
// Append: one warp per (row, token, head), both K and V.  Bound by its launch and three dependent
// loads (length, page, data): 6.1 us for 128 x 16 tokens of 8 heads of 128 (17 MB), 2.5 for one.
// ---------------------------------------------------------------------------
struct AppendArgs {
  const void *k, *v;
  int64_t sn, st, sh;
  void *kp, *vp;   // this layer's pools
  int64_t page, token, head;
  const int32_t* table;
  int64_t ld, width;   // its columns: width
  const int32_t* lens;
  int N, T, H, D, ps, pages;
  uint32_t* err;
};

// U: the unit that all rows, strides and bases are whole numbers of (16 bytes, or one element).
// Half a warp moves K and half V, so that the 256 bytes of a row of 128 bf16 leave in one
// instruction of each.
template <typename U>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
  const int64_t w = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= (int64_t)a.N * a.T * a.H) return;
  const int h = (int)(w % a.H), t = (int)(w / a.H % a.T), n = (int)(w / a.H / a.T);
  const int64_t pos = (int64_t)a.lens[n] - a.T + t;
  if (pos < 0) return;
  if (pos / a.ps >= a.width) {   // behind the row's columns
    if (lane == 0) flag(a.err, XP_ERR_LENGTH);
    return;
  }
  const int p = a.table[n * a.ld + pos / a.ps];
  if (p < 0 || p >= a.pages) {
    if (lane == 0) flag(a.err, XP_ERR_BADPAGE);
    return;
  }
  const int64_t from = n * a.sn + t * a.st + h * a.sh;
  const int64_t to = p * a.page + pos % a.ps * a.token + h * a.head;
  const U* src = (const U*)(lane < 16 ? a.k : a.v) + from;
  U* dst = (U*)(lane < 16 ? a.kp : a.vp) + to;
  for (int i = lane % 16; i < a.D; i += 16) dst[i] = src[i];
}

}  // namespace

cudaError_t xp_launch_append(const xp_cache* c, int layer, const void* k, const void* v, int64_t sn,
                             int64_t st, int64_t sh, const int32_t* table, int64_t ld,
                             int64_t width, const int32_t* lens, int N, int T, cudaStream_t s) {
  const xp_cache_desc& d = c->d;
  const size_t es = xp_elem(d.dtype);
  char *kp = (char*)d.k + layer * d.stride_layer * es, *vp = (char*)d.v + layer * d.stride_layer * es;
  if (N == 1) sn = 0;   // strides that are never used
  if (T == 1) st = 0;
  if (d.kv_heads == 1) sh = 0;
  const int64_t strides = sn | st | sh | d.stride_page | d.stride_token | d.stride_head | d.head_dim;
  const bool wide = (((uintptr_t)k | (uintptr_t)v | (uintptr_t)kp | (uintptr_t)vp) & 15) == 0 &&
                    strides * (int64_t)es % 16 == 0;
  const int64_t unit = wide ? 16 / (int64_t)es : 1;   // elements
  AppendArgs a = {k, v, sn / unit, st / unit, sh / unit, kp, vp, d.stride_page / unit,
                  d.stride_token / unit, d.stride_head / unit, table, ld, width, lens, N, T, d.kv_heads,
                  d.head_dim / (int)unit, d.page_size, d.pages, c->err};
  const int64_t warps = (int64_t)N * T * d.kv_heads;
  const unsigned grid = (unsigned)((warps + 7) / 8);
  if (wide) append_kernel<uint4><<<grid, 256, 0, s>>>(a);
  else if (d.dtype == XP_BF16) append_kernel<uint16_t><<<grid, 256, 0, s>>>(a);
  else append_kernel<uint32_t><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t xp_launch_copy_pages(const xp_cache* c, const int32_t* src, const int32_t* dst,
                                 const int32_t* tokens, int n, const int32_t* n_dev,
                                 cudaStream_t s) {
  const xp_cache_desc& d = c->d;
  const int64_t es = (int64_t)xp_elem(d.dtype);
  CopyArgs a;
  a.k = (char*)d.k;
  a.v = (char*)d.v;
  a.layer_bytes = d.stride_layer * es;
  a.page_bytes = d.stride_page * es;
  a.layers = d.layers;
  a.pages = d.pages;
  if (xp_is_quant(d.dtype)) {   // codes and scales of a token lie apart: pages move whole
    a.block_bytes = d.kv_heads * xp_quant_of(d.page_size, d.head_dim, d.dtype).head;
    a.token_bytes = a.seg_bytes = a.block_bytes;
    tokens = nullptr;
  } else {
    a.block_bytes = (int64_t)d.page_size * d.kv_heads * d.head_dim * es;
    a.token_bytes = (c->heads_outside ? 1 : d.kv_heads) * d.head_dim * es;
    a.seg_bytes = a.token_bytes * d.page_size;
  }
  a.src = src;
  a.dst = dst;
  a.tokens = tokens;
  a.n = n;
  a.n_dev = n_dev;
  a.err = c->err;
  const bool wide = ((uintptr_t)d.k | (uintptr_t)d.v | (uint64_t)a.layer_bytes |
                     (uint64_t)a.page_bytes | (uint64_t)a.token_bytes) % 16 == 0;
  const unsigned grid = (unsigned)c->num_sms * 8;
  const dim3 g(grid), b(kCopyThreads);
  return wide      ? xp_launch_pdl(copy_pages_kernel<uint4>, g, b, 0, s, a)
         : es == 4 ? xp_launch_pdl(copy_pages_kernel<uint32_t>, g, b, 0, s, a)
                   : xp_launch_pdl(copy_pages_kernel<uint16_t>, g, b, 0, s, a);
}

cudaError_t xp_launch_resize(const xp_cache* c, const int32_t* table, int64_t ld,
                             const int32_t* lens, const int32_t* new_lens, const int32_t* refs,
                             int N, int width, int32_t* table_out, int64_t ld_out,
                             int32_t* lens_out, int32_t* refs_out, cudaStream_t s) {
  ResizeArgs a = {table, ld, lens, new_lens, refs, N, width, c->d.pages, c->d.page_size,
                  table_out, ld_out, lens_out, refs_out, c->row_a, c->row_b, c->row_c, c->src,
                  c->err};
  resize_kernel<<<kCtas, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t xp_launch_fork(const xp_cache* c, const int32_t* table, int64_t ld,
                           const int32_t* lens, int rows, const int32_t* parent,
                           const int32_t* cut, int M, int width, const int32_t* refs,
                           bool in_place, int32_t* child, int64_t ld_child, int32_t* child_lens,
                           int32_t* refs_out, cudaStream_t s) {
  ForkArgs a = {table, ld, lens, rows, parent, cut, refs, M, width, c->d.pages, c->d.page_size,
                in_place, child, ld_child, child_lens, refs_out, c->row_a, c->row_b, c->row_c,
                c->row_d, c->src, c->dst, c->cnt, c->n_moves, c->err};
  fork_kernel<<<kCtas, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return xp_launch_copy_pages(c, c->src, c->dst, c->cnt, 0, c->n_moves, s);
}

cudaError_t xp_launch_compact(const xp_cache* c, const int32_t* table, int64_t ld,
                              const int32_t* lens, int N, int width, const int32_t* refs,
                              int32_t* table_out, int64_t ld_out, int32_t* refs_out, int32_t* map,
                              int32_t* live, cudaStream_t s) {
  CompactArgs a = {table, ld, lens, refs, N, width, c->d.pages, c->d.page_size, table_out, ld_out,
                   refs_out, map ? map : c->map, live, c->src, c->dst, c->n_moves, c->err};
  compact_kernel<<<kCtas, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return xp_launch_copy_pages(c, c->src, c->dst, nullptr, 0, c->n_moves, s);
}
