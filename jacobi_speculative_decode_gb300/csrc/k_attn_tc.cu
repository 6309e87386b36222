// Shared-prefix attention on tcgen05 (bf16, head_dim 64 or 128, pages of a multiple of 8
// tokens).
//
// A CTA runs two streams of (128 query rows) x (128 keys) tiles through one softmax pass:
//   S = Q K^T (tcgen05, fp32 in tensor memory), P = 2^(c S - m) rounded to bf16 over S,
//   O += P V (tcgen05, P read from tensor memory), running maximum m and sum per row.
// The streams alternate on the tensor core, so one stream's products run under the other's
// exponentials.  They are two row tiles of one kv head that share every K and V tile (the prefix,
// and blocks of more than 128 rows); one row tile of each of two kv heads; or, for the last
// head of an odd number, the even and the odd key tiles of one row tile, with a result each.
// O is rescaled only when a row's maximum grew by more than 2^8 since the last time.
//
// Warps: 0-7 and 8-15 the softmax of stream 0 and 1 (a warp is 16 query rows, four lanes a row),
// 16 and 17 issue their products, 18 loads K and V by TMA, a box of tokens of one page at a
// time, 19 cuts the work and loads the queries.
//
// What bounds it.  Two row tiles against 128 keys of 128 dims are 16.8 MFLOP, and 256 KB of
// shared memory read by the products: 2,048 cycles either way.  A pair of tiles takes 2,700 to
// 2,800, as each stream's chain is as long: S 512, softmax to the first half of P 990 and to the
// second 550, the second half of P V 256, and about 100 for each of four hand-overs.  128
// blocks of 16 tokens, 32 heads of 128 over 8, behind a shared prefix of 8192 and tails up to
// 2048 (309 GFLOP, 608 MB): 244 us with the joining kernel, back to back, 1.27 PFLOP/s, 68% of
// measured.
// A tail of few rows is bound by one tile's chain, 2,160 cycles for a tile of 128 keys of two
// heads, and by what a unit costs at its ends (about 5,000 cycles: a masked tile, the last
// product, the result's way out, code and constants that must be fetched anew).  256 single tokens,
// 64 heads of 64 over 8, a prefix of 16384 and tails up to 2000 (588 MB): 164 us, 3.6 TB/s.
// (Two streams on one head's even and odd tiles took 20% more: two results and two ends a unit.)
// A prompt's tiles are all walked, those above the diagonal too: 2,048 tokens of 32 heads of 128 over
// 8 take 77 us, 446 TFLOP/s of what the mask leaves; 8,192 take 819, 671.
//
// P is rounded to bf16, 2^-9 of each weight, because the tensor core takes both operands of a
// product in one 16-bit type, and V is bf16; the sum of a row is taken before that rounding, in fp32.
// Errors against 64 bits are 2.1e-3 to 2.3e-3 of the outputs' norm, of which the outputs' own
// rounding to bf16 is 1.7e-3.  (The rest of each weight as a second operand would cost a third
// product for every two.)
//
// Tiles of 128 x 128: a product reads 8 KB of shared memory for 64 cycles of work, which is all
// that can be read; half a tile of rows or keys would be bound by it.  Two streams: 128 columns of
// scores and D of results each fill tensor memory at D = 128.
#include <math.h>

#include <algorithm>

#include "sm100_ptx.cuh"
#include "xp_device.cuh"

typedef __nv_bfloat16 bf16;

namespace {

constexpr int kRows = 128;      // query rows of a tile (tensor memory lanes)
constexpr int kTile = 128;      // keys of a tile
constexpr int kThreads = 640;
// registers a thread: 640 x 96 at launch, moved from the issuing warpgroup to the softmax ones
constexpr int kRegsIssue = 64, kRegsSoftmax = 104;
constexpr int kChunkBytes = kTile * 128;   // 64 elements of 128 rows, 128-byte swizzle
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.0f;   // growth of the maximum (base 2) that P may carry

template <int D>
struct Cfg {
  static constexpr int CH = D / 64;
  static constexpr int TILE_BYTES = CH * kChunkBytes;
  static constexpr int STAGES = D == 128 ? 5 : 10;
  static constexpr int SMEM = (2 + STAGES) * TILE_BYTES;
};

constexpr int kFrags = 4;       // fragments announced ahead
// What a unit of work is: two row tiles of one kv head, one row tile of each of two kv heads, one
// row tile of one
enum { kRowPair, kHeadPair, kSingle, kUnitKinds };
// cost of a key tile for each, and of a unit besides its tiles (ns / 180)
constexpr int kPairCost = 8, kHeadsCost = 9, kTileCost = 5, kUnitCost = 12;
constexpr int kHeadsFewCost = 8, kFewRows = 16;   // a head pair's tiles of few rows (one warp's)
constexpr int kMinChunk = kUnitCost + kTileCost;   // least cost a CTA is given

struct Frag {
  int kind;              // 0 prefix, 1 tail, -1 no more
  int unit;              // kRowPair, kHeadPair, kSingle
  int n, hk, tile;       // sequence (tail), first kv head, first row tile
  int len;               // keys of the source
  int t0, t1;            // key tiles
  int slot;              // where its partial result goes: -1 the unit's own place, else a CTA's
};

struct Bars {
  uint64_t full[10], empty[10];
  uint64_t frag_full[kFrags], frag_empty[kFrags];
  uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_full[2];
  uint64_t drained;              // both streams' products have all run
  Frag frag[kFrags];
  int total[kThreads / 32], start_base;   // start: where this CTA's share begins
  int start_n;
  uint32_t tmem_base;
  int abort;
  int issued[2];                 // items of each stream whose products are issued
};

// The work is one line of cost: the prefix's units, then those of each sequence's tail, by kind
// (every head's row tile pairs, then the tile over of two heads each, then of the last head alone);
// a unit costs kUnitCost and its kind's cost a key tile.  CTA i does [i*chunk, (i+1)*chunk) of the
// line, so that a unit may be cut anywhere between two of its tiles and every CTA gets the
// same.  A piece that begins its unit leaves its result in the unit's place, one that does not in
// the place of its CTA, of which there is at most one.
// The costs are timed (a unit 2.2 us, two row tiles 1.4 a key tile, two heads 1.6, or 1.4 with one
// warp's rows).  With 8 or 10 for two heads many blocks of 16 tokens take 2% more, with units of 20
// as long.  With 9 or 7 for few rows 256 single tokens take 6% and 1% more; 128 blocks of 4 tokens
// (32 rows, not few) 11% more with 7 than with 9 or 10.
struct Line {
  int H, pairs, odd, T;    // kv heads; row tiles as pairs and one over; key tiles
  bool few;                // rows of the one over
  __host__ __device__ Line(int heads, int row_tiles, bool few_over, int keys)
      : H(heads), pairs(row_tiles / 2), odd(row_tiles % 2), T((keys + kTile - 1) / kTile), few(few_over) {}
  __host__ __device__ int count(int kind) const {
    return kind == kRowPair ? H * pairs : !odd ? 0 : kind == kHeadPair ? H / 2 : H % 2;
  }
  __host__ __device__ int tile_cost(int kind) const {
    return kind == kRowPair ? kPairCost : kind == kSingle ? kTileCost : few ? kHeadsFewCost : kHeadsCost;
  }
  __host__ __device__ int unit(int kind) const { return tile_cost(kind) * T + kUnitCost; }
  // cost of the units of all kinds before this one; of everything (kind = kUnitKinds)
  __host__ __device__ int before(int kind) const {
    int sum = 0;
    for (int k = 0; k < kUnitKinds; ++k) sum += k < kind ? count(k) * unit(k) : 0;
    return T ? sum : 0;
  }
  __host__ __device__ int total() const { return before(kUnitKinds); }
  // first tile of such a unit that lies behind a cost of x from its beginning
  __host__ __device__ int tile_at(int kind, int x) const {
    const int y = x - kUnitCost;   // divisors known: no division at run time
    const int t = kind == kRowPair  ? (y + kPairCost - 1) / kPairCost
                  : kind == kSingle ? (y + kTileCost - 1) / kTileCost
                  : few             ? (y + kHeadsFewCost - 1) / kHeadsFewCost
                                    : (y + kHeadsCost - 1) / kHeadsCost;
    return y <= 0 ? 0 : t > T ? T : t;
  }
};

// the same value in every lane, known to be: descriptors made from it need no per-lane registers
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 operations an instruction
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  return pair(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// V tile as the B operand of P V: rows are keys (K), 64 head dims (N) contiguous per 128-byte
// row; 8-key groups 1024 B apart, 64-dim blocks one chunk apart
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kChunkBytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// place of K tile j and of V tile j of T in the order of loading: K0 K1 V0 K2 V1 ...
__device__ __forceinline__ int pos_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int pos_v(int j, int T) { return j < T - 1 ? 2 * j + 2 : 2 * T - 1; }

// query row r of row tile `tile`: its place among the N*T*heads rows, -1 behind the end, and the
// number of keys it sees
__device__ __forceinline__ int64_t row_of(const xp_attn_args& g, const Frag& w, int hk, int tile, int r,
                                          int* n, int* t, int* h, int* limit) {
  const int per_seq = g.a.T * g.group, i = tile * g.plan.rows_tile + r;
  *limit = 0;
  if (i >= (w.kind == 0 ? g.a.N * per_seq : per_seq)) return -1;
  *n = w.kind == 0 ? i / per_seq : w.n;
  *t = i % per_seq / g.group;
  *h = hk * g.group + i % g.group;
  *limit = w.kind == 0 ? w.len : w.len - g.a.T + *t + 1;
  return ((int64_t)*n * g.a.T + *t) * g.a.heads + *h;
}

// Partial results lie in blocks of 32 query rows, [D/4][32 rows][4], so that a warp writes and
// reads them 512 bytes at a time: the prefix's by kv head, each sequence's by kv head, then stream
// 1's of the single units (the last row tile of the last kv head, where both are odd), then 8 blocks
// for every CTA's piece that does not begin its unit.
__device__ __forceinline__ int64_t block_of(const xp_attn_args& g, int kind, int n, int hk) {
  const int64_t all = g.plan.prefix_blocks;
  return kind == 0 ? hk * all : g.kv_heads * all + ((int64_t)n * g.kv_heads + hk) * g.plan.tail_blocks;
}
__device__ __forceinline__ int64_t second_block_of(const xp_attn_args& g, int kind, int n) {
  const int64_t one = min(g.plan.tail_blocks, 4);
  return block_of(g, 1, g.a.N, 0) + (kind == 0 ? 0 : 4 + n * one);
}
__device__ __forceinline__ int64_t cut_block(const xp_attn_args& g, int64_t cta, int half) {
  return block_of(g, 1, g.a.N, 0) + g.plan.second_blocks + cta * 8 + half * 4;
}

__device__ __forceinline__ int tail_len(const xp_attn_args& g, int n, bool tell) {
  int len = g.lens[n];
  if (len < 0 || len > g.a.max_len) {
    if (tell) atomicOr(g.err, XP_ERR_LENGTH);
    len = len < 0 ? 0 : g.a.max_len;
  }
  return len;
}

// Sums the tails' costs over the CTA: the chunk, and the sequence in which this CTA's share
// begins (with the cost before it).  CTA 0 leaves the chunk and every sequence's beginning for
// the kernel that joins the results.
__device__ int plan_line(const xp_attn_args& g, Bars* bars) {
  const int before = Line(g.kv_heads, g.plan.prefix_tiles, g.plan.prefix_few, g.a.prefix_len).total();
  const int N = g.a.max_len > 0 ? g.a.N : 0;
  const int per = (N + kThreads - 1) / kThreads, n0 = min(N, (int)threadIdx.x * per), n1 = min(N, n0 + per);
  auto cost = [&](int n) {
    return Line(g.kv_heads, g.plan.tail_tiles, g.plan.tail_few, tail_len(g, n, blockIdx.x == 0)).total();
  };
  int mine = 0;
  for (int n = n0; n < n1; ++n) mine += cost(n);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) bars->total[warp] = inc;
  __syncthreads();
  int base = before + inc - mine, all = before;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int t = bars->total[w];
    base += w < warp ? t : 0;
    all += t;
  }
  const int chunk = max(kMinChunk, (int)((all + gridDim.x - 1) / gridDim.x));
  const int x = blockIdx.x * chunk;
  for (int n = n0; n < n1; ++n) {
    const int c = per == 1 ? mine : cost(n);
    if (blockIdx.x == 0) g.line[1 + n] = base;
    if (c > 0 && x >= base && x < base + c) {
      bars->start_n = n;
      bars->start_base = base;
    }
    base += c;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) g.line[0] = chunk;
  __syncthreads();
  return x < all ? chunk : 0;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_q, const xp_attn_args g, int box, bool q_tma,
                   bool q_wide) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bars = reinterpret_cast<Bars*>(smem + C::SMEM);
  volatile int* abort = &bars->abort;
  const uint32_t sq = ptx::smem_u32(smem), ring = sq + 2 * C::TILE_BYTES;
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;

  const int chunk = plan_line(g, bars);
  if (chunk == 0) return;   // the line ends before this CTA's share
  if (sq & 1023u) {         // the swizzled tiles need it; the declared alignment gives it
    if (threadIdx.x == 0) atomicOr(g.err, XP_ERR_TIMEOUT);
    return;
  }

  if (threadIdx.x == 0) {
    auto init = [](uint64_t* bar, int count) { ptx::mbar_init(ptx::smem_u32(bar), count); };
    for (int s = 0; s < C::STAGES; ++s) {
      init(&bars->full[s], 1);
      init(&bars->empty[s], 2);
    }
    for (int s = 0; s < kFrags; ++s) {
      init(&bars->frag_full[s], 1);
      init(&bars->frag_empty[s], 19);   // 16 softmax warps, 2 issuing the products, 1 loading
    }
    for (int t = 0; t < 2; ++t) {
      init(&bars->q_full[t], 1);
      init(&bars->q_empty[t], 2);
      init(&bars->s_full[t], 1);
      init(&bars->p_half[t], 8);
      init(&bars->p_full[t], 8);
      init(&bars->o_full[t], 1);
    }
    init(&bars->drained, 2);
    bars->abort = 0;
    bars->issued[0] = bars->issued[1] = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 16) {
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem_base), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  auto wait = [&](uint64_t* bar, int phase) {
    const bool ok = ptx::mbar_wait(ptx::smem_u32(bar), phase & 1, abort, g.err);
    return __all_sync(0xFFFFFFFFu, ok) != 0;
  };
  // fragment f as announced; its place is free again at once
  auto next_frag = [&](int f, Frag* w) {
    if (!wait(&bars->frag_full[f % kFrags], f / kFrags)) return false;
    *w = bars->frag[f % kFrags];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->frag_empty[f % kFrags]));
    return w->kind >= 0;
  };

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 19) {
      // ---- announces the fragments and loads their query tiles: two for a pair, one of the two
      // places in turn for a single unit, so that the next one's queries are there before the
      // present one is done ----
      const int x0 = blockIdx.x * chunk, x1 = x0 + chunk;
      const Line pre(g.kv_heads, g.plan.prefix_tiles, g.plan.prefix_few, g.a.prefix_len);
      const int before = pre.total();
      const int N = g.a.max_len > 0 ? g.a.N : 0;
      const uint64_t once = ptx::policy_evict_first();
      int f = 0, splits = 0, used[2] = {0, 0};
      bool ok = true;
      auto load_q = [&](const Frag& w, int hk, int tile, int place) {
        if (!wait(&bars->q_empty[place], (used[place] & 1) ^ 1)) return false;
        ++used[place];
        uint8_t* dst = smem + place * C::TILE_BYTES;
        if (q_tma) {   // whole tokens, all the group's heads of each
          if (lane == 0) {
            const uint32_t bar = ptx::smem_u32(&bars->q_full[place]);
            const int token = (w.kind == 0 ? 0 : w.n * g.a.T) + tile * (g.plan.rows_tile / g.group);
            ptx::mbar_arrive_expect_tx(bar, g.plan.rows_tile * 128 * C::CH);
            for (int ch = 0; ch < C::CH; ++ch)
              ptx::tma_load_4d(ptx::smem_u32(dst + ch * kChunkBytes), &tm_q, bar, ch * 64, 0, hk, token,
                               once);
          }
          __syncwarp();
          return true;
        }
        for (int r = lane; r < g.plan.rows_tile; r += 32) {
          int n, t, h, lim;
          if (row_of(g, w, hk, tile, r, &n, &t, &h, &lim) < 0) break;   // rows behind the end: anything
          const uint16_t* src = (const uint16_t*)g.q + n * g.a.q_stride_n + t * g.a.q_stride_t +
                                h * g.a.q_stride_h;
          auto to = [&](int seg) {
            return dst + (seg / 8) * kChunkBytes + r * 128 + (((seg % 8) ^ (r & 7)) << 4);
          };
          if (q_wide) {
#pragma unroll 4
            for (int seg = 0; seg < D / 8; ++seg) *(uint4*)to(seg) = *(const uint4*)(src + seg * 8);
          } else {
#pragma unroll 1
            for (int seg = 0; seg < D / 8; ++seg)
#pragma unroll
              for (int e = 0; e < 8; ++e) ((uint16_t*)to(seg))[e] = src[seg * 8 + e];
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->q_full[place]));
        return true;
      };
      auto announce = [&](const Frag& w) {
        if (!wait(&bars->frag_empty[f % kFrags], ((f / kFrags) & 1) ^ 1)) return false;
        if (lane == 0) {
          bars->frag[f % kFrags] = w;
          ptx::mbar_arrive(ptx::smem_u32(&bars->frag_full[f % kFrags]));
        }
        __syncwarp();
        ++f;
        if (w.kind < 0) return true;
        const bool one = w.unit == kSingle;
#pragma unroll 1
        for (int k = 0; k < (one ? 1 : 2); ++k)
          if (!load_q(w, w.hk + (w.unit == kHeadPair ? k : 0), w.tile + (w.unit == kRowPair ? k : 0),
                      one ? splits & 1 : k))
            return false;
        splits += one;
        return true;
      };
      // the units of one source that lie in [x0, x1), from cost `at` on
      auto source = [&](const Line& l, int kind, int n, int len, int at) {
        if (l.T == 0) return true;
        for (int unit = 0; unit < kUnitKinds; ++unit) {
          const int count = l.count(unit), cost = l.unit(unit);
          int u = x0 > at ? min(count, (x0 - at) / cost) : 0;   // skip what lies before
          for (int from = at + u * cost; u < count && from < x1; ++u, from += cost) {
            const int t0 = l.tile_at(unit, x0 - from), t1 = l.tile_at(unit, min(x1 - from, cost));
            if (t0 >= t1) continue;
            const int hk = unit == kRowPair ? u / l.pairs : unit == kHeadPair ? 2 * u : l.H - 1;
            const int tile = unit == kRowPair ? 2 * (u % l.pairs) : 2 * l.pairs;
            const Frag w = {kind, unit, n, hk, tile, len, t0, t1, t0 > 0 ? (int)blockIdx.x : -1};
            if (!announce(w)) return false;
          }
          at += count * cost;
        }
        return true;
      };
      if (x0 < before) ok = source(pre, 0, 0, g.a.prefix_len, 0);
      if (x1 > before) {
        int n = x0 < before ? 0 : bars->start_n;
        int at = x0 < before ? before : bars->start_base;
        int len = n < N ? tail_len(g, n, false) : 0;
        for (; ok && n < N && at < x1; ++n) {
          const int after = n + 1 < N ? tail_len(g, n + 1, false) : 0;   // read ahead
          const Line l(g.kv_heads, g.plan.tail_tiles, g.plan.tail_few, len);
          ok = source(l, 1, n, len, at);
          at += l.total();
          len = after;
        }
      }
      if (ok) announce({-1, 0, 0, 0, 0, 0, 0, 0, 0});
      volatile int no_abort = 0;   // as with K and V below
      for (int p = 0; p < 2; ++p)
        if (used[p]) ptx::mbar_wait(ptx::smem_u32(&bars->q_full[p]), (used[p] - 1) & 1, &no_abort, g.err);
    } else if (warp == 18) {
      // ---- K and V tiles: lane (chunk, box) loads `box` tokens of one page.  The tails' rate is set
      // by how soon this warp comes to the next load: a copy takes it about 100 cycles to issue
      // (fewer where its operands are known to be one for the warp), nothing is divided from
      // tile to tile, and page ids are read two tiles ahead ----
      const uint64_t keep = ptx::policy_evict_last(), stream = ptx::policy_evict_first();
      const int per = kTile / box, in_tile = lane % per * box, chunk_of = lane / per;
      const int more = kTile / g.page_size, rest = kTile % g.page_size;   // a tile further
      const uint32_t place = ring + chunk_of * kChunkBytes + in_tile * 128;
      int issued = 0, s = 0;   // tiles loaded, the next one's stage
      Frag w;
      bool ok = true;
      for (int f = 0; ok && next_frag(f, &w); ++f) {
        const int32_t* table = w.kind == 0 ? g.prefix_table : g.table + w.n * g.ld_table;
        const int end = min(w.len, w.t1 * kTile), hk = (int)uniform(w.hk);
        const uint64_t policy = uniform(w.kind) == 0 ? keep : stream;
        // this lane's box of the next key tile to look up: where it is in the table
        int at = chunk_of < C::CH ? w.t0 * kTile + in_tile : end;
        int index = at / g.page_size, row = at - index * g.page_size;
        auto look_up = [&](int* from) {   // the page, -1 behind the end; *from: its row there
          const int page = at < end ? table[index] : -1;
          *from = at < end ? row : -1;
          at += chunk_of < C::CH ? kTile : 0;
          index += more;
          row += rest;
          if (row >= g.page_size) {
            row -= g.page_size;
            ++index;
          }
          return page;
        };
        auto check = [&](int page, int from) {   // at its first use, not when it is asked for
          if (from >= 0 && (page < 0 || page >= g.pages)) {
            atomicOr(g.err, XP_ERR_BADPAGE);
            page = page < 0 ? 0 : g.pages - 1;
          }
          return page;
        };
        // tile j of the ring: key tile j, or, of two heads in turn, key tile j / 2
        const int heads = uniform(w.unit) == kHeadPair, T = (w.t1 - w.t0) << heads;
        auto load = [&](int j, int page, int from, const CUtensorMap* map) {
          if (!wait(&bars->empty[s], ((issued / C::STAGES) & 1) ^ 1)) return false;
          const uint32_t full = uniform(ptx::smem_u32(&bars->full[s]));
          // a whole number of boxes, which are powers of two
          const int rows = (min(kTile, end - (w.t0 + (j >> heads)) * kTile) + box - 1) & -box;
          if (lane == 0) ptx::mbar_arrive_expect_tx(full, rows * 128 * C::CH);
          __syncwarp();
          if (from >= 0)
            ptx::tma_load_5d(place + s * C::TILE_BYTES, map, full, C::CH == 1 ? 0 : chunk_of * 64, from,
                             hk + (j & heads), page, g.a.layer, policy);
          ++issued;
          s = s + 1 == C::STAGES ? 0 : s + 1;
          return true;
        };
        int row0, row1, row2;
        int now = look_up(&row0), next = now, after;
        row1 = row0;
        if (!heads) next = look_up(&row1);
        now = check(now, row0);
        ok = load(0, now, row0, &tm_k);
        for (int j = 0; j < T && ok; ++j) {
          after = next, row2 = row1;
          if (!(heads && (j & 1))) after = look_up(&row2);
          if (j + 1 < T) {
            next = check(next, row1);
            ok = load(j + 1, next, row1, &tm_k);
          }
          ok = ok && load(j, now, row0, &tm_v);
          now = next, row0 = row1;
          next = after, row1 = row2;
        }
      }
      // nothing may land in shared memory after the CTA is gone: neither the loads nor the
      // products' arrivals
      volatile int no_abort = 0;
      for (int s = 0; s < C::STAGES; ++s) {
        const int n = (issued + C::STAGES - 1 - s) / C::STAGES;   // loads of this stage
        if (n > 0) {
          ptx::mbar_wait(ptx::smem_u32(&bars->full[s]), (n - 1) & 1, &no_abort, g.err);
          if (!*abort) ptx::mbar_wait(ptx::smem_u32(&bars->empty[s]), (n - 1) & 1, abort, g.err);
        }
      }
    } else {
      // ---- the products of stream t: O += P V of its item j, then S = Q K^T of item j + 1 in
      // its place.  The warp runs the loop converged, so that descriptors stay in uniform
      // registers, and a warp a stream, so that one's waits run under the other's products ----
      constexpr uint32_t kS = ptx::idesc_bf16_f32(kRows, kTile);
      constexpr uint32_t kO = ptx::idesc_bf16_f32(kRows, D) | (1u << 16);   // V: head dims contiguous
      const int t = warp - 16;
      const uint32_t s_col = uniform(tmem + t * kTile), o_col = uniform(tmem + 2 * kTile + t * D);
      const bool leader = ptx::elect_one();
      int done = 0, other = 0, pos0 = 0, splits = 0, used[2] = {0, 0};   // items of both streams
      int seen = 0;   // loads this warp has seen land
      // The streams take turns: were both to issue together, their products would end together,
      // and neither's would run under the other's exponentials.  A pause, nothing more: it
      // ends by itself, and no result depends on it.
      auto turn = [&](int j, int theirs) {
        const int want = other + min(t ? j + 1 : j, theirs);
        for (int spin = 0; spin < 100 && *(volatile int*)&bars->issued[1 - t] < want; ++spin) {}
        __syncwarp();
      };
      Frag w;
      bool ok = true;
      for (int f = 0; ok && next_frag(f, &w); ++f) {
        const bool one = w.unit == kSingle, same = w.unit == kRowPair;   // same: one ring of tiles for both
        const int keys = w.t1 - w.t0, T = w.unit == kHeadPair ? 2 * keys : keys;   // T: tiles of the ring
        const int items = one ? keys : 2 * keys, mine = (items + 1 - t) / 2;
        const int place = one ? splits & 1 : t, end = min(w.len, w.t1 * kTile);
        const uint32_t q = uniform(sq + place * C::TILE_BYTES);
        auto kv = [&](int j) { return same ? j : 2 * j + t; };
        // An mbarrier tells a phase from the one before it only.  So both warps see every load of
        // the ring land, in order, their own or not, and a stage is free again when both are
        // done with it: behind the products that read it, or at once where it is the other
        // stream's tile.  (The same holds for the places of the queries.)
        auto see = [&](int off) {
          for (; seen <= pos0 + off; ++seen) {
            const int s = seen % C::STAGES, o = seen - pos0;
            if (!wait(&bars->full[s], seen / C::STAGES)) return false;
            const int tile = o == 0 ? 0 : o == 2 * T - 1 ? T - 1 : o & 1 ? (o + 1) / 2 : o / 2 - 1;
            if (!same && (tile & 1) != t && lane == 0)
              ptx::mbar_arrive(ptx::smem_u32(&bars->empty[s]));
          }
          return true;
        };
        auto release = [&](int pos) { ptx::mma_commit(ptx::smem_u32(&bars->empty[pos % C::STAGES])); };
        auto scores = [&](int j) {
          const int pos = pos0 + pos_k(kv(j));
          const uint32_t k = uniform(ring + pos % C::STAGES * C::TILE_BYTES);
          if (leader) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = (ks / 4) * kChunkBytes + (ks % 4) * 32;
              ptx::mma_bf16(s_col, ptx::sw128_desc(q + off), ptx::sw128_desc(k + off), kS, ks > 0);
            }
            ptx::mma_commit(ptx::smem_u32(&bars->s_full[t]));
            release(pos);
            if (j == mine - 1) ptx::mma_commit(ptx::smem_u32(&bars->q_empty[place]));   // all read
          }
          __syncwarp();
        };
        for (int p = 0; p < 2 && ok; ++p) {
          if (one && p != place) continue;
          ok = wait(&bars->q_full[p], used[p]++);
          if (ok && (p != place || mine == 0) && lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->q_empty[p]));
        }
        splits += one;
        if (ok && mine > 0) {
          ok = see(pos_k(kv(0)));
          if (!ok) break;
          ptx::tc_fence_after();
          scores(0);
        }
        for (int j = 0; j < mine && ok; ++j) {
          const int pv = pos0 + pos_v(kv(j), T), valid = end - (w.t0 + (one ? kv(j) : j)) * kTile;
          // the tiles are there before the weights are
          ok = see(pv - pos0) && (j + 1 >= mine || see(pos_k(kv(j + 1))));
          if (!ok) break;
          // V rows behind the range may hold anything: cleared before the product reads them
          // (streams that share the tile both write the zeros)
          if (valid < kTile) {
            uint8_t* rows = smem + (2 + pv % C::STAGES) * C::TILE_BYTES;
            for (int i = lane; i < (kTile - valid) * C::CH * 8; i += 32) {
              const int rr = valid + i / (C::CH * 8), seg = i % (C::CH * 8);
              *(uint4*)(rows + (seg / 8) * kChunkBytes + rr * 128 + (seg % 8) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          ok = wait(&bars->p_half[t], done + j);
          if (!ok) break;
          turn(j, items - mine);
          ptx::tc_fence_after();
          const uint32_t v = uniform(ring + pv % C::STAGES * C::TILE_BYTES);
          if (leader) {
#pragma unroll
            for (int ks = 0; ks < kTile / 32; ++ks)
              ptx::mma_bf16_ts(o_col, s_col + ks * 8, v_desc(v + ks * 2048), kO, j > 0 || ks > 0);
          }
          __syncwarp();
          ok = wait(&bars->p_full[t], done + j);
          if (!ok) break;
          ptx::tc_fence_after();
          if (leader) {
#pragma unroll
            for (int ks = kTile / 32; ks < kTile / 16; ++ks)
              ptx::mma_bf16_ts(o_col, s_col + ks * 8, v_desc(v + ks * 2048), kO, 1);
            ptx::mma_commit(ptx::smem_u32(&bars->o_full[t]));
            release(pv);
          }
          __syncwarp();
          if (j + 1 < mine) scores(j + 1);
          if (leader) *(volatile int*)&bars->issued[t] = done + j + 1;
        }
        ok = ok && see(2 * T - 1);
        done += mine;
        other += items - mine;
        pos0 += 2 * T;
      }
      // whatever ended the loop, tensor memory is freed behind the last product only
      if (leader) ptx::mma_commit(ptx::smem_u32(&bars->drained));
    }
  } else {
    // ---- softmax: a warp is 16 query rows; a thread holds, of two rows 8 apart, every fourth
    // pair of columns, so that a row's maximum is two shuffles away and its sum needs none ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp / 8, quad = lane % 4;
    const int r0 = warp % 4 * 32 + warp / 4 % 2 * 16 + lane / 4;      // and r0 + 8
    const uint32_t lanes = (uint32_t)(r0 - lane / 4) << 16;
    const float c = g.a.scale * 1.44269504088896f;
    const int all_rows = g.a.N * g.a.T * g.group, RT = g.plan.rows_tile;
    int done = 0, known = -1, token[2] = {0, 0};   // the rows' tokens in a tail's row tile `known`
    Frag w;
    bool ok = true;
    for (int f = 0; ok && next_frag(f, &w); ++f) {
      const bool one = w.unit == kSingle;
      const int T = w.t1 - w.t0, mine = one ? (T + 1 - t) / 2 : T;
      const int tile = w.unit == kRowPair ? w.tile + t : w.tile;
      const int hk = w.unit == kHeadPair ? w.hk + t : w.hk;
      const int end = min(w.len, w.t1 * kTile);
      // keys its rows see: all of a prefix, a tail's by the row's token
      int limit[2];
      bool any_row = false;
      if (w.kind == 1 && tile != known) {
        known = tile;
#pragma unroll
        for (int i = 0; i < 2; ++i) token[i] = (tile * RT + r0 + 8 * i) / g.group;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool is_row = r0 + 8 * i < RT && (w.kind == 0 ? tile * RT + r0 + 8 * i < all_rows : token[i] < g.a.T);
        limit[i] = is_row && w.kind == 1 ? min(w.len - g.a.T + token[i] + 1, end) : end;
        any_row |= is_row;   // rows behind the end ask for no mask
      }
      const bool active = __any_sync(0xFFFFFFFFu, any_row);
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};   // l: of this thread's columns
      for (int j = 0; j < mine; ++j) {
        ok = wait(&bars->s_full[t], done + j);
        if (!ok) break;
        const int kt = one ? 2 * j + t : j, key = (w.t0 + kt) * kTile;
        if (!active) {   // no rows here: only the hand-over
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(ptx::smem_u32(&bars->p_half[t]));
            ptx::mbar_arrive(ptx::smem_u32(&bars->p_full[t]));
          }
          continue;
        }
        ptx::tc_fence_after();
        const uint32_t scol = tmem + lanes + t * kTile;
        uint32_t s[2][32];   // [half of the columns][4 x 8 columns: row 0 pair, row 1 pair]
        ptx::tmem_ld_16x64(scol, s[0]);
        ptx::tmem_ld_16x64(scol + 64, s[1]);
        ptx::tmem_wait_ld();
        if (__any_sync(0xFFFFFFFFu, key + kTile > min(limit[0], limit[1]))) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (key + q * 64 + x / 4 * 8 + quad * 2 + x % 2 >= limit[x / 2 % 2])
                s[q][x] = 0xFF800000u;   // -inf
        }
        // The first half's weights are computed with the maximum as it was: it rarely grows by
        // more than P may carry, and neither has to wait for the other.
        const uint64_t c2 = pair(c, c);
        uint64_t sum[2];
        uint32_t pk[16];
        auto weights = [&](int q) {   // row x % 2, columns 8 (x / 2) + 2 quad
          const float b0 = m[0] == -INFINITY ? 0.0f : m[0] * c, b1 = m[1] == -INFINITY ? 0.0f : m[1] * c;
          const uint64_t nb[2] = {pair(-b0, -b0), pair(-b1, -b1)};
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const uint64_t z = fma2(pair(s[q][2 * x], s[q][2 * x + 1]), c2, nb[x % 2]);
            const float a = ex2(low(z)), b = ex2(high(z));
            sum[x % 2] = add2(sum[x % 2], pair(a, b));
            pk[x] = pack_bf16(a, b);
          }
        };
        sum[0] = sum[1] = 0;
        if (j > 0) weights(0);
        float now[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top[2];   // two chains, three operands an instruction
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            top[q] = fmaxf(__uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1]));
#pragma unroll
            for (int x = 4; x < 32; x += 4)
              top[q] = fmaxf(fmaxf(top[q], __uint_as_float(s[q][x + 2 * i])),
                             __uint_as_float(s[q][x + 2 * i + 1]));
          }
          now[i] = fmaxf(top[0], top[1]);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            now[i] = fmaxf(now[i], __shfl_xor_sync(0xFFFFFFFFu, now[i], o));
        now[0] = fmaxf(now[0], m[0]);
        now[1] = fmaxf(now[1], m[1]);
        const bool grown0 = j == 0 || (now[0] - m[0]) * c > kLazy;   // from -inf too
        const bool grown1 = j == 0 || (now[1] - m[1]) * c > kLazy;
        if (__any_sync(0xFFFFFFFFu, grown0 || grown1)) {
          if (j > 0) {
            ok = wait(&bars->o_full[t], done + j - 1);
            if (!ok) break;
            ptx::tc_fence_after();
            const float f0 = grown0 ? ex2((m[0] - now[0]) * c) : 1.0f;
            const float f1 = grown1 ? ex2((m[1] - now[1]) * c) : 1.0f;
            const uint32_t ocol = tmem + lanes + 2 * kTile + t * D;
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[16];
              ptx::tmem_ld_16x32(ocol + q * 32, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x)
                o[x] = __float_as_uint(__uint_as_float(o[x]) * (x & 2 ? f1 : f0));
              ptx::tmem_st_16x32(ocol + q * 32, o);
            }
            ptx::tmem_wait_st();
            l[0] *= f0;
            l[1] *= f1;
          }
          if (grown0) m[0] = now[0];
          if (grown1) m[1] = now[1];
          sum[0] = sum[1] = 0;
          weights(0);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q == 1) weights(1);
          ptx::tmem_st_16x32_narrow(scol + q * 32, pk);
          // the product may start on the first half of the keys
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(q == 0 ? &bars->p_half[t] : &bars->p_full[t]));
          __syncwarp();
        }
        l[0] += low(sum[0]) + high(sum[0]);
        l[1] += low(sum[1]) + high(sum[1]);
      }
      done += mine;
      if (!ok) break;
      if (mine == 0 || !active) continue;
      ok = wait(&bars->o_full[t], done - 1);
      if (!ok) break;
      ptx::tc_fence_after();
#pragma unroll
      for (int o = 1; o < 4; o <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], o);
      const int64_t block =
          (w.slot >= 0      ? cut_block(g, w.slot, t)
           : one && t == 1 ? second_block_of(g, w.kind, w.n)
                           : block_of(g, w.kind, w.n, hk) + tile * 4) +
          warp % 4;
      const int rb = r0 % 32;   // in the block, and rb + 8
      if (quad == 0)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          ((float2*)g.stat)[block * 32 + rb + 8 * i] =
              make_float2(l[i] > 0.0f ? m[i] * c : -INFINITY, l[i]);
      __syncwarp();
      float* acc = g.acc + block * D * 32 + (quad / 2 * 32 + rb) * 4 + quad % 2 * 2;
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        uint32_t o[32];
        ptx::tmem_ld_16x64(tmem + lanes + 2 * kTile + t * D + q * 64, o);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 8; ++k)   // 8 columns: two pieces of 16 bytes a row
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *(uint2*)&acc[((q * 8 + k) * 2 * 32 + 8 * i) * 4] =
                make_uint2(o[4 * k + 2 * i], o[4 * k + 2 * i + 1]);
      }
      ptx::tc_fence_before();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    volatile int no_abort = 0;
    ptx::mbar_wait(ptx::smem_u32(&bars->drained), 0, &no_abort, g.err);
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// A row's tail from the definition, joined to what its prefix left (maximum *m in base 2, sum *l,
// weighted values o of this thread's dims).  Hidden keys weigh nothing on the tensor cores, but nothing
// times an infinite or NaN value is NaN; a row with a NaN in its result that its prefix alone does
// not have comes here, where hidden values are not read.  A thread a row: slow, and for such
// inputs only.
template <int D>
__device__ __noinline__ void tail_again(const xp_attn_args& g, int n, int hk, int t, int h, int warp,
                                        float* m, float* l, float4* o) {
  const int end = tail_len(g, n, false) - g.a.T + t + 1;
  const float c = g.a.scale * 1.44269504088896f;
  const bf16* q = (const bf16*)g.q + n * g.a.q_stride_n + t * g.a.q_stride_t + h * g.a.q_stride_h;
  for (int j = 0; j < end; ++j) {
    const int page = min(max(g.table[n * g.ld_table + j / g.page_size], 0), g.pages - 1);
    const int64_t at = page * g.kv_page + j % g.page_size * g.kv_token + hk * g.kv_head;
    const bf16 *k = (const bf16*)g.k + at, *v = (const bf16*)g.v + at;
    float z = 0.0f;
#pragma unroll 8
    for (int d = 0; d < D; ++d) z = fmaf(__bfloat162float(q[d]), __bfloat162float(k[d]), z);
    z *= c;
    const float now = fmaxf(*m, z);
    if (now == -INFINITY) continue;
    const float a = exp2f(*m - now), p = exp2f(z - now);
    *m = now;
    *l = *l * a + p;
    for (int i = 0; i < D / 32; ++i) {
      const bf16* x = v + (warp + 8 * i) * 4;
      o[i] = make_float4(o[i].x * a + p * __bfloat162float(x[0]), o[i].y * a + p * __bfloat162float(x[1]),
                         o[i].z * a + p * __bfloat162float(x[2]), o[i].w * a + p * __bfloat162float(x[3]));
    }
  }
}

// A query row's partial results: of the prefix and of its tail, each the unit's own and those of
// the CTAs at whose beginning it was cut, brought to a common maximum:
//   out = sum a_p O_p / sum a_p l_p,  a_p = 2^(m_p - m).
// A CTA joins 32 rows of (sequence, kv head, token, head) order: a thread is a row, a warp every
// eighth of its 16-byte pieces; the rows leave through shared memory.  Bound by the partial
// results' bytes, mostly from L2: 65,536 rows of 128 with two or three each, about 80 MB, in
// 20 to 29 us; with few rows by the latency of what it asks for.
// TOGETHER: partial results asked for at once.  Few rows have many (a long prefix is cut by every
// CTA) and nobody else's work to wait under: four at once take 5% off both kernels' time (one
// request of 4 tokens).  Many rows have three or four, and one at a time leaves room for more
// CTAs: 3% off (128 blocks of 16 tokens).
template <int D, int TOGETHER>
__global__ void __launch_bounds__(256) attn_tc_combine_kernel(const __grid_constant__ xp_attn_args g,
                                                              int ctas) {
  constexpr int kPer = D / 32;   // 16-byte pieces a thread
  __shared__ __align__(16) uint2 s_out[32][D / 4 + 2];   // rows 16 bytes apart in the banks
  __shared__ bf16* s_to[32];
  ptx::pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per_seq = g.a.T * g.group;
  const int64_t rows = (int64_t)g.a.N * g.a.T * g.a.heads, e = (int64_t)blockIdx.x * 32 + lane;
  bf16* to = nullptr;
  if (e < rows) {
    const int i = (int)(e % per_seq), hk = (int)(e / per_seq % g.kv_heads);
    const int n = (int)(e / per_seq / g.kv_heads), t = i / g.group, h = hk * g.group + i % g.group;
    const int chunk = g.line[0], RT = g.plan.rows_tile;
    float m = -INFINITY, l = 0.0f;
    float4 o[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) o[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto join = [&](int kind) {
      const Line ln(g.kv_heads, kind ? g.plan.tail_tiles : g.plan.prefix_tiles,
                    kind ? g.plan.tail_few : g.plan.prefix_few,
                    kind ? tail_len(g, n, false) : g.a.prefix_len);
      if (ln.T == 0) return;
      const int at_row = (kind ? 0 : n * per_seq) + i, tile = at_row / RT;
      const int unit = tile < 2 * ln.pairs ? kRowPair : hk < ln.H / 2 * 2 ? kHeadPair : kSingle;
      const int u = unit == kRowPair ? hk * ln.pairs + tile / 2 : unit == kHeadPair ? hk / 2 : 0;
      const int cost = ln.unit(unit), at = (kind ? g.line[1 + n] : 0) + ln.before(unit) + u * cost;
      // a piece of a pair has a half of each, one of a single row tile a half of each stream (the
      // second from two key tiles on)
      const bool one = unit == kSingle;
      const int mine = unit == kRowPair ? tile % 2 : hk % 2;
      const int in_tile = at_row % RT / 32, r = at_row % RT % 32;
      int cut = (at / chunk + 1) * chunk - at;   // where the unit is first cut,
      if (ln.tile_at(unit, cut) == 0) cut += chunk;       // behind its first tile
      const int first = ln.tile_at(unit, min(cut, cost)), cta0 = at / chunk + 1;
      const int cuts = max(0, min(ctas - 1, (at + cost - 1) / chunk) - cta0 + 1);
      const int64_t own = block_of(g, kind, n, hk) + tile * 4 + in_tile;
      const int64_t second = second_block_of(g, kind, n) + in_tile;
      const int64_t cut0 = cut_block(g, cta0, 0) + in_tile;
      // the block of piece q: the unit's own (and its second), then those of the CTAs; -1: none
      auto block = [&](int q) -> int64_t {
        if (q == 0) return first > 0 ? own : -1;
        if (q == 1 && one) return first > 1 ? second : -1;
        const int c = one ? (q - 2) / 2 : q - 1, half = one ? q % 2 : mine;
        const int x = (cta0 + c) * chunk - at;
        const int t0 = ln.tile_at(unit, x), t1 = ln.tile_at(unit, min(x + chunk, cost));
        return t0 == 0 || t0 >= t1 || (one && half && t1 - t0 < 2) ? -1 : cut0 + c * 8 + half * 4;
      };
      const int pieces = one ? 2 + 2 * cuts : 1 + cuts;
      for (int q = 0; q < pieces; q += TOGETHER) {
        float2 st[TOGETHER];
        float4 x[TOGETHER][kPer];
#pragma unroll
        for (int u = 0; u < TOGETHER; ++u) {
          const int64_t b = q + u < pieces ? block(q + u) : -1;
          st[u] = make_float2(0.0f, 0.0f);
          if (b < 0) continue;
          st[u] = __ldcg((const float2*)g.stat + b * 32 + r);
#pragma unroll
          for (int c = 0; c < kPer; ++c)
            x[u][c] = __ldcs((const float4*)g.acc + (b * (D / 4) + warp + 8 * c) * 32 + r);
        }
#pragma unroll
        for (int u = 0; u < TOGETHER; ++u) {
          if (st[u].y == 0.0f) continue;   // no visible key in this piece: x may be anything
          const float now = fmaxf(m, st[u].x), a = exp2f(m - now), b = exp2f(st[u].x - now);
          m = now;
          l = l * a + st[u].y * b;
#pragma unroll
          for (int c = 0; c < kPer; ++c)
            o[c] = make_float4(o[c].x * a + x[u][c].x * b, o[c].y * a + x[u][c].y * b,
                               o[c].z * a + x[u][c].z * b, o[c].w * a + x[u][c].w * b);
        }
      }
    };
    join(0);
    if (g.a.max_len > 0) {
      join(1);
      auto nans = [&]() {   // of this thread's dims, a bit each
        unsigned bits = 0;
#pragma unroll
        for (int c = 0; c < kPer; ++c)
          bits |= (o[c].x != o[c].x ? 1u : 0u) << 4 * c | (o[c].y != o[c].y ? 2u : 0u) << 4 * c |
                  (o[c].z != o[c].z ? 4u : 0u) << 4 * c | (o[c].w != o[c].w ? 8u : 0u) << 4 * c;
        return bits;
      };
      float all = 0.0f;
#pragma unroll
      for (int c = 0; c < kPer; ++c) all += o[c].x + o[c].y + o[c].z + o[c].w;
      if (all != all && l == l && g.a.T > 1) {
        const unsigned whole = nans();
        m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int c = 0; c < kPer; ++c) o[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        join(0);
        if (whole & ~nans()) {   // the tail's doing
          float m2 = m, l2 = l;
          float4 o2[kPer];
#pragma unroll
          for (int c = 0; c < kPer; ++c) o2[c] = o[c];
          tail_again<D>(g, n, hk, t, h, warp, &m2, &l2, o2);
          m = m2, l = l2;
#pragma unroll
          for (int c = 0; c < kPer; ++c) o[c] = o2[c];
        } else {   // the prefix has them too, and every row sees that
          join(1);
        }
      }
    }
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;   // NaN where a visible score is
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      s_out[lane][warp + 8 * c] = make_uint2(pack_bf16(o[c].x * inv, o[c].y * inv),
                                             pack_bf16(o[c].z * inv, o[c].w * inv));
    to = (bf16*)g.out + n * g.a.o_stride_n + t * g.a.o_stride_t + h * g.a.o_stride_h;
    if (warp == 0 && g.lse)
      g.lse[((int64_t)n * g.a.T + t) * g.a.heads + h] =
          l != 0.0f ? (m + log2f(l)) * 0.693147180559945f : -INFINITY;
  }
  if (warp == 0) s_to[lane] = to;
  __syncthreads();
  for (int x = threadIdx.x; x < 32 * (D / 8); x += 256) {
    const int r = x / (D / 8), c = x % (D / 8);
    bf16* p = s_to[r];
    if (!p) continue;
    const uint4 v = *(const uint4*)&s_out[r][2 * c];
    if (((uintptr_t)p & 15) == 0) {
      *(uint4*)(p + c * 8) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) ((uint16_t*)p)[c * 8 + k] = (uint16_t)(w[k / 2] >> (k % 2 * 16));
    }
  }
}

template <int D>
cudaError_t launch(const xp_cache* c, const xp_attn_args& g, cudaStream_t s) {
  const size_t smem = Cfg<D>::SMEM + sizeof(Bars);
  static unsigned long long allowed = 0;
  cudaError_t e = xp_allow_smem((const void*)attn_tc_kernel<D>, smem, &allowed);
  if (e != cudaSuccess) return e;
  // Queries by TMA where a tile is a whole number of tokens, one stride apart; else by loads.
  CUtensorMap tm_q = {};
  // strides that are never used (one sequence, token or head) do not count
  const int64_t sh = g.a.heads > 1 ? g.a.q_stride_h : D;
  const int64_t token = g.a.T > 1   ? g.a.q_stride_t
                        : g.a.N > 1 ? g.a.q_stride_n
                                    : (int64_t)g.a.heads * D;
  const bool q_wide = (uintptr_t)g.q % 16 == 0 &&
                      ((g.a.N > 1 ? g.a.q_stride_n : 0) | (g.a.T > 1 ? g.a.q_stride_t : 0) | sh) % 8 == 0;
  bool q_tma = q_wide && g.group <= kRows &&
               (g.a.T == 1 || g.a.N == 1 || g.a.q_stride_n == g.a.T * token) && token > 0 && sh > 0;
  if (q_tma) {
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)g.group, (cuuint64_t)g.kv_heads,
                                (cuuint64_t)g.a.N * g.a.T};
    const cuuint64_t strides[3] = {(cuuint64_t)sh * 2, (cuuint64_t)sh * 2 * g.group,
                                   (cuuint64_t)token * 2};
    const cuuint32_t boxes[4] = {64, (cuuint32_t)g.group, 1, (cuuint32_t)(g.plan.rows_tile / g.group)};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    q_tma = xp_get_encode_tiled()(&tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, (void*)g.q, dims, strides,
                                  boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  attn_tc_kernel<D><<<c->num_sms, kThreads, smem, s>>>(c->tm_k, c->tm_v, tm_q, g, c->attn_tc, q_tma, q_wide);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)g.a.N * g.a.T * g.a.heads;
  const unsigned grid = (unsigned)((rows + 31) / 32);
  return xp_launch_pdl(grid <= (unsigned)c->num_sms ? attn_tc_combine_kernel<D, 4> : attn_tc_combine_kernel<D, 1>,
                       dim3(grid), dim3(256), 0, s, g, c->num_sms);
}

}  // namespace

// Tensor maps of the pools, (dim, token, head, page, layer) with boxes of 64 dims by the largest
// power of two of tokens that divides a page (8..128): a box never leaves its page, and 128
// keys are a whole number of boxes.  0 where the shapes do not allow it.
int xp_attn_tc_maps(xp_cache* c) {
  const xp_cache_desc& d = c->d;
  if (d.dtype != XP_BF16 || (d.head_dim != 64 && d.head_dim != 128) || d.page_size % 8 != 0 ||
      !xp_get_encode_tiled())
    return 0;
  int major = 0, minor = 0;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, c->device);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, c->device);
  if (major != 10 || minor != 3) return 0;
  int box = 8;
  while (box < 128 && d.page_size % (box * 2) == 0) box *= 2;
  const cuuint64_t dims[5] = {(cuuint64_t)d.head_dim, (cuuint64_t)d.page_size,
                              (cuuint64_t)d.kv_heads, (cuuint64_t)d.pages, (cuuint64_t)d.layers};
  const cuuint64_t strides[4] = {(cuuint64_t)d.stride_token * 2, (cuuint64_t)d.stride_head * 2,
                                 (cuuint64_t)d.stride_page * 2, (cuuint64_t)d.stride_layer * 2};
  const cuuint32_t boxes[5] = {64, (cuuint32_t)box, 1, 1, 1}, es[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < 4; ++i)
    if (strides[i] % 16 != 0 || strides[i] == 0) return 0;
  void* base[2] = {d.k, d.v};
  CUtensorMap* out[2] = {&c->tm_k, &c->tm_v};
  for (int i = 0; i < 2; ++i)
    if ((uintptr_t)base[i] % 16 != 0 ||
        xp_get_encode_tiled()(out[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base[i], dims, strides,
                              boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return 0;
  return box;
}

// Row tiles only: where the work is cut is found on the device, from the lengths.
xp_attn_plan xp_attn_tc_plan(const xp_cache* c, const xp_attn* a) {
  xp_attn_plan p = {};
  p.tc = true;
  const int per_seq = a->T * (a->heads / c->d.kv_heads);
  // Whole tokens, so that a tile's queries are one box.  Loaded by one warp's plain loads instead,
  // as where tokens are not one stride apart, 80 blocks of 2 tokens of groups of 7 take 45 us and not
  // 27, 128 blocks of 16 tokens 381 and not 240 (108 and 822 off 16-byte boundaries).
  const int group = a->heads / c->d.kv_heads, RT = group <= kRows ? kRows / group * group : kRows;
  p.rows_tile = RT;
  p.prefix_tiles = (int)(((int64_t)a->N * per_seq + RT - 1) / RT);
  p.tail_tiles = (per_seq + RT - 1) / RT;
  auto few = [&](int64_t rows) { return (rows - 1) % RT < kFewRows; };
  p.prefix_few = few((int64_t)a->N * per_seq);
  p.tail_few = few(per_seq);
  auto row_blocks = [&](int64_t rows) { return (int)(rows / RT * 4 + (rows % RT + 31) / 32); };
  p.prefix_blocks = row_blocks((int64_t)a->N * per_seq);
  p.tail_blocks = row_blocks(per_seq);
  const size_t H = c->d.kv_heads, D = c->d.head_dim;
  p.second_blocks = H % 2 ? 4 + (int64_t)a->N * std::min(p.tail_blocks, 4) : 0;
  const size_t blocks = H * p.prefix_blocks + (size_t)a->N * H * p.tail_blocks + p.second_blocks +
                        (size_t)c->num_sms * 8;
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = (o + bytes + 255) / 256 * 256; return at; };
  p.line_off = take(((size_t)a->N + 1) * 4);
  p.stat_off = take(blocks * 32 * 8);
  p.acc_off = take(blocks * 32 * D * 4);
  // the line's length, at the greatest lengths, has to be an int (with room for one share more)
  auto work_of = [](const Line& l) {
    double sum = 0;
    for (int k = 0; k < kUnitKinds; ++k)
      sum += (double)l.count(k) * ((double)l.tile_cost(k) * l.T + kUnitCost);
    return sum;
  };
  const double work = work_of(Line(c->d.kv_heads, p.prefix_tiles, p.prefix_few, a->prefix_len)) +
                      work_of(Line(c->d.kv_heads, p.tail_tiles, p.tail_few, a->max_len)) * a->N;
  p.total = work < 1e9 ? o : 0;
  return p;
}

cudaError_t xp_launch_attn_tc(const xp_cache* c, const xp_attn_args& g, cudaStream_t s) {
  return g.dim == 128 ? launch<128>(c, g, s) : launch<64>(c, g, s);
}
