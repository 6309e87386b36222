// Shared-prefix attention on tcgen05 (bf16, head_dim 64 or 128, pages of a multiple of 8
// tokens).
//
// A CTA runs two streams of (128 query rows) x (128 keys) tiles through one softmax pass:
//   S = Q K^T (tcgen05, fp32 in tensor memory), P = 2^(c S - m) rounded to bf16 over S,
//   O += P V (tcgen05, P read from tensor memory), running maximum m and sum per row.
// The streams alternate on the tensor core, so one stream's products run under the other's
// exponentials.  Where a row tile has a neighbour with the same keys (the prefix, and blocks
// of more than 128 rows) the two streams are two row tiles and share every K and V tile;
// else they are the even and the odd key tiles of one row tile and are joined at the end.
// O is rescaled only when a row's maximum grew by more than 2^8 since the last time.
//
// Warps: 0-3 and 4-7 the softmax of stream 0 and 1 (a thread is a query row), 8 and 9 issue
// their products, 10 loads K and V by TMA, a box of tokens of one page at a time.
#include <math.h>

#include <algorithm>

#include "sm100_ptx.cuh"
#include "xp_device.cuh"

typedef __nv_bfloat16 bf16;

namespace {

constexpr int kRows = 128;      // query rows of a tile (tensor memory lanes)
constexpr int kTile = 128;      // keys of a tile
constexpr int kThreads = 384;
// registers a thread: 384 x 168 at launch, moved from the issuing warpgroup to the softmax ones
constexpr int kRegsIssue = 56, kRegsSoftmax = 224;
constexpr int kChunkBytes = kTile * 128;   // 64 elements of 128 rows, 128-byte swizzle
constexpr uint32_t kTmemCols = 512;
constexpr int kApart = 4;       // items of a stream from which the streams are set apart
constexpr float kLazy = 8.0f;   // growth of the maximum (base 2) that P may carry

template <int D>
struct Cfg {
  static constexpr int CH = D / 64;
  static constexpr int TILE_BYTES = CH * kChunkBytes;
  static constexpr int STAGES = D == 128 ? 5 : 10;
  static constexpr int SMEM = (2 + STAGES) * TILE_BYTES;
};

struct Bars {
  uint64_t full[10], empty[10];
  uint64_t q_full, s_full[2], p_half[2], p_full[2], o_full[2];
  uint32_t tmem_base;
  int abort;
};

struct Unit {
  bool prefix, shared;   // shared: two row tiles over the same keys
  int n, hk, tile;       // first row tile (of the batch, or of the sequence)
  int part, k0, k1;      // key range
  int len;               // keys of the source
  const int32_t* table;
};

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

__device__ __forceinline__ bool decode_unit(const xp_attn_args& g, int u, Unit* w) {
  const xp_attn_plan& p = g.plan;
  const int pairs = (p.prefix_tiles + 1) / 2, n_prefix = p.prefix_splits * pairs * g.kv_heads;
  int tiles, split, step;
  w->prefix = u < n_prefix;
  if (w->prefix) {
    w->tile = u % pairs * 2;
    w->hk = u / pairs % g.kv_heads;
    split = u / pairs / g.kv_heads;
    w->n = 0;
    w->part = split;
    w->len = g.a.prefix_len;
    w->table = g.prefix_table;
    tiles = p.prefix_tiles;
    step = p.prefix_keys;
  } else {
    u -= n_prefix;
    const int tp = (p.tail_tiles + 1) / 2;
    w->hk = u % g.kv_heads;
    w->tile = u / g.kv_heads % tp * 2;
    split = u / g.kv_heads / tp % p.tail_splits;
    w->n = u / g.kv_heads / tp / p.tail_splits;
    w->part = p.prefix_splits + split;
    w->table = g.table + w->n * g.ld_table;
    w->len = g.lens[w->n];
    if (w->len < 0 || w->len > g.a.max_len) {
      if (threadIdx.x == 0) atomicOr(g.err, XP_ERR_LENGTH);
      w->len = w->len < 0 ? 0 : g.a.max_len;
    }
    tiles = p.tail_tiles;
    step = p.tail_keys;
  }
  w->shared = w->tile + 1 < tiles;
  w->k0 = split * step;
  w->k1 = min(w->len, w->k0 + step);
  return w->k0 < w->k1;
}

// query row r of a row tile: its place among the N*T*heads rows, -1 behind the end, and the
// number of keys it sees
__device__ __forceinline__ int64_t row_of(const xp_attn_args& g, const Unit& w, int tile, int r,
                                          int* n, int* t, int* h, int* limit) {
  const int per_seq = g.a.T * g.group, i = tile * kRows + r;
  *limit = 0;
  if (i >= (w.prefix ? g.a.N * per_seq : per_seq)) return -1;
  *n = w.prefix ? i / per_seq : w.n;
  *t = i % per_seq / g.group;
  *h = w.hk * g.group + i % g.group;
  *limit = min(w.k1, w.prefix ? w.len : w.len - g.a.T + *t + 1);
  return ((int64_t)*n * g.a.T + *t) * g.a.heads + *h;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const xp_attn_args g, int box, bool q_wide) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = ptx::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + C::SMEM);
  volatile int* abort = &bars->abort;
  const uint32_t sq = ptx::smem_u32(smem), ring = sq + 2 * C::TILE_BYTES;
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;

  Unit w;
  const bool work = decode_unit(g, blockIdx.x, &w);
  const int64_t rows = (int64_t)g.a.N * g.a.T * g.a.heads;
  const int per_tile_rows =
      min(kRows * (w.shared ? 2 : 1),
          (w.prefix ? g.a.N * g.a.T * g.group : g.a.T * g.group) - w.tile * kRows);
  if (!work) {   // no key in this range: its parts are empty
    for (int r = threadIdx.x; r < per_tile_rows; r += kThreads) {
      int n, t, h, lim;
      const int64_t row = row_of(g, w, w.tile, r, &n, &t, &h, &lim);
      *(float2*)&g.stat[(w.part * rows + row) * 2] = make_float2(-INFINITY, 0.0f);
    }
    return;
  }
  const int T = (w.k1 - w.k0 + kTile - 1) / kTile;
  const int items = w.shared ? 2 * T : T;
  // softmax warps that hold rows; the others stay out of the streams
  const int active0 = min(4, (per_tile_rows + 31) / 32);
  const int active1 = w.shared ? min(4, (per_tile_rows - kRows + 31) / 32) : active0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->empty[s]), w.shared ? 2 : 1);
    }
    ptx::mbar_init(ptx::smem_u32(&bars->q_full), 8);
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bars->s_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->p_half[t]), t ? active1 : active0);
      ptx::mbar_init(ptx::smem_u32(&bars->p_full[t]), t ? active1 : active0);
      ptx::mbar_init(ptx::smem_u32(&bars->o_full[t]), 1);
    }
    bars->abort = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 8) {
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem_base), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 10) {
      // ---- K and V tiles: lane (chunk, box) loads `box` tokens of one page ----
      const uint64_t pol = w.prefix ? ptx::policy_evict_last() : ptx::policy_evict_first();
      const int per = kTile / box, chunk = lane / per, in_tile = lane % per * box;
      int issued = 0;   // tiles loaded
      // this lane's page of tile j (its box may lie behind the range: then none is loaded)
      auto page_of = [&](int j) {
        const int at = w.k0 + j * kTile + in_tile;
        if (chunk >= C::CH || at >= w.k1) return -1;
        int page = w.table[at / g.page_size];
        if (page < 0 || page >= g.pages) {
          atomicOr(g.err, XP_ERR_BADPAGE);
          page = page < 0 ? 0 : g.pages - 1;
        }
        return page;
      };
      auto load = [&](int j, int page, const CUtensorMap* map) {
        const int s = issued % C::STAGES;
        bool ok = ptx::mbar_wait(ptx::smem_u32(&bars->empty[s]), ((issued / C::STAGES) & 1) ^ 1, abort,
                                 g.err);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) return false;
        const int key = w.k0 + j * kTile;
        const int boxes = (min(kTile, w.k1 - key) + box - 1) / box;
        const uint32_t full = ptx::smem_u32(&bars->full[s]);
        if (lane == 0) ptx::mbar_arrive_expect_tx(full, boxes * box * 128 * C::CH);
        __syncwarp();
        if (page >= 0)
          ptx::tma_load_5d(ring + s * C::TILE_BYTES + chunk * kChunkBytes + in_tile * 128, map, full,
                           chunk * 64, (key + in_tile) % g.page_size, w.hk, page, g.a.layer, pol);
        ++issued;
        return true;
      };
      int now = page_of(0), next = page_of(1);   // the page ids are read ahead of the loads
      bool ok = load(0, now, &tm_k);
      for (int j = 0; j < T && ok; ++j) {
        const int after = page_of(j + 2);
        if (j + 1 < T) ok = load(j + 1, next, &tm_k);
        ok = ok && load(j, now, &tm_v);
        now = next;
        next = after;
      }
      // nothing may land in shared memory after the CTA is gone
      volatile int no_abort = 0;
      for (int s = 0; s < C::STAGES; ++s) {
        const int n = (issued + C::STAGES - 1 - s) / C::STAGES;   // loads of this stage
        if (n > 0) ptx::mbar_wait(ptx::smem_u32(&bars->full[s]), (n - 1) & 1, &no_abort, g.err);
      }
    } else if (warp < 10) {
      // ---- the products of stream t: O += P V of its item j, then S = Q K^T of item j + 1 in
      // its place.  The warp runs the loop converged, so that descriptors stay in uniform
      // registers, and a warp a stream, so that one's waits run under the other's products ----
      constexpr uint32_t kS = ptx::idesc_bf16_f32(kRows, kTile);
      constexpr uint32_t kO = ptx::idesc_bf16_f32(kRows, D) | (1u << 16);   // V: head dims contiguous
      const int t = warp - 8, mine = (items + 1 - t) / 2;
      const uint32_t q = sq + (w.shared ? t * C::TILE_BYTES : 0);
      const uint32_t s_col = tmem + t * kTile, o_col = tmem + 2 * kTile + t * D;
      const bool leader = ptx::elect_one();
      auto wait = [&](uint64_t* bar, int phase) {
        const bool ok = ptx::mbar_wait(ptx::smem_u32(bar), phase & 1, abort, g.err);
        return __all_sync(0xFFFFFFFFu, ok) != 0;
      };
      auto loaded = [&](int pos) { return wait(&bars->full[pos % C::STAGES], pos / C::STAGES); };
      auto kv = [&](int j) { return w.shared ? j : 2 * j + t; };
      // the stage of load `pos` is free again, where another load waits for it (a commit that
      // nobody waits for could land behind the CTA's end)
      auto release = [&](int pos) {
        if (pos + C::STAGES < 2 * T) ptx::mma_commit(ptx::smem_u32(&bars->empty[pos % C::STAGES]));
      };
      auto scores = [&](int pos) {
        const uint32_t k = ring + pos % C::STAGES * C::TILE_BYTES;
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = (ks / 4) * kChunkBytes + (ks % 4) * 32;
            ptx::mma_bf16(s_col, ptx::sw128_desc(q + off), ptx::sw128_desc(k + off), kS, ks > 0);
          }
          ptx::mma_commit(ptx::smem_u32(&bars->s_full[t]));
          release(pos);
        }
        __syncwarp();
      };
      bool ok = mine > 0 && wait(&bars->q_full, 0) && loaded(pos_k(kv(0)));
      // the streams run half a period apart (started together they would stay together, and
      // neither's products would run under the other's exponentials)
      if (ok && t == 1 && mine >= kApart) ok = wait(&bars->p_half[0], 0);
      if (ok) {
        ptx::tc_fence_after();
        scores(pos_k(kv(0)));
      }
      for (int j = 0; j < mine && ok; ++j) {
        const int pv = pos_v(kv(j), T), pk = pos_k(kv(j + 1));
        const uint32_t v = ring + pv % C::STAGES * C::TILE_BYTES;
        // the tiles are there before the weights are
        ok = loaded(pv) && (j + 1 >= mine || loaded(pk));
        ok = ok && wait(&bars->p_half[t], j);
        if (!ok) break;
        ptx::tc_fence_after();
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < kTile / 32; ++ks)
            ptx::mma_bf16_ts(o_col, s_col + ks * 8, v_desc(v + ks * 2048), kO, j > 0 || ks > 0);
        }
        __syncwarp();
        ok = wait(&bars->p_full[t], j);
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
        if (j + 1 < mine) scores(pk);
      }
    }
  } else {
    // ---- softmax ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp / 4, r = threadIdx.x - t * 128;
    const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;
    const int tile = w.shared ? w.tile + t : w.tile;
    // the query tile, 16 bytes at a time, in the swizzled layout of the A operand
    if (t == 0 || w.shared) {
      constexpr int SEG = D / 8;
      for (int i = r; i < kRows * SEG; i += 128) {
        const int rr = i / SEG, seg = i % SEG;
        int n, tt, h, lim;
        uint4 val = make_uint4(0, 0, 0, 0);
        if (row_of(g, w, tile, rr, &n, &tt, &h, &lim) >= 0) {
          const bf16* src = (const bf16*)g.q + n * g.a.q_stride_n + tt * g.a.q_stride_t +
                            h * g.a.q_stride_h + seg * 8;
          if (q_wide) {
            val = *(const uint4*)src;
          } else {
            uint16_t e[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) e[x] = ((const uint16_t*)src)[x];
            val = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                             e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
          }
        }
        const int c = seg / 8;
        *(uint4*)(smem + t * C::TILE_BYTES + c * kChunkBytes + rr * 128 +
                  (((seg % 8) ^ (rr & 7)) << 4)) = val;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->q_full));

    const bool active = warp % 4 < (t ? active1 : active0);
    int n, tt, h, limit;
    const int64_t row = row_of(g, w, tile, r, &n, &tt, &h, &limit);
    if (row < 0) limit = w.k1;   // rows behind the end ask for no mask of their own
    const float c = g.a.scale * 1.44269504088896f;
    const int mine = active ? (items + 1 - t) / 2 : 0;   // items of this stream
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < mine; ++j) {
      ok = ptx::mbar_wait(ptx::smem_u32(&bars->s_full[t]), j & 1, abort, g.err);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t scol = tmem + lanes + t * kTile;
      uint32_t s[4][32];
#pragma unroll
      for (int q = 0; q < 4; ++q) ptx::tmem_ld32(scol + q * 32, s[q]);
      ptx::tmem_wait_ld();
      const int kt = w.shared ? j : 2 * j + t;
      const int key = w.k0 + kt * kTile;
      if (__any_sync(0xFFFFFFFFu, key + kTile > limit)) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (key + q * 32 + x >= limit) s[q][x] = 0xFF800000u;   // -inf
      }
      float top[4];   // four chains, three operands an instruction
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        top[q] = fmaxf(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]));
#pragma unroll
        for (int x = 2; x < 32; x += 2)
          top[q] = fmaxf(fmaxf(top[q], __uint_as_float(s[q][x])), __uint_as_float(s[q][x + 1]));
      }
      const float now = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), m);
      if (j == 0) {
        m = now;
      } else {
        const bool grown = (now - m) * c > kLazy;   // from -inf too
        if (__any_sync(0xFFFFFFFFu, grown)) {
          ok = ptx::mbar_wait(ptx::smem_u32(&bars->o_full[t]), (j - 1) & 1, abort, g.err);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          ptx::tc_fence_after();
          const float f = grown ? ex2((m - now) * c) : 1.0f;
          const uint32_t ocol = tmem + lanes + 2 * kTile + t * D;
#pragma unroll
          for (int q = 0; q < D / 16; ++q) {
            uint32_t o[16];
            ptx::tmem_ld16(ocol + q * 16, o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
            ptx::tmem_st16(ocol + q * 16, o);
          }
          ptx::tmem_wait_st();
          l *= f;
          if (grown) m = now;
        }
      }
      // V rows behind the range may hold anything: cleared before this stream's product reads
      // them (streams that share the tile both write the zeros)
      const int valid = w.k1 - key;
      if (valid < kTile) {
        const int pos = pos_v(kt, T), st = pos % C::STAGES;
        ok = ptx::mbar_wait(ptx::smem_u32(&bars->full[st]), (pos / C::STAGES) & 1, abort, g.err);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const int aw = t ? active1 : active0;
        uint8_t* v = smem + (2 + st) * C::TILE_BYTES;
        for (int i = (warp % 4) * 32 + lane; i < (kTile - valid) * C::CH * 8; i += aw * 32) {
          const int rr = valid + i / (C::CH * 8), seg = i % (C::CH * 8);
          *(uint4*)(v + (seg / 8) * kChunkBytes + rr * 128 + (seg % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      const float base = m == -INFINITY ? 0.0f : m * c;
      const uint64_t c2 = pair(c, c), nb2 = pair(-base, -base);
      uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t pk[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const uint64_t z = fma2(pair(s[q][2 * x], s[q][2 * x + 1]), c2, nb2);
          const float a = ex2(low(z)), b = ex2(high(z));
          sum[x % 4] = add2(sum[x % 4], pair(a, b));
          pk[x] = pack_bf16(a, b);
        }
        ptx::tmem_st16(scol + q * 16, pk);
        if (q == 1) {   // the product may start on the first half of the keys
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->p_half[t]));
        }
      }
      sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
      l += low(sum[0]) + high(sum[0]);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->p_full[t]));
    }
    if (mine > 0 && ok) {
      ok = ptx::mbar_wait(ptx::smem_u32(&bars->o_full[t]), (mine - 1) & 1, abort, g.err);
      ok = __all_sync(0xFFFFFFFFu, ok);
    }
    ptx::tc_fence_after();
    // a row's keys are the whole range (shared) or every second tile: join the two streams
    float f0 = 1.0f, f1 = 0.0f, mm = m, ll = l;
    if (!w.shared) {
      float2* stat = (float2*)(smem + C::TILE_BYTES);   // the second query tile's room is free
      stat[t * kRows + r] = make_float2(m, mine > 0 ? l : 0.0f);
      ptx::tc_fence_before();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      ptx::tc_fence_after();
      const float m0 = stat[r].x, l0 = stat[r].y;
      const float m1 = stat[kRows + r].x, l1 = stat[kRows + r].y;
      mm = fmaxf(l0 > 0.0f ? m0 : -INFINITY, l1 > 0.0f ? m1 : -INFINITY);
      f0 = l0 > 0.0f ? ex2((m0 - mm) * c) : 0.0f;
      f1 = l1 > 0.0f ? ex2((m1 - mm) * c) : 0.0f;
      ll = f0 * l0 + f1 * l1;
    }
    // each stream writes its rows, or (joined) its half of the head dims
    if (active && ok && !*abort) {
      const int q0 = w.shared ? 0 : t * (D / 64), q1 = w.shared ? D / 32 : q0 + D / 64;
      float* acc = g.acc + (w.part * rows + (row < 0 ? 0 : row)) * D;
      if (row >= 0 && (w.shared || t == 0))
        *(float2*)&g.stat[(w.part * rows + row) * 2] =
            make_float2(ll > 0.0f ? mm * c : -INFINITY, ll);
      for (int q = q0; q < q1; ++q) {
        uint32_t o[32];
        ptx::tmem_ld32(tmem + lanes + 2 * kTile + (w.shared ? t * D : 0) + q * 32, o);
        if (w.shared || items == 1) {
          ptx::tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f0);
        } else {
          uint32_t b[32];
          ptx::tmem_ld32(tmem + lanes + 2 * kTile + D + q * 32, b);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x)
            o[x] = __float_as_uint(__uint_as_float(o[x]) * f0 + __uint_as_float(b[x]) * f1);
        }
        if (row >= 0 && ll > 0.0f) {
#pragma unroll
          for (int x = 0; x < 32; x += 4)
            *(uint4*)(acc + q * 32 + x) = make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch(const xp_cache* c, const xp_attn_args& g, unsigned grid, cudaStream_t s) {
  const size_t smem = Cfg<D>::SMEM + sizeof(Bars) + 1024;
  static unsigned long long allowed = 0;
  const cudaError_t e = xp_allow_smem((const void*)attn_tc_kernel<D>, smem, &allowed);
  if (e != cudaSuccess) return e;
  const bool wide = ((uintptr_t)g.q | (uint64_t)g.a.q_stride_n * 2 | (uint64_t)g.a.q_stride_t * 2 |
                     (uint64_t)g.a.q_stride_h * 2) % 16 == 0;
  attn_tc_kernel<D><<<grid, kThreads, smem, s>>>(c->tm_k, c->tm_v, g, c->attn_tc, wide);
  return cudaGetLastError();
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

xp_attn_plan xp_attn_tc_plan(const xp_cache* c, const xp_attn* a) {
  xp_attn_plan p = {};
  const int group = a->heads / c->d.kv_heads, per_seq = a->T * group;
  p.rows_tile = kRows;
  p.prefix_tiles = (int)(((int64_t)a->N * per_seq + kRows - 1) / kRows);
  p.tail_tiles = (per_seq + kRows - 1) / kRows;
  // ranges of whole key tiles, so that about one CTA an SM has work, of at least two tiles
  auto splits = [&](int64_t units, int keys, int* range) {
    if (keys <= 0) return 0;
    const int tiles = (keys + kTile - 1) / kTile;
    int64_t s = std::max<int64_t>(1, c->num_sms / std::max<int64_t>(1, units));
    s = std::min<int64_t>(s, std::max(1, tiles / 2));
    *range = (int)((tiles + s - 1) / s) * kTile;
    return (keys + *range - 1) / *range;
  };
  p.prefix_splits = splits((int64_t)(p.prefix_tiles + 1) / 2 * c->d.kv_heads, a->prefix_len,
                           &p.prefix_keys);
  p.tail_splits = splits((int64_t)a->N * ((p.tail_tiles + 1) / 2) * c->d.kv_heads, a->max_len,
                         &p.tail_keys);
  p.parts = p.prefix_splits + p.tail_splits;
  return p;
}

cudaError_t xp_launch_attn_tc(const xp_cache* c, const xp_attn_args& g, cudaStream_t s) {
  const xp_attn_plan& p = g.plan;
  const unsigned grid = (unsigned)(((int64_t)p.prefix_splits * ((p.prefix_tiles + 1) / 2) +
                                    (int64_t)g.a.N * ((p.tail_tiles + 1) / 2) * p.tail_splits) *
                                   g.kv_heads);
  if (grid == 0) return cudaSuccess;
  return g.dim == 128 ? launch<128>(c, g, grid, s) : launch<64>(c, g, grid, s);
}
