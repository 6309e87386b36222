// Shared-prefix attention over a quantised cache (8 or 4 bits), from the packed bytes.
//
//   out = softmax(scale q . k^) v^ with k^ = c s, v^ = c s the values held.
//
// Few queries see each key (one token, or a drafted block, of a group of heads), so the cache's bytes and
// what it costs to widen them bound the call, not the products.  Keys are the rows of a product's tile and
// queries its 8 columns: S^T = K^ Q^T, then O^T = V^^T P^T (mma.sync m16n8k16, fp16 operands, fp32 sums), so
// that 4 queries fill half a tile and not a quarter or less.  (tcgen05 takes its operands from shared or
// tensor memory: widened values would be written there and read again, 512 bytes a key and head of
// 128, where here they go from a register to a product.)  A product sums over its k index in any order, so
// a lane takes the dims and keys whose codes lie side by side: 32 dims of a key for K^, 16 dims
// of four keys for V^, each one or two vector loads from shared memory.
//
// What bounds it: no one thing, but a warp's own chain of instructions.  A warp's step of 32 keys of 128 dims in 4
// bits is 4.6 KB, 206 cycles of an SM's share of HBM, and 700 instructions, 175 cycles of its four issue slots;
// 290 of them, mostly what picks codes out of words, are the logic pipe's, which takes one every other cycle.  16
// single tokens, 32 heads of 128 over 8, contexts of 1000 to 32768 (311 MB): 75 us, 4.1 TB/s, 61% of measured,
// and 4 more with the joining; issue slots are busy in 57% of the cycles, the logic pipe in 48%, the tensor pipe in 24%.
// An SM's 14 warps, 3.5 a scheduler, issue every 6 cycles each: 1.2 of them wait for the instruction before,
// 1.6 for a pipe's turn, 0.9 for memory, 1.1 for another warp.  Without its loads it takes 62 us.  In 8 bits (589 MB)
// 118 us for both kernels, 73% of measured.
//
// A value held is exact in fp16 (quant.cuh).  Queries are bf16, scaled by a power of two a row so that
// their largest is in [1, 4) (4 bits: 128 times that, and 1/16 in odd pairs): exact but for what lies 2^-14 and more
// below it, which loses less than 2^-25 of the largest.  Weights are 2^(z - m + 6), rounded to fp16 (2^-12 of
// each, and 2^-31 of the largest where that is more): as the second product's operand they have to be 16 bits,
// and fp16 leaves an eighth of bf16's error.  Sums are taken before that rounding, in fp32, as are all statistics.
//
// Work is one line, cut into equal shares of as many CTAs as the GPU holds (plan_line).  A CTA is four warps on
// one unit at a time: a row tile of 8 NQ queries of a kv head and a range of keys.  Every warp
// takes every fourth step of 32 keys, through a ring of its own in shared memory (cp.async, no barrier
// between warps), and the four results are joined at the end.  Results go to the workspace, and
// attn_quant_combine_kernel joins those of a row.
#include <limits.h>

#include <algorithm>

#include "quant.cuh"
#include "sm100_ptx.cuh"
#include "xp_device.cuh"

typedef __nv_bfloat16 bf16;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 32;             // keys of a warp's step
constexpr float kLazy = 8.0f;         // growth of the maximum (base 2) that weights may carry
constexpr float kLift = 6.0f;         // weights are 2^(z - m + kLift): at most 2^14
constexpr unsigned kAll = 0xFFFFFFFFu;

constexpr int kRound = kWarps * kStep;   // keys of a round of the four warps
constexpr int kUnitCost = 1;          // what a unit costs besides its keys, in rounds
constexpr int kMostResident = 5;      // CTAs an SM
constexpr int kMinChunk = 2;          // least work of a CTA, in rounds

struct Quant {
  int code, scale, scale_at;   // bytes of a token's codes and scales; where a head's scales begin
  bool q_wide;                 // queries by 16 bytes
  // 16 tokens from a multiple of 16 on lie side by side, as in the ring, and pages less than 2^32 bytes apart
  bool runs;
};

// The work is one line of cost: the prefix's units (kv head by kv head, row tile by row tile), then those
// of each sequence's tail.  A unit costs its rounds of keys and kUnitCost; CTA i does [i*chunk, (i+1)*chunk) of
// the line, so that every CTA gets the same whatever the lengths are.  A piece that begins its unit leaves
// its result in the unit's place, one that does not in its CTA's, of which there is at most one.
__host__ __device__ inline int rounds_of(int keys) { return (keys + kRound - 1) / kRound; }
__host__ __device__ inline int cost_of(int keys) { return keys > 0 ? rounds_of(keys) + kUnitCost : 0; }
// first round of a unit of T that lies behind a cost of x from its beginning
__device__ __forceinline__ int round_at(int64_t x, int T) {
  const int64_t y = x - kUnitCost;
  return y <= 0 ? 0 : y > T ? T : (int)y;
}
__device__ __forceinline__ int tail_len(const xp_attn_args& g, int n, bool tell) {
  int len = g.lens[n];
  if (len < 0 || len > g.a.max_len) {
    if (tell) atomicOr(g.err, XP_ERR_LENGTH);
    len = len < 0 ? 0 : g.a.max_len;
  }
  return len;
}
// what the prefix costs that is attended over here
__device__ __forceinline__ int64_t prefix_cost(const xp_attn_args& g) {
  return (int64_t)g.kv_heads * g.plan.prefix_tiles * cost_of(g.a.prefix_len);
}

struct Start {
  int64_t total[kWarps], base;   // where the sequence in which this CTA begins has its beginning
  int n;
};
// Sums the tails' costs over the CTA: the chunk (0 where the line ends before this CTA's share), and where
// the share begins.  CTA 0 leaves the chunk and every sequence's beginning for the kernel that joins.
__device__ __forceinline__ int64_t plan_line(const xp_attn_args& g, Start* s) {
  const int64_t before = prefix_cost(g);
  const int N = g.a.max_len > 0 ? g.a.N : 0, units = g.kv_heads * g.plan.tail_tiles;
  const int per = (N + kThreads - 1) / kThreads, n0 = min(N, (int)threadIdx.x * per), n1 = min(N, n0 + per);
  auto cost = [&](int n) { return (int64_t)units * cost_of(tail_len(g, n, blockIdx.x == 0)); };
  int64_t mine = 0;
  for (int n = n0; n < n1; ++n) mine += cost(n);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(kAll, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) s->total[warp] = inc;
  __syncthreads();
  int64_t base = before + inc - mine, all = before;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    base += w < warp ? s->total[w] : 0;
    all += s->total[w];
  }
  const int64_t chunk = max((int64_t)kMinChunk, (all + gridDim.x - 1) / gridDim.x), x = blockIdx.x * chunk;
  int64_t* line = (int64_t*)g.line;
  for (int n = n0; n < n1; ++n) {
    const int64_t c = per == 1 ? mine : cost(n);
    if (blockIdx.x == 0) line[1 + n] = base;
    if (x >= base && x < base + c) {
      s->n = n;
      s->base = base;
    }
    base += c;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) line[0] = chunk;
  __syncthreads();
  return x < all ? chunk : 0;
}

template <int BITS, int DP, int NQ> struct Cfg {
  static constexpr int CODE = DP * BITS / 8;              // bytes a token of the ring
  static constexpr int SCALE = DP / 16;
  static constexpr int STAGE = kStep * 2 * (CODE + SCALE);
  static constexpr int STAGES = STAGE > 8000 ? 2 : 3;
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int PITCH = DP + 4;                    // floats of a row of the joined results
  static constexpr int JOIN = kWarps * 8 * PITCH * 4;
  static constexpr int QUERIES = NQ == 4 ? NQ * (DP / 16) * 32 * 8 : 0;   // held in shared memory
  static constexpr int SMEM = (RING > JOIN ? RING : JOIN) + QUERIES;
  // CTAs an SM, which registers (results: 4 NQ KS a thread) and shared memory have room for: the line is cut into as
  // many pieces, which all run at once.  Heads of 128 in 8 bits: three with two stages and two with three,
  // contexts of 1000 to 32768 behind 1 token 116 and 123 us, behind 4 134 and 147 (in 4 bits, behind 4: three and two
  // 115 both).  Heads of 64 in 8 bits, 64 over 8: three 64 us, four 67, five with two stages 66; of 256, where one
  // fits, 150.
  static constexpr int RESIDENT = DP == 64    ? (NQ == 1 ? (BITS == 4 ? 5 : 3) : NQ == 2 ? 4 : 2)
                                  : DP == 128 ? (BITS == 4 ? (NQ == 1 ? 4 : 2) : NQ < 4 ? 3 : 2)
                                              : (BITS == 4 ? 2 : 1);
  // an SM's shared memory, of which every CTA takes 1 KB besides its own
  static constexpr int STATIC = sizeof(Start) + kWarps * 8 * NQ * 8;
  static_assert(RESIDENT * (SMEM + STATIC + 1024) <= 228 * 1024, "more CTAs than fit");
  // 4 bits: values are widened 2^-7 times as large (see widen4), queries are 2^7 times, to 512 (1/16 of them keeps
  // more than in 8 bits), so that a product is as large and its factor as far from fp32's ends
  static constexpr float UNIT = BITS == 4 ? 128.0f : 1.0f;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void copy_async(uint32_t to, const char* from, int bytes) {
  if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else if (bytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void wait_groups() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *(const uint32_t*)&v;
}
__device__ __forceinline__ __half2 h2(uint32_t v) { return *(const __half2*)&v; }
__device__ __forceinline__ uint32_t u32(__half2 v) { return *(const uint32_t*)&v; }
// two scales as fp16: the bytes lo and hi (by multiplies: what widens codes fills the logic pipe)
__device__ __forceinline__ __half2 scales(uint32_t lo, uint32_t hi) { return h2((hi * 65536u + lo) * 128u); }

// w & mask | magic in one instruction: of two constants one has to be in a register, and the compiler, where it
// sees both, takes two instructions (which cost long contexts 10% of their time)
__device__ __forceinline__ uint32_t pick(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(magic));
  return r;
}
__device__ __forceinline__ uint32_t in_register(uint32_t v) {
  asm volatile("" : "+r"(v));
  return v;
}

// Codes of 4 bits as they are held, c + 8 = 0..15, times a scale: pairs j = 0..3 of either half of w.
// 8 + c/128 and 8 + 16 c/128 are fp16 numbers with c in their last bits, so one multiply-add gives
// (8 + c/128) s - 8 s = c s / 128, exactly (8 s is finite, and c s down to the least scale is whole 2^-17).
// Odd pairs come 16 times too large: the queries' dims there are 1/16 of the others', and the results' are
// divided at the end.  What the 8 too much brings is one product more for every 16 keys: 8 sum_d s q_d for
// scores, 8 sum_j s p_j for results.
struct Scale4 {
  __half2 s, base;
};
__device__ __forceinline__ Scale4 scale4(__half2 s) { return {s, __hmul2(s, h2(0xC800C800u))}; }   // -8
__device__ __forceinline__ void widen4(uint32_t w, Scale4 f, uint32_t magic, uint32_t (&out)[4]) {   // 0x48004800
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    out[2 * i] = u32(__hfma2(h2(pick(w, 0x000F000Fu, magic)), f.s, f.base));
    out[2 * i + 1] = u32(__hfma2(h2(pick(w, 0x00F000F0u, magic)), f.s, f.base));
    w >>= 8;
  }
}
// one pair of codes of 8 bits: the low byte of either half of w
__device__ __forceinline__ uint32_t widen8(uint32_t w, __half2 s, uint32_t magic) {   // 0x64006400: 1024 + c + 128
  return u32(__hmul2(__hadd2(h2(pick(w, 0x00FF00FFu, magic)), h2(0xE480E480u)), s));   // -1152
}

// NW 32-bit words of shared memory, from a boundary of their size
template <int NW> __device__ __forceinline__ void load_words(const char* p, uint32_t (&w)[NW]) {
  if constexpr (NW == 1) {
    w[0] = *(const uint32_t*)p;
  } else if constexpr (NW == 2) {
    const uint2 v = *(const uint2*)p;
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < NW / 4; ++i) {
      const uint4 v = ((const uint4*)p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}

template <int BITS, int DP, int NQ>
__global__ void __launch_bounds__(kThreads, Cfg<BITS, DP, NQ>::RESIDENT)
    attn_quant_kernel(const __grid_constant__ xp_attn_args g, const Quant z) {
  using C = Cfg<BITS, DP, NQ>;
  constexpr int KS = DP / 16;             // k steps of the first product, row tiles of the second
  constexpr int KW = DP / 4 * BITS / 32;  // words of a lane's 1/4 of a key
  constexpr int VW = DP / 8 * BITS / 32;  // and of its 1/8 of a value
  constexpr int WPG = 16 * BITS / 32;     // words of 16 dims
  constexpr int KG = KS / 4;              // groups of 16 dims of a lane's 1/4 of a key
  constexpr int VG = DP <= 128 ? 1 : 2;   // and of its 1/8 of a value
  constexpr int KB = BITS == 4 ? (KG + 1) / 2 : 0;   // products for the 8 too much: of scores,
  constexpr bool VB = BITS == 4;                     // of results
  constexpr bool QREGS = NQ < 4;
  constexpr int KT = NQ * KS >= 32 ? 1 : 2;          // tiles of 16 keys at a time
  extern __shared__ __align__(16) char smem[];
  __shared__ float s_m[kWarps][8 * NQ], s_l[kWarps][8 * NQ];
  __shared__ Start s_start;

  const xp_attn_plan& pl = g.plan;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gr = lane >> 2, t4 = lane & 3;   // row group and place in it of a product's fragments
  const int per_seq = g.a.T * g.group, RT = 8 * NQ;
  const int64_t chunk = plan_line(g, &s_start);
  if (chunk == 0) return;
  const int64_t x0 = blockIdx.x * chunk, x1 = x0 + chunk, prefix_units = (int64_t)g.kv_heads * pl.prefix_tiles;

  // the unit in which this CTA's share begins: unit u of the prefix (n < 0) or of sequence n
  int n, keys, u;
  int64_t at;
  if (x0 < prefix_cost(g)) {
    n = -1, keys = g.a.prefix_len;
    u = (int)(x0 / cost_of(keys));
    at = (int64_t)u * cost_of(keys);
  } else {
    n = s_start.n, keys = tail_len(g, n, false);
    u = (int)((x0 - s_start.base) / cost_of(keys));
    at = s_start.base + (int64_t)u * cost_of(keys);
  }
  const uint32_t magic = in_register(BITS == 4 ? 0x48004800u : 0x64006400u);
  const int more = kRound / g.page_size, rest = kRound % g.page_size;   // a round further in a table

  while (true) {   // unit by unit; the same in every thread
  const bool prefix = n < 0;
  const int tiles = prefix ? pl.prefix_tiles : pl.tail_tiles, T = rounds_of(keys);
  const int r0 = round_at(x0 - at, T), r1 = round_at(min(x1 - at, (int64_t)cost_of(keys)), T);
  if (r0 < r1) {
  const int hk = u / tiles, tile = u % tiles;
  const int32_t* table = prefix ? g.prefix_table : g.table + n * g.ld_table;
  const int64_t slot = r0 > 0 ? pl.units + blockIdx.x
                       : prefix ? u
                                : prefix_units + (int64_t)n * g.kv_heads * pl.tail_tiles + u;
  const int k0 = r0 * kRound, k1 = min(keys, r1 * kRound);
  const int D = g.dim;
  auto row_at = [&](int r, int* rn, int* rt, int* rj) {   // false behind the end
    const int i = tile * RT + r;
    if (i >= (prefix ? g.a.N * per_seq : per_seq)) return false;
    *rn = prefix ? i / per_seq : n;
    *rt = i % per_seq / g.group;
    *rj = i % g.group;
    return true;
  };

  // The loads of a step.  A lane asks for the page of its key (where 16 tokens lie side by side: of the first key
  // of its half of the step) a step ahead, and looks at the answer when the loads are made.
  char* ring = smem + warp * (C::STAGES * C::STAGE);
  const uint32_t ring_at = ptx::smem_u32(ring);
  const int64_t head_at = hk * g.kv_head;
  const int in_run = z.runs ? lane & 15 : 0;
  int key = k0 + warp * kStep + lane - in_run, col = key / g.page_size, at_page = key - col * g.page_size;
  int page = 0, in_page = 0, left = 0;   // left: keys of the range from there on
  auto find = [&]() {   // the next step's
    left = k1 - key;
    if (left > 0) page = table[col];
    in_page = at_page;
    key += kRound;
    col += more;
    at_page += rest;
    if (at_page >= g.page_size) at_page -= g.page_size, ++col;
  };
  const char *k_head = (const char*)g.k + head_at, *v_head = (const char*)g.v + head_at;
  auto load = [&](int stage) {
    const uint32_t to = ring_at + stage * C::STAGE;
    if (left > 0 && (unsigned)page >= (unsigned)g.pages) {
      atomicOr(g.err, XP_ERR_BADPAGE);
      page = page < 0 ? 0 : g.pages - 1;
    }
    // a key behind the end: scales of 0, so that whatever codes the ring holds there are worth nothing
    const uint32_t ds = to + 2 * kStep * C::CODE + lane * C::SCALE;
    auto no_scale = [&]() {
#pragma unroll
      for (int p = 0; p < C::SCALE; p += 4) {
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(ds + p), "r"(0) : "memory");
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(ds + kStep * C::SCALE + p), "r"(0) : "memory");
      }
    };
    if (z.runs) {   // half a warp copies its half's 16 tokens, a lane 16 bytes
      const uint64_t page_at = (uint64_t)(unsigned)page * (unsigned)g.kv_page;
      const unsigned code_at = in_page * C::CODE + in_run * 16;
      const unsigned scale_at = z.scale_at + (in_page + in_run) * C::SCALE;
      const char *k = k_head + page_at, *v = v_head + page_at;
      if (left > 0) {
        const uint32_t d = to + (lane & 16) * C::CODE + in_run * 16;
#pragma unroll
        for (int i = 0; i < C::CODE / 16; ++i) {
          copy_async(d + i * 256, k + code_at + i * 256, 16);
          copy_async(d + kStep * C::CODE + i * 256, v + code_at + i * 256, 16);
        }
      }
      if (left > in_run) {
        copy_async(ds, k + scale_at, C::SCALE);
        copy_async(ds + kStep * C::SCALE, v + scale_at, C::SCALE);
      } else {
        no_scale();
      }
      return;
    }
    const int64_t page_at = page * g.kv_page, code_at = page_at + (int64_t)in_page * z.code;
    const uint32_t in = __ballot_sync(kAll, left > 0);
    auto codes = [&](auto piece_bytes) {
      constexpr int PB = decltype(piece_bytes)::value, PIECES = C::CODE / PB;   // of a token
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int piece = i * 32 + lane, of = piece / PIECES, p = piece % PIECES;
        const int64_t from = __shfl_sync(kAll, code_at, of) + p * PB;
        if ((in >> of & 1) && p * PB < z.code) {
          const uint32_t d = to + of * C::CODE + p * PB;
          copy_async(d, k_head + from, PB);
          copy_async(d + kStep * C::CODE, v_head + from, PB);
        }
      }
    };
    if (z.code % 16 == 0) codes(std::integral_constant<int, 16>());
    else codes(std::integral_constant<int, 8>());
    if (left > 0) {
      const int64_t scale_at = page_at + z.scale_at + (int64_t)in_page * z.scale;
#pragma unroll
      for (int p = 0; p < C::SCALE; p += 4)
        if (p < z.scale) {
          copy_async(ds + p, k_head + scale_at + p, 4);
          copy_async(ds + kStep * C::SCALE + p, v_head + scale_at + p, 4);
        }
    } else {
      no_scale();
    }
  };
  const int steps = k1 > k0 ? (k1 - k0 + kStep - 1) / kStep : 0;
  const int mine = steps > warp ? (steps - warp + kWarps - 1) / kWarps : 0;   // this warp's
  auto base_of = [&](int i) { return k0 + (warp + i * kWarps) * kStep; };
  int found = 0;
  if (mine > 0) find();
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) {
    if (i < mine) {
      load(i);
      if (++found < mine) find();
    }
    commit();
  }

  // Queries: lane (gr, t4) holds dims t4 DP/4.. of query gr of every column tile, as fp16 pairs
  uint32_t qr[QREGS ? NQ : 1][QREGS ? 2 * KS : 1];
  uint2* sq = (uint2*)(smem + (C::SMEM - C::QUERIES));
  uint32_t qb[NQ][KB > 0 ? 2 * KB : 1];   // -8 times the sums of groups of 16 dims, as two fp16 each
  float cz[NQ][2];       // of queries 2 t4 and 2 t4 + 1: score to base 2,
  int limit[NQ][2];      // keys it sees
  int least = k1;        // and the least of them
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    int rn, rt, rj;
    const bool is_row = row_at(q * 8 + gr, &rn, &rt, &rj);
    const bf16* src = is_row ? (const bf16*)g.q + rn * g.a.q_stride_n + rt * g.a.q_stride_t +
                                   (int64_t)(hk * g.group + rj) * g.a.q_stride_h
                             : nullptr;
    float x[DP / 4], top = 0.0f;
#pragma unroll
    for (int i = 0; i < DP / 4; i += 8) {
      const int d = t4 * (DP / 4) + i;
      if (is_row && d < D && z.q_wide) {
        const uint4 v = *(const uint4*)(src + d);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i + j] = __uint_as_float(j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i + j] = is_row && d < D ? __bfloat162float(src[d + j]) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[i + j]));
    }
    top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
    top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
    float up;
    const float down = C::UNIT * xpq::row_scale(top, &up);
#pragma unroll
    for (int i = 0; i < KS; ++i) {   // of a k step: dims 4 i.. of the lane's
      const uint32_t b0 = pack(x[4 * i] * down, x[4 * i + 1] * down);
      const float odd = BITS == 4 ? down * 0.0625f : down;
      const uint32_t b1 = pack(x[4 * i + 2] * odd, x[4 * i + 3] * odd);
      if constexpr (QREGS) qr[q][2 * i] = b0, qr[q][2 * i + 1] = b1;
      else if (warp == 0) sq[(q * KS + i) * 32 + lane] = make_uint2(b0, b1);
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) {   // k of the product: (group, group + 1) as fp16, then what that leaves
      float sum[2] = {0.0f, 0.0f};
#pragma unroll
      for (int e = 0; e < (KG > 1 ? 2 : 1); ++e)
#pragma unroll
        for (int j = 0; j < 16; ++j) sum[e] += x[(2 * i + e) * 16 + j] * down;
      const float h0 = -8.0f / C::UNIT * sum[0], h1 = -8.0f / C::UNIT * sum[1];
      const uint32_t hi = pack(h0, h1);
      qb[q][2 * i] = hi;
      qb[q][2 * i + 1] = pack(h0 - __low2float(h2(hi)), h1 - __high2float(h2(hi)));
    }
    const float c = xpq::row_factor(up, g.a.scale * 1.44269504088896f);
    const int lim = !is_row ? k1 : min(k1, prefix ? keys : keys - g.a.T + rt + 1);
    least = min(least, lim);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      cz[q][i] = __shfl_sync(kAll, c, (2 * t4 + i) * 4);
      limit[q][i] = __shfl_sync(kAll, lim, (2 * t4 + i) * 4);
    }
  }
  least = __reduce_min_sync(kAll, least);
  if constexpr (!QREGS) __syncthreads();

  float o[NQ][KS][4], ob[NQ][4], m[NQ][2], l[NQ][2];   // ob: sum_j s p_j of the lane's groups
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[q][i][e] = ob[q][e] = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) m[q][i] = -INFINITY, l[q][i] = 0.0f;
  }
  const int groups = D / 16;
  // the groups of a lane's key that there are, as bytes
  const int k_count = min(max(groups - t4 * KG, 0), KG);
  const uint32_t k_groups = k_count >= 4 ? 0xFFFFFFFFu : (1u << k_count * 8) - 1;

  for (int it = 0; it < mine; ++it) {
    wait_groups<C::STAGES - 2>();
    __syncwarp();   // every lane's copies are in, and every lane is done with the stage to be refilled
    if (it + C::STAGES - 1 < mine) {
      load((it + C::STAGES - 1) % C::STAGES);
      if (++found < mine) find();
    }
    commit();
    const char* st = ring + it % C::STAGES * C::STAGE;
    const char *sk = st, *sv = st + kStep * C::CODE;
    const uint8_t* ks = (const uint8_t*)st + 2 * kStep * C::CODE;
    const uint8_t* vs = ks + kStep * C::SCALE;
    const int kb = base_of(it);

    // 16 KT keys at a time: where the results of 32 queries fill the registers, half a step's scores fit beside them
#pragma unroll(KT == 2 ? 2 : 1)
    for (int kh = 0; kh < 2; kh += KT) {
    // S^T: 16 KT keys by 8 NQ queries
    float s[KT][NQ][4];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[kt][q][e] = 0.0f;
      uint32_t w[2][KW], bytes[2];   // scales of the lane's groups
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int key = (kh + kt) * 16 + r * 8 + gr;
        load_words<KW>(sk + key * C::CODE + t4 * (C::CODE / 4), w[r]);
        const uint8_t* from = ks + key * C::SCALE + t4 * KG;
        bytes[r] = (KG == 1 ? *from : KG == 2 ? *(const uint16_t*)from : *(const uint32_t*)from) & k_groups;
      }
      Scale4 sc4[2][KG];
      __half2 sc8[2][KG];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < KG; ++i) {
          sc8[r][i] = KG == 1 ? h2(bytes[r] * 0x00800080u)
                              : h2(__byte_perm(bytes[r], 0, 0x4040 + 0x0101 * i) * 128u);
          if constexpr (BITS == 4) sc4[r][i] = scale4(sc8[r][i]);
        }
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        uint32_t f[4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
          f[r] = f[2 + r] = __byte_perm(u32(sc4[r][2 * i].s), KG > 1 ? u32(sc4[r][KG > 1 ? 2 * i + 1 : 0].s) : 0, 0x5410);
#pragma unroll
        for (int q = 0; q < NQ; ++q) mma(s[kt][q], f, qb[q][2 * i], qb[q][2 * i + 1]);
      }
#pragma unroll
      for (int i = 0; i < KS; i += 2) {   // two k steps: 8 dims of the lane
        uint32_t a[2][4];                 // [row][pair]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (BITS == 4) {
            widen4(w[r][i / 2], sc4[r][i / 4], magic, a[r]);
          } else {
#pragma unroll
            for (int p = 0; p < 4; ++p)   // bytes 0, 1 or 2, 3 of a word, one in each half
              a[r][p] = widen8(__byte_perm(w[r][i + p / 2], 0, p % 2 ? 0x4342 : 0x4140), sc8[r][i / 4], magic);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t f[4] = {a[0][2 * h], a[1][2 * h], a[0][2 * h + 1], a[1][2 * h + 1]};
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if constexpr (QREGS) {
              mma(s[kt][q], f, qr[q][2 * (i + h)], qr[q][2 * (i + h) + 1]);
            } else {
              const uint2 b = sq[(q * KS + i + h) * 32 + lane];
              mma(s[kt][q], f, b.x, b.y);
            }
          }
        }
      }
    }

    // scores in base 2; element e of a tile: key gr + 8 (e / 2), query 2 t4 + e % 2
    bool grew = false;
    float top[NQ][2];
    if (kb + kStep > least) {   // some are hidden (never so but in the last steps)
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (kb + (kh + kt) * 16 + e / 2 * 8 + gr >= limit[q][e % 2]) s[kt][q][e] = -INFINITY;
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      top[q][0] = top[q][1] = -INFINITY;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[kt][q][e] *= cz[q][e % 2];   // positive, so -inf stays
          top[q][e % 2] = fmaxf(top[q][e % 2], s[kt][q][e]);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) grew |= top[q][i] > m[q][i] + kLazy;
    }
    if (__any_sync(kAll, grew)) {
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v = top[q][i];
#pragma unroll
          for (int x = 4; x < 32; x *= 2) v = fmaxf(v, __shfl_xor_sync(kAll, v, x));
          v = fmaxf(v, m[q][i]);
          const float f = v == m[q][i] ? 1.0f : ex2(m[q][i] - v);
          m[q][i] = v;
          l[q][i] *= f;
#pragma unroll
          for (int j = 0; j < KS; ++j) o[q][j][i] *= f, o[q][j][2 + i] *= f;
          if (VB) ob[q][i] *= f, ob[q][2 + i] *= f;
        }
    }
    uint32_t p[KT][NQ][2];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      float base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) base[i] = (m[q][i] == -INFINITY ? 0.0f : m[q][i]) - kLift;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = ex2(s[kt][q][e] - base[e % 2]);
          l[q][e % 2] += v[e];
        }
        p[kt][q][0] = transpose8(pack(v[0], v[1]));   // keys 2 t4, 2 t4 + 1 of query gr
        p[kt][q][1] = transpose8(pack(v[2], v[3]));   // and those 8 on
      }
    }

    // O^T: a lane's rows are dims 2 i and 2 i + 1 of its DP / 8, its keys 2 t4, 2 t4 + 1 and those 8 on
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      uint32_t w[4][VW];
      Scale4 sc4[2][VG];   // of a pair of keys
      __half2 sc8[2][VG];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        load_words<VW>(sv + ((kh + kt) * 16 + 2 * t4 + r / 2 * 8 + r % 2) * C::CODE + gr * (C::CODE / 8), w[r]);
#pragma unroll
      for (int i = 0; i < VG; ++i) {
        const int group = DP == 64 ? gr / 2 : DP == 128 ? gr : 2 * gr + i;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t* from = vs + ((kh + kt) * 16 + 2 * t4 + r * 8) * C::SCALE + group;
          sc8[r][i] = scales(group < groups ? from[0] : 0, group < groups ? from[C::SCALE] : 0);
          if constexpr (BITS == 4) sc4[r][i] = scale4(sc8[r][i]);
        }
      }
      if constexpr (VB) {   // rows: the lane's groups
        const uint32_t f[4] = {u32(sc4[0][0].s), VG > 1 ? u32(sc4[0][VG - 1].s) : 0, u32(sc4[1][0].s),
                               VG > 1 ? u32(sc4[1][VG - 1].s) : 0};
#pragma unroll
        for (int q = 0; q < NQ; ++q) mma(ob[q], f, p[kt][q][0], p[kt][q][1]);
      }
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const int gi = VG == 1 ? 0 : i / WPG;
        uint32_t a[2][8];   // [keys 2 t4.. or those 8 on][dim of the word]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (BITS == 4) {
            uint32_t even[4], odd[4];
            widen4(__byte_perm(w[2 * r][i], w[2 * r + 1][i], 0x5410), sc4[r][gi], magic, even);
            widen4(__byte_perm(w[2 * r][i], w[2 * r + 1][i], 0x7632), sc4[r][gi], magic, odd);
#pragma unroll
            for (int j = 0; j < 4; ++j) a[r][2 * j] = even[j], a[r][2 * j + 1] = odd[j];
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              a[r][j] = widen8(__byte_perm(w[2 * r][i], w[2 * r + 1][i], 0x0400 + 0x0101 * j), sc8[r][gi], magic);
          }
        }
#pragma unroll
        for (int j = 0; j < (BITS == 4 ? 4 : 2); ++j) {
          const uint32_t f[4] = {a[0][2 * j], a[0][2 * j + 1], a[1][2 * j], a[1][2 * j + 1]};
#pragma unroll
          for (int q = 0; q < NQ; ++q)
            mma(o[q][i * (BITS == 4 ? 4 : 2) + j], f, p[kt][q][0], p[kt][q][1]);
        }
      }
    }
    }
  }
  wait_groups<0>();

  // the four warps' results at a common maximum
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int x = 4; x < 32; x *= 2) l[q][i] += __shfl_xor_sync(kAll, l[q][i], x);
      if (gr == 0) {
        s_m[warp][q * 8 + 2 * t4 + i] = m[q][i];
        s_l[warp][q * 8 + 2 * t4 + i] = l[q][i];
      }
    }
  __syncthreads();   // the rings are read no more either
  float* join = (float*)smem;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = q * 8 + 2 * t4 + i;
      const float all = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
      const float f = m[q][i] == all ? 1.0f : ex2(m[q][i] - all);
      float* to = join + (warp * 8 + 2 * t4 + i) * C::PITCH + gr * (DP / 8);
      // 4 bits: row tiles in pairs, of which the second came 16 times too large; a lane's first and second
      // half have a group each where it has two
      const float even = C::UNIT * f, odd = BITS == 4 ? even * 0.0625f : even;
#pragma unroll
      for (int j = 0; j < KS; j += 2) {
        const float over = VB ? 8.0f * f * ob[q][VG > 1 && j >= KS / 2 ? 2 + i : i] : 0.0f;
        *(float4*)(to + 2 * j) = make_float4(o[q][j][i] * even - over, o[q][j][2 + i] * even - over,
                                             o[q][j + 1][i] * odd - over, o[q][j + 1][2 + i] * odd - over);
      }
    }
    __syncthreads();
    for (int u = threadIdx.x; u < 8 * (DP / 4); u += kThreads) {
      const int r = u / (DP / 4), d = u % (DP / 4) * 4;
      int rn, rt, rj;
      if (d >= D || !row_at(q * 8 + r, &rn, &rt, &rj)) continue;
      float all = s_m[0][q * 8 + r], sum = 0.0f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) all = fmaxf(all, s_m[w][q * 8 + r]);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = s_m[w][q * 8 + r];
        sum += s_l[w][q * 8 + r] * (mw == all ? 1.0f : ex2(mw - all));
        const float4 x = *(const float4*)(join + (w * 8 + r) * C::PITCH + d);
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
      }
      const int64_t row = slot * RT + q * 8 + r;
      if (d == 0) *(float2*)&g.stat[row * 2] = make_float2(all - kLift, sum);
      if (sum != 0.0f) *(float4*)&g.acc[row * D + d] = v;
    }
    __syncthreads();
  }
  }

  at += cost_of(keys);
  if (++u == g.kv_heads * tiles) {
    u = 0;
    const int N = g.a.max_len > 0 ? g.a.N : 0;
    do ++n;
    while (n < N && (keys = tail_len(g, n, false)) == 0);
    if (n >= N) return;
  }
  if (at >= x1) return;
  }
}

// L lanes a query row (32, or 16 for heads to 64): what tcgen05 left of its prefix, and the pieces of its prefix
// and of its tail (the unit's own and those of the CTAs at whose beginning it was cut), brought to a common maximum:
//   out = sum_p a_p O_p / sum_p a_p l_p,  a_p = 2^(m_p - m).
// A lane holds E dims.  Bound by the latency of what it asks for, so four pieces are asked for at once, and where
// there are few rows, which have many pieces, W warps share a row's.
template <int E, int L, int W>
__global__ void __launch_bounds__(256) attn_quant_combine_kernel(const __grid_constant__ xp_attn_args g) {
  ptx::pdl_wait();
  const int64_t rows = (int64_t)g.a.N * g.a.T * g.a.heads;
  const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / (L * W);
  if (row >= rows) return;
  const int lane = threadIdx.x % L, warp = W == 1 ? 0 : threadIdx.x / L, D = g.dim, RT = g.plan.rows_tile, per_seq = g.a.T * g.group;
  const int h = (int)(row % g.a.heads), t = (int)(row / g.a.heads % g.a.T);
  const int n = (int)(row / g.a.heads / g.a.T), hk = h / g.group, i = t * g.group + h % g.group;
  const int64_t* line = (const int64_t*)g.line;
  const int64_t chunk = line[0], begin = g.a.max_len > 0 ? line[1 + n] : 0;
  const bool dims = lane * E < D;
  const unsigned row_lanes = L == 32 ? kAll : 0xFFFFu << (threadIdx.x & 16);

  float o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int c = 0; c < E; ++c) o[c] = 0.0f;
  auto load = [&](const float* acc, float (&x)[E]) {
#pragma unroll
    for (int c = 0; c < E; c += 4) {
      const float4 v = __ldcg((const float4*)(acc + lane * E + c));
      x[c] = v.x, x[c + 1] = v.y, x[c + 2] = v.z, x[c + 3] = v.w;
    }
  };
  auto add = [&](float2 st, const float (&x)[E]) {   // a piece that has a visible key
    const float now = fmaxf(m, st.x), a = exp2f(m - now), b = exp2f(st.x - now);
    m = now;
    l = l * a + st.y * b;
#pragma unroll
    for (int c = 0; c < E; ++c) o[c] = o[c] * a + x[c] * b;
  };
  auto pieces = [&](int keys, int64_t at, int64_t unit, int r) {
    const int T = rounds_of(keys), cost = cost_of(keys);
    const int64_t c0 = at / chunk, c1 = (at + cost - 1) / chunk;
    for (int64_t first = c0 + warp; first <= c1; first += L * W) {   // a lane a CTA
      const int64_t c = first + lane * W;
      int64_t from = 0;
      float2 st = make_float2(0.0f, 0.0f);   // of no piece, and where no key was visible: acc may hold anything
      if (c <= c1) {
        const int r0 = round_at(c * chunk - at, T), r1 = round_at(min((c + 1) * chunk - at, (int64_t)cost), T);
        if (r0 < r1) {
          from = (r0 > 0 ? g.plan.units + c : unit) * RT + r;
          st = __ldcg((const float2*)g.stat + from);
        }
      }
      const int count = (int)min((int64_t)L, (c1 - first) / W + 1);
      for (int k = 0; k < count; k += 4) {
        float2 s[4];
        float x[4][E];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t f = __shfl_sync(row_lanes, from, min(k + j, L - 1), L);
          s[j] = make_float2(__shfl_sync(row_lanes, st.x, min(k + j, L - 1), L), __shfl_sync(row_lanes, st.y, min(k + j, L - 1), L));
          if (k + j >= count) s[j].y = 0.0f;
          if (dims && s[j].y != 0.0f) load(g.acc + f * D, x[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (s[j].y != 0.0f) add(s[j], x[j]);
      }
    }
  };
  if (g.part_stat && warp == 0) {
    const float2 st = __ldcg((const float2*)g.part_stat + row);
    float x[E];
    if (dims) load(g.part_acc + row * D, x);
    if (st.y != 0.0f) add(st, x);
  }
  const int units = g.kv_heads * g.plan.prefix_tiles;
  if (units > 0 && g.a.prefix_len > 0) {
    const int at_row = n * per_seq + i, u = hk * g.plan.prefix_tiles + at_row / RT;
    pieces(g.a.prefix_len, (int64_t)u * cost_of(g.a.prefix_len), u, at_row % RT);
  }
  if (g.a.max_len > 0) {
    const int keys = tail_len(g, n, false), u = hk * g.plan.tail_tiles + i / RT;
    if (keys > 0)
      pieces(keys, begin + (int64_t)u * cost_of(keys), units + (int64_t)n * g.kv_heads * g.plan.tail_tiles + u, i % RT);
  }
  if constexpr (W > 1) {   // the warps', in the first
    __shared__ float2 s_st[W];
    __shared__ float s_o[W][E][L];
    if (lane == 0) s_st[warp] = make_float2(m, l);
#pragma unroll
    for (int c = 0; c < E; ++c) s_o[warp][c][lane] = o[c];
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < W; ++w) {
      float x[E];
#pragma unroll
      for (int c = 0; c < E; ++c) x[c] = s_o[w][c][lane];
      if (s_st[w].y != 0.0f) add(s_st[w], x);
    }
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;   // NaN where a visible score is
  bf16* out = (bf16*)g.out + n * g.a.o_stride_n + t * g.a.o_stride_t + h * g.a.o_stride_h + lane * E;
  if (dims) {
    if ((uintptr_t)out % (2 * E) == 0) {
      uint32_t v[E / 2];
#pragma unroll
      for (int c = 0; c < E; c += 2) {
        const __nv_bfloat162 w = __floats2bfloat162_rn(o[c] * inv, o[c + 1] * inv);
        v[c / 2] = *(const uint32_t*)&w;
      }
      if constexpr (E == 4) *(uint2*)out = make_uint2(v[0], v[1]);
      else *(uint4*)out = make_uint4(v[0], v[1], v[E / 2 - 2], v[E / 2 - 1]);
    } else {
#pragma unroll
      for (int c = 0; c < E; ++c) out[c] = __float2bfloat16_rn(o[c] * inv);
    }
  }
  if (lane == 0 && g.lse) g.lse[row] = l != 0.0f ? (m + log2f(l)) * 0.693147180559945f : -INFINITY;
}

template <int BITS, int DP, int NQ>
cudaError_t launch(const xp_attn_args& g, const Quant& z, int sms, cudaStream_t s) {
  using C = Cfg<BITS, DP, NQ>;
  static unsigned long long allowed = 0;
  const cudaError_t e = xp_allow_smem((const void*)attn_quant_kernel<BITS, DP, NQ>, C::SMEM, &allowed);
  if (e != cudaSuccess) return e;
  static_assert(C::RESIDENT <= kMostResident, "places for pieces");
  attn_quant_kernel<BITS, DP, NQ><<<sms * C::RESIDENT, kThreads, C::SMEM, s>>>(g, z);
  return cudaGetLastError();
}
template <int BITS, int DP>
cudaError_t launch_rows(const xp_attn_args& g, const Quant& z, int sms, cudaStream_t s) {
  switch (g.plan.rows_tile) {
    case 8: return launch<BITS, DP, 1>(g, z, sms, s);
    case 16: return launch<BITS, DP, 2>(g, z, sms, s);
    default:
      if constexpr (DP <= 128) return launch<BITS, DP, 4>(g, z, sms, s);
      else return cudaErrorInvalidValue;
  }
}
template <int BITS> cudaError_t launch_dims(const xp_attn_args& g, const Quant& z, int sms, cudaStream_t s) {
  return g.dim <= 64 ? launch_rows<BITS, 64>(g, z, sms, s)
         : g.dim <= 128 ? launch_rows<BITS, 128>(g, z, sms, s)
                        : launch_rows<BITS, 256>(g, z, sms, s);
}

}  // namespace

// Many queries of each key are the tensor cores' work, not that of widening: from so many of a kv head on,
// what they see is widened to fp16 in the workspace once (exactly, as here) and attended over on tcgen05.
// 32 sequences of 1, 2, 4 tokens behind 8192, 8 kv heads of 4 x 128, widened and not: in 4 bits 128 rows 40 and
// 39 us, 256 rows 36 and 55, 512 rows 41 and 92; in 8 bits 40 and 41, 38 and 61, 42 and 104; heads of 64 in 4 bits
// 33 and 27, 29 and 35, 30 and 52, in 8 bits 33 and 28, 29 and 37, 30 and 56.  32 tails of 17 to 1500 tokens, rows
// of one: in 4 bits 16 take 52 and 33, 32 take 54 and 57, 64 take 59 and 95; in 8 bits 54 and 35, 56 and 58, 60 and
// 96; heads of 64 in 4 bits 38 and 18, 41 and 33, 44 and 54, in 8 bits 38 and 20, 41 and 37, 44 and 61.  Tails
// beside a widened prefix, which spare a kernel and a second joining: 32 rows 89 and 119 us, 16 rows 80 and 81 (128
// sequences: 223 and 173), 8 rows 117 and 79.
constexpr int kWidePrefixRows = 256, kWideTailRows = 64;
constexpr size_t kWideTailBytes = (size_t)1 << 30;   // of tails that may be widened

// The cache that the widened tokens are: heads outside, one layer.  False where its maps cannot be made.
static bool wide_cache(const xp_cache* c, const xp_attn_plan& p, int64_t pages, char* ws, xp_cache* w) {
  const int D = c->d.head_dim;
  *w = *c;
  w->d.dtype = XP_BF16;
  w->d.pages = (int)pages;
  w->d.page_size = kWidePage;
  w->d.layers = 1;
  w->d.stride_token = D;
  w->d.stride_page = (int64_t)kWidePage * D;
  w->d.stride_head = p.wide_plane;
  w->d.stride_layer = w->d.stride_head * c->d.kv_heads;
  w->d.k = ws + p.wide_k;
  w->d.v = ws + p.wide_v;
  w->heads_outside = true;
  w->attn_tc = xp_attn_tc_maps(w);
  return w->attn_tc != 0;
}
// the call that the tcgen05 form does: all of it, or the prefix alone
static xp_attn wide_call(const xp_attn& a, const xp_attn_plan& p) {
  xp_attn w = a;
  w.layer = 0;
  if (!p.tc) w.max_len = 0;
  return w;
}

// Row tiles of 8, 16 or 32 queries (heads wider than 128: 8 or 16, their results fill the registers): the
// least that hold a sequence's rows of one kv head, or where there is a prefix the batch's, or fewer in small
// calls.  Where the work is cut is found on the device, from the lengths.
xp_attn_plan xp_attn_quant_plan(const xp_cache* c, const xp_attn* a) {
  xp_attn_plan p = {};
  const int group = a->heads / c->d.kv_heads, per_seq = a->T * group, D = c->d.head_dim;
  auto pages = [](int keys) { return (keys + kWidePage - 1) / kWidePage; };
  const size_t page_bytes = (size_t)kWidePage * c->d.kv_heads * D * 4;
  const bool prefix = c->attn_tc && a->prefix_len > 0 && (int64_t)a->N * per_seq >= kWidePrefixRows;
  // Tails beside a widened prefix are widened too where they are no longer than it all together: a kernel of
  // their own and a second joining take 20 us.
  const size_t tail_pages = (size_t)a->N * pages(a->max_len);
  const bool tails = c->attn_tc && a->max_len > 0 && tail_pages * page_bytes <= kWideTailBytes &&
                     ((per_seq >= (prefix ? kWideTailRows / 2 : kWideTailRows) && (prefix || a->prefix_len == 0)) ||
                      (prefix && tail_pages <= 2 * (size_t)pages(a->prefix_len)));
  if (prefix || tails) {
    p.wide_prefix = prefix ? pages(a->prefix_len) : 0;
    p.wide_tail = tails ? pages(a->max_len) : 0;
    p.tc = (prefix || a->prefix_len == 0) && (tails || a->max_len == 0);
    const int64_t count = p.wide_prefix + (int64_t)a->N * p.wide_tail;
    p.wide_plane = count * kWidePage * D;
    size_t o = 0;
    auto take = [&](size_t bytes) { size_t at = o; o = (o + bytes + 255) / 256 * 256; return at; };
    p.wide_k = take(count * page_bytes / 2);
    p.wide_v = take(count * page_bytes / 2);
    p.wide_table = take(count * 4);
    p.wide_q = take((size_t)a->N * a->T * a->heads * D * 2);
    p.wide_factor = take((size_t)a->N * a->T * a->heads * 4);
    const xp_attn w = wide_call(*a, p);
    const xp_attn_plan tc = xp_attn_tc_plan(c, &w);
    if (tc.total && count < INT_MAX / kWidePage) {
      const size_t at = take(tc.total);
      p.wide_line = at + tc.line_off;
      p.wide_stat = at + tc.stat_off;
      p.wide_acc = at + tc.acc_off;
      p.total = o;
      if (p.tc) return p;
    } else {
      p = {};   // more work than the tcgen05 form's line can count
    }
  }

  // what is not widened
  const int prefix_len = p.wide_prefix ? 0 : a->prefix_len;
  const int64_t seen = (int64_t)per_seq * (prefix_len > 0 ? a->N : 1);
  p.rows_tile = seen <= 8 ? 8 : seen <= 16 || D > 128 ? 16 : 32;
  // Where that leaves less than a round for every CTA at once, fewer queries a tile are quicker: 4 single tokens
  // behind 512 keys 16.6 us in tiles of 16 and 14.5 of 8, 16 of them 23.9 in tiles of 32 and 18.6 of 8.
  auto line = [&](int rows) {
    return c->d.kv_heads * (((int64_t)a->N * per_seq + rows - 1) / rows * cost_of(prefix_len) +
                            (int64_t)a->N * ((per_seq + rows - 1) / rows) * cost_of(a->max_len));
  };
  while (p.rows_tile > 8 && line(p.rows_tile) < (int64_t)c->num_sms * 4) p.rows_tile /= 2;
  p.prefix_tiles = prefix_len > 0 ? (int)(((int64_t)a->N * per_seq + p.rows_tile - 1) / p.rows_tile) : 0;
  p.tail_tiles = (per_seq + p.rows_tile - 1) / p.rows_tile;
  const size_t H = c->d.kv_heads;
  p.units = H * p.prefix_tiles + (a->max_len > 0 ? (size_t)a->N * H * p.tail_tiles : 0);
  const size_t places = ((size_t)p.units + (size_t)c->num_sms * kMostResident) * p.rows_tile;
  size_t o = p.total;
  auto take = [&](size_t bytes) { size_t at = o; o = (o + bytes + 255) / 256 * 256; return at; };
  p.line_off = take(((size_t)a->N + 1) * 8);
  p.stat_off = take(places * 8);
  p.acc_off = take(places * D * 4);
  if (p.wide_prefix) {
    p.part_stat = take((size_t)a->N * a->T * a->heads * 8);
    p.part_acc = take((size_t)a->N * a->T * a->heads * D * 4);
  }
  p.total = o;
  return p;
}

cudaError_t xp_launch_attn_quant(const xp_cache* c, const xp_attn_args& g, cudaStream_t s) {
  const xp_attn_plan& p = g.plan;
  if (p.wide_prefix || p.wide_tail) {
    const int64_t count = p.wide_prefix + (int64_t)g.a.N * p.wide_tail;
    xp_cache wide;
    if (!wide_cache(c, p, count, g.ws, &wide)) return cudaErrorInvalidValue;
    int32_t* table = (int32_t*)(g.ws + p.wide_table);
    cudaError_t e = xp_launch_widen(c, g, p.wide_prefix, p.wide_tail, wide.d.k, wide.d.v, p.wide_plane, table,
                                    g.ws + p.wide_q, (float*)(g.ws + p.wide_factor), s);
    if (e != cudaSuccess) return e;
    xp_attn_args w = g;
    w.a = wide_call(g.a, p);
    w.q = g.ws + p.wide_q;
    w.q_factor = (float*)(g.ws + p.wide_factor);
    w.a.q_stride_h = g.dim;
    w.a.q_stride_t = (int64_t)g.a.heads * g.dim;
    w.a.q_stride_n = g.a.T * w.a.q_stride_t;
    w.page_size = kWidePage;
    w.pages = (int)count;
    w.k = wide.d.k;
    w.v = wide.d.v;
    w.kv_page = wide.d.stride_page;
    w.kv_token = wide.d.stride_token;
    w.kv_head = wide.d.stride_head;
    w.prefix_table = table;
    w.table = table + p.wide_prefix;
    w.ld_table = p.wide_tail;
    w.plan = xp_attn_tc_plan(c, &w.a);
    w.line = (int*)(g.ws + p.wide_line);
    w.stat = (float*)(g.ws + p.wide_stat);
    w.acc = (float*)(g.ws + p.wide_acc);
    if (!p.tc) {
      w.part_stat = (float*)(g.ws + p.part_stat);
      w.part_acc = (float*)(g.ws + p.part_acc);
    }
    e = xp_launch_attn_tc(&wide, w, s);
    if (e != cudaSuccess || p.tc) return e;
  }
  xp_attn_args q = g;
  if (p.wide_prefix) {
    q.part_stat = (float*)(g.ws + p.part_stat);
    q.part_acc = (float*)(g.ws + p.part_acc);
  }
  const xp_quant_sizes size = xp_quant_of(c->d.page_size, c->d.head_dim, c->d.dtype);
  const int64_t strides = (g.a.N > 1 ? g.a.q_stride_n : 0) | (g.a.T > 1 ? g.a.q_stride_t : 0) |
                          (g.a.heads > 1 ? g.a.q_stride_h : 0);
  const int D = c->d.head_dim;
  const Quant z = {size.code, size.scale, c->d.page_size * size.code, (uintptr_t)g.q % 16 == 0 && strides % 8 == 0,
                   c->d.page_size % 16 == 0 && (D == 64 || D == 128 || D == 256) &&
                       c->d.stride_page <= UINT_MAX};
  const cudaError_t e = c->d.dtype == XP_Q8 ? launch_dims<8>(q, z, c->num_sms, s) : launch_dims<4>(q, z, c->num_sms, s);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)g.a.N * g.a.T * g.a.heads;
  if (rows <= c->num_sms * 4)
    return xp_launch_pdl(D <= 128 ? attn_quant_combine_kernel<4, 32, 8> : attn_quant_combine_kernel<8, 32, 8>,
                         dim3((unsigned)rows), dim3(256), 0, s, q);
  return xp_launch_pdl(D <= 64    ? attn_quant_combine_kernel<4, 16, 1>
                       : D <= 128 ? attn_quant_combine_kernel<4, 32, 1>
                                  : attn_quant_combine_kernel<8, 32, 1>,
                       dim3((unsigned)((rows * (D <= 64 ? 16 : 32) + 255) / 256)), dim3(256), 0, s, q);
}
