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
// A value held is exact in fp16 (quant.cuh).  Queries are bf16, scaled by a power of two a row so that
// their largest is in [1, 4): exact but for what lies 2^-14 and more below it, which loses less than 2^-25 of the
// largest.  Weights are 2^(z - m + 6), rounded to fp16 (2^-12 of each, and 2^-31 of the largest where that
// is more): as the second product's operand they have to be 16 bits, and fp16 leaves an eighth of
// bf16's error.  Sums are taken before that rounding, in fp32, as are all statistics.
//
// A CTA is four warps on one unit: a row tile of 8 NQ queries of a kv head and a range of keys.  Every warp
// takes every fourth step of 32 keys, through a ring of its own in shared memory (cp.async, no barrier
// between warps), and the four results are joined at the end.  A unit's result goes to the workspace, and
// attn_combine_kernel joins the units of a row; where a row has one unit it is written out at once.
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

struct Quant {
  int code, scale, scale_at;   // bytes of a token's codes and scales; where a head's scales begin
};

template <int BITS, int DP, int NQ> struct Cfg {
  static constexpr int CODE = DP * BITS / 8;              // bytes a token of the ring
  static constexpr int SCALE = DP / 16;
  static constexpr int STAGE = kStep * 2 * (CODE + SCALE);
  static constexpr int STAGES = STAGE > 9000 ? 2 : 3;
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int PITCH = DP + 4;                    // floats of a row of the joined results
  static constexpr int JOIN = kWarps * 8 * PITCH * 4;
  static constexpr int QUERIES = NQ == 4 ? NQ * (DP / 16) * 32 * 8 : 0;   // held in shared memory
  static constexpr int SMEM = (RING > JOIN ? RING : JOIN) + QUERIES;
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
// two scales as fp16: the bytes lo and hi
__device__ __forceinline__ __half2 scales(uint32_t lo, uint32_t hi) { return h2(lo << 7 | hi << 23); }

// Four pairs of codes of 4 bits: bits 4j.. of either half of w, times s.  1024 + c and 1024 + 16 c are fp16
// numbers with c in their last bits.
__device__ __forceinline__ void widen4(uint32_t w, __half2 s, uint32_t (&out)[4]) {
  const __half2 sixteenth = h2(0x2C002C00u), low = h2(0xE408E408u), high = h2(0xD480D480u);   // 1/16, -1032, -72
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 a = h2((w & 0x000F000Fu) | 0x64006400u), b = h2((w & 0x00F000F0u) | 0x64006400u);
    out[2 * i] = u32(__hmul2(__hadd2(a, low), s));
    out[2 * i + 1] = u32(__hmul2(__hfma2(b, sixteenth, high), s));
    w >>= 8;
  }
}
// one pair of codes of 8 bits: the low byte of either half of w
__device__ __forceinline__ uint32_t widen8(uint32_t w, __half2 s) {
  return u32(__hmul2(__hadd2(h2((w & 0x00FF00FFu) | 0x64006400u), h2(0xE480E480u)), s));   // -1152
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
__global__ void __launch_bounds__(kThreads) attn_quant_kernel(const __grid_constant__ xp_attn_args g,
                                                              const Quant z) {
  using C = Cfg<BITS, DP, NQ>;
  constexpr int KS = DP / 16;             // k steps of the first product, row tiles of the second
  constexpr int KW = DP / 4 * BITS / 32;  // words of a lane's 1/4 of a key
  constexpr int VW = DP / 8 * BITS / 32;  // and of its 1/8 of a value
  constexpr int WPG = 16 * BITS / 32;     // words of 16 dims
  constexpr bool QREGS = NQ < 4;
  extern __shared__ __align__(16) char smem[];
  __shared__ float s_m[kWarps][8 * NQ], s_l[kWarps][8 * NQ];

  const xp_attn_plan& pl = g.plan;
  const int hk = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gr = lane >> 2, t4 = lane & 3;   // row group and place in it of a product's fragments
  const int per_seq = g.a.T * g.group, RT = 8 * NQ;
  int unit = blockIdx.x;
  const bool prefix = unit < pl.prefix_tiles * pl.prefix_splits;
  int tile, split, n = 0, part, keys;
  const int32_t* table = g.prefix_table;
  if (prefix) {
    tile = unit / pl.prefix_splits;
    split = unit % pl.prefix_splits;
    part = split;
    keys = g.a.prefix_len;
  } else {
    unit -= pl.prefix_tiles * pl.prefix_splits;
    split = unit % pl.tail_splits;
    tile = unit / pl.tail_splits % pl.tail_tiles;
    n = unit / pl.tail_splits / pl.tail_tiles;
    part = pl.prefix_splits + split;
    table = g.table + n * g.ld_table;
    keys = g.lens[n];
    if (keys < 0 || keys > g.a.max_len) {
      if (threadIdx.x == 0) atomicOr(g.err, XP_ERR_LENGTH);
      keys = keys < 0 ? 0 : g.a.max_len;
    }
  }
  const int range = prefix ? pl.prefix_keys : pl.tail_keys;
  const int k0 = split * range, k1 = k0 + min(range, keys - k0);   // none where keys < k0

  const int D = g.dim;
  auto row_at = [&](int r, int* rn, int* rt, int* rj) {   // false behind the end
    const int i = tile * RT + r;
    if (i >= (prefix ? g.a.N * per_seq : per_seq)) return false;
    *rn = prefix ? i / per_seq : n;
    *rt = i % per_seq / g.group;
    *rj = i % g.group;
    return true;
  };

  // The loads of a step.  A lane finds the place of the key that it is for, a step ahead.
  char* ring = smem + warp * (C::STAGES * C::STAGE);
  const uint32_t ring_at = ptx::smem_u32(ring);
  int64_t key_at = 0;   // of this lane's key in the step to be loaded: its codes,
  int scale_at = 0;     // and its scales from there
  bool key_in = false;
  auto find = [&](int kb) {
    const int key = kb + lane;
    key_in = key < k1;
    if (!key_in) return;
    const int col = key / g.page_size, at = key - col * g.page_size;
    int p = table[col];
    if (p < 0 || p >= g.pages) {
      atomicOr(g.err, XP_ERR_BADPAGE);
      p = p < 0 ? 0 : g.pages - 1;
    }
    key_at = p * g.kv_page + hk * g.kv_head + (int64_t)at * z.code;
    scale_at = z.scale_at + at * (z.scale - z.code);
  };
  auto load = [&](int stage) {
    const uint32_t to = ring_at + stage * C::STAGE;
    const uint32_t in = __ballot_sync(kAll, key_in);
    auto codes = [&](auto piece_bytes) {
      constexpr int PB = decltype(piece_bytes)::value, PIECES = C::CODE / PB;   // of a token
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int at = i * 32 + lane, key = at / PIECES, p = at % PIECES;
        const int64_t from = __shfl_sync(kAll, key_at, key) + p * PB;
        if ((in >> key & 1) && p * PB < z.code) {
          const uint32_t d = to + key * C::CODE + p * PB;
          copy_async(d, (const char*)g.k + from, PB);
          copy_async(d + kStep * C::CODE, (const char*)g.v + from, PB);
        }
      }
    };
    if (z.code % 16 == 0) codes(std::integral_constant<int, 16>());
    else codes(std::integral_constant<int, 8>());
    // a key behind the end: scales of 0, so that whatever codes the ring holds there are worth nothing
    const uint32_t d = to + 2 * kStep * C::CODE + lane * C::SCALE, dv = d + kStep * C::SCALE;
    if (key_in) {
      const char *k = (const char*)g.k + key_at + scale_at, *v = (const char*)g.v + key_at + scale_at;
      if (C::SCALE >= 8 && z.scale % 8 == 0) {
#pragma unroll
        for (int p = 0; p < C::SCALE; p += 8)
          if (p < z.scale) {
            copy_async(d + p, k + p, 8);
            copy_async(dv + p, v + p, 8);
          }
      } else {
#pragma unroll
        for (int p = 0; p < C::SCALE; p += 4)
          if (p < z.scale) {
            copy_async(d + p, k + p, 4);
            copy_async(dv + p, v + p, 4);
          }
      }
    } else {
#pragma unroll
      for (int p = 0; p < C::SCALE; p += 4) {
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(d + p), "r"(0) : "memory");
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(dv + p), "r"(0) : "memory");
      }
    }
  };
  const int steps = k1 > k0 ? (k1 - k0 + kStep - 1) / kStep : 0;
  const int mine = steps > warp ? (steps - warp + kWarps - 1) / kWarps : 0;   // this warp's
  auto base_of = [&](int i) { return k0 + (warp + i * kWarps) * kStep; };
  int found = 0;
  if (mine > 0) find(base_of(0));
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) {
    if (i < mine) {
      load(i);
      if (++found < mine) find(base_of(found));
    }
    commit();
  }

  // Queries: lane (gr, t4) holds dims t4 DP/4.. of query gr of every column tile, as fp16 pairs
  uint32_t qr[QREGS ? NQ : 1][QREGS ? 2 * KS : 1];
  uint2* sq = (uint2*)(smem + (C::SMEM - C::QUERIES));
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
    for (int i = 0; i < DP / 4; ++i) {
      const int d = t4 * (DP / 4) + i;
      x[i] = is_row && d < D ? __bfloat162float(src[d]) : 0.0f;
      top = fmaxf(top, fabsf(x[i]));
    }
    top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
    top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
    float up;
    const float down = xpq::row_scale(top, &up);
#pragma unroll
    for (int i = 0; i < KS; ++i) {   // of a k step: dims 4 i.. of the lane's
      const uint32_t b0 = pack(x[4 * i] * down, x[4 * i + 1] * down);
      const uint32_t b1 = pack(x[4 * i + 2] * down, x[4 * i + 3] * down);
      if constexpr (QREGS) qr[q][2 * i] = b0, qr[q][2 * i + 1] = b1;
      else if (warp == 0) sq[(q * KS + i) * 32 + lane] = make_uint2(b0, b1);
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

  float o[NQ][KS][4], m[NQ][2], l[NQ][2];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[q][i][e] = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) m[q][i] = -INFINITY, l[q][i] = 0.0f;
  }
  const int groups = D / 16;

  for (int it = 0; it < mine; ++it) {
    wait_groups<C::STAGES - 2>();
    __syncwarp();   // every lane's copies are in, and every lane is done with the stage to be refilled
    if (it + C::STAGES - 1 < mine) {
      load((it + C::STAGES - 1) % C::STAGES);
      if (++found < mine) find(base_of(found));
    }
    commit();
    const char* st = ring + it % C::STAGES * C::STAGE;
    const char *sk = st, *sv = st + kStep * C::CODE;
    const uint8_t* ks = (const uint8_t*)st + 2 * kStep * C::CODE;
    const uint8_t* vs = ks + kStep * C::SCALE;
    const int kb = base_of(it);

    // S^T: 32 keys by 8 NQ queries
    float s[2][NQ][4];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[kt][q][e] = 0.0f;
      uint32_t w[2][KW];
      __half2 sc[2][KS / 4];   // scales of the lane's KS/4 groups
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int key = kt * 16 + r * 8 + gr;
        load_words<KW>(sk + key * C::CODE + t4 * (C::CODE / 4), w[r]);
#pragma unroll
        for (int i = 0; i < KS / 4; ++i) {
          const int group = t4 * (KS / 4) + i;
          const uint32_t b = group < groups ? ks[key * C::SCALE + group] : 0;
          sc[r][i] = scales(b, b);
        }
      }
#pragma unroll
      for (int i = 0; i < KS; i += 2) {   // two k steps: 8 dims of the lane
        uint32_t a[2][4];                 // [row][pair]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (BITS == 4) {
            widen4(w[r][i / 2], sc[r][i / 4], a[r]);
          } else {
#pragma unroll
            for (int p = 0; p < 4; ++p)   // bytes 0, 1 or 2, 3 of a word, one in each half
              a[r][p] = widen8(__byte_perm(w[r][i + p / 2], 0, p % 2 ? 0x4342 : 0x4140), sc[r][i / 4]);
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
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      top[q][0] = top[q][1] = -INFINITY;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s[kt][q][e] * cz[q][e % 2];
          if (kb + kStep > least && kb + kt * 16 + e / 2 * 8 + gr >= limit[q][e % 2]) v = -INFINITY;
          s[kt][q][e] = v;
          top[q][e % 2] = fmaxf(top[q][e % 2], v);
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
        }
    }
    uint32_t p[2][NQ][2];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      float base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) base[i] = (m[q][i] == -INFINITY ? 0.0f : m[q][i]) - kLift;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
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
    for (int kt = 0; kt < 2; ++kt) {
      uint32_t w[4][VW];
      __half2 sc[2][DP <= 128 ? 1 : 2];   // scales of a pair of keys
#pragma unroll
      for (int r = 0; r < 4; ++r)
        load_words<VW>(sv + (kt * 16 + 2 * t4 + r / 2 * 8 + r % 2) * C::CODE + gr * (C::CODE / 8), w[r]);
#pragma unroll
      for (int i = 0; i < (DP <= 128 ? 1 : 2); ++i) {
        const int group = DP == 64 ? gr / 2 : DP == 128 ? gr : 2 * gr + i;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t* at = vs + (kt * 16 + 2 * t4 + r * 8) * C::SCALE + group;
          sc[r][i] = scales(group < groups ? at[0] : 0, group < groups ? at[C::SCALE] : 0);
        }
      }
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const int gi = DP <= 128 ? 0 : i / WPG;
        uint32_t a[2][8];   // [keys 2 t4.. or those 8 on][dim of the word]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (BITS == 4) {
            uint32_t even[4], odd[4];
            widen4(__byte_perm(w[2 * r][i], w[2 * r + 1][i], 0x5410), sc[r][gi], even);
            widen4(__byte_perm(w[2 * r][i], w[2 * r + 1][i], 0x7632), sc[r][gi], odd);
#pragma unroll
            for (int j = 0; j < 4; ++j) a[r][2 * j] = even[j], a[r][2 * j + 1] = odd[j];
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              a[r][j] = widen8(__byte_perm(w[2 * r][i], w[2 * r + 1][i], 0x0400 + 0x0101 * j), sc[r][gi]);
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
  const int64_t rows = (int64_t)g.a.N * g.a.T * g.a.heads;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = q * 8 + 2 * t4 + i;
      const float all = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
      const float f = m[q][i] == all ? 1.0f : ex2(m[q][i] - all);
      float* to = join + (warp * 8 + 2 * t4 + i) * C::PITCH + gr * (DP / 8);
#pragma unroll
      for (int j = 0; j < KS; j += 2)
        *(float4*)(to + 2 * j) = make_float4(o[q][j][i] * f, o[q][j][2 + i] * f, o[q][j + 1][i] * f,
                                             o[q][j + 1][2 + i] * f);
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
      const int h = hk * g.group + rj;
      const int64_t row = ((int64_t)rn * g.a.T + rt) * g.a.heads + h;
      if (pl.parts == 1) {
        const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;   // NaN where a visible score is
        bf16* out = (bf16*)g.out + rn * g.a.o_stride_n + rt * g.a.o_stride_t + h * g.a.o_stride_h + d;
        out[0] = __float2bfloat16_rn(v.x * inv), out[1] = __float2bfloat16_rn(v.y * inv);
        out[2] = __float2bfloat16_rn(v.z * inv), out[3] = __float2bfloat16_rn(v.w * inv);
        if (d == 0 && g.lse)
          g.lse[row] = sum != 0.0f ? (all - kLift + log2f(sum)) * 0.693147180559945f : -INFINITY;
      } else {
        if (d == 0) *(float2*)&g.stat[(part * rows + row) * 2] = make_float2(all - kLift, sum);
        if (sum != 0.0f) *(float4*)&g.acc[(part * rows + row) * D + d] = v;
      }
    }
    __syncthreads();
  }
}

template <int BITS, int DP, int NQ>
cudaError_t launch(const xp_attn_args& g, const Quant& z, cudaStream_t s) {
  using C = Cfg<BITS, DP, NQ>;
  static unsigned long long allowed = 0;
  const cudaError_t e = xp_allow_smem((const void*)attn_quant_kernel<BITS, DP, NQ>, C::SMEM, &allowed);
  if (e != cudaSuccess) return e;
  const xp_attn_plan& p = g.plan;
  const dim3 grid(p.prefix_tiles * p.prefix_splits + g.a.N * p.tail_tiles * p.tail_splits, g.kv_heads);
  attn_quant_kernel<BITS, DP, NQ><<<grid, kThreads, C::SMEM, s>>>(g, z);
  return cudaGetLastError();
}
template <int BITS, int DP>
cudaError_t launch_rows(const xp_attn_args& g, const Quant& z, cudaStream_t s) {
  switch (g.plan.rows_tile) {
    case 8: return launch<BITS, DP, 1>(g, z, s);
    case 16: return launch<BITS, DP, 2>(g, z, s);
    default:
      if constexpr (DP <= 128) return launch<BITS, DP, 4>(g, z, s);
      else return cudaErrorInvalidValue;
  }
}
template <int BITS> cudaError_t launch_dims(const xp_attn_args& g, const Quant& z, cudaStream_t s) {
  return g.dim <= 64 ? launch_rows<BITS, 64>(g, z, s)
         : g.dim <= 128 ? launch_rows<BITS, 128>(g, z, s)
                        : launch_rows<BITS, 256>(g, z, s);
}

}  // namespace

// Many queries of each key are the tensor cores' work, not that of widening: from so many of a kv head on,
// what they see is widened to fp16 in the workspace once (exactly, as here) and attended over on tcgen05.
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
// least that hold a sequence's rows of one kv head, or where there is a prefix the batch's.  Key ranges of
// whole rounds of the four warps, so that the units fill the GPU about four times over.
xp_attn_plan xp_attn_quant_plan(const xp_cache* c, const xp_attn* a) {
  xp_attn_plan p = {};
  const int group = a->heads / c->d.kv_heads, per_seq = a->T * group, D = c->d.head_dim;
  auto pages = [](int keys) { return (keys + kWidePage - 1) / kWidePage; };
  const size_t page_bytes = (size_t)kWidePage * c->d.kv_heads * D * 4;
  const bool prefix = c->attn_tc && a->prefix_len > 0 && (int64_t)a->N * per_seq >= kWidePrefixRows;
  const bool tails = c->attn_tc && a->max_len > 0 && per_seq >= kWideTailRows &&
                     (prefix || a->prefix_len == 0) &&
                     (size_t)a->N * pages(a->max_len) * page_bytes <= kWideTailBytes;
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
  const int round = kWarps * kStep;
  p.prefix_tiles = p.wide_prefix ? 0 : (int)(((int64_t)a->N * per_seq + p.rows_tile - 1) / p.rows_tile);
  p.tail_tiles = (per_seq + p.rows_tile - 1) / p.rows_tile;
  auto rounds = [&](int keys) { return ((int64_t)keys + round - 1) / round; };
  const int64_t all = (p.prefix_tiles * rounds(prefix_len) +
                       (int64_t)a->N * p.tail_tiles * rounds(a->max_len)) * c->d.kv_heads;
  const int64_t want = (int64_t)c->num_sms * 16, each = std::max<int64_t>(1, (all + want - 1) / want);
  auto splits = [&](int keys, int* range) {
    *range = (int)(std::min<int64_t>(each, std::max<int64_t>(1, rounds(keys))) * round);
    return keys > 0 ? (keys - 1) / *range + 1 : 0;
  };
  p.prefix_splits = p.wide_prefix ? 1 : splits(prefix_len, &p.prefix_keys);   // 1: what tcgen05 leaves
  p.tail_splits = splits(a->max_len, &p.tail_keys);
  p.parts = p.prefix_splits + p.tail_splits;
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
    if (!p.tc) w.part_stat = g.stat, w.part_acc = g.acc;   // the first range
    e = xp_launch_attn_tc(&wide, w, s);
    if (e != cudaSuccess || p.tc) return e;
  }
  const xp_quant_sizes q = xp_quant_of(c->d.page_size, c->d.head_dim, c->d.dtype);
  const Quant z = {q.code, q.scale, c->d.page_size * q.code};
  cudaError_t e = cudaSuccess;
  if (p.parts > (p.wide_prefix ? 1 : 0)) e = c->d.dtype == XP_Q8 ? launch_dims<8>(g, z, s) : launch_dims<4>(g, z, s);
  // a row of one range is written out by that kernel
  return e == cudaSuccess && p.parts != 1 ? xp_launch_attn_combine(g, s) : e;
}
