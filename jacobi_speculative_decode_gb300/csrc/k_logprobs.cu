// Log probabilities of given tokens, the entropy, the token's rank and the best alternatives: one pass
// over the row.
//
// A row, or a part of one, is a CTA's.  Every thread keeps a base m, near its running maximum, S = sum 2^((l - m) c)
// and W = sum (l - m) c 2^((l - m) c), c = log2(e) / t; then, all joined at the row's maximum,
//   log p(x) = (l_x - m) / t - log S,   H = log S - log(2) W / S.
// Differences are taken before they are scaled, so that neither large logits nor small temperatures lose
// digits.
// Bound by the row's bytes in fp32: 2048 rows of 151647, 1.24 GB, 199 to 202 us, 6.2 TB/s, 91% of measured.  In bf16 by
// instructions: 2048 rows of 151647, 621 MB, 117 us, 78%.  One CTA
// a row leaves few rows to as many CTAs: 410 rows (125 MB) with 20 alternatives 39 us, with none 31.
// The best ids.  On the way a thread only writes down the greatest of every batch of four 16-byte vectors.  The `top`-th of the
// 256 threads' greatest is a bound: there are `top` elements that are not below it, and few that are above.
// The batches that reach it are read again (from L2, some 25 of a row's, by the threads they are of, all at once:
// warp by warp 42 us, not 39), their elements that do go to a buffer,
// and an element of the buffer counts those before it and so knows its place.  Where the buffer overflows, as
// for a row of equal logits, every warp reads its part of the row again into a sorted list.
// (Looked at on the way, under a bound that follows, the same rows took 62 us where 44 are taken without.)
#include <float.h>
#include <math.h>

#include <algorithm>

#include "xp_device.cuh"

using namespace xpd;
typedef __nv_bfloat16 bf16;
typedef unsigned long long u64;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLoads = 4;             // 16-byte vectors of a thread in flight
constexpr int kResident = 4;          // CTAs an SM
constexpr int kMostParts = 10;        // of a row
constexpr int kCand = 1024;           // places of the buffer
static_assert(kMostParts * 32 <= kCand, "the parts of a row leave what the buffer holds");
constexpr int kBatches = 64;          // of which the greatest is held; all behind them share the last place
constexpr int kLeastVectors = kThreads * kLoads;   // of a part of a row
constexpr float kLazy = 8.0f;         // how far (base 2) a logit may lie above the base of its thread's sums
constexpr float kLog2e = 1.44269504088896f;
constexpr unsigned kAll = 0xFFFFFFFFu;

struct Args {
  const void* logits;
  int64_t sn, sb;
  const int64_t* tokens;
  const float* temperature;
  int B, V, top, parts, rows;   // rows: 0 where they are taken as they come
  float *logprob, *entropy;
  int32_t* rank;
  int64_t* top_ids;
  float* top_logprobs;
  uint32_t* err;
  unsigned* tickets;     // a row's finished parts; zero between calls
  float4* stat;          // (m, S, W, ids ahead) of a part
  u64* best;             // its list
};

struct Stat {
  float m, s, w;   // m: -FLT_MAX at least
  int ahead;
};
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 operations an instruction
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// the sums of a at a maximum m that is not below its own
__device__ __forceinline__ void rebase(Stat& a, float m, float c) {
  if (a.s > 0.0f) {
    const float d = (a.m - m) * c, f = ex2(d);
    a.w = f > 0.0f ? (a.w + d * a.s) * f : 0.0f;
    a.s *= f;
  }
  a.m = m;
}
__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
  const float m = fmaxf(a.m, b.m);
  rebase(a, m, c);
  rebase(b, m, c);
  return {m, a.s + b.s, a.w + b.w, a.ahead + b.ahead};
}

// 16 bytes of logits.  W: what greatest values and counts are kept in, two halves of bf16 or one float.
template <typename T> struct Vec;
template <> struct Vec<bf16> {
  static constexpr int N = 8;
  static constexpr float kLeast = -3.38953139e38f;   // the least finite value
  typedef __nv_bfloat162 W;
  static __device__ __forceinline__ W word(const uint4& x, int i) {
    const uint32_t w = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
    return *(const W*)&w;
  }
  static __device__ __forceinline__ W all(float v) { return __float2bfloat162_rn(v); }
  static __device__ __forceinline__ W join(W a, W b) { return __hmax2(a, b); }   // NaN left out
  static __device__ __forceinline__ W top(const uint4& x) {
    return join(join(word(x, 0), word(x, 1)), join(word(x, 2), word(x, 3)));
  }
  static __device__ __forceinline__ float most(W a) { return fmaxf(__low2float(a), __high2float(a)); }
  // a value of the type that is not above v
  static __device__ __forceinline__ float round_down(float v) {
    return __bfloat162float(__float2bfloat16_rd(fmaxf(v, kLeast)));
  }
  // elements, those below `least` (and NaN) as that
  static __device__ __forceinline__ void get(const uint4& x, float least, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const W v = join(word(x, i), all(least));
      const uint32_t u = *(const uint32_t*)&v;
      f[2 * i] = __uint_as_float(u * 65536u);   // a multiply: the logic pipe has enough to do
      f[2 * i + 1] = __uint_as_float(u & 0xFFFF0000u);
    }
  }
  // elements above v
  static __device__ __forceinline__ W count(const uint4& x, float v) {
    W n = __hgt2(word(x, 0), all(v));
#pragma unroll
    for (int i = 1; i < 4; ++i) n = __hadd2(n, __hgt2(word(x, i), all(v)));
    return n;
  }
  // the greatest value of the type that reads less than v does
  static __device__ __forceinline__ float before(float v) {
    const uint32_t u = __float_as_uint(v);
    return v == 0.0f ? __uint_as_float(0x80010000u) : __uint_as_float(v > 0.0f ? u - 0x10000u : u + 0x10000u);
  }
  static __device__ __forceinline__ W add(W a, W b) { return __hadd2(a, b); }   // counts to 256 are exact
  static __device__ __forceinline__ float sum(W a) { return __low2float(a) + __high2float(a); }
};
template <> struct Vec<float> {
  static constexpr int N = 4;
  static constexpr float kLeast = -FLT_MAX;
  typedef float W;
  static __device__ __forceinline__ float word(const uint4& x, int i) {
    return __uint_as_float(i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w);
  }
  static __device__ __forceinline__ W join(W a, W b) { return fmaxf(a, b); }
  static __device__ __forceinline__ W top(const uint4& x) {
    return fmaxf(fmaxf(word(x, 0), word(x, 1)), fmaxf(word(x, 2), word(x, 3)));
  }
  static __device__ __forceinline__ float most(W a) { return a; }
  static __device__ __forceinline__ float round_down(float v) { return fmaxf(v, kLeast); }
  static __device__ __forceinline__ void get(const uint4& x, float least, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = fmaxf(word(x, i), least);
  }
  static __device__ __forceinline__ W count(const uint4& x, float v) {
    W n = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) n += word(x, i) > v ? 1.0f : 0.0f;
    return n;
  }
  static __device__ __forceinline__ float before(float v) { return nextafterf(fminf(v, FLT_MAX), -INFINITY); }
  static __device__ __forceinline__ W add(W a, W b) { return a + b; }
  static __device__ __forceinline__ float sum(W a) { return a; }
};
// as the softmax reads a logit: NaN as -inf, +inf as the largest finite value
template <typename T> __device__ __forceinline__ float read_logit(T l) {
  return fminf(fmaxf(to_f(l), -INFINITY), FLT_MAX);
}

// A list of the 32 best (value, lowest id first) of a warp, lane i its entry i; 0: none.
__device__ __forceinline__ void insert(u64& list, u64 key, int lane) {
  const int at = __popc(__ballot_sync(kAll, list > key));   // entries that stay ahead
  const u64 up = __shfl_up_sync(kAll, list, 1);
  if (lane >= at) list = lane == at ? key : up;
}
// A value that k of the 256 are not below, at most 2^-7 under the k-th largest: by halving, the same in all
// lanes of a warp.
__device__ __forceinline__ float kth_of(const float* v, int k, int lane) {
  uint32_t key[kThreads / 32], low = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) key[i] = f2key(v[i * 32 + lane]);
  for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit >>= 1) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) n += key[i] >= (low | bit);
    if (__reduce_add_sync(kAll, n) >= k) low |= bit;
  }
  return fmaxf(key2f(low), -FLT_MAX);
}

// The i-th row in an order that has those with a token first: where all CTAs run at once, SMs get as many of them
// each, but for one.
__device__ __forceinline__ void in_order(const Args& a, int i, int lane, int warp, int* row) {
  __shared__ int s_live[kWarps];
  const int per = (a.rows + kThreads - 1) / kThreads, r0 = min(a.rows, (int)threadIdx.x * per), r1 = min(a.rows, r0 + per);
  auto has = [&](int r) { return a.tokens[r] >= 0 && a.tokens[r] < a.V; };
  int mine = 0;
  for (int r = r0; r < r1; ++r) mine += has(r);
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kAll, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) s_live[warp] = inc;
  if (threadIdx.x == 0) *row = i;   // a row at any rate, were the tokens written to meanwhile
  __syncthreads();
  int live = inc - mine, all = 0;   // before this thread's, and all
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    live += w < warp ? s_live[w] : 0;
    all += s_live[w];
  }
  int none = all + r0 - live;
  for (int r = r0; r < r1; ++r)
    if ((has(r) ? live++ : none++) == i) *row = r;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, kResident) logprobs_kernel(const Args a) {
  constexpr int E = Vec<T>::N;
  __shared__ Stat s_stat[kWarps];
  __shared__ u64 s_best[32];
  __shared__ float s_peak[TOP ? kThreads : 1], s_bound;   // the threads' greatest; a bound of the best
  __shared__ u64 s_cand[TOP ? kCand : 1];
  __shared__ bf16 s_most[TOP ? kBatches : 1][TOP ? kThreads : 1];   // rounded up
  __shared__ int s_count, s_row;
  __shared__ int s_last;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % a.parts;
  if (a.rows) in_order(a, blockIdx.x / a.parts, lane, warp, &s_row);
  else if (threadIdx.x == 0) s_row = blockIdx.x / a.parts;
  __syncthreads();
  const int row = s_row, n = row / a.B, b = row % a.B;
  const int64_t x = a.tokens[row];
  if (x < 0 || x >= a.V) {   // none: nothing is read
    if (part != 0) return;
    if (threadIdx.x == 0) {
      if (x != -1) atomicOr(a.err, XP_ERR_BADTOKEN);
      if (a.logprob) a.logprob[row] = 0.0f;
      if (a.entropy) a.entropy[row] = 0.0f;
      if (a.rank) a.rank[row] = 0;
    }
    if (TOP && (int)threadIdx.x < a.top) {
      if (a.top_ids) a.top_ids[(int64_t)row * a.top + threadIdx.x] = -1;
      if (a.top_logprobs) a.top_logprobs[(int64_t)row * a.top + threadIdx.x] = 0.0f;
    }
    return;
  }
  const T* l = (const T*)a.logits + n * a.sn + b * a.sb;
  const float heat = a.temperature ? a.temperature[n] : 1.0f;
  const bool greedy = !(heat >= FLT_MIN);   // of a smaller one 1 / t is not finite
  const float inv_t = greedy ? 1.0f : fmaxf(1.0f / heat, FLT_MIN), c = inv_t * kLog2e;
  const float mine = read_logit(l[x]), raw_mine = fmaxf(to_f(l[x]), -INFINITY);
  // an id at -inf has all lower ids ahead of it, and of the higher ones those above -inf
  const bool low_id = mine == -INFINITY;

  // vectors from the first 16-byte boundary on; this CTA's are [v0, v1)
  const int head = min(a.V, (int)((16 - ((uintptr_t)l & 15)) % 16 / sizeof(T)));
  const int vectors = (a.V - head) / E;
  const int v0 = (int)((int64_t)vectors * part / a.parts), v1 = (int)((int64_t)vectors * (part + 1) / a.parts);
  const uint4* body = (const uint4*)(l + head);

  typedef Vec<T> Vt;
  // what an id before x is above if it is ahead, and one behind
  const float below = low_id ? INFINITY : Vt::before(raw_mine), above = mine < FLT_MAX ? raw_mine : INFINITY;
  Stat st = {-FLT_MAX, 0.0f, 0.0f, 0};
  // Of this thread's sums: above `limit` the base has to follow, what is not above `least` adds nothing.
  float peak = -FLT_MAX, limit = -INFINITY, least = -INFINITY, ahead_of = 0.0f;
  uint64_t s2 = 0, w2 = 0;   // the sums while the row is read, of even and odd elements
  const uint64_t c2 = pair(c, c);
  u64 list = 0;
  float bound = -FLT_MAX;   // what the best are not below

  auto follow = [&](float most) {   // the base
    const float d = (st.m - most) * c, by = ex2(d);
    const uint64_t by2 = pair(by, by);
    w2 = by > 0.0f ? mul2(fma2(pair(d, d), s2, w2), by2) : 0ull;
    s2 = mul2(s2, by2);
    st.m = most;
    limit = most + kLazy / c;
    least = Vt::round_down(__fsub_rd(most, 200.0f / c));   // 2^-200 is nothing
    // one by one where there is no such value, or the next one below is so far away that its difference is infinite
    if (least == Vt::kLeast || (least - most) * c == -INFINITY) least = -INFINITY;
  };
  auto add = [&](float lo, float hi) {   // neither infinite
    const uint64_t d = mul2(add2(pair(lo, hi), pair(-st.m, -st.m)), c2);
    const uint64_t e = pair(ex2(low(d)), ex2(high(d)));
    s2 = add2(s2, e);
    w2 = fma2(d, e, w2);
  };
  auto add_one = [&](float v) {
    if (!(v > -INFINITY)) return;
    const float d = (v - st.m) * c, e = ex2(d);
    s2 = add2(s2, pair(e, 0.0f));
    if (e > 0.0f) w2 = fma2(pair(d, 0.0f), pair(e, 0.0f), w2);
  };
  auto push = [&](float v, int id) {   // one that may be among the best
    if (!(v >= bound)) return;
    const int at = atomicAdd(&s_count, 1);
    if (at < kCand) s_cand[at] = pack_best(v, (uint32_t)id);
  };
  // ids before the first boundary and behind the last vector: one a lane of warp 0
  auto ends = [&](int from, int to) {
    const int id = from + lane;
    if (id >= to) return;
    const float v = read_logit(l[id]);
    peak = fmaxf(peak, v);
    if (v > limit) follow(v);
    add_one(v);
    ahead_of += (low_id ? v > mine && id > x : v > mine || (v == mine && id < x)) ? 1.0f : 0.0f;
    if (TOP) push(v, id);
  };
  // one id a lane into the warp's sorted list; *own: its last entry of `top`
  auto put = [&](float v, int id, float* own) {
    const u64 key = pack_best(v, (uint32_t)id);
    unsigned good = __ballot_sync(kAll, v >= bound && v > *own);
    while (good) {
      const int i = __ffs(good) - 1;
      good &= good - 1;
      insert(list, __shfl_sync(kAll, key, i), lane);
      const u64 last = __shfl_sync(kAll, list, a.top - 1);
      if (last) *own = packed_val(last);
      good &= __ballot_sync(kAll, v > *own);
    }
  };

  uint4 raw[kLoads];
  auto load = [&](int v) {
    const uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;   // -inf
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int at = v + u * kThreads + lane;
      raw[u] = at < v1 ? __ldcs(body + at) : make_uint4(none, none, none, none);
    }
  };
  const int first = v0 + warp * 32;
  load(first);
  if (TOP) {
    if (threadIdx.x == 0) s_count = 0;
    if (threadIdx.x < 32) s_best[threadIdx.x] = 0;
    __syncthreads();
  }
  if (warp == 0 && part == 0 && head > 0) ends(0, head);

  int batch = 0;
  for (int v = first; v < v1; v += kThreads * kLoads) {
    uint4 now[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) now[u] = raw[u];
    load(v + kThreads * kLoads);   // the next ones are on their way meanwhile
    typename Vt::W top[kLoads], of_all;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      top[u] = Vt::top(now[u]);
      of_all = u == 0 ? top[0] : Vt::join(of_all, top[u]);
    }
    const float raw_most = fmaxf(Vt::most(of_all), -INFINITY), most = fminf(raw_most, FLT_MAX);
    auto id_of = [&](int u) { return head + (v + u * kThreads + lane) * E; };
    peak = fmaxf(peak, most);
    // Where all are NaN or -inf, or too small to add anything, nothing is added.
    if (most > least) {
      if (most > limit) follow(most);
      if (least > -INFINITY && raw_most <= FLT_MAX) {
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          float f[E];
          Vt::get(now[u], least, f);
#pragma unroll
          for (int i = 0; i < E; i += 2) add(f[i], f[i + 1]);
        }
      } else {   // an infinity, or one that would not be told from the least value: one by one
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          float f[E];
          Vt::get(now[u], -INFINITY, f);
#pragma unroll
          for (int i = 0; i < E; ++i) add_one(fminf(f[i], FLT_MAX));
        }
      }
    }
    // ids ahead of x; x's own vector is put right at the end
    if (sizeof(T) == 2 || most >= mine) {
      typename Vt::W n;
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const typename Vt::W k = Vt::count(now[u], id_of(u) + E <= x ? below : above);
        n = u == 0 ? k : Vt::add(n, k);
      }
      ahead_of += Vt::sum(n);
    }
    if (TOP) {
      bf16* to = &s_most[min(batch, kBatches - 1)][threadIdx.x];
      *to = __float2bfloat16_ru(batch < kBatches ? most : fmaxf(most, to_f(*to)));
      ++batch;
    }
  }
  if (warp == 0 && part == a.parts - 1 && head + vectors * E < a.V) ends(head + vectors * E, a.V);

  // the keys in the buffer to their places
  auto place = [&](int count) {
    for (int i = threadIdx.x; i < count; i += kThreads) {
      const u64 key = s_cand[i];
      int ahead = 0;
#pragma unroll 8
      for (int j = 0; j < count; ++j) ahead += s_cand[j] > key;
      if (key && ahead < a.top) s_best[ahead] = key;
    }
    __syncthreads();
  };
  if (TOP) {
    s_peak[threadIdx.x] = peak;
    __syncthreads();
    if (warp == 0) {
      bound = kth_of(s_peak, a.top, lane);
      if (lane == 0) s_bound = bound;
    }
    __syncthreads();
    bound = s_bound;
    // every lane its own batches, all lanes' first ones together
    u64 reach = 0;
    for (int i = 0; i < min(batch, kBatches); ++i) reach |= (u64)(to_f(s_most[i][threadIdx.x]) >= bound) << i;
    int behind = 0;   // of the batches that share the last place
    while (__any_sync(kAll, reach != 0)) {
      const int i = __ffsll(reach) - 1;
      const int v = i < 0 ? v1 : first + (i + behind) * (kThreads * kLoads);
      if (i < kBatches - 1 || ++behind == batch - i) reach &= reach - 1;
      load(v);
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        if (!(Vt::most(Vt::top(raw[u])) >= bound)) continue;
        float f[E];
        Vt::get(raw[u], -INFINITY, f);
#pragma unroll
        for (int i = 0; i < E; ++i) push(fminf(f[i], FLT_MAX), head + (v + u * kThreads + lane) * E + i);
      }
    }
    __syncthreads();
    int count = s_count;
    if (count > kCand) {
      // a list a warp, in ascending order of ids, so that what only equals its last entry is passed over
      float own = -INFINITY;
      if (warp == 0 && part == 0) put(lane < head ? read_logit(l[lane]) : -INFINITY, lane, &own);
      for (int id0 = head + v0 * E + warp * 32; id0 < a.V; id0 += kThreads) {
        const int id = id0 + lane, end = part == a.parts - 1 ? a.V : head + v1 * E;
        if (id0 >= end) break;
        put(id < end ? read_logit(l[id]) : -INFINITY, id, &own);
      }
      __syncthreads();   // count has been read by all
      s_cand[threadIdx.x] = list;
      __syncthreads();
      count = kThreads;
    }
    place(count);
  }
  // x's own vector was counted by what is above it: of the ids before x, equal ones are ahead too
  const int own_vector = x < head || x >= head + vectors * E ? -1 : (int)(x - head) / E;
  if (own_vector >= v0 && own_vector < v1) {
    const int from = head + own_vector * E;
    if (warp == 0 && from + lane < x) {
      const float v = read_logit(l[from + lane]);
      ahead_of += low_id ? (v > mine ? -1.0f : 0.0f) : v == mine ? 1.0f : 0.0f;
    }
  }
  st.ahead = (int)ahead_of;
  st.s = low(s2) + high(s2);
  st.w = low(w2) + high(w2);
  // the CTA's, in warp 0
  auto gather = [&]() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      st = join(st, {__shfl_xor_sync(kAll, st.m, o), __shfl_xor_sync(kAll, st.s, o),
                     __shfl_xor_sync(kAll, st.w, o), __shfl_xor_sync(kAll, st.ahead, o)}, c);
    if (lane == 0) s_stat[warp] = st;
    __syncthreads();
    if (warp == 0) {
      st = s_stat[0];
      for (int w = 1; w < kWarps; ++w) st = join(st, s_stat[w], c);
    }
  };
  gather();

  if (a.parts > 1) {
    const int row = s_row;   // again, so that no register holds it all the way
    const int64_t at = (int64_t)row * a.parts;
    if (warp == 0) {
      if (lane == 0) __stcg(a.stat + at + part, make_float4(st.m, st.s, st.w, __int_as_float(st.ahead)));
      if (TOP && lane < a.top) __stcg(a.best + (at + part) * a.top + lane, s_best[lane]);
      __threadfence();
    }
    if (!arrive_last(a.tickets + row, a.parts, &s_last)) return;
    if (threadIdx.x == 0) a.tickets[row] = 0;
    st = {-FLT_MAX, 0.0f, 0.0f, 0};
    for (int p = threadIdx.x; p < a.parts; p += kThreads) {
      const float4 v = __ldcg(a.stat + at + p);
      st = join(st, {v.x, v.y, v.z, __float_as_int(v.w)}, c);
    }
    if (TOP) {
      if (threadIdx.x < 32) s_best[threadIdx.x] = 0;
      const int count = a.parts * a.top;   // at most the places of the buffer
      for (int i = threadIdx.x; i < count; i += kThreads) s_cand[i] = __ldcg(a.best + at * a.top + i);
      __syncthreads();
      place(count);
    }
    gather();
  }
  if (warp != 0) return;

  if (TOP) list = s_best[lane];
  const int out = s_row;
  const float log_s = logf(st.s);   // s = 0: nothing above -inf
  const int ahead = st.ahead + (low_id ? (int)x : 0);
  auto log_p = [&](float v) { return greedy ? -INFINITY : (v - st.m) * inv_t - log_s; };
  if (lane == 0) {
    if (!(st.s > 0.0f)) atomicOr(a.err, XP_ERR_EMPTY);
    if (a.logprob) a.logprob[out] = !(st.s > 0.0f) ? -INFINITY : greedy && ahead == 0 ? 0.0f : log_p(mine);
    if (a.entropy) a.entropy[out] = greedy || !(st.s > 0.0f) ? 0.0f : log_s - st.w / st.s * 0.693147180559945f;
    if (a.rank) a.rank[out] = ahead + 1;
  }
  if (TOP && lane < a.top) {
    const int64_t at = (int64_t)out * a.top + lane;
    if (a.top_ids) a.top_ids[at] = list ? (int64_t)packed_idx(list) : -1;
    if (a.top_logprobs)
      a.top_logprobs[at] = !list ? -INFINITY : greedy && lane == 0 ? 0.0f : log_p(packed_val(list));
  }
}

}  // namespace

// Tickets of the most rows that are cut (at a place of their own, so that it does not move with the
// call), then what parts leave.
xp_logprobs_ws xp_logprobs_layout(const xp_head* h, int rows, int top) {
  (void)rows;
  const size_t cut = (size_t)h->num_sms * kResident;
  xp_logprobs_ws L;
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = (o + bytes + 255) / 256 * 256; return at; };
  L.tickets = take(cut * 4);
  L.stat = take(cut * sizeof(float4));
  L.best = take(cut * 8 * (size_t)top);
  L.total = o;
  return L;
}

cudaError_t xp_launch_logprobs(const xp_head* h, const xp_logprobs_args& g, cudaStream_t s) {
  const int es = (int)xp_elem(g.dtype), rows = g.N * g.B, cut = h->num_sms * kResident;
  Args a;
  a.logits = g.logits;
  a.sn = g.sn, a.sb = g.sb;
  a.tokens = g.tokens, a.temperature = g.temperature;
  a.B = g.B, a.V = h->V, a.top = g.top;
  // As many parts as run at once: 32 rows of 151936 in fp32 45 us whole, 25 in 10 parts, 31 in 18; 200 rows 50 whole,
  // 42 in 3, 56 in 4; 456 rows 65 whole, 85 in 2.
  a.parts = std::max(1, std::min({h->V / (16 / es) / kLeastVectors, cut / rows, kMostParts}));
  // An order, which takes a microsecond, where SMs have more than one CTA and all run at once
  a.rows = rows <= cut && rows * a.parts > h->num_sms ? rows : 0;
  a.logprob = g.logprob, a.entropy = g.entropy, a.rank = g.rank;
  a.top_ids = g.top_ids, a.top_logprobs = g.top_logprobs;
  a.err = h->err;
  a.tickets = g.tickets, a.stat = (float4*)g.stat, a.best = g.best;
  const unsigned grid = (unsigned)(rows * a.parts);
  if (g.dtype == XP_BF16) {
    if (a.top) logprobs_kernel<bf16, true><<<grid, kThreads, 0, s>>>(a);
    else logprobs_kernel<bf16, false><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (a.top) logprobs_kernel<float, true><<<grid, kThreads, 0, s>>>(a);
    else logprobs_kernel<float, false><<<grid, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}
