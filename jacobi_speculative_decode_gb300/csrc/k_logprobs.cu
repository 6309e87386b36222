// Log probabilities of given tokens, the entropy, the token's rank and the best alternatives: one pass
// over the row.
//
// A row, or a part of one, is a CTA's.  Every thread keeps a base m, near its running maximum, S = sum 2^((l - m) c)
// and W = sum (l - m) c 2^((l - m) c), c = log2(e) / t; then, all joined at the row's maximum,
//   log p(x) = (l_x - m) / t - log S,   H = log S - log(2) W / S.
// Differences are taken before they are scaled, so that neither large logits nor small temperatures lose
// digits.
// The best ids.  Of the 256 threads' greatest elements so far, each warp's ceil(top / 8)-th is a bound: there are
// `top` elements that are not below the least of the eight.  What reaches it goes to a buffer in shared
// memory (some 40 elements whenever as many more have been read as before), and the buffer is sorted at
// the end.  Where it overflows, as it does for a row that rises from end to end, the row is read again and
// every element above the last of a sorted list put in its place there.
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
constexpr int kMostParts = 4;         // parts of cut rows, all together, per CTA that runs at once
constexpr float kPartCost = 0.03f;    // what a part costs besides its elements, in rows of a usual vocabulary
constexpr int kCand = 2048;           // places of the buffer: elements of fewer than 227 vectors all fit,
                                      // and from there on every warp has its share of them
constexpr int kLeastVectors = kThreads * kLoads;   // of a part of a row
constexpr float kLazy = 8.0f;         // how far (base 2) a logit may lie above the base of its thread's sums
constexpr float kLog2e = 1.44269504088896f;
constexpr unsigned kAll = 0xFFFFFFFFu;

struct Args {
  const void* logits;
  int64_t sn, sb;
  const int64_t* tokens;
  const float* temperature;
  int B, V, top, parts;
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

// 16 bytes of logits as floats, NaN as -inf
template <typename T> struct Vec;
template <> struct Vec<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    const __nv_bfloat162 least = __float2bfloat162_rn(-INFINITY);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __hmax2(*(const __nv_bfloat162*)&w[i], least);
      const uint32_t u = *(const uint32_t*)&v;
      f[2 * i] = __uint_as_float(u * 65536u);   // a multiply: the logic pipe has enough to do
      f[2 * i + 1] = __uint_as_float(u & 0xFFFF0000u);
    }
  }
};
template <> struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& x, float (&f)[4]) {
    f[0] = fmaxf(__uint_as_float(x.x), -INFINITY), f[1] = fmaxf(__uint_as_float(x.y), -INFINITY);
    f[2] = fmaxf(__uint_as_float(x.z), -INFINITY), f[3] = fmaxf(__uint_as_float(x.w), -INFINITY);
  }
};
// as the softmax reads a logit: NaN as -inf, +inf as the largest finite value
__device__ __forceinline__ float read_logit(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX); }

// A list of the 32 best (value, lowest id first) of a warp, lane i its entry i; 0: none.
__device__ __forceinline__ void insert(u64& list, u64 key, int lane) {
  const int at = __popc(__ballot_sync(kAll, list > key));   // entries that stay ahead
  const u64 up = __shfl_up_sync(kAll, list, 1);
  if (lane >= at) list = lane == at ? key : up;
}
// the 32 best of two lists
__device__ __forceinline__ u64 merge(u64 a, u64 b, int lane) {
  const u64 r = __shfl_sync(kAll, b, 31 - lane);
  u64 v = a > r ? a : r;   // the 32 best, rising and falling
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 w = __shfl_xor_sync(kAll, v, o);
    v = ((lane & o) == 0) == (v > w) ? v : w;
  }
  return v;
}

// 32 entries sorted, the best first
__device__ __forceinline__ u64 sorted(u64 v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int o = size / 2; o > 0; o >>= 1) {
      const u64 w = __shfl_xor_sync(kAll, v, o);
      v = (((lane & o) == 0) == ((lane & size) == 0)) == (v > w) ? v : w;
    }
  return v;
}
// The k-th largest of the lanes' values.
__device__ __forceinline__ float kth_of_lanes(float v, int k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int o = size / 2; o > 0; o >>= 1) {
      const float w = __shfl_xor_sync(kAll, v, o);
      v = ((lane & o) == 0) == ((lane & size) == 0) ? fmaxf(v, w) : fminf(v, w);
    }
  return __shfl_sync(kAll, v, k - 1);
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, kResident) logprobs_kernel(const Args a) {
  constexpr int E = Vec<T>::N;
  __shared__ Stat s_stat[kWarps];
  __shared__ u64 s_best[kWarps][32];
  __shared__ float s_bound[kWarps];
  __shared__ u64 s_cand[TOP ? kCand : 1];
  __shared__ int s_count;
  __shared__ int s_last;

  const int row = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const int n = row / a.B, b = row % a.B;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
  const float mine = read_logit(to_f(l[x]));
  // an id at -inf has all lower ids ahead of it, and of the higher ones those above -inf
  const bool low_id = mine == -INFINITY;

  // vectors from the first 16-byte boundary on; this CTA's are [v0, v1)
  const int head = min(a.V, (int)((16 - ((uintptr_t)l & 15)) % 16 / sizeof(T)));
  const int vectors = (a.V - head) / E;
  const int v0 = (int)((int64_t)vectors * part / a.parts), v1 = (int)((int64_t)vectors * (part + 1) / a.parts);
  const uint4* body = (const uint4*)(l + head);

  Stat st = {-FLT_MAX, 0.0f, 0.0f, 0};
  float peak = -FLT_MAX, limit = -FLT_MAX;   // running maximum; where the base has to follow it
  uint64_t s2 = 0, w2 = 0;   // its sums while the row is read, of even and odd elements
  const uint64_t c2 = pair(c, c);
  const float below = low_id ? INFINITY : nextafterf(mine, -INFINITY);   // what an id before x has to be above
  u64 list = 0;
  float bound = -INFINITY;    // what the best are not below
  const int share = (a.top + kWarps - 1) / kWarps;   // entries a warp brings to the bound
  volatile float* bounds = s_bound;

  // E elements of ids from `id` on; before: x is behind them
  auto take = [&](float (&f)[E], int id, bool before) {
    float most = f[0];
#pragma unroll
    for (int i = 1; i < E; ++i) most = fmaxf(most, f[i]);
    if (most > FLT_MAX) {
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = fminf(f[i], FLT_MAX);
      most = FLT_MAX;
    }
    peak = fmaxf(peak, most);
    if (most > limit) {   // sums to the new base
      const float d = (st.m - most) * c, by = ex2(d);
      const uint64_t by2 = pair(by, by);
      w2 = by > 0.0f ? mul2(fma2(pair(d, d), s2, w2), by2) : 0ull;
      s2 = mul2(s2, by2);
      st.m = most;
      limit = most + kLazy / c;
    }
    const uint64_t off = pair(-st.m, -st.m);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const uint64_t d = mul2(add2(pair(f[i], f[i + 1]), off), c2);
      const uint64_t e = pair(ex2(low(d)), ex2(high(d)));
      s2 = add2(s2, e);
      w2 = fma2(pair(fmaxf(low(d), -FLT_MAX), fmaxf(high(d), -FLT_MAX)), e, w2);   // nothing of -inf
    }
    if (most >= mine) {
      const float t = before ? below : mine;   // the vector with x in it is put right at the end
#pragma unroll
      for (int i = 0; i < E; ++i) st.ahead += f[i] > t;
    }
    if (TOP && most >= bound) {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (f[i] >= bound && f[i] > -INFINITY) {
          const int at = atomicAdd(&s_count, 1);
          if (at < kCand) s_cand[at] = pack_best(f[i], (uint32_t)(id + i));
        }
    }
  };
  // ids before the first boundary and behind the last vector: one element a lane of warp 0
  auto ends = [&](int from, int to) {
    const int id = from + lane;
    float f[E];
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = -INFINITY;
    if (id < to) f[0] = fmaxf(to_f(l[id]), -INFINITY);
    take(f, id, id < x);
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
  load(v0 + warp * 32);
  auto tighten = [&](float most) {   // this lane's greatest so far
    const float mine = kth_of_lanes(most, share, lane);
    if (lane == 0) bounds[warp] = mine;
  };
  auto read_bound = [&]() {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) bound = w == 0 ? bounds[0] : fminf(bound, bounds[w]);
  };
  if (TOP) {
    float most = -INFINITY;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      float f[E];
      Vec<T>::get(raw[u], f);
#pragma unroll
      for (int i = 0; i < E; ++i) most = fmaxf(most, f[i]);
    }
    tighten(fminf(most, FLT_MAX));
    if (threadIdx.x == 0) s_count = 0;
    __syncthreads();
    read_bound();
  }
  if (warp == 0 && part == 0 && head > 0) ends(0, head);

  int batch = 0;
  for (int v = v0 + warp * 32; v < v1; v += kThreads * kLoads) {
    uint4 now[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) now[u] = raw[u];
    load(v + kThreads * kLoads);   // the next ones are on their way meanwhile
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      float f[E];
      Vec<T>::get(now[u], f);
      const int id = head + (v + u * kThreads + lane) * E;
      take(f, id, id + E <= x);
    }
    if (TOP && (++batch & (batch - 1)) == 0) {   // after 1, 2, 4, ... of them; another warp's word may be its last one
      tighten(peak);
      __syncwarp();
      read_bound();
    }
  }
  if (warp == 0 && part == a.parts - 1 && head + vectors * E < a.V) ends(head + vectors * E, a.V);

  if (TOP) {
    __syncthreads();
    const int count = s_count;
    if (count <= kCand) {
      for (int i = warp * 32; i < count; i += kThreads) {
        const u64 more = sorted(i + lane < count ? s_cand[i + lane] : 0, lane);
        list = i == warp * 32 ? more : merge(list, more, lane);
      }
    } else {
      // a list a warp, in ascending order of ids, so that what only equals its last entry is passed over
      read_bound();
      float own = -INFINITY;
      if (warp == 0 && part == 0) put(lane < head ? read_logit(to_f(l[lane])) : -INFINITY, lane, &own);
      for (int id0 = head + v0 * E + warp * 32; id0 < a.V; id0 += kThreads) {
        const int id = id0 + lane, end = part == a.parts - 1 ? a.V : head + v1 * E;
        if (id0 >= end) break;
        put(id < end ? read_logit(to_f(l[id])) : -INFINITY, id, &own);
      }
    }
  }
  // x's own vector was counted by what is above it: of the ids before x, equal ones are ahead too
  const int own_vector = x < head || x >= head + vectors * E ? -1 : (int)(x - head) / E;
  if (own_vector >= v0 && own_vector < v1) {
    const int from = head + own_vector * E;
    if (warp == 0 && from + lane < x) {
      const float v = read_logit(to_f(l[from + lane]));
      st.ahead += low_id ? -(v > mine) : v == mine;
    }
  }
  st.s = low(s2) + high(s2);
  st.w = low(w2) + high(w2);
  // the CTA's, in warp 0
  auto gather = [&]() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      st = join(st, {__shfl_xor_sync(kAll, st.m, o), __shfl_xor_sync(kAll, st.s, o),
                     __shfl_xor_sync(kAll, st.w, o), __shfl_xor_sync(kAll, st.ahead, o)}, c);
    if (lane == 0) s_stat[warp] = st;
    if (TOP) s_best[warp][lane] = list;
    __syncthreads();
    if (TOP) {
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) {
        if (warp < o) s_best[warp][lane] = list = merge(list, s_best[warp + o][lane], lane);
        __syncthreads();
      }
    }
    if (warp == 0) {
      st = s_stat[0];
      for (int w = 1; w < kWarps; ++w) st = join(st, s_stat[w], c);
    }
  };
  gather();

  if (a.parts > 1) {
    const int64_t at = (int64_t)row * a.parts;
    if (warp == 0) {
      if (lane == 0) __stcg(a.stat + at + part, make_float4(st.m, st.s, st.w, __int_as_float(st.ahead)));
      if (TOP && lane < a.top) __stcg(a.best + (at + part) * a.top + lane, list);
      __threadfence();
    }
    if (!arrive_last(a.tickets + row, a.parts, &s_last)) return;
    if (threadIdx.x == 0) a.tickets[row] = 0;
    st = {-FLT_MAX, 0.0f, 0.0f, 0};
    for (int p = threadIdx.x; p < a.parts; p += kThreads) {
      const float4 v = __ldcg(a.stat + at + p);
      st = join(st, {v.x, v.y, v.z, __float_as_int(v.w)}, c);
    }
    list = 0;
    if (TOP)
      for (int p = warp; p < a.parts; p += kWarps)
        list = merge(list, lane < a.top ? __ldcg(a.best + (at + p) * a.top + lane) : 0ull, lane);
    gather();
  }
  if (warp != 0) return;

  const float log_s = logf(st.s);   // s = 0: nothing above -inf
  const int ahead = st.ahead + (low_id ? (int)x : 0);
  auto log_p = [&](float v) { return greedy ? -INFINITY : (v - st.m) * inv_t - log_s; };
  if (lane == 0) {
    if (!(st.s > 0.0f)) atomicOr(a.err, XP_ERR_EMPTY);
    if (a.logprob) a.logprob[row] = !(st.s > 0.0f) ? -INFINITY : greedy && ahead == 0 ? 0.0f : log_p(mine);
    if (a.entropy) a.entropy[row] = greedy || !(st.s > 0.0f) ? 0.0f : log_s - st.w / st.s * 0.693147180559945f;
    if (a.rank) a.rank[row] = ahead + 1;
  }
  if (TOP && lane < a.top) {
    const int64_t at = (int64_t)row * a.top + lane;
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
  L.stat = take(kMostParts * cut * sizeof(float4));
  L.best = take(kMostParts * cut * 8 * (size_t)top);
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
  // Parts so that the CTAs come in whole turns: the least turns * (1 / parts + kPartCost).  Rows that fill the
  // GPU by themselves are not cut.
  const int most = std::min(std::max(1, h->V / (16 / es) / kLeastVectors), kMostParts * cut / std::max(1, rows));
  a.parts = 1;
  float best = FLT_MAX;
  for (int parts = 1; rows < cut && parts <= most; ++parts) {
    const float time = (float)((rows * parts + cut - 1) / cut) * (1.0f / parts + kPartCost);
    if (time < best) best = time, a.parts = parts;
  }
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
