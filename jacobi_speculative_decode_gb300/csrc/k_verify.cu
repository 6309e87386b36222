// Verification of drafted blocks.  Two kernels:
//  verify_stats_kernel  softmax statistics (max, sum) of the target's and the draft's rows,
//                       and each slot's test u q(x) < p(x);
//  verify_draw_kernel   the one token each block draws, at the slot where it ended.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "sm100_ptx.cuh"
#include "xp_device.cuh"

using namespace xpd;
typedef __nv_bfloat16 bf16;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLoads = 4;           // 16-byte loads a thread has in flight
constexpr int kResident = 3;        // CTAs an SM: 48 KB of loads in flight
constexpr float kLog2e = 1.44269504088896f;

// a logit as the softmax reads it: scaled, NaN as -inf, +inf as the largest finite value
__device__ __forceinline__ float read_logit(float l, float inv_t) {
  return fminf(fmaxf(l * inv_t, -INFINITY), FLT_MAX);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Softmax statistics of part of a row: its maximum (a raw logit) and the sum of
// 2^((l - m) c), c = log2(e) / temperature.
struct Stat {
  float m, s;
};
// 2^((l - m) c) for m = base_of(a maximum): NaN gives 0, +inf gives 1, the maximum itself 1
__device__ __forceinline__ float weight(float l, float c, float m) {
  return __saturatef(ex2((l - m) * c));
}
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
  const Stat r = {fmaxf(a.m, b.m), 0.0f};
  const float m = base_of(r.m);
  return {r.m, a.s * weight(a.m, c, m) + b.s * weight(b.m, c, m)};
}
__device__ __forceinline__ Stat warp_join(Stat v, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = join(v, {__shfl_xor_sync(0xFFFFFFFFu, v.m, o), __shfl_xor_sync(0xFFFFFFFFu, v.s, o)}, c);
  return v;
}

__device__ __forceinline__ float heat_of(const xp_verify_args& a, int n) {
  const float t = a.temperature ? a.temperature[n] : 1.0f;
  return t > 0.0f ? t : 0.0f;
}
__device__ __forceinline__ int drafts_of(const xp_verify_args& a, int n, bool tell) {
  if (!a.n_draft) return a.B - 1;
  const int d = a.n_draft[n];
  if (d < 0 || d > a.B - 1) {
    if (tell) atomicOr(a.err, XP_ERR_LENGTH);
    return d < 0 ? 0 : a.B - 1;
  }
  return d;
}

// 16 bytes of logits as floats
template <typename T> struct Vec;
template <> struct Vec<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    const uint32_t w = i / 2 == 0 ? v.x : i / 2 == 1 ? v.y : i / 2 == 2 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
};
template <> struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
};

// elements before the first 16-byte boundary of a row
template <typename T>
__device__ __forceinline__ int head_of(const T* row, int V) {
  return min(V, (int)(((16 - ((uintptr_t)row & 15)) & 15) / sizeof(T)));
}

// Chunk c of a row (its 16-byte aligned vectors [c*chunk, (c+1)*chunk) elements behind the head;
// the first chunk also takes the head, the last one what is left of the row), a thread's share:
// statistics, and with TOP the lowest id of the maximum.
template <typename T, bool TOP>
__device__ __forceinline__ Stat thread_stat(const T* row, int V, int chunk, int c, bool last, float k,
                                            int* top) {
  constexpr int VN = Vec<T>::N;
  const int head = head_of(row, V), vecs = (V - head) / VN;
  const int v0 = c * (chunk / VN), v1 = last ? vecs : min(vecs, v0 + chunk / VN);
  const uint4* at = (const uint4*)(row + head);
  Stat st = {-INFINITY, 0.0f};
  int id = 0x7FFFFFFF;
  // at most one single element a thread: of the head, or behind the last vector
  const int rest = V - head - vecs * VN;
  int one = -1;
  if (c == 0 && (int)threadIdx.x < head) one = threadIdx.x;
  if (last && threadIdx.x >= 32 && (int)threadIdx.x < 32 + rest)
    one = head + vecs * VN + threadIdx.x - 32;
  if (one >= 0) {
    st.m = read_logit(to_f(row[one]), 1.0f);
    st.s = st.m > -INFINITY ? 1.0f : 0.0f;
    id = one;
  }
  for (int i0 = v0 + (int)threadIdx.x; i0 < v1; i0 += kThreads * kLoads) {
    uint4 x[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (i0 + u * kThreads < v1) x[u] = __ldcs(at + i0 + u * kThreads);
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (i0 + u * kThreads < v1)
#pragma unroll
        for (int e = 0; e < VN; ++e) m = fmaxf(m, Vec<T>::get(x[u], e));
    m = fminf(m, FLT_MAX);
    if (TOP && m >= st.m) {
#pragma unroll
      for (int u = kLoads - 1; u >= 0; --u)
        if (i0 + u * kThreads < v1)
#pragma unroll
          for (int e = VN - 1; e >= 0; --e) {
            const int v = head + (i0 + u * kThreads) * VN + e;
            // an equal maximum of a later vector does not count, one of the row's end does
            if (read_logit(Vec<T>::get(x[u], e), 1.0f) == m && (m > st.m || v < id)) id = v;
          }
    }
    const float now = fmaxf(st.m, m), base = base_of(now);
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (i0 + u * kThreads < v1)
#pragma unroll
        for (int e = 0; e < VN; e += 2) {
          s0 += weight(Vec<T>::get(x[u], e), k, base);
          s1 += weight(Vec<T>::get(x[u], e + 1), k, base);
        }
    st.s = st.s * weight(st.m, k, base) + s0 + s1;
    st.m = now;
  }
  if (TOP) *top = id;
  return st;
}

// the row's chunk over the CTA; warp 0's result counts
template <typename T, bool TOP>
__device__ Stat chunk_stat(const T* row, int V, int chunk, int c, bool last, float k, int* top,
                           Stat* s_warp, int* s_top) {
  Stat st = thread_stat<T, TOP>(row, V, chunk, c, last, k, top);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (TOP) {
    float m = st.m;
    warp_argmax(m, *top);
    if (lane == 0) s_top[w] = *top;
  }
  st = warp_join(st, k);
  if (lane == 0) s_warp[w] = st;
  __syncthreads();
  if (w == 0) {
    st = lane < kWarps ? s_warp[lane] : Stat{-INFINITY, 0.0f};
    if (TOP) {
      float m = st.m;
      *top = lane < kWarps ? s_top[lane] : 0x7FFFFFFF;
      warp_argmax(m, *top);
    }
    st = warp_join(st, k);
  }
  __syncthreads();
  return st;
}

// Work items (slot, block, chunk), slots outermost, dealt out over a resident grid: the rows of
// early slots are done first, and a row behind a slot that was rejected by then is skipped.
// Nothing waits for that: a row read in vain changes no result.
template <typename T>
__global__ void __launch_bounds__(kThreads, kResident) verify_stats_kernel(const xp_verify_args a, int chunk,
                                                                int chunks) {
  __shared__ Stat s_warp[kWarps];
  __shared__ int s_top[kWarps];
  __shared__ unsigned s_next;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t items = (int64_t)a.B * a.N * chunks;
  int64_t it = blockIdx.x;
  while (it < items) {
    // a thread an item: the next one of this CTA's that is still wanted
    if (threadIdx.x == 0) s_next = kThreads;
    __syncthreads();
    {
      const int64_t mine = it + (int64_t)threadIdx.x * gridDim.x;
      bool wanted = false;
      if (mine < items) {
        const int n = (int)(mine / chunks % a.N), b = (int)(mine / chunks / a.N);
        // marks[n] = B - (first rejected slot known so far), 0 when none is
        const int done = a.B - (int)__ldcg(&a.marks[n]);
        wanted = b <= drafts_of(a, n, b == 0) && b <= done;
      }
      const unsigned any = __ballot_sync(0xFFFFFFFFu, wanted);
      if (lane == 0 && any) atomicMin(&s_next, w * 32 + __ffs(any) - 1);
    }
    __syncthreads();
    const unsigned skip = s_next;
    it += (int64_t)skip * gridDim.x;
    if (skip == kThreads) continue;

    const int c = (int)(it % chunks);
    const int n = (int)(it / chunks % a.N), b = (int)(it / chunks / a.N);
    it += gridDim.x;
    const int drafts = drafts_of(a, n, false);
    const float heat = heat_of(a, n);
    const float inv_t = heat > 0.0f ? 1.0f / heat : 1.0f, k = inv_t * kLog2e;
    const bool last = c == chunks - 1, two = a.draft && heat > 0.0f && b < drafts;
    const int64_t row = (int64_t)n * a.B + b;
    const T* t_row = (const T*)a.target + n * a.sn + b * a.sb;
    const float* d_row = two ? a.draft + ((int64_t)n * (a.B - 1) + b) * a.ld_draft : nullptr;
    Stat d = {0.0f, 1.0f}, t;
    int top = -1;
    if (heat > 0.0f)
      t = chunk_stat<T, false>(t_row, a.V, chunk, c, last, k, nullptr, s_warp, s_top);
    else
      t = chunk_stat<T, true>(t_row, a.V, chunk, c, last, k, &top, s_warp, s_top);
    if (two) d = chunk_stat<float, false>(d_row, a.V, chunk, c, last, k, nullptr, s_warp, s_top);
    if (w != 0) continue;
    // the rest is warp 0's: the row's last chunk joins them all and tests the slot
    float* out = a.part + (row * chunks + c) * 5;
    unsigned ticket = 0;
    if (lane == 0) {
      __stcg(out, t.m);
      __stcg(out + 1, t.s);
      __stcg(out + 2, d.m);
      __stcg(out + 3, d.s);
      __stcg(out + 4, __int_as_float(top));
      asm volatile("atom.add.acq_rel.gpu.u32 %0, [%1], 1;"
                   : "=r"(ticket)
                   : "l"(&a.tickets[row])
                   : "memory");
    }
    ticket = __shfl_sync(0xFFFFFFFFu, ticket, 0);
    if (ticket != (unsigned)chunks - 1) continue;
    __threadfence();
    t = d = {-INFINITY, 0.0f};
    float m = -INFINITY;
    top = 0x7FFFFFFF;
    for (int i = lane; i < chunks; i += 32) {
      const float* in = a.part + (row * chunks + i) * 5;
      const Stat x = {__ldcg(in), __ldcg(in + 1)};
      const int id = __float_as_int(__ldcg(in + 4));
      if (better(x.m, id, m, top)) { m = x.m; top = id; }
      t = join(t, x, k);
      if (two) d = join(d, {__ldcg(in + 2), __ldcg(in + 3)}, k);
    }
    warp_argmax(m, top);
    t = warp_join(t, k);
    if (two) d = warp_join(d, k);
    if (lane != 0) continue;
    float* out_row = a.row + row * 5;
    out_row[0] = t.m;
    out_row[1] = t.s;
    out_row[2] = d.m;
    out_row[3] = d.s;
    out_row[4] = __int_as_float(t.m > -INFINITY ? top : -1);
    if (b >= drafts) continue;
    const int64_t x = a.blk[(int64_t)n * a.B + 1 + b];
    float px = 0.0f, qx = 1.0f;
    if (x < 0 || x >= a.V) {
      atomicOr(a.err, XP_ERR_BADTOKEN);
    } else if (t.m > -INFINITY) {
      if (heat == 0.0f) {
        px = x == top ? 1.0f : 0.0f;
      } else {
        px = expf(read_logit(to_f(t_row[x]), inv_t) - read_logit(t.m, inv_t)) / t.s;
        if (two)
          qx = d.m > -INFINITY
                   ? expf(read_logit(d_row[x], inv_t) - read_logit(d.m, inv_t)) / d.s
                   : 0.0f;
      }
    }
    const float u = a.u[(int64_t)n * (a.B - 1) + b];
    if (a.prob) a.prob[(int64_t)n * (a.B - 1) + b] = px > 0.0f ? fminf(px / qx, 1.0f) : 0.0f;
    if (!(u * qx < px)) atomicMax(&a.marks[n], (unsigned)(a.B - b));
  }
}

// The race of one id: w / e with w = max(p - q, 0).  Most ids are far behind the best, so a
// quick form (approximate exponential and reciprocal: relative error below 2^-15 of p and q,
// the exponent's rounding at most 150 * 2^-23) decides first whether the exact one, which
// alone counts, is worth computing.
struct Race {
  float inv_t, inv_s, tz, inv_d, dz;   // dz, inv_d: the draft's, where it has a row
  int64_t x;                           // a one-hot draft's id, -1
  unsigned long long best;
  float best_f;

  __device__ __forceinline__ float exact(float l, bool two, float d, float e, int v) const {
    const float p = expf(read_logit(l, inv_t) - tz) * inv_s;
    const float q = two ? expf(read_logit(d, inv_t) - dz) * inv_d : v == x ? 1.0f : 0.0f;
    return p > q ? (p - q) / e : 0.0f;
  }
  template <bool TWO>
  __device__ __forceinline__ void take(float l, float d, float e, int v) {
    constexpr float kMore = 1.0f + 1.0f / 16384, kLess = 1.0f - 1.0f / 16384;
    float w = __saturatef(ex2((l * inv_t - tz) * kLog2e)) * inv_s * kMore;
    if (TWO) w -= __saturatef(ex2((d * inv_t - dz) * kLog2e)) * inv_d * kLess;
    if (w > 0.0f && __fdividef(w, e) * kMore >= best_f) {
      const float r = exact(l, TWO, d, e, v);
      if (r > 0.0f) {
        best = max(best, pack_best(r, (uint32_t)v));
        best_f = packed_val(best);
      }
    }
  }
};

// Chunk c of a block's race: rows of target, draft and noise need not share an alignment, so
// ids are taken in vectors of the noise row (fp32); the others come with plain loads where
// theirs differs.
template <typename T, bool TWO>
__device__ void race_chunk(Race& r, const T* t_row, const float* d_row, const float* e_row, int V,
                           int lo, int hi) {
  // common case: all three rows on 16-byte boundaries from the same id on
  const bool wide = (((uintptr_t)(t_row + lo) | (uintptr_t)(e_row + lo) |
                      (TWO ? (uintptr_t)(d_row + lo) : 0)) & 15) == 0;
  int v = lo;
  if (wide) {
    constexpr int W = 8;
    const int vecs = (hi - lo) / W;
    for (int i = threadIdx.x; i < vecs; i += kThreads) {
      const int at = lo + i * W;
      uint4 tx[sizeof(T) / 2], ex[2], dx[2];
#pragma unroll
      for (int u = 0; u < (int)sizeof(T) / 2; ++u) tx[u] = __ldcs((const uint4*)(t_row + at) + u);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        ex[u] = __ldcs((const uint4*)(e_row + at) + u);
        if (TWO) dx[u] = __ldcs((const uint4*)(d_row + at) + u);
      }
#pragma unroll
      for (int e = 0; e < W; ++e)
        r.take<TWO>(Vec<T>::get(tx[e / Vec<T>::N], e % Vec<T>::N),
                    TWO ? Vec<float>::get(dx[e / 4], e % 4) : 0.0f, Vec<float>::get(ex[e / 4], e % 4),
                    at + e);
    }
    v = lo + vecs * W;
  }
  for (v += (int)threadIdx.x; v < hi; v += kThreads)
    r.take<TWO>(to_f(t_row[v]), TWO ? d_row[v] : 0.0f, e_row[v], v);
}

// Work items (block, chunk): the race of every id of the chunk, merged into the block's best;
// the block's last chunk writes its tokens and clears its counters for the next call.
template <typename T>
__global__ void __launch_bounds__(kThreads) verify_draw_kernel(const xp_verify_args a, int chunk) {
  __shared__ unsigned long long s_best[kWarps];
  __shared__ int s_last;
  ptx::pdl_wait();
  const int n = blockIdx.y, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int drafts = drafts_of(a, n, false);
  const unsigned mark = a.marks[n];
  const bool rejected = mark != 0;
  const int end = rejected ? min(drafts, a.B - (int)mark) : drafts;   // slots accepted
  const int64_t row = (int64_t)n * a.B + end;
  const float heat = heat_of(a, n);
  const float tm = a.row[row * 5];
  const bool empty = !(tm > -INFINITY);
  const T* t_row = (const T*)a.target + n * a.sn + end * a.sb;
  const float* e_row = a.noise + n * a.ld_noise;
  Race r = {};
  if (heat > 0.0f && !empty) {
    r.inv_t = 1.0f / heat;
    r.inv_s = 1.0f / a.row[row * 5 + 1];
    r.tz = read_logit(tm, r.inv_t);
    r.x = rejected && !a.draft ? a.blk[(int64_t)n * a.B + 1 + end] : -1;
    const float dm = a.row[row * 5 + 2];
    const bool two = a.draft && rejected && dm > -INFINITY;
    const float* d_row = two ? a.draft + ((int64_t)n * (a.B - 1) + end) * a.ld_draft : nullptr;
    const int lo = blockIdx.x * chunk, hi = min(a.V, lo + chunk);
    if (two) {
      r.inv_d = 1.0f / a.row[row * 5 + 3];
      r.dz = read_logit(dm, r.inv_t);
      race_chunk<T, true>(r, t_row, d_row, e_row, a.V, lo, hi);
    } else {
      race_chunk<T, false>(r, t_row, nullptr, e_row, a.V, lo, hi);
    }
    unsigned long long best = r.best;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
    if (lane == 0) s_best[w] = best;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < kWarps; ++i) best = max(best, s_best[i]);
      if (best) atomicMax(&a.packed[n], best);
    }
  }
  if (!arrive_last(&a.draw_ticket[n], gridDim.x, &s_last)) return;
  int64_t last = -1;
  if (empty) {
    if (threadIdx.x == 0) atomicOr(a.err, XP_ERR_EMPTY);
  } else if (heat == 0.0f) {
    last = __float_as_int(a.row[row * 5 + 4]);
  } else {
    unsigned long long best = __ldcg(&a.packed[n]);
    if (!best) {   // rounding left no positive residual: p itself is raced, by this CTA alone
      r.x = -1;
      r.best = 0;
      r.best_f = 0.0f;
      race_chunk<T, false>(r, t_row, nullptr, e_row, a.V, 0, a.V);
      best = r.best;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
      if (lane == 0) s_best[w] = best;
      __syncthreads();
      for (int i = 0; i < kWarps; ++i) best = max(best, s_best[i]);
    }
    last = packed_idx(best);
  }
  __syncthreads();   // read by everyone before thread 0 clears
  for (int b = threadIdx.x; b < a.B; b += kThreads) {
    a.tokens[(int64_t)n * a.B + b] =
        b < end ? a.blk[(int64_t)n * a.B + 1 + b] : b == end ? last : -1;
    a.tickets[(int64_t)n * a.B + b] = 0;
    // slots behind the end may have been tested by rows that ran ahead
    if (a.prob && b < a.B - 1 && (b > end || b >= drafts)) a.prob[(int64_t)n * (a.B - 1) + b] = 0.0f;
  }
  if (threadIdx.x == 0) {
    a.counts[n] = end + (last >= 0 ? 1 : 0);
    a.marks[n] = 0;
    a.packed[n] = 0;
    a.draw_ticket[n] = 0;
  }
}

// Vocabulary ids of one work item: 16384 where that leaves every SM several items, less
// (down to 2048) for few rows, whose latency counts.
int chunk_of(int64_t rows, int V, int sms) {
  int chunk = 16384;
  while (chunk > 2048 && rows * ((V + chunk - 1) / chunk) < (int64_t)sms * 4) chunk /= 2;
  return chunk;
}

}  // namespace

xp_verify_ws xp_verify_layout(const xp_head* h, int N) {
  (void)N;
  const size_t rows = (size_t)h->max_N * h->B, n = (size_t)h->max_N;
  xp_verify_ws L;
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = (o + bytes + 255) / 256 * 256; return at; };
  L.marks = take(n * 4);
  L.tickets = take(rows * 4);
  L.packed = take(n * 8);
  L.draw_ticket = take(n * 4);
  L.part = take(rows * (((size_t)h->V + 2047) / 2048) * 20);
  L.row = take(rows * 20);
  L.total = o;
  return L;
}

template <typename T>
static cudaError_t launch_verify(const xp_head* h, const xp_verify_args& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.N * a.B;
  const int chunk = chunk_of(rows, a.V, h->num_sms), chunks = (a.V + chunk - 1) / chunk;
  const unsigned grid = (unsigned)std::min<int64_t>(rows * chunks, (int64_t)h->num_sms * kResident);
  verify_stats_kernel<T><<<grid, kThreads, 0, s>>>(a, chunk, chunks);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int draw = chunk_of(a.N, a.V, h->num_sms);
  return xp_launch_pdl(verify_draw_kernel<T>, dim3((a.V + draw - 1) / draw, a.N), dim3(kThreads), 0, s,
                       a, draw);
}

cudaError_t xp_launch_verify(const xp_head* h, const xp_verify_args& a, cudaStream_t s) {
  return h->dtype == XP_BF16 ? launch_verify<bf16>(h, a, s) : launch_verify<float>(h, a, s);
}
