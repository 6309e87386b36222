// Verification of drafted blocks.  Two kernels:
//  verify_stats_kernel  softmax statistics (max, sum) of the target's and the draft's rows,
//                       and each slot's test u q(x) < p(x);
//  verify_draw_kernel   the one token each block draws, at the slot where it ended.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "xp_device.cuh"

using namespace xpd;
typedef __nv_bfloat16 bf16;

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;        // vocabulary ids of one work item
constexpr int kDrawChunk = 8192;

// a logit as the softmax reads it: scaled, NaN as -inf, +inf as the largest finite value
__device__ __forceinline__ float read_logit(float l, float inv_t) {
  return fminf(fmaxf(l * inv_t, -INFINITY), FLT_MAX);
}

struct Stat {
  float m, s;   // maximum, sum of exp(z - m)
};
__device__ __forceinline__ float minus(float z, float m) { return m == -INFINITY ? 0.0f : z - m; }
__device__ __forceinline__ Stat join(Stat a, Stat b) {
  const float m = fmaxf(a.m, b.m);
  Stat r = {m, 0.0f};
  if (m > -INFINITY) r.s = a.s * __expf(a.m - m) + b.s * __expf(b.m - m);
  return r;
}
__device__ __forceinline__ void warp_join(Stat& v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat t = {__shfl_xor_sync(0xFFFFFFFFu, v.m, o), __shfl_xor_sync(0xFFFFFFFFu, v.s, o)};
    v = join(v, t);
  }
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

// Per chunk (5 floats): target max, sum, draft max, sum, lowest id of the target's max.
struct Part {
  Stat t, d;
  int top;
};

// the softmax statistics of one chunk of a row over the CTA; thread 0's result counts
template <typename T>
__device__ Stat chunk_stat(const T* row, int lo, int hi, float inv_t, int* top, Stat* s_warp,
                           int* s_top) {
  Stat st = {-INFINITY, 0.0f};
  int id = 0x7FFFFFFF;
  for (int v = lo + (int)threadIdx.x; v < hi; v += kThreads) {
    const float z = read_logit(to_f(row[v]), inv_t);
    if (z > st.m) {
      st.s = st.s * __expf(minus(st.m, z)) + 1.0f;
      st.m = z;
      id = v;
    } else if (z > -INFINITY) {
      st.s += __expf(z - st.m);
    }
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (top) {
    float m = st.m;
    int i = id;
    warp_argmax(m, i);
    if (lane == 0) s_top[w] = i;
  }
  warp_join(st);
  if (lane == 0) s_warp[w] = st;
  __syncthreads();
  if (threadIdx.x == 0) {
    Stat r = s_warp[0];
    int best = top ? s_top[0] : 0;
    for (int k = 1; k < kThreads / 32; ++k) {
      if (top && better(s_warp[k].m, s_top[k], r.m, best)) best = s_top[k];
      r = join(r, s_warp[k]);
    }
    st = r;
    if (top) *top = best;
  }
  __syncthreads();
  return st;
}

// Work items (slot, block, chunk), slots outermost, spread over a resident grid: the rows of
// early slots are done first, and a row behind a slot that was rejected by then is skipped.
// Nothing waits for that: a row read in vain changes no result.
template <typename T>
__global__ void __launch_bounds__(kThreads) verify_stats_kernel(const xp_verify_args a) {
  __shared__ Stat s_warp[kThreads / 32];
  __shared__ int s_top[kThreads / 32];
  __shared__ int s_last;
  const int chunks = (a.V + kChunk - 1) / kChunk;
  const int64_t items = (int64_t)a.B * a.N * chunks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int c = (int)(it % chunks);
    const int n = (int)(it / chunks % a.N), b = (int)(it / chunks / a.N);
    const int drafts = drafts_of(a, n, c == 0 && b == 0 && threadIdx.x == 0);
    // marks[n] = B - (first rejected slot known so far), 0 when none is
    __syncthreads();
    if (threadIdx.x == 0)
      s_last = b > drafts || a.B - (int)*(volatile unsigned*)&a.marks[n] < b;
    __syncthreads();
    if (s_last) continue;
    const float heat = heat_of(a, n);
    const float inv_t = heat > 0.0f ? 1.0f / heat : 1.0f;
    const int lo = c * kChunk, hi = min(a.V, lo + kChunk);
    const int64_t row = (int64_t)n * a.B + b;
    Part p;
    p.t = chunk_stat((const T*)a.target + n * a.sn + b * a.sb, lo, hi, inv_t, &p.top, s_warp, s_top);
    const bool two = a.draft && heat > 0.0f && b < drafts;
    p.d = {0.0f, 1.0f};
    if (two)
      p.d = chunk_stat(a.draft + ((int64_t)n * (a.B - 1) + b) * a.ld_draft, lo, hi, inv_t, nullptr,
                       s_warp, s_top);
    float* out = a.part + (row * chunks + c) * 5;
    if (threadIdx.x == 0) {
      __stcg(out, p.t.m);
      __stcg(out + 1, p.t.s);
      __stcg(out + 2, p.d.m);
      __stcg(out + 3, p.d.s);
      __stcg(out + 4, __int_as_float(p.top));
    }
    if (!arrive_last(&a.tickets[row], chunks, &s_last)) continue;
    // the row's last chunk: join them all and test the slot
    if (threadIdx.x < 32) {
      Stat t = {-INFINITY, 0.0f}, d = {-INFINITY, 0.0f};
      float m = -INFINITY;
      int top = 0x7FFFFFFF;
      for (int k = threadIdx.x; k < chunks; k += 32) {
        const float* in = a.part + (row * chunks + k) * 5;
        const Stat x = {__ldcg(in), __ldcg(in + 1)};
        const int id = __float_as_int(__ldcg(in + 4));
        if (better(x.m, id, m, top)) { m = x.m; top = id; }
        t = join(t, x);
        if (two) d = join(d, {__ldcg(in + 2), __ldcg(in + 3)});
      }
      warp_argmax(m, top);
      warp_join(t);
      if (two) warp_join(d);
      if (threadIdx.x == 0) {
        float* out_row = a.row + row * 5;
        out_row[0] = t.m;
        out_row[1] = t.s;
        out_row[2] = d.m;
        out_row[3] = d.s;
        out_row[4] = __int_as_float(t.m > -INFINITY ? top : -1);
        if (b < drafts) {
          const int64_t x = a.blk[(int64_t)n * a.B + 1 + b];
          float px = 0.0f, qx = 1.0f;
          if (x < 0 || x >= a.V) {
            atomicOr(a.err, XP_ERR_BADTOKEN);
          } else if (t.m > -INFINITY) {
            if (heat == 0.0f) {
              px = x == top ? 1.0f : 0.0f;
            } else {
              px = expf(read_logit(to_f(((const T*)a.target)[n * a.sn + b * a.sb + x]), inv_t) - t.m) / t.s;
              if (two) {
                const float z =
                    read_logit(a.draft[((int64_t)n * (a.B - 1) + b) * a.ld_draft + x], inv_t);
                qx = d.m > -INFINITY ? expf(z - d.m) / d.s : 0.0f;
              }
            }
          }
          const float u = a.u[(int64_t)n * (a.B - 1) + b];
          if (a.prob)
            a.prob[(int64_t)n * (a.B - 1) + b] = px > 0.0f ? fminf(px / qx, 1.0f) : 0.0f;
          if (!(u * qx < px)) atomicMax(&a.marks[n], (unsigned)(a.B - b));
        }
      }
    }
  }
}

// Work items (block, chunk): the race of every id of the chunk, merged into the block's best;
// the block's last chunk writes its tokens and clears its counters for the next call.
template <typename T>
__global__ void __launch_bounds__(kThreads) verify_draw_kernel(const xp_verify_args a) {
  __shared__ unsigned long long s_best[2][kThreads / 32];
  __shared__ int s_last;
  const int n = blockIdx.y, c = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int drafts = drafts_of(a, n, false);
  const unsigned mark = a.marks[n];
  const int end = mark ? min(drafts, a.B - (int)mark) : drafts;   // slots accepted
  const bool rejected = mark != 0;
  const int64_t row = (int64_t)n * a.B + end;
  const float heat = heat_of(a, n);
  const float tm = a.row[row * 5], ts = a.row[row * 5 + 1];
  const bool empty = !(tm > -INFINITY);
  if (heat > 0.0f && !empty) {
    const float inv_t = 1.0f / heat, inv_s = 1.0f / ts;
    const bool two = a.draft && rejected;
    const float dm = two ? a.row[row * 5 + 2] : 0.0f, ds = two ? a.row[row * 5 + 3] : 1.0f;
    const bool q_any = two && dm > -INFINITY;
    const float inv_d = 1.0f / ds;
    const T* t_row = (const T*)a.target + n * a.sn + end * a.sb;
    const float* d_row = two ? a.draft + ((int64_t)n * (a.B - 1) + end) * a.ld_draft : nullptr;
    const float* e_row = a.noise + n * a.ld_noise;
    const int64_t x = rejected && !a.draft ? a.blk[(int64_t)n * a.B + 1 + end] : -1;
    const int lo = c * kDrawChunk, hi = min(a.V, lo + kDrawChunk);
    // best of the residual, and of p itself for the case that no residual is positive
    unsigned long long best = 0, back = 0;
    for (int v = lo + (int)threadIdx.x; v < hi; v += kThreads) {
      const float p = expf(read_logit(to_f(t_row[v]), inv_t) - tm) * inv_s;
      float q = v == x ? 1.0f : 0.0f;
      if (q_any) q = expf(read_logit(d_row[v], inv_t) - dm) * inv_d;
      const float e = e_row[v];
      if (p > 0.0f) back = max(back, pack_best(p / e, (uint32_t)v));
      if (p > q) best = max(best, pack_best((p - q) / e, (uint32_t)v));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
      back = max(back, __shfl_xor_sync(0xFFFFFFFFu, back, o));
    }
    if (lane == 0) {
      s_best[0][w] = best;
      s_best[1][w] = back;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      unsigned long long m = 0;
      for (int k = 0; k < kThreads / 32; ++k) m = max(m, s_best[threadIdx.x][k]);
      if (m) atomicMax(&a.packed[2 * n + threadIdx.x], m);
    }
  }
  if (!arrive_last(&a.draw_ticket[n], gridDim.x, &s_last)) return;
  int64_t last = -1;
  if (empty) {
    if (threadIdx.x == 0) atomicOr(a.err, XP_ERR_EMPTY);
  } else if (heat == 0.0f) {
    last = __float_as_int(a.row[row * 5 + 4]);
  } else {
    unsigned long long m = __ldcg(&a.packed[2 * n]);
    if (!m) m = __ldcg(&a.packed[2 * n + 1]);
    last = packed_idx(m);
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
    a.packed[2 * n] = a.packed[2 * n + 1] = 0;
    a.draw_ticket[n] = 0;
  }
}

}  // namespace

xp_verify_ws xp_verify_layout(const xp_head* h, int N) {
  (void)N;
  const size_t rows = (size_t)h->max_N * h->B, n = (size_t)h->max_N;
  const size_t chunks = ((size_t)h->V + kChunk - 1) / kChunk;
  xp_verify_ws L;
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = (o + bytes + 255) / 256 * 256; return at; };
  L.marks = take(n * 4);
  L.tickets = take(rows * 4);
  L.packed = take(n * 16);
  L.draw_ticket = take(n * 4);
  L.part = take(rows * chunks * 20);
  L.row = take(rows * 20);
  L.total = o;
  return L;
}

cudaError_t xp_launch_verify(const xp_head* h, const xp_verify_args& a, cudaStream_t s) {
  const int64_t items = (int64_t)a.B * a.N * ((a.V + kChunk - 1) / kChunk);
  const unsigned grid = (unsigned)std::min<int64_t>(items, (int64_t)h->num_sms * 8);
  const dim3 draw((a.V + kDrawChunk - 1) / kDrawChunk, a.N);
  if (h->dtype == XP_BF16) {
    verify_stats_kernel<bf16><<<grid, kThreads, 0, s>>>(a);
    verify_draw_kernel<bf16><<<draw, kThreads, 0, s>>>(a);
  } else {
    verify_stats_kernel<float><<<grid, kThreads, 0, s>>>(a);
    verify_draw_kernel<float><<<draw, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}
