// Verification of drafted blocks.  Two kernels:
//  verify_stats_kernel  softmax statistics (max, sum) of the target's and the draft's rows,
//                       and each slot's test u q(x) < p(x);
//  verify_draw_kernel   the one token each block draws, at the slot where it ended.
#include <float.h>
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "sm100_ptx.cuh"
#include "xp_device.cuh"

using namespace xpd;
typedef __nv_bfloat16 bf16;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLoads = 4;               // 16-byte vectors of a stage a thread reads
constexpr int kStageBytes = kThreads * kLoads * 16;   // 16 KB
constexpr int kStages = 4;              // 64 KB in flight a CTA
constexpr int kResident = 2;            // CTAs an SM
constexpr float kLog2e = 1.44269504088896f;

// a logit as the softmax reads it: NaN as -inf, +inf as the largest finite value
__device__ __forceinline__ float read_logit(float l) {
  return fminf(fmaxf(l, -INFINITY), FLT_MAX);
}
// e^((l - m) / t) for a row's maximum m.  The difference is taken before it is scaled: l / t and m / t
// apart would be rounded at their own size, and clipped where t is small.
__device__ __forceinline__ float share(float l, float m, float inv_t) {
  return expf((read_logit(l) - m) * inv_t);
}
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
  return t >= FLT_MIN ? t : 0.0f;   // of a smaller one 1 / t is not finite, or its product with log2 e
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

// 16 bytes of logits
template <typename T> struct Vec;
template <> struct Vec<bf16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = 0xFF80FF80u;   // -inf, twice
  static __device__ __forceinline__ float get(uint32_t w, int i) {
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
  static __device__ __forceinline__ float top(const uint4 (&x)[kLoads]) {   // NaN left out
    __nv_bfloat162 m = __float2bfloat162_rn(-INFINITY);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    }
    return fmaxf(__low2float(m), __high2float(m));
  }
};
template <> struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
  static __device__ __forceinline__ float get(uint32_t w, int) { return __uint_as_float(w); }
  static __device__ __forceinline__ float top(const uint4 (&x)[kLoads]) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(x[u].x), __uint_as_float(x[u].y)),
                         fmaxf(__uint_as_float(x[u].z), __uint_as_float(x[u].w))));
    return m;
  }
};
template <typename T>
__device__ __forceinline__ float element(const uint4& x, int i) {
  constexpr int P = Vec<T>::N / 4;   // logits a word
  const uint32_t w = i / P == 0 ? x.x : i / P == 1 ? x.y : i / P == 2 ? x.z : x.w;
  return Vec<T>::get(w, i % P);
}

// elements before the first 16-byte boundary of a row
template <typename T>
__device__ __forceinline__ int head_of(const T* row, int V) {
  return min(V, (int)(((16 - ((uintptr_t)row & 15)) & 15) / sizeof(T)));
}

// One batch of a row, kLoads vectors a thread (those behind the row hold -inf), into running
// statistics.  Returns the batch's maximum.
template <typename T>
__device__ __forceinline__ float batch_stat(const uint4 (&x)[kLoads], float k, Stat& st) {
  constexpr int VN = Vec<T>::N;
  const float m = fminf(Vec<T>::top(x), FLT_MAX), now = fmaxf(st.m, m), base = base_of(now);
  // two logits an instruction: 2^(l k - bk), bk = base k rounded; what that rounding took, at most
  // 2^-11, is given back to the sum: 2^(bk - base k) = 1 + ln 2 (bk - base k), within 2^-23
  uint64_t sum[2] = {0, 0};
  const float bk = __fmul_rn(base, k);
  float back = fmaf(fmaf(-base, k, bk), 0.693147180559945f, 1.0f);
  const uint64_t k2 = pair(k, k), b2 = pair(-bk, -bk);
#pragma unroll
  for (int u = 0; u < kLoads; ++u)
#pragma unroll
    for (int e = 0; e < VN; e += 2) {
      const uint64_t z = fma2(pair(element<T>(x[u], e), element<T>(x[u], e + 1)), k2, b2);
      sum[e / 2 % 2] = add2(sum[e / 2 % 2], pair(ex2(low(z)), ex2(high(z))));
    }
  sum[0] = add2(sum[0], sum[1]);
  float s = low(sum[0]) + high(sum[0]);
  // NaN or +inf among them, or a base whose rounding is more: logit by logit
  if (!(s <= (float)(kLoads * VN + 1)) || fabsf(bk) > 16384.0f) {
    s = 0.0f;
    back = 1.0f;
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
#pragma unroll 1
      for (int e = 0; e < VN; ++e) s += weight(element<T>(x[u], e), k, base);
  }
  st.s = fmaf(s, back, st.s * weight(st.m, k, base));
  st.m = now;
  return m;
}

// The maximum of a greedy row as it is met: its value, the first vector of the batch that held
// it (-1: none), and a logit that no vector holds.  The id is looked up at the item's end, by
// the few lanes that hold the item's maximum.
struct Top {
  float m;
  int batch;
  float single;
  int single_id;
};
template <typename T>
__device__ __forceinline__ int id_of(const T* row, int V, int v1, const Top& t, float m) {
  constexpr int VN = Vec<T>::N;
  const int head = head_of(row, V);
  int id = t.single == m ? t.single_id : 0x7FFFFFFF;
  if (t.m == m && t.batch >= 0)
    for (int u = kLoads - 1; u >= 0; --u) {
      const int at = t.batch + (int)threadIdx.x + u * kThreads;
      if (at < v1)
        for (int e = VN - 1; e >= 0; --e) {
          const int v = head + at * VN + e;
          if (read_logit(to_f(row[v])) == m) id = min(id, v);
        }
    }
  return id;
}
// vectors [*v0, *v1) of chunk c of a row
template <typename T>
__device__ __forceinline__ void vectors_of(const T* row, int V, int chunk, int chunks, int c, int* v0,
                                           int* v1) {
  constexpr int VN = Vec<T>::N;
  const int vecs = (V - head_of(row, V)) / VN;
  *v0 = min(vecs, c * (chunk / VN));
  *v1 = c == chunks - 1 ? vecs : min(vecs, *v0 + chunk / VN);
}

// What a stage of the ring holds: `bytes` of the item's target or draft row, behind `first` vectors
struct Stage {
  int item, kind;     // kind: of the draft's row, first of its row's chunk, last of the item, ...
  int first, bytes;   // first vector of the stage in the row
};
constexpr int kDraft = 1, kOpens = 2, kEnds = 4, kStop = 8, kDropped = 16;

constexpr int kItems = 4;
struct Ring {
  uint64_t full[kStages], empty[kStages];
  Stage stage[kStages];
  // finished items on their way to the joining warp: statistics (target, draft) of every warp
  uint64_t written[kItems], read[kItems];
  Stat stat[kItems][kWarps][2];
  int top[kItems][kWarps];
  int item[kItems];          // -1: there are no more
  int abort;
};

// The statistics of every wanted row, in items (slot, block, chunk) with the slots outermost: the
// rows of early slots are done first, and a row behind a slot that was rejected by then is
// skipped.  Nothing waits for that: a row read in vain changes no result.
// Warp 8 claims the items from a counter and streams the rows into a ring by bulk copies, ahead
// over the items' ends; warps 0-7 sum what it holds; warp 9 writes the items' results, and
// where an item is its row's last joins them and tests the slot.
// What bounds it: rows read in vain, and the ends of items.  Two items a CTA are claimed and under
// way, close to a slot of a large batch, and a rejection is known only when its row is done.  So
// the streaming warp looks at the block's mark again with every stage and leaves a row in the
// middle (7 us of 75 for the drafter's logits below).  256 blocks of 16 slots, 151,936 ids, bf16,
// one-hot drafts of which 0.7 are accepted: 111 us for 472 MB, a quarter of it in vain, 4.3 TB/s (63%
// of measured; instructions issue in 53% of the cycles).  Both kernels take 154 there, 67 for 32
// blocks with the drafter's logits.
// Smaller items reach a rejection sooner but end more often, which costs more than it saves (what of
// it is not hidden is not known): with 32768, 16384 and 8192 ids instead of 65536 the large batch took
// 23, 70 and 157 us more.  Two CTAs of 64 KB in flight an SM: one of 512 threads and 96 to 192 KB
// took 10 to 30 us more.  Claims of several items at once, for the slots where most are not wanted,
// leave some CTAs with several rows at the end: 10 to 190 us more.
template <typename T>
__global__ void __launch_bounds__(kThreads + 64, kResident) verify_stats_kernel(
    const xp_verify_args a, int chunk, int chunks) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ Ring sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per_slot = a.N * chunks;
  volatile int* abort = &sh.abort;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&sh.full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&sh.empty[s]), kWarps);
    }
    for (int h = 0; h < kItems; ++h) {
      ptx::mbar_init(ptx::smem_u32(&sh.written[h]), kWarps);
      ptx::mbar_init(ptx::smem_u32(&sh.read[h]), 1);
    }
    sh.abort = 0;
    ptx::fence_barrier_init();
  }
  __syncthreads();

  if (warp == kWarps) {
    const int items = a.B * per_slot;
    int issued = 0;
    bool ok = true;
    // marks[n] = B - (first rejected slot known so far), 0 when none is.  Other CTAs raise it
    // meanwhile: lane 0 reads it and the warp takes its value, where it is used.
    auto mark_of = [&](int i) {
      return lane == 0 && i < items ? (int)__ldcg(&a.marks[i / chunks % a.N]) : a.B;
    };
    // room for the next stage
    auto room = [&]() {
      const int s = issued % kStages;
      ok = ptx::mbar_wait(ptx::smem_u32(&sh.empty[s]), ((issued / kStages) & 1) ^ 1, abort, a.err);
      ok = __all_sync(0xFFFFFFFFu, ok);
      return s;
    };
    auto post = [&](int s, const Stage& st, const void* from) {
      if (lane == 0) {
        sh.stage[s] = st;
        const uint32_t full = ptx::smem_u32(&sh.full[s]);
        if (st.bytes > 0) {
          ptx::mbar_arrive_expect_tx(full, st.bytes);
          ptx::bulk_load(ptx::smem_u32(ring + s * kStageBytes), from, st.bytes, full);
        } else {
          ptx::mbar_arrive(full);
        }
      }
      __syncwarp();
      ++issued;
    };
    // The stages of one row's chunk; false where the row was found to lie behind a rejection on the
    // way (it can never be wanted, and its item leaves no result).
    auto stream = [&](auto* row, int item, int c, int kind, int ends) {
      using E = typename std::remove_const<typename std::remove_pointer<decltype(row)>::type>::type;
      constexpr int VN = Vec<E>::N, kPer = kStageBytes / 16;
      const int head = head_of(row, a.V);
      int v, v1, opens = kOpens, seen = 0;
      vectors_of(row, a.V, chunk, chunks, c, &v, &v1);
      do {
        const int n = min(kPer, v1 - v), s = room();
        if (!ok) return false;
        if (item / per_slot > a.B - __shfl_sync(0xFFFFFFFFu, seen, 0)) {
          post(s, {item, kDropped, 0, 0}, nullptr);
          return false;
        }
        post(s, {item, kind | opens | (v + n == v1 ? ends : 0), v, n * 16}, row + head + (int64_t)v * VN);
        seen = mark_of(item);   // there by the time of the next stage
        v += n;
        opens = 0;
      } while (v < v1);
      return true;
    };
    // A CTA's first item is its own number, the others come from the counter.  The counter and
    // the next item's mark are read while this one streams.
    auto claim = [&]() {
      unsigned i = 0;
      if (lane == 0) i = min(gridDim.x + atomicAdd(a.next, 1u), (unsigned)items);
      return (int)i;
    };
    int next = blockIdx.x, mark = mark_of(next);
    int claimed = claim();
    while (ok && next < items) {
      const int i = next, c = i % chunks, n = i / chunks % a.N, b = i / per_slot;
      const int drafts = drafts_of(a, n, c == 0 && b == 0 && lane == 0);
      const bool wanted = b <= a.B - __shfl_sync(0xFFFFFFFFu, mark, 0) && b <= drafts;
      next = __shfl_sync(0xFFFFFFFFu, claimed, 0);
      mark = mark_of(next);
      claimed = claim();
      if (!wanted) continue;
      const bool two = a.draft && heat_of(a, n) > 0.0f && b < drafts;
      if (stream((const T*)a.target + n * a.sn + b * a.sb, i, c, 0, two ? 0 : kEnds) && two)
        stream(a.draft + ((int64_t)n * (a.B - 1) + b) * a.ld_draft, i, c, kDraft, kEnds);
    }
    if (ok) {
      const int s = room();
      if (ok) post(s, {0, kStop, 0, 0}, nullptr);
    }
    // nothing may land in shared memory after the CTA is gone
    volatile int no_abort = 0;
    for (int s = 0; s < kStages; ++s) {
      const int n = (issued + kStages - 1 - s) / kStages;
      if (n > 0) ptx::mbar_wait(ptx::smem_u32(&sh.full[s]), (n - 1) & 1, &no_abort, a.err);
    }
    return;
  }

  if (warp == kWarps + 1) {
    for (int done = 0;; ++done) {
      const int h = done % kItems;
      const bool ok = ptx::mbar_wait(ptx::smem_u32(&sh.written[h]), (done / kItems) & 1, abort, a.err);
      if (!__all_sync(0xFFFFFFFFu, ok)) return;
      const int item = sh.item[h];
      if (item < 0) return;
      const int c = item % chunks, n = item / chunks % a.N, b = item / per_slot, row = n * a.B + b;
      const int drafts = drafts_of(a, n, false);
      const float heat = heat_of(a, n);
      const float inv_t = heat > 0.0f ? 1.0f / heat : 1.0f, k = inv_t * kLog2e;
      const bool draft = a.draft && heat > 0.0f && b < drafts;
      Stat t = {-INFINITY, 0.0f}, d = t;
      int top = 0x7FFFFFFF;
      if (lane < kWarps) {
        t = sh.stat[h][lane][0];
        d = sh.stat[h][lane][1];
        top = sh.top[h][lane];
      }
      float m = t.m;
      warp_argmax(m, top);
      t = warp_join(t, k);
      d = draft ? warp_join(d, k) : Stat{0.0f, 1.0f};
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.read[h]));
      float* out = a.part + ((int64_t)row * chunks + c) * 5;
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
      // the row's last item
      __threadfence();
      t = d = {-INFINITY, 0.0f};
      m = -INFINITY;
      top = 0x7FFFFFFF;
      for (int i = lane; i < chunks; i += 32) {
        const float* in = a.part + ((int64_t)row * chunks + i) * 5;
        const Stat x = {__ldcg(in), __ldcg(in + 1)};
        const int id = __float_as_int(__ldcg(in + 4));
        if (better(x.m, id, m, top)) { m = x.m; top = id; }
        t = join(t, x, k);
        if (draft) d = join(d, {__ldcg(in + 2), __ldcg(in + 3)}, k);
      }
      warp_argmax(m, top);
      t = warp_join(t, k);
      if (draft) d = warp_join(d, k);
      if (lane != 0) continue;
      float* out_row = a.row + (int64_t)row * 5;
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
          const T* t_row = (const T*)a.target + n * a.sn + b * a.sb;
          px = share(to_f(t_row[x]), t.m, inv_t) / t.s;
          if (draft) {
            const float* d_row = a.draft + ((int64_t)n * (a.B - 1) + b) * a.ld_draft;
            qx = d.m > -INFINITY ? share(d_row[x], d.m, inv_t) / d.s : 0.0f;
          }
        }
      }
      const float u = a.u[(int64_t)n * (a.B - 1) + b];
      if (a.prob) a.prob[(int64_t)n * (a.B - 1) + b] = px > 0.0f ? fminf(px / qx, 1.0f) : 0.0f;
      if (!(u * qx < px)) atomicMax(&a.marks[n], (unsigned)(a.B - b));
    }
  }

  Stat st = {-INFINITY, 0.0f}, kept = {-INFINITY, 0.0f};   // of the row in progress; of the target
  Top tp = {-INFINITY, -1, -INFINITY, 0x7FFFFFFF};
  int n = 0, b = 0, c = 0, done = 0;   // done: items finished
  float heat = 1.0f, k = kLog2e;
  for (int pos = 0;; ++pos) {
    const int s = pos % kStages;
    bool ok = ptx::mbar_wait(ptx::smem_u32(&sh.full[s]), (pos / kStages) & 1, abort, a.err);
    if (!__all_sync(0xFFFFFFFFu, ok)) break;
    const Stage sg = sh.stage[s];
    if (sg.kind & kStop) {
      const int h = done % kItems;
      ok = ptx::mbar_wait(ptx::smem_u32(&sh.read[h]), ((done / kItems) & 1) ^ 1, abort, a.err);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      if (lane == 0) {
        if (warp == 0) sh.item[h] = -1;
        ptx::mbar_arrive(ptx::smem_u32(&sh.written[h]));
      }
      break;
    }
    if (sg.kind & kDropped) {
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[s]));
      continue;
    }
    const bool draft = sg.kind & kDraft;
    if (sg.kind & kOpens) {
      if (!draft) {
        c = sg.item % chunks;
        n = sg.item / chunks % a.N;
        b = sg.item / per_slot;
        heat = heat_of(a, n);
        k = (heat > 0.0f ? 1.0f / heat : 1.0f) * kLog2e;
        tp = {-INFINITY, -1, -INFINITY, 0x7FFFFFFF};
      } else {
        kept = st;
      }
      st = {-INFINITY, 0.0f};
    }
    uint4 x[kLoads];
    const uint32_t none = draft ? Vec<float>::kNone : Vec<T>::kNone;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int at = (threadIdx.x + u * kThreads) * 16;
      x[u] = at < sg.bytes ? *(const uint4*)(ring + s * kStageBytes + at)
                           : make_uint4(none, none, none, none);
    }
    float m;
    if (draft) {
      m = batch_stat<float>(x, k, st);
    } else if (heat > 0.0f) {
      m = batch_stat<T>(x, k, st);
    } else {
      m = fminf(Vec<T>::top(x), FLT_MAX);
      if (m > tp.m) {
        tp.m = m;
        tp.batch = sg.first;
      }
    }
    // given back only when every lane's loads have returned: the arrival hangs on a value (always
    // true) that is made from all of them
    if (__any_sync(0xFFFFFFFFu, m >= -INFINITY) && lane == 0)
      ptx::mbar_arrive(ptx::smem_u32(&sh.empty[s]));
    if (sg.kind & kOpens) {   // what no 16-byte vector holds: the row's head and end
      auto single = [&](auto* row) {
        using E = typename std::remove_const<typename std::remove_pointer<decltype(row)>::type>::type;
        const int head = head_of(row, a.V), rest = (a.V - head) % Vec<E>::N, i = threadIdx.x;
        const int v = c == 0 && i < head                                      ? i
                      : c == chunks - 1 && i >= 32 && i < 32 + rest ? a.V - rest + i - 32
                                                                    : -1;
        if (v < 0) return;
        const float l = read_logit(to_f(row[v]));
        if (heat == 0.0f) {
          tp.single = l;
          tp.single_id = v;
        } else {
          st = join(st, {l, l > -INFINITY ? 1.0f : 0.0f}, k);
        }
      };
      if (draft) single(a.draft + ((int64_t)n * (a.B - 1) + b) * a.ld_draft);
      else single((const T*)a.target + n * a.sn + b * a.sb);
    }
    if (!(sg.kind & kEnds)) continue;

    // the item's end: this warp's results go to the joining warp
    Stat t = draft ? kept : st, d = {0.0f, 1.0f};
    int top = 0x7FFFFFFF;
    if (heat > 0.0f) {
      t = warp_join(t, k);
      if (draft) d = warp_join(st, k);
    } else {
      m = fmaxf(tp.m, tp.single);
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const T* row = (const T*)a.target + n * a.sn + b * a.sb;
      int v0, v1;
      vectors_of(row, a.V, chunk, chunks, c, &v0, &v1);
      if (tp.m == m || tp.single == m) top = id_of(row, a.V, v1, tp, m);
      for (int o = 16; o > 0; o >>= 1) top = min(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      t = {m, m > -INFINITY ? 1.0f : 0.0f};
    }
    const int h = done % kItems;
    ok = ptx::mbar_wait(ptx::smem_u32(&sh.read[h]), ((done / kItems) & 1) ^ 1, abort, a.err);
    if (!__all_sync(0xFFFFFFFFu, ok)) break;
    ++done;
    if (lane == 0) {
      sh.stat[h][warp][0] = t;
      sh.stat[h][warp][1] = d;
      sh.top[h][warp] = top;
      if (warp == 0) sh.item[h] = sg.item;
      ptx::mbar_arrive(ptx::smem_u32(&sh.written[h]));
    }
    __syncwarp();
  }
}

// The race of one id is w / e with w = max(p - q, 0).  One pass takes an upper bound of it
// from quick exponentials and logarithms, and keeps each thread's highest bound and the one
// after it; the exact form, which alone counts, is computed for the highest, and for the
// others only where their bound reaches the best exact value of the CTA.
//  one row (TWO false): log2(p / e) + log2 s = (l - m) k - log2 e
//  two rows: (p (1 + d) - q (1 - d)) / e
// Both forms take the same rounded difference l - m (of p down to 2^-150) and scale it by factors
// that differ by 2^-22 at most: 4e-5 in the exponent.  `slack` = 2e-4 and d = 2^-14 cover that, and
// the errors of ex2, lg2 (2^-22 of |log2 e|) and expf.
struct Race {
  static constexpr float slack = 2e-4f;
  float inv_t, inv_s, m, inv_d, dm;    // dm, inv_d: the draft's, where it has a row
  float k, shift;
  int64_t x;                           // a one-hot draft's id, -1

  __device__ __forceinline__ void start(float heat, float tm, float ts) {
    inv_t = 1.0f / heat;
    inv_s = 1.0f / ts;
    m = tm;
    k = inv_t * kLog2e;
    shift = log2f(ts);
  }
  template <bool TWO>
  __device__ __forceinline__ float bound(float l, float d, float e) const {
    if (TWO) {
      constexpr float kMore = 1.0f + 1.0f / 16384, kLess = 1.0f - 1.0f / 16384;
      const float p = weight(l, k, m) * inv_s, q = weight(d, k, dm) * inv_d;
      return __fdividef(p * kMore - q * kLess, e) * kMore;
    }
    float lg;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(e));
    return fmaf(l - m, k, -lg);
  }
  // the bound that an exact value of `best` asks for
  template <bool TWO>
  __device__ __forceinline__ float asks(unsigned long long best) const {
    if (!best) return TWO ? 0.0f : -FLT_MAX;
    const float r = packed_val(best);
    return TWO ? r : log2f(r) + shift - slack;
  }
  template <bool TWO>
  __device__ __forceinline__ unsigned long long exact(float l, float d, float e, int v) const {
    const float p = share(l, m, inv_t) * inv_s;
    const float q = TWO ? share(d, dm, inv_t) * inv_d : v == x ? 1.0f : 0.0f;
    return p > q && (p - q) / e > 0.0f ? pack_best((p - q) / e, (uint32_t)v) : 0ull;
  }
};

// f(l, d, e, v) for this thread's ids of [lo, hi)
template <typename T, bool TWO, typename F>
__device__ __forceinline__ void each_id(const T* t_row, const float* d_row, const float* e_row, int lo,
                                        int hi, F&& f) {
  // vectors where all rows are on 16-byte boundaries from the same id on
  const bool wide = (((uintptr_t)(t_row + lo) | (uintptr_t)(e_row + lo) |
                      (TWO ? (uintptr_t)(d_row + lo) : 0)) & 15) == 0;
  int v = lo;
  if (wide) {
    constexpr int W = 8, TV = (int)sizeof(T) / 2;
    const int vecs = (hi - lo) / W;
#pragma unroll 2
    for (int i = threadIdx.x; i < vecs; i += kThreads) {
      const int at = lo + i * W;
      uint4 tx[TV], ex[2], dx[2];
#pragma unroll
      for (int u = 0; u < TV; ++u) tx[u] = __ldcs((const uint4*)(t_row + at) + u);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        ex[u] = __ldcs((const uint4*)(e_row + at) + u);
        if (TWO) dx[u] = __ldcs((const uint4*)(d_row + at) + u);
      }
#pragma unroll
      for (int e = 0; e < W; ++e)
        f(element<T>(tx[e / Vec<T>::N], e % Vec<T>::N), TWO ? element<float>(dx[e / 4], e % 4) : 0.0f,
          element<float>(ex[e / 4], e % 4), at + e);
    }
    v = lo + vecs * W;
  }
  for (v += (int)threadIdx.x; v < hi; v += kThreads)
    f(to_f(t_row[v]), TWO ? d_row[v] : 0.0f, e_row[v], v);
}

// the race of ids [lo, hi) over the CTA: every thread gets the best, 0 when no weight is positive
template <typename T, bool TWO>
__device__ unsigned long long race(const Race& r, const T* t_row, const float* d_row,
                                   const float* e_row, int lo, int hi, unsigned long long* s_best) {
  float top = -INFINITY, second = -INFINITY;
  int at = -1;
  each_id<T, TWO>(t_row, d_row, e_row, lo, hi, [&](float l, float d, float e, int v) {
    const float u = r.bound<TWO>(l, d, e);   // NaN: no
    const bool more = u > top;
    second = fmaxf(second, more ? top : u);
    top = more ? u : top;
    at = more ? v : at;
  });
  if (threadIdx.x == 0) *s_best = 0;
  __syncthreads();
  unsigned long long best = 0;
  if (at >= 0) best = r.exact<TWO>(to_f(t_row[at]), TWO ? d_row[at] : 0.0f, e_row[at], at);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
  if ((threadIdx.x & 31) == 0 && best) atomicMax(s_best, best);
  __syncthreads();
  best = *s_best;
  const float asked = r.asks<TWO>(best);
  __syncthreads();
  if (second >= asked) {   // rare: another of this thread's ids may be the one
    each_id<T, TWO>(t_row, d_row, e_row, lo, hi, [&](float l, float d, float e, int v) {
      if (r.bound<TWO>(l, d, e) >= asked) best = max(best, r.exact<TWO>(l, d, e, v));
    });
    if (best) atomicMax(s_best, best);
  }
  __syncthreads();
  best = *s_best;
  __syncthreads();
  return best;
}

// Work items (block, chunk): the race of every id of the chunk, merged into the block's best;
// the block's last chunk writes its tokens and clears its counters for the next call.
// Bound by its loads, at 71% of HBM's rate: 224 blocks' target row and noise, 220 MB read in 46 us
// (4.8 TB/s) with five CTAs an SM and items of 32768 ids (3 us more with the four that its registers
// would leave; 8192, 16384 and 65536 ids: 4, 1 and 5 us more).  Where few blocks would leave SMs idle
// an item is down to 2048 ids.
template <typename T>
__global__ void __launch_bounds__(kThreads, 5) verify_draw_kernel(const xp_verify_args a, int chunk) {
  __shared__ unsigned long long s_best;
  __shared__ int s_last;
  ptx::pdl_wait();
  const int n = blockIdx.y;
  if (blockIdx.x == 0 && n == 0 && threadIdx.x == 0) *a.next = 0;
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
    r.start(heat, tm, a.row[row * 5 + 1]);
    r.x = rejected && !a.draft ? a.blk[(int64_t)n * a.B + 1 + end] : -1;
    const float dm = a.row[row * 5 + 2];
    const bool two = a.draft && rejected && dm > -INFINITY;
    const float* d_row = two ? a.draft + ((int64_t)n * (a.B - 1) + end) * a.ld_draft : nullptr;
    const int lo = blockIdx.x * chunk, hi = min(a.V, lo + chunk);
    unsigned long long best;
    if (two) {
      r.inv_d = 1.0f / a.row[row * 5 + 3];
      r.dm = dm;
      best = race<T, true>(r, t_row, d_row, e_row, lo, hi, &s_best);
    } else {
      best = race<T, false>(r, t_row, nullptr, e_row, lo, hi, &s_best);
    }
    if (threadIdx.x == 0 && best) atomicMax(&a.packed[n], best);
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
      best = race<T, false>(r, t_row, nullptr, e_row, 0, a.V, &s_best);
    }
    if (best) last = packed_idx(best);
    else if (threadIdx.x == 0) atomicOr(a.err, XP_ERR_EMPTY);   // noise that lets no id win
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

// Vocabulary ids of one work item of `workers` that share `rows` rows: from `most` down to
// `least` where few rows would leave workers idle.
int chunk_of(int64_t rows, int V, int64_t workers, int most, int least) {
  int chunk = most;
  while (chunk > least && rows * ((V + chunk - 1) / chunk) < workers) chunk /= 2;
  return chunk;
}
constexpr int kMostIds = 65536, kLeastIds = 8192;
constexpr int kMostRace = 32768, kLeastRace = 2048;

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
  L.next = take(4);
  L.part = take(rows * (((size_t)h->V + kLeastIds - 1) / kLeastIds) * 20);
  L.row = take(rows * 20);
  L.total = o;
  return L;
}

template <typename T>
static cudaError_t launch_verify(const xp_head* h, const xp_verify_args& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.N * a.B, ctas = (int64_t)h->num_sms * kResident;
  // a batch of requests rarely needs the rows of more than a few slots
  const int chunk =
      chunk_of(std::min<int64_t>(rows, (int64_t)a.N * 4), a.V, ctas * 3 / 2, kMostIds, kLeastIds);
  const int chunks = (a.V + chunk - 1) / chunk;
  if (rows * chunks > INT_MAX / 2) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)std::min(rows * chunks, ctas);
  const int smem = kStages * kStageBytes;
  static unsigned long long allowed = 0;
  const cudaError_t f = xp_allow_smem((const void*)verify_stats_kernel<T>, smem, &allowed);
  if (f != cudaSuccess) return f;
  verify_stats_kernel<T><<<grid, kThreads + 64, smem, s>>>(a, chunk, chunks);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int race = chunk_of(a.N, a.V, (int64_t)h->num_sms * 4, kMostRace, kLeastRace);
  return xp_launch_pdl(verify_draw_kernel<T>, dim3((a.V + race - 1) / race, a.N), dim3(kThreads), 0, s,
                       a, race);
}

cudaError_t xp_launch_verify(const xp_head* h, const xp_verify_args& a, cudaStream_t s) {
  return h->dtype == XP_BF16 ? launch_verify<bf16>(h, a, s) : launch_verify<float>(h, a, s);
}
