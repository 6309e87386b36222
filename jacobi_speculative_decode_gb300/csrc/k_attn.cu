// Shared-prefix attention on plain CUDA cores (fp32 caches, and shapes the tensor-core
// kernel does not tile), and the kernel that joins partial results.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "sm100_ptx.cuh"
#include "xp_device.cuh"

using namespace xpd;
typedef __nv_bfloat16 bf16;

namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 64;    // keys of one step

// query row r of a tile -> its (sequence, token, head within the group); false behind the end
struct Row {
  int n, t, j;
};
__device__ __forceinline__ bool row_of(const xp_attn_args& g, bool prefix, int tile, int r, int n,
                                       int rows_tile, Row* out) {
  const int i = tile * rows_tile + r;
  const int per_seq = g.a.T * g.group;
  if (i >= (prefix ? g.a.N * per_seq : per_seq)) return false;
  out->n = prefix ? i / per_seq : n;
  out->t = i % per_seq / g.group;
  out->j = i % g.group;
  return true;
}

// four consecutive elements as floats; wide: 16 (fp32) or 8 (bf16) bytes at once
__device__ __forceinline__ float4 load4(const float* p, bool wide, int n) {
  if (wide) return *(const float4*)p;
  return make_float4(p[0], n > 1 ? p[1] : 0.0f, n > 2 ? p[2] : 0.0f, n > 3 ? p[3] : 0.0f);
}
__device__ __forceinline__ float4 load4(const bf16* p, bool wide, int n) {
  if (wide) {
    const uint2 v = *(const uint2*)p;
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
  }
  return make_float4(to_f(p[0]), n > 1 ? to_f(p[1]) : 0.0f, n > 2 ? to_f(p[2]) : 0.0f,
                     n > 3 ? to_f(p[3]) : 0.0f);
}

// A CTA holds BM query rows and walks over its keys 64 at a time: scores from shared memory (RM
// x 4 a thread), one pass of the softmax in base 2 with a running maximum and sum, weights times
// values.  A warp loads eight keys and values at once, a lane four dims.
// Large calls wait for shared memory: 64 rows a CTA leave 8 warps an SM, which issue in 57% of the
// cycles with that pipe 59% and the multiply-adds 44% busy.  32 blocks of 16 tokens, 32 heads of 128
// over 8, prefix 8192, tails up to 1500, fp32: 2,646 us, 28.8 TFLOP/s, 36% of 152 SMs' fp32 rate;
// bf16 of heads that the tensor cores' form does not take is no faster (heads of 96: 18.4, pages of
// 20 tokens: 23.9).  Small ones are bound by the latency of a step's loads (page ids, then keys and
// values), so key ranges are as short as one step of 64 keys until two CTAs an SM have work:
// 7 sequences of 5 tokens, 12 heads of 96 over 3, prefix 1001, tails up to 333: 33.3 us both kernels
// (84 with loads of single elements and longer ranges).
template <typename T, int RM, int NC>
__global__ void __launch_bounds__(kThreads, RM <= 2 ? 2 : 1) attn_simt_kernel(const xp_attn_args g,
                                                             bool wide) {
  constexpr int BM = 16 * RM;
  extern __shared__ __align__(16) float smem[];
  const int D = g.dim, DP = (D + 3) / 4 * 4, LD = DP + 4;
  float* sq = smem;                      // [BM][LD]
  float* sk = sq + BM * LD;              // [kKeys][LD]
  float* sv = sk + kKeys * LD;           // [kKeys][DP]; dims behind a row's end: the next row's, or sp
  float* sp = sv + kKeys * DP;           // [BM][kKeys + 4]
  constexpr int LP = kKeys + 4;
  __shared__ int s_limit[BM];            // keys each row sees
  __shared__ int64_t s_at[kKeys];        // where each key begins in the pools, -1 behind the range

  const xp_attn_plan& pl = g.plan;
  const int hk = blockIdx.y, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
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
      if (tid == 0) atomicOr(g.err, XP_ERR_LENGTH);
      keys = keys < 0 ? 0 : g.a.max_len;
    }
  }
  const int step = prefix ? pl.prefix_keys : pl.tail_keys;
  const int k0 = split * step, k1 = k0 + min(step, keys - k0);   // none where keys < k0

  for (int i = tid; i < BM; i += kThreads) {
    Row r;
    int lim = 0;
    if (row_of(g, prefix, tile, i, n, BM, &r)) lim = prefix ? keys : keys - g.a.T + r.t + 1;
    s_limit[i] = min(lim, k1);
  }
  // queries, scaled so that the softmax runs in base 2
  const float scale = g.a.scale * 1.44269504088896f;
  for (int r = tid >> 5; r < BM; r += kThreads / 32) {
    Row w;
    const bool is_row = row_of(g, prefix, tile, r, n, BM, &w);
    const T* src = is_row ? (const T*)g.q + w.n * g.a.q_stride_n + w.t * g.a.q_stride_t +
                                (int64_t)(hk * g.group + w.j) * g.a.q_stride_h
                          : nullptr;
    for (int d = tid & 31; d < LD; d += 32) sq[r * LD + d] = is_row && d < D ? to_f(src[d]) * scale : 0.0f;
  }
  float o[RM][NC * 4], m[RM], l[RM];
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.0f;
#pragma unroll
    for (int c = 0; c < NC * 4; ++c) o[i][c] = 0.0f;
  }

  for (int kb = k0; kb < k1; kb += kKeys) {
    __syncthreads();
    if (tid < kKeys) {
      int64_t at = -1;
      if (kb + tid < k1) {
        const int key = kb + tid, page = key / g.page_size;
        int p = table[page];
        if (p < 0 || p >= g.pages) {
          atomicOr(g.err, XP_ERR_BADPAGE);
          p = p < 0 ? 0 : g.pages - 1;
        }
        at = p * g.kv_page + (key - page * g.page_size) * g.kv_token + hk * g.kv_head;
      }
      s_at[tid] = at;
    }
    __syncthreads();
    for (int d = (tid & 31) * 4; d < DP; d += 128) {
      float4 kx[kKeys / 8], vx[kKeys / 8];
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i) {
        const int64_t at = s_at[(tid >> 5) + 8 * i];
        kx[i] = vx[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (at >= 0) {   // tokens behind the length are not read
          kx[i] = load4((const T*)g.k + at + d, wide, D - d);
          vx[i] = load4((const T*)g.v + at + d, wide, D - d);
        }
      }
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i) {
        const int j = (tid >> 5) + 8 * i;
        *(float4*)&sk[j * LD + d] = kx[i];
        *(float4*)&sv[j * DP + d] = vx[i];
      }
    }
    __syncthreads();
    // scores: rows ty*RM.., keys tx + 16 j
    float s[RM][4];
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
    for (int d = 0; d < DP; d += 4) {
      float4 qa[RM], ka[4];
#pragma unroll
      for (int i = 0; i < RM; ++i) qa[i] = *(const float4*)&sq[(ty * RM + i) * LD + d];
#pragma unroll
      for (int j = 0; j < 4; ++j) ka[j] = *(const float4*)&sk[(tx + 16 * j) * LD + d];
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = fmaf(qa[i].x, ka[j].x, s[i][j]);
          s[i][j] = fmaf(qa[i].y, ka[j].y, s[i][j]);
          s[i][j] = fmaf(qa[i].z, ka[j].z, s[i][j]);
          s[i][j] = fmaf(qa[i].w, ka[j].w, s[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int lim = s_limit[ty * RM + i];
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kb + tx + 16 * j >= lim) s[i][j] = -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
      const float now = fmaxf(m[i], top);
      const float base = now == -INFINITY ? 0.0f : now;   // a row that sees none of these keys
      const float keep = exp2f(m[i] - base);
      m[i] = now;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[i][j] - base);
        sp[(ty * RM + i) * LP + tx + 16 * j] = e;
        sum += e;
      }
      l[i] = l[i] * keep + sum;   // this thread's keys only
#pragma unroll
      for (int c = 0; c < NC * 4; ++c) o[i][c] *= keep;
    }
    __syncwarp();   // a row's 16 threads are in one warp
    // weights times values: dims 4 tx + 64 c.  Where the mask hides keys of this step from some
    // rows, a hidden key's value is left out, not multiplied by zero: it may be infinite or NaN.
    auto add = [&](auto some_hidden) {
      for (int j = 0; j < kKeys; j += 4) {
        float pa[RM][4];
#pragma unroll
        for (int i = 0; i < RM; ++i) {
          const float4 x = *(const float4*)&sp[(ty * RM + i) * LP + j];
          pa[i][0] = x.x; pa[i][1] = x.y; pa[i][2] = x.z; pa[i][3] = x.w;
        }
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float4 x = *(const float4*)&sv[(j + jj) * DP + c * 64 + tx * 4];
#pragma unroll
            for (int i = 0; i < RM; ++i) {
              if (decltype(some_hidden)::value && kb + j + jj >= s_limit[ty * RM + i]) continue;
              o[i][c * 4 + 0] = fmaf(pa[i][jj], x.x, o[i][c * 4 + 0]);
              o[i][c * 4 + 1] = fmaf(pa[i][jj], x.y, o[i][c * 4 + 1]);
              o[i][c * 4 + 2] = fmaf(pa[i][jj], x.z, o[i][c * 4 + 2]);
              o[i][c * 4 + 3] = fmaf(pa[i][jj], x.w, o[i][c * 4 + 3]);
            }
          }
      }
    };
    if (prefix || kb + kKeys <= keys - g.a.T + 1)
      add(std::false_type());
    else
      add(std::true_type());
  }
  const int64_t rows = (int64_t)g.a.N * g.a.T * g.a.heads;
#pragma unroll
  for (int i = 0; i < RM; ++i) {
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], x);
    Row w;
    if (!row_of(g, prefix, tile, ty * RM + i, n, BM, &w)) continue;
    const int64_t row = ((int64_t)w.n * g.a.T + w.t) * g.a.heads + hk * g.group + w.j;
    if (tx == 0) {
      g.stat[(part * rows + row) * 2] = m[i];
      g.stat[(part * rows + row) * 2 + 1] = l[i];
    }
    float* acc = g.acc + (part * rows + row) * D;
    if (l[i] != 0.0f) {   // NaN where a visible score is
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c * 64 + tx * 4 + e < D) acc[c * 64 + tx * 4 + e] = o[i][c * 4 + e];
    }
  }
}

// One warp a query row: partial results (maximum, sum, weighted values) of all its key
// ranges, brought to a common maximum.  Bound by the latency of its two rounds of loads: 5 us for
// the 420 rows above.  out = sum_p a_p O_p / sum_p a_p l_p, a_p = 2^(m_p - m).
template <typename T>
__global__ void __launch_bounds__(256) attn_combine_kernel(const xp_attn_args g) {
  ptx::pdl_wait();
  const int64_t rows = (int64_t)g.a.N * g.a.T * g.a.heads;
  const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31, parts = g.plan.parts, D = g.dim;
  if (row >= rows) return;
  float m = -INFINITY;
  for (int p = lane; p < parts; p += 32) {
    const float2 st = *(const float2*)&g.stat[(p * rows + row) * 2];
    if (st.y != 0.0f) m = fmaxf(m, st.x);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
  float o[8], l = 0.0f;
#pragma unroll
  for (int c = 0; c < 8; ++c) o[c] = 0.0f;
  for (int p0 = 0; p0 < parts; p0 += 32) {   // a lane a range's weight, then all ranges' results
    float2 st = make_float2(0.0f, 0.0f);
    if (p0 + lane < parts) st = *(const float2*)&g.stat[((p0 + lane) * rows + row) * 2];
    // 0: no key of this range.  A weight that underflows is the least number instead, so that an
    // infinite or NaN result still shows.
    const float mine = st.y != 0.0f ? fmaxf(exp2f(st.x - m), 1.4e-45f) : 0.0f;
    l += mine * st.y;
    const int n = min(32, parts - p0);
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
      const float w = __shfl_sync(0xFFFFFFFFu, mine, p);
      const float* acc = g.acc + ((p0 + p) * rows + row) * D;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (w != 0.0f && c * 32 + lane < D) o[c] = fmaf(w, acc[c * 32 + lane], o[c]);
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
  const int h = (int)(row % g.a.heads), t = (int)(row / g.a.heads % g.a.T);
  const int n = (int)(row / g.a.heads / g.a.T);
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  T* out = (T*)g.out + n * g.a.o_stride_n + t * g.a.o_stride_t + h * g.a.o_stride_h;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (c * 32 + lane < D) out[c * 32 + lane] = from_f<T>(o[c] * inv);
  if (lane == 0 && g.lse) g.lse[row] = l != 0.0f ? (m + log2f(l)) * 0.693147180559945f : -INFINITY;
}

size_t simt_smem(int rm, int D) {
  const int DP = (D + 3) / 4 * 4, LD = DP + 4, BM = 16 * rm;
  return sizeof(float) * ((size_t)BM * LD + kKeys * LD + kKeys * DP + BM * (kKeys + 4));
}

template <typename T, int RM, int NC>
cudaError_t launch(const xp_attn_args& g, cudaStream_t s) {
  const size_t smem = simt_smem(RM, g.dim);
  // the widest head of this instantiation, so that one call covers them all
  static unsigned long long allowed = 0;
  const cudaError_t e = xp_allow_smem((const void*)attn_simt_kernel<T, RM, NC>,
                                      simt_smem(RM, NC * 64), &allowed);
  if (e != cudaSuccess) return e;
  const xp_attn_plan& p = g.plan;
  const dim3 grid(p.prefix_tiles * p.prefix_splits + g.a.N * p.tail_tiles * p.tail_splits,
                  g.kv_heads);
  const uint64_t unit = 4 * sizeof(T);
  const bool wide = g.dim % 4 == 0 && ((uintptr_t)g.k | (uintptr_t)g.v | (uint64_t)g.kv_page * sizeof(T) |
                                       (uint64_t)g.kv_token * sizeof(T) |
                                       (uint64_t)g.kv_head * sizeof(T)) % unit == 0;
  attn_simt_kernel<T, RM, NC><<<grid, kThreads, smem, s>>>(g, wide);
  return cudaGetLastError();
}
template <typename T, int RM>
cudaError_t launch_nc(const xp_attn_args& g, cudaStream_t s) {
  switch ((g.dim + 63) / 64) {
    case 1: return launch<T, RM, 1>(g, s);
    case 2: return launch<T, RM, 2>(g, s);
    case 3: return launch<T, RM, 3>(g, s);
    default: return launch<T, RM, 4>(g, s);
  }
}

}  // namespace

// Row tiles of 16, 32 or 64 query rows, the least that hold a sequence's rows of one kv head: a
// tile's keys are read once for all its rows, and rows that are not there cost as much as rows that
// are.  Key ranges so that about two CTAs an SM have work.
xp_attn_plan xp_attn_simt_plan(const xp_cache* c, const xp_attn* a) {
  xp_attn_plan p = {};
  const int group = a->heads / c->d.kv_heads, per_seq = a->T * group;
  p.rows_tile = per_seq > 32 ? 64 : per_seq > 16 ? 32 : 16;
  const int64_t want = (int64_t)c->num_sms * 2;
  // both sources share the CTAs by their keys; a range is a whole number of steps
  const int64_t all_steps =
      (((int64_t)a->N * per_seq + p.rows_tile - 1) / p.rows_tile * ((a->prefix_len + kKeys - 1) / kKeys) +
       (int64_t)a->N * ((per_seq + p.rows_tile - 1) / p.rows_tile) * ((a->max_len + kKeys - 1) / kKeys)) *
      c->d.kv_heads;
  const int64_t steps = std::max<int64_t>(1, (all_steps + want - 1) / want);
  auto splits = [&](int keys, int* range) {
    const int64_t r = std::min<int64_t>(steps * kKeys, ((int64_t)keys + kKeys - 1) / kKeys * kKeys);
    *range = (int)std::max<int64_t>(kKeys, r);
    return keys > 0 ? (keys - 1) / *range + 1 : 0;
  };
  p.prefix_tiles = (int)(((int64_t)a->N * per_seq + p.rows_tile - 1) / p.rows_tile);
  p.tail_tiles = (per_seq + p.rows_tile - 1) / p.rows_tile;
  p.prefix_splits = splits(a->prefix_len, &p.prefix_keys);
  p.tail_splits = splits(a->max_len, &p.tail_keys);
  p.parts = p.prefix_splits + p.tail_splits;
  return p;
}

cudaError_t xp_launch_attn_simt(const xp_cache* c, const xp_attn_args& g, cudaStream_t s) {
  if (g.plan.parts == 0) return cudaSuccess;
  const int rm = g.plan.rows_tile / 16;
  if (c->d.dtype == XP_BF16)
    return rm == 1 ? launch_nc<bf16, 1>(g, s) : rm == 2 ? launch_nc<bf16, 2>(g, s) : launch_nc<bf16, 4>(g, s);
  return rm == 1 ? launch_nc<float, 1>(g, s) : rm == 2 ? launch_nc<float, 2>(g, s) : launch_nc<float, 4>(g, s);
}

cudaError_t xp_launch_attn_combine(const xp_attn_args& g, cudaStream_t s) {
  const int64_t rows = (int64_t)g.a.N * g.a.T * g.a.heads;
  const dim3 grid((unsigned)((rows + 7) / 8)), block(256);
  return g.a.dtype == XP_BF16 ? xp_launch_pdl(attn_combine_kernel<bf16>, grid, block, 0, s, g)
                               : xp_launch_pdl(attn_combine_kernel<float>, grid, block, 0, s, g);
}
