// Rows into a quantised cache, and rows of any cache back out.
//
// A CTA takes kTokens tokens of one sequence and finds their pages once; a thread is one piece of a token's
// row (8 dims of K or V written, 16 bytes of them read) and walks over the tokens, so that nothing is divided
// inside.  8 prompts of 4096 tokens, 8 heads of 128, fp32 in 8 bits: written in 64 us (340 MB, 5.3 TB/s, between
// HBM and what quantising costs), read back in 62 (5.5 TB/s, 81% of measured); 32 sequences to 3000 tokens out of 4
// bits as bf16 75 us, 6.0 TB/s, 88%.  Rows of bf16 are half the bytes and more instructions, 79 us of 30 that their
// bytes take: they are widened to fp32 and quantised element by element as those are.
#include <algorithm>

#include "quant.cuh"
#include "xp_device.cuh"

using namespace xpd;
typedef __nv_bfloat16 bf16;

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;

struct RowArgs {
  char *kp, *vp;                // this layer's pools
  int64_t page, token, head;    // strides: bytes of a quantised pool, elements of another
  int scale_at, scale;          // quantised: where a head's scales begin, and a token's bytes of them
  void *k, *v;                  // the dense rows
  int64_t sn, st, sh;
  const int32_t* table;
  int64_t ld, width;
  const int32_t *lens, *first;
  int N, T, H, D, ps, pages;
  uint32_t* err;
};

// Where the CTA's tokens lie: their page's beginning (-1: nowhere) and place in the page.  `len`: the
// sequence's end.
struct Places {
  int64_t page[kTokens];
  int at[kTokens];
};
__device__ __forceinline__ void find_pages(const RowArgs& a, int n, int t0, int64_t pos0, int64_t len,
                                           Places* s) {
  if (threadIdx.x < kTokens) {
    const int t = t0 + (int)threadIdx.x;
    const int64_t pos = pos0 + t;
    int page = -1, at = 0;
    if (t < a.T && pos >= 0 && pos < len) {
      const int64_t col = pos / a.ps;
      at = (int)(pos - col * a.ps);
      if (col >= a.width) {
        atomicOr(a.err, XP_ERR_LENGTH);
      } else {
        page = a.table[n * a.ld + col];
        if (page < 0 || page >= a.pages) {
          atomicOr(a.err, XP_ERR_BADPAGE);
          page = -1;
        }
      }
    }
    s->page[threadIdx.x] = page < 0 ? -1 : page * a.page;
    s->at[threadIdx.x] = at;
  }
  __syncthreads();
}

template <typename T> struct Piece {              // elements of 16 bytes
  static constexpr int N = 16 / sizeof(T);
};
// 8 consecutive elements; wide: from a 16-byte boundary
template <typename T> struct Eight {
  uint4 v[8 / Piece<T>::N];
  __device__ __forceinline__ void load(const T* p, bool wide) {
    if (wide) {
#pragma unroll
      for (int i = 0; i < 8 / Piece<T>::N; ++i) v[i] = __ldcs((const uint4*)p + i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) ((T*)v)[i] = p[i];
    }
  }
};
__device__ __forceinline__ void floats_of(const Eight<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.v[i].x), x[4 * i + 1] = __uint_as_float(r.v[i].y);
    x[4 * i + 2] = __uint_as_float(r.v[i].z), x[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}
__device__ __forceinline__ void floats_of(const Eight<bf16>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN where either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float reciprocal(float x) {   // nearly
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// tokens of a thread whose loads are on their way together; to append, the next while one is quantised (both calls
// of the prompts 126 us, 128 with two and two together; with four, which leave two CTAs an SM, 8 us more)
constexpr int kAppendBatch = 2, kReadBatch = 4;

// What a thread does of a row: piece `e` of head `h` of K or V, for every lanes-th token from `lane` on.
struct Part {
  int e, h, is_v, lane, lanes;
};
template <typename F> __device__ __forceinline__ void for_parts(const RowArgs& a, int elements, F f) {
  const int pieces = (a.D + elements - 1) / elements, units = 2 * a.H * pieces;
  Part p;
  p.lanes = max(1, kThreads / units);   // tokens at once where a row is short
  p.lane = units < kThreads ? threadIdx.x / units : 0;
  if (p.lane >= p.lanes) return;
  for (int u = units < kThreads ? threadIdx.x % units : threadIdx.x; u < units; u += kThreads) {
    p.e = u % pieces * elements;
    p.h = u / pieces % a.H;
    p.is_v = u / pieces / a.H;
    f(p);
  }
}

// ---------------------------------------------------------------------------
// Quantised append.  A thread has 8 dims, and its neighbour the other 8 of their scale: with 4, as 16-byte loads
// would have it of fp32, what a scale costs is too much (the prompts above took 102 us and not 80).
// ---------------------------------------------------------------------------
template <int BITS, typename T>
__global__ void __launch_bounds__(kThreads, 4) append_quant_kernel(const RowArgs a, bool wide) {
  __shared__ Places s;
  const int chunks = (a.T + kTokens - 1) / kTokens;
  const int n = blockIdx.x / chunks, t0 = (int)(blockIdx.x % chunks) * kTokens;
  find_pages(a, n, t0, (int64_t)a.lens[n] - a.T, INT64_MAX, &s);

  const int count = min(kTokens, a.T - t0);
  const unsigned both = 3u << (threadIdx.x & 30);   // the two of a group: rows are a whole number of groups
  for_parts(a, 8, [&](const Part& part) {
    const T* from = (const T*)(part.is_v ? a.v : a.k) + n * a.sn + t0 * a.st + part.h * a.sh + part.e;
    char* pool = (part.is_v ? a.vp : a.kp) + part.h * a.head;
    const int g = part.e / 16;
    Eight<T> raw[kAppendBatch];
    int64_t page[kAppendBatch];
    auto load = [&](int k, int i) {
      page[k] = i < count ? s.page[i] : -1;
      if (page[k] >= 0) raw[k].load(from + i * a.st, wide);
    };
#pragma unroll
    for (int k = 0; k < kAppendBatch; ++k) load(k, part.lane + k * part.lanes);
    for (int i0 = part.lane; i0 < count; i0 += kAppendBatch * part.lanes) {
#pragma unroll
      for (int k = 0; k < kAppendBatch; ++k) {
        const int64_t to_page = page[k];
        float x[8], top = 0.0f;
        floats_of(raw[k], x);
        load(k, i0 + (k + kAppendBatch) * part.lanes);
        if (to_page < 0) continue;   // the same in both
        const int at = s.at[i0 + k * part.lanes];
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max_nan(top, fabsf(x[j]));
        top = max_nan(top, __shfl_xor_sync(both, top, 1));
        if (top != top) {   // a NaN is held as 0
          top = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] = x[j] != x[j] ? 0.0f : x[j];
            top = fmaxf(top, fabsf(x[j]));
          }
          top = fmaxf(top, __shfl_xor_sync(both, top, 1));
          atomicOr(a.err, XP_ERR_RANGE);
        }
        bool over;
        const unsigned b = xpq::scale_byte<BITS>(top, &over);
        const float step = xpq::scale_of(b), r = b ? reciprocal(step) : 0.0f;   // b = 0: all are 0
        if (over) {
          const float most = xpq::Codes<BITS>::kMost * step;
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = fminf(fmaxf(x[j], -most), most);
          atomicOr(a.err, XP_ERR_RANGE);
        }
        char* head = pool + to_page;
        char* scale = head + a.scale_at + at * a.scale;
        if (part.e % 16 == 0) scale[g] = (char)b;
        if (part.e + 8 == a.D)   // the padding behind the scales
          for (int p = g + 1; p < a.scale; ++p) scale[p] = 0;
        uint32_t c[8];
        xpq::codes_of<BITS>(x, step, r, c);
        char* to = head + at * a.token + part.e / 8 * BITS;
        if constexpr (BITS == 8) {
          *(uint2*)to = make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
        } else {
          uint32_t w = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) w |= c[j] << (j / 2 + j % 2 * 4) * 4;
          *(uint32_t*)to = w;
        }
      }
    }
  });
}

// ---------------------------------------------------------------------------
// Read back: BITS of a code, or 16 / 32 for a cache of bf16 / fp32.  Those are read one element a load, as their
// strides may be any: the prompts above out of bf16 as bf16 55 us of 40, out of fp32 as fp32 99 of 79.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void store(float* p, bool wide, const float (&x)[4], int n) {
  if (wide) {
    __stcs((float4*)p, make_float4(x[0], x[1], x[2], x[3]));
  } else {
    for (int i = 0; i < n; ++i) p[i] = x[i];
  }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *(const uint32_t*)&v;
}
__device__ __forceinline__ void store(bf16* p, bool wide, const float (&x)[8], int n) {
  if (wide) {
    __stcs((uint4*)p, make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])));
  } else {
    for (int i = 0; i < n; ++i) p[i] = from_f<bf16>(x[i]);
  }
}
// N pairs of codes times a scale, two dims an operation and exactly: 1024 + c is an fp16 number with c in its
// last bits.  4 bits: pair j is nibbles j and j + 4 of w.x; 8 bits: bytes 2j and 2j + 1 of w.
template <int BITS, int N>
__device__ __forceinline__ void widen(uint2 w, unsigned scale, __half2 (&out)[N]) {
  const uint32_t s = scale * 0x00800080u, zero = BITS == 4 ? 0xE408E408u : 0xE480E480u;   // -1024 - 8, -1024 - 128
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t pair = BITS == 4 ? (w.x >> 4 * j & 0x000F000Fu) | 0x64006400u
                                    : __byte_perm(j < 2 ? w.x : w.y, 0x64646464u, j % 2 ? 0x4342 : 0x4140);
    out[j] = __hmul2(__hadd2(*(const __half2*)&pair, *(const __half2*)&zero), *(const __half2*)&s);
  }
}

// 8 codes of 4 bits as bf16: 128 + c is a bf16 number with c in its last bits
__device__ __forceinline__ uint4 widen_bf16(uint32_t w, unsigned scale) {
  const __nv_bfloat162 s = __float2bfloat162_rn(xpq::scale_of(scale)), zero = __float2bfloat162_rn(-136.0f);
  uint32_t out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t pair = (w >> 4 * j & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 v = __hmul2(__hadd2(*(const __nv_bfloat162*)&pair, zero), s);
    out[j] = *(const uint32_t*)&v;
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int BITS, typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(const RowArgs a, bool wide) {
  constexpr int E = Piece<T>::N;
  __shared__ Places s;
  const int chunks = (a.T + kTokens - 1) / kTokens;
  const int n = blockIdx.x / chunks, t0 = (int)(blockIdx.x % chunks) * kTokens;
  find_pages(a, n, t0, a.first ? a.first[n] : 0, a.lens[n], &s);

  const int count = min(kTokens, a.T - t0);
  for_parts(a, E, [&](const Part& part) {
    const int e = part.e, live = min(E, a.D - e);
    T* to = (T*)(part.is_v ? a.v : a.k) + n * a.sn + t0 * a.st + part.h * a.sh + e;
    const char* pool = part.is_v ? a.vp : a.kp;
    if (BITS <= 8) pool += part.h * a.head;
    for (int i0 = part.lane; i0 < count; i0 += kReadBatch * part.lanes) {
      if constexpr (BITS <= 8) {
        uint2 code[kReadBatch];
        unsigned scale[kReadBatch];
#pragma unroll
        for (int k = 0; k < kReadBatch; ++k) {
          const int i = i0 + k * part.lanes;
          const int64_t page = i < count ? s.page[i] : -1;
          code[k] = make_uint2(0, 0);
          scale[k] = 0;   // what lies nowhere reads as 0
          if (page >= 0) {
            const char* head = pool + page;
            scale[k] = (uint8_t)head[a.scale_at + s.at[i] * a.scale + e / 16];
            const char* from = head + s.at[i] * a.token + e / 8 * BITS;
            if constexpr (BITS == 4) code[k].x = *(const uint32_t*)from >> e % 8 * 2;   // fp32: the first four or the last
            else if constexpr (E == 4) code[k].x = *(const uint32_t*)(from + e % 8);
            else code[k] = *(const uint2*)from;
          }
        }
#pragma unroll
        for (int k = 0; k < kReadBatch; ++k) {
          if (i0 + k * part.lanes >= count) break;
          if constexpr (BITS == 4 && E == 8) {   // c s is exact in bf16 too: no way by fp32
            if (wide) {
              __stcs((uint4*)(to + (i0 + k * part.lanes) * a.st), widen_bf16(code[k].x, scale[k]));
              continue;
            }
          }
          __half2 v[E / 2];
          widen<BITS>(code[k], scale[k], v);
          float x[E];
#pragma unroll
          for (int j = 0; j < E / 2; ++j) {
            const float2 f = __half22float2(v[j]);
            x[2 * j] = f.x, x[2 * j + 1] = f.y;
          }
          store(to + (i0 + k * part.lanes) * a.st, wide, x, live);
        }
      } else {
#pragma unroll
        for (int k = 0; k < kReadBatch; ++k) {
          const int i = i0 + k * part.lanes;
          if (i >= count) break;
          float x[E] = {};
          if (s.page[i] >= 0) {
            const int64_t at = s.page[i] + s.at[i] * a.token + part.h * a.head + e;
#pragma unroll
            for (int j = 0; j < E; ++j)
              if (j < live) x[j] = BITS == 16 ? to_f(((const bf16*)pool)[at + j]) : ((const float*)pool)[at + j];
          }
          store(to + i * a.st, wide, x, live);
        }
      }
    }
  });
}

// ---------------------------------------------------------------------------
// A quantised cache's tokens as fp16 (exactly) for attention on tcgen05, which many queries of each key are
// better done by: pools [head][page of kWidePage tokens][dim] and the table that names their pages in order.
// Behind a sequence's end its last page is zeros.  A CTA is 32 tokens of a head.  Bound by what it writes: 8192 and 32
// times 17 to 1500 tokens, 8 heads of 128 in 8 bits, 70 MB in, 135 out to L2 and past it, 33 us (64 tokens a CTA 1 us
// more, 128 5 us).  The CTAs behind the pages' make the queries fp16, a warp a row, scaled by the power of two that
// brings the row's largest into [1, 4).
// ---------------------------------------------------------------------------
constexpr int kWideTokens = 32;
struct WidenArgs {
  RowArgs r;                      // r.table, r.ld, r.lens: the tails'
  const int32_t* prefix_table;
  int prefix, prefix_pages, tail_pages, max_len;   // tokens; pages of it and of a tail; longest tail
  int64_t plane;                  // elements of a head in either pool
  int32_t* table;                 // [prefix_pages], then [N][tail_pages]
  int page_ctas;
  const bf16* q;
  int64_t q_n, q_t, q_h;
  int T, heads, group;
  float scale;                    // of the scores, to base 2
  __half* q_out;                  // [N][T][heads][dim]
  float* q_factor;                // [kv heads][N][T][group]
};

__device__ __forceinline__ void widen_queries(const WidenArgs& w) {
  const int64_t rows = (int64_t)w.r.N * w.T * w.heads;
  const int64_t cta = ((int64_t)blockIdx.x - w.page_ctas) * gridDim.y + blockIdx.y;
  const int64_t row = cta * (kThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x % 32, D = w.r.D;
  if (row >= rows) return;
  const int h = (int)(row % w.heads), t = (int)(row / w.heads % w.T), n = (int)(row / w.heads / w.T);
  const bf16* q = w.q + n * w.q_n + t * w.q_t + h * w.q_h;
  float x[4], top = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = lane * 2 + i % 2 + i / 2 * 64;
    x[i] = d < D ? to_f(q[d]) : 0.0f;
    top = fmaxf(top, fabsf(x[i]));
  }
  top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));
  float up;
  const float down = xpq::row_scale(top, &up);
#pragma unroll
  for (int i = 0; i < 4; i += 2)
    if (i * 32 < D)
      *(__half2*)(w.q_out + row * D + lane * 2 + i * 32) = __floats2half2_rn(x[i] * down, x[i + 1] * down);
  if (lane == 0) {
    const int64_t per_head = (int64_t)w.r.N * w.T * w.group;
    w.q_factor[h / w.group * per_head + ((int64_t)n * w.T + t) * w.group + h % w.group] =
        xpq::row_factor(up, w.scale);
  }
}

template <int BITS, int D>
__global__ void __launch_bounds__(kThreads) widen_kernel(const __grid_constant__ WidenArgs w) {
  const RowArgs& a = w.r;
  if ((int)blockIdx.x >= w.page_ctas) return widen_queries(w);
  constexpr int per = kWidePage / kWideTokens;
  const int page = blockIdx.x / per, t0 = (int)(blockIdx.x % per) * kWideTokens, h = blockIdx.y;
  const int tail = page - w.prefix_pages, n = tail < 0 ? 0 : tail / w.tail_pages;
  const int32_t* table = tail < 0 ? w.prefix_table : a.table + n * a.ld;
  int len = tail < 0 ? w.prefix : a.lens[n];
  if (tail >= 0 && (len < 0 || len > w.max_len)) len = len < 0 ? 0 : w.max_len;   // told by the attention
  const int pos0 = (tail < 0 ? page : tail % w.tail_pages) * kWidePage;
  if (pos0 >= len) return;
  if (h == 0 && t0 == 0 && threadIdx.x == 0) w.table[page] = page;

  // where the CTA's tokens begin in either pool, and their scales; behind the end -1
  __shared__ int64_t s_code[kWideTokens], s_scale[kWideTokens];
  if (threadIdx.x < kWideTokens) {
    const int pos = pos0 + t0 + (int)threadIdx.x;
    int64_t code = -1, scale = 0;
    if (pos < len) {
      const int col = pos / a.ps, at = pos - col * a.ps;
      int p = table[col];
      if (p < 0 || p >= a.pages) {
        atomicOr(a.err, XP_ERR_BADPAGE);
        p = p < 0 ? 0 : a.pages - 1;
      }
      const int64_t from = p * a.page + h * a.head;
      code = from + at * a.token;
      scale = from + a.scale_at + at * a.scale;
    }
    s_code[threadIdx.x] = code;
    s_scale[threadIdx.x] = scale;
  }
  __syncthreads();

  // A thread takes a piece of 8 dims of every 256 / (D/8)-th token: all codes, then all stores.
  constexpr int kPieces = D / 8, kStep = kThreads / kPieces, kEach = kWideTokens / kStep;
  const int e = threadIdx.x % kPieces * 8, i0 = threadIdx.x / kPieces;
  const char *k_code = a.kp + e / 8 * BITS, *v_code = a.vp + e / 8 * BITS;
  const char *k_scale = a.kp + e / 16, *v_scale = a.vp + e / 16;
  uint2 code[kEach][2];
  unsigned scale[kEach][2];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int64_t at = s_code[i0 + k * kStep], of_scale = s_scale[i0 + k * kStep];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      code[k][kv] = make_uint2(0, 0);
      scale[k][kv] = 0;
      if (at >= 0) {
        scale[k][kv] = (uint8_t)(kv ? v_scale : k_scale)[of_scale];
        const char* c = (kv ? v_code : k_code) + at;
        if (BITS == 4) code[k][kv].x = __ldcs((const unsigned*)c);
        else code[k][kv] = __ldcs((const uint2*)c);
      }
    }
  }
  __half* to = (__half*)a.k + h * w.plane + ((int64_t)page * kWidePage + t0 + i0) * D + e;
  const int64_t to_v = (__half*)a.v - (__half*)a.k;
#pragma unroll
  for (int k = 0; k < kEach; ++k)
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      __half2 v[4];
      widen<BITS>(code[k][kv], scale[k][kv], v);
      *(uint4*)(to + (kv ? to_v : 0) + k * kStep * D) = *(const uint4*)v;
    }
}

template <typename T> bool wide_rows(const RowArgs& a) {
  const int64_t strides = a.sn | a.st | a.sh | a.D;
  return (((uintptr_t)a.k | (uintptr_t)a.v) & 15) == 0 && strides * (int64_t)sizeof(T) % 16 == 0;
}

RowArgs row_args(const xp_cache* c, int layer, void* k, void* v, int64_t sn, int64_t st, int64_t sh,
                 const int32_t* table, int64_t ld, int64_t width, const int32_t* lens,
                 const int32_t* first, int N, int T) {
  const xp_cache_desc& d = c->d;
  const int64_t es = (int64_t)xp_elem(d.dtype);
  RowArgs a = {};
  a.kp = (char*)d.k + layer * d.stride_layer * es;
  a.vp = (char*)d.v + layer * d.stride_layer * es;
  a.page = d.stride_page, a.token = d.stride_token, a.head = d.stride_head;
  if (xp_is_quant(d.dtype)) {
    const xp_quant_sizes q = xp_quant_of(d.page_size, d.head_dim, d.dtype);
    a.scale_at = d.page_size * q.code;
    a.scale = q.scale;
  }
  a.k = k, a.v = v;
  a.sn = N == 1 ? 0 : sn, a.st = T == 1 ? 0 : st, a.sh = d.kv_heads == 1 ? 0 : sh;   // 0: never used
  a.table = table, a.ld = ld, a.width = width, a.lens = lens, a.first = first;
  a.N = N, a.T = T, a.H = d.kv_heads, a.D = d.head_dim, a.ps = d.page_size, a.pages = d.pages;
  a.err = c->err;
  return a;
}
unsigned row_grid(int N, int T) { return (unsigned)((int64_t)N * ((T + kTokens - 1) / kTokens)); }

template <int BITS> cudaError_t append(const RowArgs& a, xp_dtype rows, cudaStream_t s) {
  if (rows == XP_BF16) append_quant_kernel<BITS, bf16><<<row_grid(a.N, a.T), kThreads, 0, s>>>(a, wide_rows<bf16>(a));
  else append_quant_kernel<BITS, float><<<row_grid(a.N, a.T), kThreads, 0, s>>>(a, wide_rows<float>(a));
  return cudaGetLastError();
}
template <int BITS> cudaError_t read(const RowArgs& a, xp_dtype rows, cudaStream_t s) {
  if (rows == XP_BF16) read_kernel<BITS, bf16><<<row_grid(a.N, a.T), kThreads, 0, s>>>(a, wide_rows<bf16>(a));
  else read_kernel<BITS, float><<<row_grid(a.N, a.T), kThreads, 0, s>>>(a, wide_rows<float>(a));
  return cudaGetLastError();
}

}  // namespace

cudaError_t xp_launch_append_quant(const xp_cache* c, int layer, const void* k, const void* v, int64_t sn,
                                   int64_t st, int64_t sh, xp_dtype rows, const int32_t* table, int64_t ld,
                                   int64_t width, const int32_t* lens, int N, int T, cudaStream_t s) {
  const RowArgs a = row_args(c, layer, (void*)k, (void*)v, sn, st, sh, table, ld, width, lens, nullptr, N, T);
  return c->d.dtype == XP_Q8 ? append<8>(a, rows, s) : append<4>(a, rows, s);
}

cudaError_t xp_launch_widen(const xp_cache* c, const xp_attn_args& g, int prefix_pages, int tail_pages,
                            void* k, void* v, int64_t plane, int32_t* table, void* q, float* q_factor,
                            cudaStream_t s) {
  WidenArgs w;
  w.r = row_args(c, g.a.layer, k, v, 0, 0, 0, g.table, g.ld_table, 0, g.lens, nullptr, g.a.N, 0);
  w.prefix_table = g.prefix_table;
  w.prefix = g.a.prefix_len, w.prefix_pages = prefix_pages, w.tail_pages = tail_pages;
  w.max_len = g.a.max_len;
  w.plane = plane, w.table = table;
  w.page_ctas = (int)((prefix_pages + (int64_t)g.a.N * tail_pages) * (kWidePage / kWideTokens));
  w.q = (const bf16*)g.q;
  w.q_n = g.a.q_stride_n, w.q_t = g.a.q_stride_t, w.q_h = g.a.q_stride_h;
  w.T = g.a.T, w.heads = g.a.heads, w.group = g.group;
  w.scale = g.a.scale * 1.44269504088896f;
  w.q_out = (__half*)q, w.q_factor = q_factor;
  const int64_t rows = (int64_t)g.a.N * g.a.T * g.a.heads, each = (int64_t)g.kv_heads * (kThreads / 32);
  const dim3 grid((unsigned)(w.page_ctas + (rows + each - 1) / each), g.kv_heads);
  const bool narrow = c->d.head_dim == 64;   // or 128
  if (c->d.dtype == XP_Q8) {
    if (narrow) widen_kernel<8, 64><<<grid, kThreads, 0, s>>>(w);
    else widen_kernel<8, 128><<<grid, kThreads, 0, s>>>(w);
  } else {
    if (narrow) widen_kernel<4, 64><<<grid, kThreads, 0, s>>>(w);
    else widen_kernel<4, 128><<<grid, kThreads, 0, s>>>(w);
  }
  return cudaGetLastError();
}

cudaError_t xp_launch_cache_read(const xp_cache* c, int layer, const int32_t* table, int64_t ld,
                                 int64_t width, const int32_t* lens, const int32_t* first, int N, int T,
                                 void* k, void* v, int64_t sn, int64_t st, int64_t sh, xp_dtype rows,
                                 cudaStream_t s) {
  const RowArgs a = row_args(c, layer, k, v, sn, st, sh, table, ld, width, lens, first, N, T);
  switch (c->d.dtype) {
    case XP_BF16: return read<16>(a, rows, s);
    case XP_F32: return read<32>(a, rows, s);
    case XP_Q8: return read<8>(a, rows, s);
    default: return read<4>(a, rows, s);
  }
}
