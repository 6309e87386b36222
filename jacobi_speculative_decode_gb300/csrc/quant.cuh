// The quantised cache's format: sizes of its pieces, and codes and scales on the device.
//
// 16 dims of a token's head share a scale s, the 16-bit float whose bits are a byte << 7 (5 bits of
// exponent, 3 of mantissa); an element is c s, c a whole number of 8 or 4 bits.  c s has at most 7 + 4
// bits, so 16-bit floats hold it exactly: products on tensor cores take it without a rounding of
// their own (and in 4 bits, 3 + 4, bf16 does too).
#pragma once

#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "xp_internal.h"

// bytes of a token's codes and of its scales, and of one head of a page
struct xp_quant_sizes {
  int code, scale;
  int64_t head;
};
inline bool xp_is_quant(xp_dtype t) { return t == XP_Q8 || t == XP_Q4; }
inline xp_quant_sizes xp_quant_of(int page_size, int head_dim, xp_dtype t) {
  xp_quant_sizes q;
  q.code = t == XP_Q8 ? head_dim : head_dim / 2;
  q.scale = (head_dim / 16 + 3) / 4 * 4;
  q.head = ((int64_t)page_size * (q.code + q.scale) + 15) / 16 * 16;
  return q;
}

constexpr int kWidePage = 128;   // tokens of a page of a cache widened for tcgen05

#ifdef __CUDACC__
namespace xpq {

template <int BITS> struct Codes {
  static constexpr int kMost = (1 << (BITS - 1)) - 1;   // greatest code
  static constexpr int kZero = 1 << (BITS - 1);         // how code 0 is held
  // greatest scale: the last for which kMost * s is a finite 16-bit float (512); of 4 bits 7680, for which
  // 1024 * s * 2^-7 is
  static constexpr unsigned kTop = BITS == 4 ? 0xDFu : 0xC0u;
};

__device__ __forceinline__ float scale_of(unsigned byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// A query row of largest magnitude `top` as fp16: times 2^-e, e its exponent, 2^-119 at least (what is
// not finite stays so), which is exact but for what lies 2^-14 and more below the largest; *up: 2^e.
__device__ __forceinline__ float row_scale(float top, float* up) {
  const int e = min(max((int)(__float_as_uint(top) >> 23), 8), 253);   // so that 2^-e times 16 is finite too
  *up = __uint_as_float((uint32_t)e << 23);
  return __uint_as_float((uint32_t)(254 - e) << 23);
}
// What a product of that row is multiplied by to be a score in base 2.  Never 0: a hidden key's -inf times it
// has to stay -inf.
__device__ __forceinline__ float row_factor(float up, float scale) {
  return fmaxf(fminf(scale * up, 3.0e38f), FLT_MIN);
}

// The least scale that reaches `top`, a group's largest magnitude; *over where none does.
template <int BITS> __device__ __forceinline__ unsigned scale_byte(float top, bool* over) {
  constexpr float most = Codes<BITS>::kMost;
  const unsigned h = __half_as_ushort(__float2half_ru(top / most));
  unsigned b = min((h + 127u) >> 7, Codes<BITS>::kTop);
  // the quotient may have been rounded down onto a scale just short of it; products are exact
  if (b < Codes<BITS>::kTop && scale_of(b) * most < top) ++b;
  *over = scale_of(b) * most < top;
  return b;
}

// x over s to the nearest whole number, ties to even, at most +-kMost (s = 0: every x of its group is 0)
template <int BITS> __device__ __forceinline__ int code_of(float x, float s) {
  constexpr float most = Codes<BITS>::kMost;
  if (s == 0.0f) return 0;
  float n = fminf(fmaxf(rintf(x / s), -most), most);
  // The quotient may have been rounded onto a tie that is none.  What is left is exact.
  const float rest = fmaf(-n, s, x);
  n += rest > 0.5f * s ? 1.0f : rest < -0.5f * s ? -1.0f : 0.0f;
  return (int)fminf(fmaxf(n, -most), most);
}

}  // namespace xpq
#endif
