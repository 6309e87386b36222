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
  const int e = min(max((int)(__float_as_uint(top) >> 23), 8), 253);   // so that 2^-e times 128 is finite too
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
  constexpr float most = Codes<BITS>::kMost, least = 6.103515625e-05f;   // 2^-14, the least that is not subnormal
  // A quotient that is not above the true one; in the scales' bits, rounded up.  A subnormal one, whole 2^-17,
  // is taken 2^-14 higher, where the spacing is the same, and 8 places back.
  const float q = __fmul_rd(fminf(top, 65536.0f), BITS == 4 ? 0x1.249248p-3f : 0x1.020408p-7f);
  const bool low = q < least;
  const unsigned bits = __float_as_uint(low ? __fadd_rd(q, least) : q) - (112u << 23);
  unsigned b = ((bits + 0xFFFFFu) >> 20) - (low ? 8u : 0u);
  b = min(b, Codes<BITS>::kTop);
  if (b < Codes<BITS>::kTop && scale_of(b) * most < top) ++b;   // products are exact
  *over = scale_of(b) * most < top;
  return b;
}

// E elements x over s (|x| at most kMost * s) to the nearest whole numbers, ties to even, as they are held; r: about
// 1/s.  A product with r may lie across a half, or on one; what a code leaves of x is exact, and where it is
// half of s or more the code is looked at again.
template <int BITS, int E>
__device__ __forceinline__ void codes_of(const float (&x)[E], float s, float r, uint32_t (&code)[E]) {
  constexpr float magic = 12582912.0f + Codes<BITS>::kZero;   // 1.5 * 2^23: a sum's last bits are the whole number
  const float half = 0.5f * s;
  bool look = false;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const float t = fmaf(x[j], r, magic);
    look |= fabsf(fmaf(magic - t, s, x[j])) >= half;
    code[j] = __float_as_uint(t) & 0xFFu;
  }
  if (look && s > 0.0f) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int whole = (int)code[j] - Codes<BITS>::kZero;
      const float rest = fmaf(-(float)whole, s, x[j]);
      if (fabsf(rest) > half || (fabsf(rest) == half && (whole & 1))) code[j] += rest > 0.0f ? 1 : -1;
    }
  }
}

}  // namespace xpq
#endif
