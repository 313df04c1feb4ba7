// Rows of 16-bit floats as 8-bit integers with one scale (gfx950), shared by the
// products in 8-bit integers and the cache:
//
//   top = max |x|,   code = rint(127 x / top),   scale = top / 127
//
// A row of zeros has codes and scale zero; a row that holds an infinity or NaN has
// codes zero and the scale NaN, so that everything made of it is NaN.
#ifndef DFH_QUANT_H
#define DFH_QUANT_H

#include "dfh_gemm.h"

namespace dfh {
namespace {

// The bits above which a magnitude is an infinity or NaN.
__device__ __forceinline__ constexpr uint32_t finite_bits(BF16) { return 0x7F7Fu; }
__device__ __forceinline__ constexpr uint32_t finite_bits(F16) { return 0x7BFFu; }

// The larger of two pairs of 16-bit magnitudes (bits, so a NaN is the largest).
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t most_pair(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t most_bits(u32x4 v, uint32_t so_far) {
#pragma unroll
  for (int i = 0; i < 4; i++) so_far = most_pair(so_far, v[i] & 0x7FFF7FFFu);
  return so_far;
}
__device__ __forceinline__ uint32_t joined(uint32_t pair) {
  return (pair & 0xFFFFu) > pair >> 16 ? pair & 0xFFFFu : pair >> 16;
}

// Quantises by a row's largest magnitude.  127 x / top has to be rounded as the
// quotient itself is: of two 16-bit floats it is either half way between two
// integers or at least 2^-19 of itself away from there (|254 X - odd A| >= 1 over
// 254 X, X < 2^11), so any quotient within 2^-22 rounds right where it is no tie, and
// the step of Newton's below makes a quotient that FP32 holds, as a tie is, exact.
// Exponents are taken off first: 127 x then neither overflows nor loses bits that a
// code could see.
struct Quantiser {
  float top, inv, scale;
  int down;
  template <class T>
  __device__ __forceinline__ void init(T, uint32_t bits) {
    const bool good = bits <= finite_bits(T{});
    const float t = from_bits(T{}, (uint16_t)bits);
    scale = good ? t / 127.f : __builtin_nanf("");
    down = good && t > 0.f ? -__builtin_amdgcn_frexp_expf(t) : 0;
    top = good && t > 0.f ? __builtin_ldexpf(t, down) : 1.f;
    inv = good && t > 0.f ? 1.f / top : 0.f;
  }
  // the code in the low byte
  __device__ __forceinline__ uint32_t code(float x) const {
    const float y = 127.f * __builtin_ldexpf(x, down);
    float q = y * inv;
    q = __builtin_fmaf(__builtin_fmaf(-q, top, y), inv, q);
    // an integer's two's complement in the low bits of 1.5 2^23 + it
    return __float_as_uint(q + 12582912.f);
  }
  template <class T>
  __device__ __forceinline__ u32x2 codes(T, u32x4 v) const {
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      c[2 * i] = code(from_bits(T{}, (uint16_t)v[i]));
      c[2 * i + 1] = code(from_bits(T{}, (uint16_t)(v[i] >> 16)));
    }
    u32x2 o;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const uint32_t lo = __builtin_amdgcn_perm(c[4 * i + 1], c[4 * i], 0x0C0C0400u);
      const uint32_t hi = __builtin_amdgcn_perm(c[4 * i + 3], c[4 * i + 2], 0x0C0C0400u);
      o[i] = lo | hi << 16;
    }
    // infinities and NaN times zero are no numbers, whose low bits are no code
    return inv == 0.f ? u32x2{0, 0} : o;
  }
};

}  // namespace
}  // namespace dfh

#endif
