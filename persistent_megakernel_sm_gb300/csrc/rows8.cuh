// 8-bit rows: what one group of a row is held as.  The formulas are those of
// moe_rows8_quantize (moe.h); rows8.cu converts whole tensors with them, norm.cu
// keeps rows as it writes them.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace moe {

// The larger of |v| so far, as bits: they order as the magnitudes do, an
// infinity above every number and a NaN above that.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// A group's scale from the bits of its largest magnitude: max / 127 as bf16, NaN
// for a group with an infinity or a NaN in it.  A bf16 number over 127 is never near
// halfway between two bf16 numbers (127 times an odd number of 9 bits is odd and has
// more than 8), so that a product gives the quotient's bf16; fp32 is divided.
template <typename T>
__device__ __forceinline__ __nv_bfloat16 rows8_scale(uint32_t most) {
  if (most >= 0x7f800000u) return __ushort_as_bfloat16(0x7fffu);
  const float m = __uint_as_float(most);
  return __float2bfloat16_rn(sizeof(T) == 2 ? m * (1.f / 127.f) : __fdiv_rn(m, 127.f));
}

// Codes of 8 values by the definition: divisions.
__device__ __forceinline__ uint2 rows8_by_division(const float2 (&v)[4], float s) {
  const float div = s == 0.f ? 1.f : s;
  uint2 word = make_uint2(0, 0);
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const float2 p = i < 4 ? (i < 2 ? v[0] : v[1]) : (i < 6 ? v[2] : v[3]);
    const uint32_t c = (uint32_t)(__float2int_rn(fminf(fmaxf(__fdiv_rn(i & 1 ? p.y : p.x, div), -127.f), 127.f)) & 255) << (i % 4 * 8);
    if (i < 4) word.x |= c;
    else word.y |= c;
  }
  return word;
}

// Codes of 8 values v (rounded to the type T that they are held in, if that is bf16)
// over the scale s, packed four to a word.  Adding 1.5 2^23 to a quotient below 2^22
// rounds it to an integer, half to even, whose low byte is the code: none is over
// 127 (1 + 2^-8), which rounds to 127.  The quotient:
// - bf16 values: v and s have 8 bits each, so one that is not halfway between two
//   integers is at least 2^-9 from it.  v times an approximate reciprocal (within
//   2^-22) is off by less than 2^-14; adding 1.5 2^13 first rounds it to a multiple of
//   2^-10, which makes those exact that are halfway and leaves the others on their side.
// - fp32 values: one correction by the remainder, with the reciprocal correctly
//   rounded, gives the correctly rounded quotient (Markstein), unless the remainder is
//   too small to be exact.
// Scales that are zero or that small are divided; NaN gives zeros.
template <typename T>
__device__ __forceinline__ uint2 rows8_codes(const float2 (&v)[4], __nv_bfloat16 scale) {
  const float s = __bfloat162float(scale);
  if (!(s == s)) return make_uint2(0, 0);
  if (s < (sizeof(T) == 2 ? 1.17549435e-38f : 7.9e-31f))  // 2^-126, 2^-100
    return rows8_by_division(v, s);
  constexpr float kGrid = 12288.f, kInteger = 12582912.f;
  float2 c[4];
  if constexpr (sizeof(T) == 2) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = __fadd2_rn(__ffma2_rn(v[i], make_float2(inv, inv), make_float2(kGrid, kGrid)), make_float2(kInteger - kGrid, kInteger - kGrid));
  } else {
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = __fmul2_rn(v[i], make_float2(inv, inv));
      const float2 left = __ffma2_rn(q, make_float2(-s, -s), v[i]);
      c[i] = __fadd2_rn(__ffma2_rn(left, make_float2(inv, inv), q), make_float2(kInteger, kInteger));
    }
  }
  auto bits = [](float x) { return __float_as_uint(x); };
  auto four = [&](float2 a, float2 b) {
    return __byte_perm(__byte_perm(bits(a.x), bits(a.y), 0x0040), __byte_perm(bits(b.x), bits(b.y), 0x0040), 0x5410);
  };
  return make_uint2(four(c[0], c[1]), four(c[2], c[3]));
}

// The four codes of a word as fp32, exactly: 2^23 + 128 + code, less 2^23 + 128.
__device__ __forceinline__ void rows8_floats(uint32_t word, float2 (&v)[2]) {
  const uint32_t u = word ^ 0x80808080u;  // code + 128
  auto at = [&](int i) { return __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 | i)); };
  const float2 base = make_float2(-8388736.f, -8388736.f);
  v[0] = __fadd2_rn(make_float2(at(0), at(1)), base);
  v[1] = __fadd2_rn(make_float2(at(2), at(3)), base);
}

}  // namespace moe
