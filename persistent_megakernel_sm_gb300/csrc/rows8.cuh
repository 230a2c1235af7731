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

// Codes of N values v (already rounded to the type T that they are held in) over
// the scale s, packed four to a word.
//
// bf16 values: v and s have 8 bits each, so a quotient below 128 that is not
// halfway between two integers is at least 2^-9 from it.  v times an approximate
// reciprocal (within 2^-22) is off by less than 2^-14; adding 1.5 2^13 rounds it
// to a multiple of 2^-10, which makes those exact that are halfway and leaves the
// others on their side; adding on to 1.5 2^23 rounds to the integer, half to
// even, whose low byte is the code: no quotient is over 127 (1 + 2^-8), which
// rounds to 127.  fp32 values, and scales that are zero or subnormal, are divided.
template <typename T, int N>
__device__ __forceinline__ void rows8_codes(const float (&v)[N], __nv_bfloat16 scale, uint32_t (&word)[N / 4]) {
  const float s = __bfloat162float(scale);
  uint32_t c[N];
  if (sizeof(T) == 2 && s >= 1.17549435e-38f) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    constexpr float kGrid = 12288.f, kInteger = 12582912.f;
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = __float_as_uint(fmaf(v[i], inv, kGrid) + (kInteger - kGrid));
  } else if (s == s) {
    const float div = s == 0.f ? 1.f : s;
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = (uint32_t)__float2int_rn(fminf(fmaxf(__fdiv_rn(v[i], div), -127.f), 127.f));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = 0;
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    word[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
}

// The four codes of a word as fp32, exactly: 2^23 + 128 + code, less 2^23 + 128.
__device__ __forceinline__ void rows8_floats(uint32_t word, float* v) {
  const uint32_t u = word ^ 0x80808080u;  // code + 128
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 | i)) - 8388736.f;
}

}  // namespace moe
